// host_state.h - host-side state and helpers shared by the library's translation units
// (defined in squad_api.cu): per-device facts, the error word, tensor-map encoding.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "squad.h"

// Returns SQUAD_ERR_CUDA from the calling function where a CUDA call fails.
#define SQ_CUDA(call)                                          \
  do {                                                         \
    cudaError_t e_ = (call);                                   \
    if (e_ != cudaSuccess) return sq::host_cuda_fail(int(e_)); \
  } while (0)

#define SQ_HIDDEN __attribute__((visibility("hidden")))

namespace sq {

constexpr uint64_t kWaitTimeoutNs = 2000000000ull;  // 2 s per wait, where no wait lasts longer than a job

struct HostDevice {
  int device;
  int sms;
  int* err;  // device address of the library's error word
};

// Facts of the current device; binds its primary context to this thread.
SQ_HIDDEN squad_status host_device(HostDevice* out);
// Remembers a failing CUDA call's code for squad_last_cuda_error.
SQ_HIDDEN squad_status host_cuda_fail(int code);
// Tiled bf16 tensor map with the 128-byte swizzle (taken from the cache where it was made
// before); call host_device first.
SQ_HIDDEN squad_status host_encode_bf16(CUtensorMap* m, int device, int rank, const void* base,
                                        const uint64_t* dims, const uint64_t* strides, const uint32_t* box);

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sq
