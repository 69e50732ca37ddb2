// Host model of the barriers of the cross-attention kernels on the tensor cores (cross_fwd_tc.cuh, cross_bwd_tc.cuh): each
// warp's role as a coroutine with the waits and arrivals of the kernel, one CTA at a time over the items of the real
// work plan, run in random order. Copies land at random times; products run in the order of their issue, and read and
// write what they do when they run. Checked: a wait by parity returns for the phase that it was meant for and no other,
// no barrier gets more arrivals than it counts, every product and every role finds the tile, the scores, the mask, the
// statistics or the sum that it should, nothing is overwritten before its last reader, and every role comes to its end.
//
// Not in the model: the epilogue's staging buffers (each warp's own, in the order of its stores), and what a role does
// when a wait gives up.
//
// cross_protocol_check [runs] [seed] [plant]: plant > 0 leaves out a wait (see PLANT; forward 1 to 8, dQ 11 to 18, dK
// and dV 21 to 28) and has to be found.
#include <algorithm>
#include <coroutine>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <memory>
#include <string>
#include <vector>

#include "cross_plan.h"

static int g_plant = 0;
static std::string g_what;  // the run, for messages

[[noreturn]] static void fail(const std::string& why) {
  std::printf("FAIL %s: %s\n", g_what.c_str(), why.c_str());
  std::exit(1);
}
static void check(bool ok, const char* why) {
  if (!ok) fail(why);
}

struct Rng {
  unsigned s;
  int operator()(int n) {
    s = s * 1664525u + 1013904223u;
    return int((s >> 8) % unsigned(n));
  }
};

struct Bar {
  int count = 1, pending = 1, tx = 0, phase = 0;
  void init(int n) { count = pending = n; }
  void settle() {
    if (pending == 0 && tx == 0) {
      ++phase;
      pending = count;
    }
  }
  void arrive() {
    check(pending > 0, "an arrival beyond the barrier's count");
    --pending;
    settle();
  }
  void expect() {
    ++tx;
    arrive();
  }
  void landed() {
    --tx;
    settle();
  }
  // A wait for phase `want` (-1: passes on a fresh barrier), by its parity.
  bool ready(int want) const {
    const bool passes = (phase & 1) != (want & 1);
    check(passes ? phase == want + 1 : phase == want, "a wait meets another phase of its parity");
    return passes;
  }
};

struct Task {
  struct promise_type {
    const Bar* bar = nullptr;  // waits for it, or for its turn
    int want = 0;
    Task get_return_object() { return Task{std::coroutine_handle<promise_type>::from_promise(*this)}; }
    std::suspend_always initial_suspend() noexcept { return {}; }
    std::suspend_always final_suspend() noexcept { return {}; }
    void return_void() {}
    void unhandled_exception() { std::abort(); }
  };
  std::coroutine_handle<promise_type> h;
};
struct On {  // co_await On{bar, want}: the wait of a role
  const Bar* bar;
  int want;
  bool await_ready() const noexcept { return false; }
  void await_suspend(std::coroutine_handle<Task::promise_type> h) const noexcept {
    h.promise().bar = bar;
    h.promise().want = want;
  }
  void await_resume() const noexcept {}
};
static On turn() { return On{nullptr, 0}; }
#define WAIT(bar, want) co_await On{&(bar), int(want)}
#define PLANT(id, bar, want) \
  if (g_plant != kPlants + (id)) co_await On{&(bar), int(want)}

struct Cta {
  Rng& rnd;
  explicit Cta(Rng& r) : rnd(r) {}
  std::vector<std::function<void()>> copies;             // in flight, land in any order
  std::vector<std::function<void()>> pipe;               // products and commits, in order
  size_t done = 0;
  std::vector<std::coroutine_handle<Task::promise_type>> roles;
  std::vector<int> weight;
  void add(Task t) {
    roles.push_back(t.h);
    weight.push_back(rnd(4) ? 32 : 1);  // some roles are slow
  }
  void commit(Bar& b) {
    pipe.push_back([&b] { b.arrive(); });
  }
  void run() {
    const int slow_copies = rnd(3) ? 24 : 1, slow_pipe = rnd(3) ? 24 : 1;
    for (;;) {
      std::vector<std::pair<int, int>> can;  // (what, weight)
      int total = 0;
      bool live = false;
      for (size_t i = 0; i < roles.size(); ++i) {
        if (roles[i].done()) continue;
        live = true;
        auto& p = roles[i].promise();
        if (p.bar != nullptr && !p.bar->ready(p.want)) continue;
        can.push_back({int(i), weight[i]});
        total += weight[i];
      }
      if (!copies.empty()) can.push_back({-1, slow_copies}), total += slow_copies;
      if (done < pipe.size()) can.push_back({-2, slow_pipe}), total += slow_pipe;
      if (can.empty()) {
        if (live) fail("no role can go on");
        break;
      }
      int at = rnd(total), what = 0;
      for (auto& c : can) {
        if (at < c.second) {
          what = c.first;
          break;
        }
        at -= c.second;
      }
      if (what == -1) {
        const int i = rnd(int(copies.size()));
        auto f = copies[i];
        copies.erase(copies.begin() + i);
        f();
      } else if (what == -2) {
        auto f = pipe[done];
        pipe[done++] = nullptr;
        f();
      } else {
        roles[what].promise().bar = nullptr;
        roles[what].resume();
      }
    }
    for (auto h : roles) h.destroy();
  }
};

struct Tile {
  int item = -1, block = -1;  // whose
  char kind = ' ';            // 'K', 'V', 'Q', 'O' (dO)
  bool there = false, zeroed = false;
  bool is(char k, int i, int b) const { return there && kind == k && item == i && block == b; }
};

struct Shape {
  int B, heads, kv_heads, n, m;
  std::vector<int> len;
  int mask;  // 0: none, 1: lengths, 2: a byte for each key
};

// ==================================================================== forward
struct Forward : Cta {
  static constexpr int kPlants = 0;
  const Shape& sh;
  const sq::CrossPlan plan;
  const int d, nkv, ns, first, step;
  std::vector<sq::CrossItem> items;
  std::vector<sq::CrossRange> ranges;
  std::vector<int> lens;
  int count, size;  // rings
  std::vector<Bar> kvf, kve, rdy, wf;
  Bar qf[2], qe[2], sf[2], pf[2], of[2], oe[2], lf[2], le[2], drain;
  std::vector<Tile> slots;
  std::vector<std::pair<int, int>> bias, words;  // (item, block) of every operand and word place
  std::vector<int> word_reads;                   // of a place, still to come
  Tile q[2];
  struct Scores {
    int item = -1, k = -1, warps = 0;  // of P
    bool used = true;                  // by P V
  } s[2];
  struct Out {
    int item = -1, blocks = 0, drained = 4;
  } o[2];
  int stat[2][4];

  Forward(Rng& r, const Shape& shape, int dim, int cta, int ctas)
      : Cta(r), sh(shape), plan(sq::make_cross_plan(shape.B, shape.heads, shape.kv_heads, shape.n, shape.m)), d(dim),
        nkv(dim == 128 ? 4 : shape.mask == 2 ? 8 : 10), ns(nkv / 2), first(cta), step(ctas) {
    for (int i = first; i < plan.items; i += step) {
      items.push_back(sq::cross_item(plan, sh.heads, i));
      lens.push_back(sh.mask ? sh.len[items.back().b] : sh.m);
      ranges.push_back(sq::cross_range(plan, lens.back(), items.back().sp[0]));
    }
    count = plan.splits > 1 ? 2 : 1;
    size = count == 2 ? ns : nkv;
    kvf.resize(nkv);
    kve.resize(nkv);
    rdy.resize(nkv);
    wf.resize(16);
    slots.resize(nkv);
    bias.assign(nkv / 2, {-1, -1});
    words.assign(16, {-1, -1});
    word_reads.assign(16, 0);
    for (int x = 0; x < 2; ++x) {
      pf[x].init(4);
      oe[x].init(4);
      lf[x].init(4);
      le[x].init(4);
      for (int& w : stat[x]) w = -1;
    }
  }
  int slot(int x, int n) const { return (count == 2 ? x * size : 0) + n % size; }
  int block(int j, int x, int k) const { return ranges[j].k0 + (count == 2 ? x * ranges[j].nk : 0) + k; }

  Task loader() {
    int e[2] = {0, 0};
    for (int j = 0; j < int(items.size()); ++j)
      for (int k = 0; k <= ranges[j].nk; ++k)
        for (int x = 0; x < count; ++x)
          for (int v = 1; v >= 0; --v) {  // values of block k - 1, then keys of block k
            if (v ? k == 0 : k == ranges[j].nk) continue;
            const int n = e[x]++, at = slot(x, n), b = block(j, x, k - v);
            PLANT(1, kve[at], n / size - 1);
            const bool cut = v && (b + 1) * 128 > lens[j];
            Bar& full = sh.mask == 1 && cut ? rdy[at] : kvf[at];
            full.expect();
            slots[at] = Tile{};
            copies.push_back([this, at, j, b, v, &full] {
              slots[at] = Tile{j, b, v ? 'V' : 'K', true, false};
              full.landed();
            });
          }
    for (int x = 0; x < count; ++x)
      for (int i = 0; i < size; ++i)
        if (e[x] > i) WAIT(kvf[x * size + i], (e[x] - 1 - i) / size);
  }
  Task lengths() {  // the mask warp where a length is all there is
    int e[2] = {0, 0};
    std::vector<int> seen(nkv, 0);
    for (int j = 0; j < int(items.size()); ++j) {
      const int cut = lens[j] >> 7, nk = ranges[j].nk, k0 = ranges[j].k0;
      for (int k = std::max(0, cut - (k0 + (count - 1) * nk)); k < nk; ++k)
        for (int x = 0; x < count; ++x) {
          const int b = k0 + x * nk + k;
          if (b < cut) continue;
          const int at = slot(x, e[x] + 2 * k + 1);
          PLANT(2, rdy[at], seen[at]);
          ++seen[at];
          check(slots[at].is('V', j, b), "the mask warp zeroes another tile");
          slots[at].zeroed = true;
          co_await turn();
          kvf[at].arrive();
        }
      e[0] += 2 * nk;
      e[1] += 2 * nk;
    }
  }
  Task keys() {  // the mask warp with a mask of each key
    int e[2] = {0, 0}, blocks[2] = {0, 0};
    for (int j = 0; j < int(items.size()); ++j)
      for (int k = 0; k <= ranges[j].nk; ++k)
        for (int x = 0; x < count; ++x)
          for (int v = 1; v >= 0; --v) {
            if (v ? k == 0 : k == ranges[j].nk) continue;
            const int n = e[x]++, at = slot(x, n), b = block(j, x, k - v);
            WAIT(kvf[at], n / size);
            check(slots[at].is(v ? 'V' : 'K', j, b), "the mask warp zeroes another tile");
            slots[at].zeroed = true;
            if (!v) {
              const int w = x * 8 + blocks[x]++ % 8;
              bias[at >> 1] = {j, b};
              check(word_reads[w] == 0, "a mask is overwritten before its last reader");
              words[w] = {j, b};
              word_reads[w] = count == 2 ? 4 : items[j].qt[1] >= 0 ? 8 : 4;
              wf[w].arrive();
              co_await turn();
            }
            rdy[at].arrive();
          }
  }
  Task queries() {
    int n[2] = {0, 0};
    for (int j = 0; j < int(items.size()); ++j)
      for (int x = 0; x < 2; ++x) {
        if (items[j].qt[x] < 0) continue;
        PLANT(3, qe[x], n[x] - 1);
        ++n[x];
        qf[x].expect();
        q[x] = Tile{};
        copies.push_back([this, x, j] {
          q[x] = Tile{j, items[j].qt[x], 'Q', true, false};
          qf[x].landed();
        });
      }
    for (int x = 0; x < 2; ++x)
      if (n[x]) WAIT(qf[x], n[x] - 1);
  }
  Task issuer() {
    struct Pending {
      bool on = false, first = false, last = false, fresh = false, done = false;
      int item = 0, k = 0, v = 0;  // entry of its value tile
    } pend[2];
    int pos[2] = {0, 0}, kpos = 0, products[2] = {0, 0}, jobs[2] = {0, 0}, tiles[2] = {0, 0};
    std::vector<Bar>& full = sh.mask == 2 ? rdy : kvf;
    const bool own = count == 2;
    for (int j = 0;; ++j) {
      const bool more = j < int(items.size());
      const int nk = more ? ranges[j].nk : 1;
      const bool two = more && items[j].qt[1] >= 0;
      for (int k = 0; k < nk; ++k)
        for (int x = 0; x < 2; ++x) {
          const bool scores = more && (x == 0 || two);
          const Pending p = pend[x];
          const int ring = own ? x : 0;
          if (p.on) {
            if (p.fresh) WAIT(full[slot(ring, p.v)], p.v / size);
            if (p.first) {
              if (jobs[x] > 0) PLANT(4, oe[x], jobs[x] - 1);
              ++jobs[x];
            }
          }
          const bool fresh = own || x == 0, done = own || x == 1 || !two;
          if (scores) {
            if (fresh) {
              kpos = pos[ring];
              pos[ring] += 2;
              WAIT(full[slot(ring, kpos)], kpos / size);
            }
            if (k == 0) {
              WAIT(qf[x], tiles[x]);
              ++tiles[x];
            }
          }
          if (p.on) {  // P V of the block before
            PLANT(5, pf[x], products[x]);
            ++products[x];
            const int at = slot(ring, p.v), b = block(p.item, x, p.k), len = lens[p.item];
            pipe.push_back([this, x, p, at, b, len] {
              check(slots[at].is('V', p.item, b), "P V reads another tile");
              check(slots[at].zeroed || sh.mask == 0 || (sh.mask == 1 && (b + 1) * 128 <= len), "P V reads masked values");
              check(s[x].item == p.item && s[x].k == p.k && s[x].warps == 4 && !s[x].used, "P V reads another P");
              s[x].used = true;
              if (p.first) {
                check(o[x].drained == 4, "O is overwritten before the epilogue has read it");
                o[x] = Out{p.item, 0, 0};
              }
              check(o[x].item == p.item && o[x].blocks == p.k, "P V adds to another O");
              ++o[x].blocks;
            });
            if (p.done) commit(kve[at]);
            if (p.last) commit(of[x]);
            pend[x].on = false;
          }
          if (!scores) continue;
          const int at = slot(ring, kpos), b = block(j, x, k);
          pipe.push_back([this, x, j, k, at, b] {
            check(slots[at].is('K', j, b), "S reads another tile");
            check(sh.mask != 2 || (slots[at].zeroed && bias[at >> 1] == std::make_pair(j, b)), "S reads another mask");
            check(q[x].is('Q', j, items[j].qt[x]), "S reads other queries");
            check(s[x].used, "S overwrites a P that is still to be used");
            s[x] = Scores{j, k, 0, false};
          });
          commit(sf[x]);
          if (done) commit(kve[at]);
          if (k == nk - 1) commit(qe[x]);
          pend[x] = Pending{true, k == 0, k == nk - 1, fresh, done, j, k, kpos + 1};
        }
      if (!more) break;
    }
    commit(drain);
    WAIT(drain, 0);
  }
  Task softmax(int x, int w) {
    int seen = 0, jobs = 0, at = 0;
    for (int j = 0; j < int(items.size()); ++j) {
      if (items[j].qt[x] < 0) {
        at += ranges[j].nk;
        continue;
      }
      for (int k = 0; k < ranges[j].nk; ++k) {
        PLANT(6, sf[x], seen);
        ++seen;
        check(s[x].item == j && s[x].k == k && !s[x].used, "the softmax reads other scores");
        if (sh.mask == 2) {
          const int place = (count == 2 ? x * 8 : 0) + at % 8;
          WAIT(wf[place], at / 8);
          ++at;
          check(words[place] == std::make_pair(j, block(j, x, k)), "the softmax reads another mask");
          --word_reads[place];
        }
        // O is rescaled where the maximum grows: every product before has run
        check(k == 0 || (o[x].item == j && o[x].blocks == k), "O is rescaled under a product");
        co_await turn();
        ++s[x].warps;
        pf[x].arrive();
        co_await turn();
      }
      PLANT(7, le[x], jobs - 1);
      ++jobs;
      check(stat[x][w] == -1, "statistics are overwritten before the epilogue has read them");
      stat[x][w] = j;
      co_await turn();
      lf[x].arrive();
    }
  }
  Task epilogue(int w) {
    int jobs[2] = {0, 0};
    for (int j = 0; j < int(items.size()); ++j)
      for (int x = 0; x < 2; ++x) {
        if (items[j].qt[x] < 0) continue;
        const int job = jobs[x]++;
        WAIT(lf[x], job);
        check(stat[x][w] == j, "the epilogue reads other statistics");
        stat[x][w] = -1;
        co_await turn();
        le[x].arrive();
        PLANT(8, of[x], job);
        check(o[x].item == j && o[x].blocks == ranges[j].nk && o[x].drained < 4, "the epilogue reads another O");
        co_await turn();
        check(o[x].item == j && o[x].blocks == ranges[j].nk, "O changes under the epilogue");
        ++o[x].drained;
        oe[x].arrive();
      }
  }
  void go() {
    add(loader());
    add(queries());
    add(issuer());
    if (sh.mask == 1) add(lengths());
    if (sh.mask == 2) add(keys());
    for (int x = 0; x < 2; ++x)
      for (int w = 0; w < 4; ++w) add(softmax(x, w));
    for (int w = 0; w < 4; ++w) add(epilogue(w));
    run();
    for (int x = 0; x < 2; ++x) check(s[x].used && o[x].drained == 4, "something is left over");
  }
};

// ==================================================================== dQ
struct BackwardDq : Cta {
  static constexpr int kPlants = 10;
  const Shape& sh;
  const int nk_, nv_, qtiles, kblocks, splits;  // ring sizes; the plan
  struct Item {
    int b, qt, sp, len, nk;
  };
  std::vector<Item> items;
  std::vector<Bar> kf, ke, kr, vf, ve, vr, wf;
  Bar qf, qe, dof, doe, sf[2], dpf, dsf, of, oe, df[2], de[2], xd[4], drain;
  std::vector<Tile> ks, vs;
  Tile q, dout;
  std::vector<std::pair<int, int>> words;
  std::vector<int> word_reads;
  struct Scores {
    int t = -1, warps = 0;  // of dS
    bool used = true;
  } s[2];
  struct {
    int t = -1, reads = 8;
  } dp;
  struct {
    int item = -1, blocks = 0, drained = 4;
  } acc;
  std::vector<int> d_made;
  int halves[2][2][4];  // [parity][half][warp]: the tile whose half sum lies there

  BackwardDq(Rng& r, const Shape& shape, int d, int cta, int ctas)
      : Cta(r), sh(shape), nk_(d == 128 ? 3 : 4), nv_(d == 128 ? 2 : 4), qtiles((shape.n + 127) / 128),
        kblocks((shape.m + 127) / 128),
        splits(sq::cross_dq_splits((long long)shape.B * shape.heads * qtiles, kblocks, true)) {
    const int all = sh.B * sh.heads * qtiles * splits;
    for (int i = cta; i < all; i += ctas) {
      Item it;
      const int bh = i / (qtiles * splits), rest = i % (qtiles * splits);
      it.b = bh / sh.heads;
      it.qt = rest / splits;
      it.sp = rest % splits;
      it.len = sh.mask ? sh.len[it.b] : sh.m;
      const int nb = (it.len + 127) >> 7;
      it.nk = std::max(1, (nb + splits - 1) / splits);
      items.push_back(it);
    }
    for (auto* v : {&kf, &ke, &kr}) v->resize(nk_);
    for (auto* v : {&vf, &ve, &vr}) v->resize(nv_);
    wf.resize(8);
    ks.resize(nk_);
    vs.resize(nv_);
    words.assign(8, {-1, -1});
    word_reads.assign(8, 0);
    d_made.assign(items.size(), 0);
    dsf.init(8);
    oe.init(4);
    for (int i = 0; i < 2; ++i) {
      df[i].init(4);
      de[i].init(8);
    }
    for (Bar& b : xd) b.init(2);
    for (auto& a : halves)
      for (auto& h : a)
        for (int& w : h) w = -1;
  }
  bool exact(int j) const { return splits == 1 && items[j].nk == 1; }

  Task loader(bool values) {
    int e = 0, n = 0;
    const int size = values ? nv_ : nk_;
    auto &full = values ? vf : kf, &empty = values ? ve : ke;
    auto& ring = values ? vs : ks;
    Bar &xf = values ? dof : qf, &xe = values ? doe : qe;
    Tile& x = values ? dout : q;
    for (int j = 0; j < int(items.size()); ++j)
      for (int k = 0; k < items[j].nk; ++k) {
        const int at = e % size, b = items[j].sp * items[j].nk + k;
        PLANT(1, empty[at], e / size - 1);
        ++e;
        full[at].expect();
        ring[at] = Tile{};
        copies.push_back([&ring, at, j, b, values, &full] {
          ring[at] = Tile{j, b, values ? 'V' : 'K', true, false};
          full[at].landed();
        });
        if (k == 0) {
          PLANT(3, xe, n - 1);
          ++n;
          xf.expect();
          x = Tile{};
          copies.push_back([&x, &xf, j, values] {
            x = Tile{j, 0, values ? 'O' : 'Q', true, false};
            xf.landed();
          });
        }
      }
    for (int i = 0; i < size; ++i)
      if (e > i) WAIT(full[i], (e - i + size - 1) / size - 1);
    if (n) WAIT(xf, n - 1);
  }
  Task masks() {
    int t = 0;
    for (int j = 0; j < int(items.size()); ++j)
      for (int k = 0; k < items[j].nk; ++k, ++t) {
        const int b = items[j].sp * items[j].nk + k, a = t % nk_, c = t % nv_;
        PLANT(2, kf[a], t / nk_);
        check(ks[a].is('K', j, b), "the mask warp zeroes another key tile");
        ks[a].zeroed = true;
        if (sh.mask == 2) {
          check(word_reads[t % 8] == 0, "a mask is overwritten before its last reader");
          words[t % 8] = {j, b};
          word_reads[t % 8] = 8;
          wf[t % 8].arrive();
          co_await turn();
        }
        kr[a].arrive();
        WAIT(vf[c], t / nv_);
        check(vs[c].is('V', j, b), "the mask warp zeroes another value tile");
        vs[c].zeroed = true;
        co_await turn();
        vr[c].arrive();
      }
  }
  void dq(int t, int j, int k) {  // issue of dQ(t)
    const int at = t % nk_, b = items[j].sp * items[j].nk + k;
    pipe.push_back([this, t, j, k, at, b] {
      check(ks[at].is('K', j, b), "dQ reads another key tile");
      check(s[t & 1].t == t && s[t & 1].warps == 8 && !s[t & 1].used, "dQ reads another dS");
      s[t & 1].used = true;
      if (k == 0) {
        check(acc.drained == 4, "dQ is overwritten before the epilogue has read it");
        acc = {j, 0, 0};
      }
      check(acc.item == j && acc.blocks == k, "dQ adds to another tile's");
      ++acc.blocks;
    });
    commit(ke[at]);
    if (k == items[j].nk - 1) commit(of);
  }
  Task issuer() {
    auto &kready = sh.mask ? kr : kf, &vready = sh.mask ? vr : vf;
    int t = 0, pj = -1, pk = 0;
    for (int j = 0; j < int(items.size()); ++j)
      for (int k = 0; k < items[j].nk; ++k, ++t) {
        const bool first = k == 0, last = k == items[j].nk - 1;
        const int a = t % nk_, c = t % nv_, b = items[j].sp * items[j].nk + k;
        WAIT(kready[a], t / nk_);
        if (first) WAIT(qf, j);
        pipe.push_back([this, t, j, a, b] {
          check(ks[a].is('K', j, b) && (ks[a].zeroed || !sh.mask), "S reads another key tile");
          check(q.is('Q', j, 0), "S reads other queries");
          check(s[t & 1].used, "S overwrites a dS that is still to be used");
          s[t & 1] = Scores{t, 0, false};
        });
        commit(sf[t & 1]);
        if (last) commit(qe);
        if (!first) WAIT(vready[c], t / nv_);
        if (pj >= 0) PLANT(5, dsf, t - 1);
        if (first) {
          if (pj >= 0) {
            if (pk == 0 && pj > 0) PLANT(4, oe, pj - 1);
            dq(t - 1, pj, pk);
          }
          WAIT(vready[c], t / nv_);
          WAIT(dof, j);
        }
        pipe.push_back([this, t, j, c, b] {
          check(vs[c].is('V', j, b) && (vs[c].zeroed || !sh.mask), "dP reads another value tile");
          check(dout.is('O', j, 0), "dP reads another dO");
          check(dp.reads == 8, "dP is overwritten before its last reader");
          dp = {t, 0};
        });
        commit(dpf);
        commit(ve[c]);
        if (last) commit(doe);
        if (!first) {
          if (pk == 0 && pj > 0) PLANT(4, oe, pj - 1);
          dq(t - 1, pj, pk);
        }
        pj = j;
        pk = k;
      }
    if (pj >= 0) {
      WAIT(dsf, t - 1);
      if (pk == 0 && pj > 0) WAIT(oe, pj - 1);
      dq(t - 1, pj, pk);
    }
    commit(drain);
    WAIT(drain, 0);
  }
  Task epilogue(int) {
    int made = 0;
    for (int j = -1; j < int(items.size()); ++j) {
      const int nx = j + 1;  // D of the next tile, then dQ of this one
      if (nx < int(items.size()) && !exact(nx)) {
        WAIT(de[made & 1], (made >> 1) - 1);
        co_await turn();
        ++d_made[nx];
        df[made & 1].arrive();
        ++made;
      }
      if (j < 0) continue;
      PLANT(8, of, j);
      check(acc.item == j && acc.blocks == items[j].nk && acc.drained < 4, "the epilogue reads another dQ");
      co_await turn();
      check(acc.item == j, "dQ changes under the epilogue");
      ++acc.drained;
      oe.arrive();
    }
  }
  Task softmax(int g, int w) {
    int t = 0, made = 0, summed = 0;
    for (int j = 0; j < int(items.size()); ++j) {
      const bool idle = items[j].qt * 128 + w * 32 >= sh.n;
      for (int k = 0; k < items[j].nk; ++k, ++t) {
        PLANT(6, sf[t & 1], t >> 1);
        check(s[t & 1].t == t, "the softmax reads other scores");
        if (sh.mask == 2) {
          WAIT(wf[t % 8], t / 8);
          check(words[t % 8] == std::make_pair(j, items[j].sp * items[j].nk + k), "the softmax reads another mask");
          --word_reads[t % 8];
        }
        co_await turn();
        if (k == 0 && !exact(j)) {
          PLANT(7, df[made & 1], made >> 1);
          check(d_made[j] == 4, "D is not made yet");
          co_await turn();
          de[made & 1].arrive();
          ++made;
        }
        WAIT(dpf, t);
        check(dp.t == t, "dS reads another dP");
        if (exact(j) && !idle) {
          halves[summed & 1][g][w] = j;
          co_await turn();
          xd[w].arrive();
          WAIT(xd[w], summed);
          check(halves[summed & 1][g ^ 1][w] == j, "the other half's sum is another tile's");
          ++summed;
        }
        co_await turn();
        check(dp.t == t, "dP changes under the softmax");
        ++dp.reads;
        ++s[t & 1].warps;
        dsf.arrive();
        co_await turn();
      }
    }
  }
  void go() {
    add(loader(false));
    add(loader(true));
    add(issuer());
    if (sh.mask) add(masks());
    for (int w = 0; w < 4; ++w) {
      add(epilogue(w));
      for (int g = 0; g < 2; ++g) add(softmax(g, w));
    }
    run();
    check(acc.drained == 4 && s[0].used && s[1].used, "something is left over");
  }
};

// ==================================================================== dK, dV
struct BackwardDkdv : Cta {
  static constexpr int kPlants = 20;
  const Shape& sh;
  const int nq, ndo, group, qtiles, kblocks, splits;
  struct Unit {
    int t0, t1;
  };
  std::vector<Unit> units;  // those without a tile to add up too
  std::vector<Bar> qf, qe, dof, doe;
  Bar kf, ke, vf, ve, sf, pf, dpf, dsf, accf, acce, vecf[2], vece[2], drain;
  std::vector<Tile> qs, dos;
  Tile key, value;
  struct Scores {  // S^T and P^T, dP^T and dS^T
    int e = -1, warps = 0;
    bool used = true;
  } s, dp;
  struct {
    int unit = -1, tiles = 0, drained = 4;
  } dk, dv;
  struct {
    int e = -1, reads = 8;
  } vec[2];

  BackwardDkdv(Rng& r, const Shape& shape, int d, int cta, int ctas)
      : Cta(r), sh(shape), nq(d == 128 ? 3 : 4), ndo(d == 128 ? 2 : 4), group(shape.heads / shape.kv_heads),
        qtiles((shape.n + 127) / 128), kblocks((shape.m + 127) / 128),
        splits(sq::cross_dkv_splits((long long)shape.B * shape.kv_heads * kblocks, group * qtiles)) {
    const int per = sh.B * sh.kv_heads * kblocks, tiles = group * qtiles, part = (tiles + splits - 1) / splits;
    for (int i = cta; i < per * splits; i += ctas) {
      const int sp = i / per, j = i % per, kb = j % kblocks, b = j / kblocks / sh.kv_heads;
      Unit u{std::min(sp * part, tiles), std::min(sp * part + part, tiles)};
      if ((sh.mask ? sh.len[b] : sh.m) - kb * 128 <= 0) u.t1 = u.t0;
      units.push_back(u);
    }
    qf.resize(nq);
    qe.resize(nq);
    dof.resize(ndo);
    doe.resize(ndo);
    qs.resize(nq);
    dos.resize(ndo);
    pf.init(8);
    dsf.init(8);
    acce.init(4);
    vece[0].init(8);
    vece[1].init(8);
  }
  Task loader(bool grads) {
    int e = 0, n = 0;
    const int size = grads ? ndo : nq;
    auto &full = grads ? dof : qf, &empty = grads ? doe : qe;
    auto& ring = grads ? dos : qs;
    Bar &xf = grads ? vf : kf, &xe = grads ? ve : ke;
    Tile& x = grads ? value : key;
    for (int i = 0; i < int(units.size()); ++i) {
      if (units[i].t0 >= units[i].t1) continue;
      for (int t = units[i].t0; t < units[i].t1; ++t) {
        if (t == units[i].t0) {
          PLANT(3, xe, n - 1);
          ++n;
          xf.expect();
          x = Tile{};
          copies.push_back([&x, &xf, i, grads] {
            x = Tile{i, 0, grads ? 'V' : 'K', true, false};
            xf.landed();
          });
        }
        const int at = e % size;
        PLANT(1, empty[at], e / size - 1);
        full[at].expect();
        ring[at] = Tile{};
        copies.push_back([&ring, at, i, t, grads, &full] {
          ring[at] = Tile{i, t, grads ? 'O' : 'Q', true, false};
          full[at].landed();
        });
        ++e;
      }
    }
    if (n) WAIT(xf, n - 1);
    for (int i = 0; i < size; ++i)
      if (e > i) WAIT(full[i], (e - i + size - 1) / size - 1);
  }
  Task statistics() {
    int e = 0;
    for (auto& u : units)
      for (int t = u.t0; t < u.t1; ++t, ++e) {
        PLANT(7, vece[e & 1], (e >> 1) - 1);
        check(vec[e & 1].reads == 8, "statistics are overwritten before their last reader");
        vec[e & 1] = {e, 0};
        co_await turn();
        vecf[e & 1].arrive();
      }
  }
  Task issuer() {
    struct Step {
      int i = 0, t = 0, unit = 0;  // unit: number among those with tiles
      bool ok = false;
    };
    auto seek = [this](int i, int unit) {
      for (; i < int(units.size()); ++i)
        if (units[i].t0 < units[i].t1) return Step{i, units[i].t0, unit, true};
      return Step{i, 0, unit, false};
    };
    Step cur{}, nxt = seek(0, 0);
    int e = 0;
    while (cur.ok || nxt.ok) {
      const bool first = cur.ok && cur.t == units[cur.i].t0, last = cur.ok && cur.t == units[cur.i].t1 - 1;
      const int n = cur.ok ? e + 1 : 0;
      const bool nfirst = nxt.ok && nxt.t == units[nxt.i].t0, nlast = nxt.ok && nxt.t == units[nxt.i].t1 - 1;
      if (cur.ok) {  // dV(e)
        if (first && cur.unit > 0) PLANT(4, acce, cur.unit - 1);
        PLANT(5, pf, e);
        const int z = e % ndo;
        pipe.push_back([this, cur, e, z, first] {
          check(dos[z].is('O', cur.i, cur.t), "dV reads another dO");
          check(s.e == e && s.warps == 8 && !s.used, "dV reads another P");
          s.used = true;
          if (first) {
            check(dv.drained == 4, "dV is overwritten before the epilogue has read it");
            dv = {cur.i, 0, 0};
          }
          check(dv.unit == cur.i && dv.tiles == cur.t - units[cur.i].t0, "dV adds to another unit's");
          ++dv.tiles;
        });
        commit(doe[z]);
      }
      if (nxt.ok) {  // S(n)
        const int z = n % nq;
        if (nfirst) WAIT(kf, nxt.unit);
        WAIT(qf[z], n / nq);
        pipe.push_back([this, nxt, n, z] {
          check(key.is('K', nxt.i, 0) && qs[z].is('Q', nxt.i, nxt.t), "S reads another tile");
          check(s.used, "S overwrites a P that is still to be used");
          s = Scores{n, 0, false};
        });
        commit(sf);
        if (nlast) commit(ke);
      }
      if (cur.ok) {  // dK(e)
        WAIT(dsf, e);
        const int z = e % nq;
        pipe.push_back([this, cur, e, z, first] {
          check(qs[z].is('Q', cur.i, cur.t), "dK reads other queries");
          check(dp.e == e && dp.warps == 8 && !dp.used, "dK reads another dS");
          dp.used = true;
          if (first) {
            check(dk.drained == 4, "dK is overwritten before the epilogue has read it");
            dk = {cur.i, 0, 0};
          }
          check(dk.unit == cur.i && dk.tiles == cur.t - units[cur.i].t0, "dK adds to another unit's");
          ++dk.tiles;
        });
        commit(qe[z]);
        if (last) commit(accf);
      }
      if (nxt.ok) {  // dP(n)
        const int z = n % ndo;
        if (nfirst) WAIT(vf, nxt.unit);
        WAIT(dof[z], n / ndo);
        pipe.push_back([this, nxt, n, z] {
          check(value.is('V', nxt.i, 0) && dos[z].is('O', nxt.i, nxt.t), "dP reads another tile");
          check(dp.used, "dP overwrites a dS that is still to be used");
          dp = Scores{n, 0, false};
        });
        commit(dpf);
        if (nlast) commit(ve);
      }
      if (cur.ok) ++e;
      cur = nxt;
      if (cur.ok) {
        if (cur.t + 1 < units[cur.i].t1)
          nxt.t = cur.t + 1;
        else
          nxt = seek(cur.i + 1, cur.unit + 1);
      }
    }
    commit(drain);
    WAIT(drain, 0);
  }
  Task epilogue(int) {
    int n = 0;
    for (int i = 0; i < int(units.size()); ++i) {
      const int tiles = units[i].t1 - units[i].t0;
      if (tiles <= 0) continue;
      PLANT(8, accf, n);
      check(dk.unit == i && dv.unit == i && dk.tiles == tiles && dv.tiles == tiles, "the epilogue reads other sums");
      co_await turn();
      check(dk.unit == i && dv.unit == i, "dK, dV change under the epilogue");
      ++dk.drained;
      ++dv.drained;
      acce.arrive();
      ++n;
    }
  }
  Task softmax() {
    int e = 0;
    for (auto& u : units)
      for (int t = u.t0; t < u.t1; ++t, ++e) {
        WAIT(vecf[e & 1], e >> 1);
        check(vec[e & 1].e == e, "the softmax reads other statistics");
        PLANT(6, sf, e);
        check(s.e == e && !s.used, "the softmax reads other scores");
        co_await turn();
        ++s.warps;
        pf.arrive();
        WAIT(dpf, e);
        check(dp.e == e && !dp.used && vec[e & 1].e == e, "dS reads another dP");
        co_await turn();
        ++dp.warps;
        ++vec[e & 1].reads;
        dsf.arrive();
        vece[e & 1].arrive();
        co_await turn();
      }
  }
  void go() {
    add(loader(false));
    add(loader(true));
    add(statistics());
    add(issuer());
    for (int w = 0; w < 4; ++w) add(epilogue(w));
    for (int w = 0; w < 8; ++w) add(softmax());
    run();
    check(dk.drained == 4 && dv.drained == 4 && s.used && dp.used, "something is left over");
  }
};

int main(int argc, char** argv) {
  const int runs = argc > 1 ? std::atoi(argv[1]) : 300;
  Rng rnd{unsigned(argc > 2 ? std::atoi(argv[2]) : 1)};
  g_plant = argc > 3 ? std::atoi(argv[3]) : 0;
  int whole[3] = {}, split[3] = {};
  for (int t = 0; t < runs; ++t) {
    Shape sh;
    sh.mask = t % 3;
    sh.B = 1 + rnd(4);
    const int kind = rnd(3);  // pairs of query tiles, single tiles, keys split over jobs
    sh.kv_heads = kind == 0 ? 12 + rnd(30) : 1 + rnd(4);
    sh.heads = sh.kv_heads * (1 + rnd(3));
    sh.n = kind == 0 ? 300 + rnd(900) : kind == 1 ? 1 + rnd(500) : 1 + rnd(140);
    sh.m = kind == 2 ? 1024 + rnd(6000) : 1 + rnd(900);
    for (int b = 0; b < sh.B; ++b) {
      const int any = rnd(sh.m + 1);
      const int choice[6] = {any, sh.m, any & ~127, 0, 1, any};
      sh.len.push_back(choice[rnd(6)]);
    }
    const int d = rnd(2) ? 128 : 64;
    const sq::CrossPlan p = sq::make_cross_plan(sh.B, sh.heads, sh.kv_heads, sh.n, sh.m);
    (p.splits > 1 ? split : whole)[sh.mask]++;
    auto ctas = [&](int items) { return std::max(1, items / (1 + rnd(7))); };  // one to seven items each
    char name[200];
    std::snprintf(name, sizeof name, "run %d: B %d heads %d (%d) n %d m %d d %d mask %d splits %d", t, sh.B, sh.heads,
                  sh.kv_heads, sh.n, sh.m, d, sh.mask, p.splits);
    {
      g_what = std::string("forward, ") + name;
      const int c = ctas(p.items);
      Forward(rnd, sh, d, rnd(c), c).go();
    }
    {
      g_what = std::string("dq, ") + name;
      const int qtiles = (sh.n + 127) / 128;
      const int c = ctas(sh.B * sh.heads * qtiles * sq::cross_dq_splits((long long)sh.B * sh.heads * qtiles, (sh.m + 127) / 128, true));
      BackwardDq(rnd, sh, d, rnd(c), c).go();
    }
    {
      g_what = std::string("dk, dv, ") + name;
      const int c = ctas(sh.B * sh.kv_heads * ((sh.m + 127) / 128));
      BackwardDkdv(rnd, sh, d, rnd(c), c).go();
    }
  }
  if (runs >= 100)
    for (int i = 0; i < 3; ++i) check(whole[i] > 0 && split[i] > 0, "a mask was not run with whole and split keys");
  std::printf("ok\n");
  return 0;
}
