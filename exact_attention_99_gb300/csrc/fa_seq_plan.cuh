// The division of work of the calls on sequences of different lengths, made
// on the device (the lengths are there) by one block before the main kernel.
//
// Work is counted in tile products. The forward's unit is up to two tiles of
// query rows of a sequence and its n key tiles; the backward's is a key tile
// and its n tiles of query rows; either for every kv head. A tile of query
// rows holds `tok` = 128 / group tokens with all query heads of the group
// (row = token * group + head), so that they share the key tiles.
//
// Two divisions, whichever promises the earlier end:
//   sorted: the units by n, longest first, in rounds of one to each CTA, in
//           each round the longest to the CTA that has least so far;
//   split : all tile products laid end to end (sequence, kv head, unit), an
//           equal share to each CTA. A unit that a boundary falls into is
//           done in parts, and a last kernel joins them in the CTAs' order.
// Sorted order leaves no parts, ends within its shortest units where there
// are many, and lets the CTAs walk the same keys at the same time; few units
// (a chunk of new tokens over long caches) would leave CTAs idle, and are
// split. Every unit costs kItemCost products beside its own: Q's load, the
// first S that nothing overlaps, the epilogue.
#pragma once
#include <atomic>

#include "fa_seq.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace seq {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;    // of the sort by n: a length to each, or more where the longest passes them
constexpr int kMaxWorkers = 256;  // CTAs of a main kernel
constexpr int kItemCost = 2;

// An item is a unit, or a part of one, for one kv head.
struct __align__(16) FwdItem {
  int q0;     // first packed token
  int count;  // tokens (at most 2 * tok, in the low 16 bits) and the flags below
  int kvh;
  int kbase;  // packed: the sequence's first key row; paged: the sequence
  int klen;
  int pos;    // place of the first token among the keys (klen - qlen + its place in the sequence)
  int kt, nt; // key tiles [kt, kt + nt)
  __device__ __forceinline__ int ntok() const { return count & 0xffff; }
};
static_assert(sizeof(FwdItem) == 32, "two 16-byte loads");

struct __align__(16) BwdItem {
  int krow;   // first packed key row of the tile
  int count;  // its keys (at most 128, in the low 16 bits) and the flags below
  int kvh;
  int q0, qlen;  // the sequence's queries
  int rel;       // place of its first token among the tile's keys: klen - qlen - 128 * (tile)
  int tiles;     // first row tile of the sequence in the padded arrays
  int i0, n;     // row tiles [i0, i0 + n) of the sequence
  int pad[3];
  __device__ __forceinline__ int nkey() const { return count & 0xffff; }
};
static_assert(sizeof(BwdItem) == 48, "three 16-byte loads");

// Forward, at most `tok` tokens (one tile of rows): the two stages of the
// pipeline take alternate key tiles of the same rows; else each has rows of its own.
constexpr int kKeyMode = 1 << 16;
// The item is part of a unit: its results go to a slot, to be joined with the
// other parts'. kCont: not the unit's first part.
constexpr int kPart = 1 << 17;
constexpr int kCont = 1 << 18;

// A unit divided between the workers c0 .. c1: parts in slot 2 * c0 + 1 and,
// for the others that have a share, slot 2 * c. Kept at index c0 + 1.
struct Cut {
  int row0, count, kvh, c0, c1;  // c1 < 0: nothing
  int pad[3];
};

struct PlanHead {
  int n_items;
  int step;     // worker c takes items first[c], first[c] + step, ... up to last[c]
  int bad;      // the lengths say something that the tensors cannot hold
  int pad;
};

template <class Item>
struct Plan {
  PlanHead* head;
  int* first;       // [G]
  int* last;        // [G]
  Cut* cuts;        // [G]
  int* ustart;      // [B + 1] first unit of each sequence
  int* tstart;      // [B + 1] first row tile of each sequence
  long long* cost;  // [units + 1] cost of the units before
  int* order;       // [units] longest first
  Item* items;      // [units * Hkv + G]
  int max_units;
};

// A kernel's dynamic shared memory limit, set on each context's first launch
// (one object per kernel; `done` holds the context of each device's last).
struct SmemLimit {
  std::atomic<unsigned long long> done[64] = {};
  template <class Kernel>
  cudaError_t set(Kernel kernel, int bytes) {
    int dev = -1;
    const cudaError_t g = cudaGetDevice(&dev);
    if (g != cudaSuccess) return g;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const unsigned long long ctx = context_id();
    if (ctx != 0 && done[dev].load(std::memory_order_relaxed) == ctx) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev].store(ctx, std::memory_order_relaxed);
    return e;
  }
};

// Takes pieces of a workspace, 256-byte aligned (base null: sizes alone).
struct Carver {
  uint8_t* base;
  size_t at;
  template <class T>
  T* take(size_t n) {
    uint8_t* r = base == nullptr ? nullptr : base + at;
    at += (n * sizeof(T) + 255) & ~size_t(255);
    return reinterpret_cast<T*>(r);
  }
};
template <class Item>
Plan<Item> carve_plan(Carver& c, int B, long long units, int Hkv, int G) {
  Plan<Item> p{};
  p.max_units = int(units);
  p.head = c.take<PlanHead>(1);
  p.first = c.take<int>(G);
  p.last = c.take<int>(G);
  p.cuts = c.take<Cut>(G);
  p.ustart = c.take<int>(size_t(B) + 1);
  p.tstart = c.take<int>(size_t(B) + 1);
  p.cost = c.take<long long>(size_t(units) + 1);
  p.order = c.take<int>(size_t(units));
  p.items = c.take<Item>(size_t(units) * Hkv + G);
  return p;
}

#ifdef __CUDACC__

struct Range {
  int first, n;
};

struct FwdSide {
  using Item = FwdItem;
  // One causal sequence of 16384 tokens (32 query heads, 8 kv heads) took 6 %
  // longer split, packed prompts of 16 to 4096 tokens 44 % (at 2 % less in the count).
  static constexpr int kSplitGain = 9;
  // Of divided units: the parts' stores and the last kernel, in tile products.
  // (40 tokens of 8 heads, 2 kv heads over 600 keys, 5 products: 20.6 us
  // divided, 16.6 whole; over 800, 7 products: 21.6 divided, 19.8 whole.)
  static constexpr int kPartsCost = 9;
  static constexpr int kRanked = 2;  // many units of few tiles: back and forth is even enough
  int tok, wl, wr, paged;
  __device__ __forceinline__ int units(const Seq& s) const { return (s.qlen + 2 * tok - 1) / (2 * tok); }
  __device__ __forceinline__ int row_tiles(const Seq&) const { return 0; }
  // key tiles seen by unit j's tokens
  __device__ __forceinline__ Range range(const Seq& s, int j) const {
    const int t0 = j * 2 * tok, ntok = min(2 * tok, s.qlen - t0), pos = s.klen - s.qlen + t0;
    const int lo = wl >= 0 ? max(0, pos - wl) : 0;
    const int hi = wr >= 0 ? min(s.klen - 1, pos + ntok - 1 + wr) : s.klen - 1;
    if (hi < lo) return Range{0, 0};
    return Range{lo >> 7, (hi >> 7) - (lo >> 7) + 1};
  }
  __device__ __forceinline__ Item item(const Seq& s, int b, int j, int kvh, int) const {
    Item it;
    const int t0 = j * 2 * tok, ntok = min(2 * tok, s.qlen - t0);
    it.q0 = s.q0 + t0;
    it.count = ntok | (ntok <= tok ? kKeyMode : 0);
    it.kvh = kvh;
    it.kbase = paged ? b : s.k0;
    it.klen = s.klen;
    it.pos = s.klen - s.qlen + t0;
    return it;
  }
  __device__ __forceinline__ static void set_range(Item& it, int first, int n) {
    it.kt = first;
    it.nt = n;
  }
  __device__ __forceinline__ static int row0(const Item& it) { return it.q0; }
};

struct BwdSide {
  using Item = BwdItem;
  // Split, the CTAs of a sequence add into dQ rows far apart: one causal
  // sequence of 16384 tokens took 5.8 instead of 3.9 ms.
  static constexpr int kSplitGain = 12;
  static constexpr int kPartsCost = 6;  // (at 9 a training step on 2115 tokens took 54 instead of 48 us)
  // Units of many tiles: the documents of a packed training step are 6 % from
  // even back and forth, 1 % ranked (step 1.68 -> 1.53 ms).
  static constexpr int kRanked = 12;
  int tok, wl, wr;
  __device__ __forceinline__ int units(const Seq& s) const { return (s.klen + 127) >> 7; }
  __device__ __forceinline__ int row_tiles(const Seq& s) const { return (s.qlen + tok - 1) / tok; }
  // row tiles with a token that sees a key of tile j
  __device__ __forceinline__ Range range(const Seq& s, int j) const {
    const int off = s.klen - s.qlen, k0 = j * 128, k1 = min(k0 + 127, s.klen - 1);
    const int lo = wr >= 0 ? max(0, k0 - off - wr) : 0;
    const int hi = wl >= 0 ? min(s.qlen - 1, k1 - off + wl) : s.qlen - 1;
    if (hi < lo) return Range{0, 0};
    return Range{lo / tok, hi / tok - lo / tok + 1};
  }
  __device__ __forceinline__ Item item(const Seq& s, int, int j, int kvh, int tiles) const {
    Item it;
    it.krow = s.k0 + j * 128;
    it.count = min(128, s.klen - j * 128);
    it.kvh = kvh;
    it.q0 = s.q0;
    it.qlen = s.qlen;
    it.rel = s.klen - s.qlen - j * 128;
    it.tiles = tiles;
    return it;
  }
  __device__ __forceinline__ static void set_range(Item& it, int first, int n) {
    it.i0 = first;
    it.n = n;
  }
  __device__ __forceinline__ static int row0(const Item& it) { return it.krow; }
};

template <class Side>
struct PlanArgs {
  Lens L;
  Plan<typename Side::Item> P;
  Side side;
  int Hkv, G;
  unsigned* status;
};

// inclusive scan over the block (kPlanThreads threads); total in `sum`
static __device__ __noinline__ long long block_scan(long long v, long long* warp_sums, long long& sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    long long x = warp_sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += o;
    }
    warp_sums[lane] = x;
  }
  __syncthreads();
  sum = warp_sums[31];
  return v + (w > 0 ? warp_sums[w - 1] : 0);
}

// the last b in [0, B) with start[b] * scale <= x
__device__ __forceinline__ int find_seq(const int* start, int B, int scale, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] * scale <= x) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// What the planning block keeps at hand; larger batches than that are read
// from device memory.
constexpr int kNearSeqs = 512, kNearUnits = 1024;

template <class Side>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs<Side> a) {
  using Item = typename Side::Item;
  __shared__ long long sums[32];
  __shared__ int hist[kBuckets];
  __shared__ long long share[kMaxWorkers + 1];
  __shared__ Seq near_seq[kNearSeqs];
  __shared__ int near_ustart[kNearSeqs + 1];
  __shared__ long long near_cost[kNearUnits + 1];
  __shared__ int near_order[kNearUnits];
  __shared__ __align__(16) unsigned load[kMaxWorkers];
  __shared__ int rank[kMaxWorkers], taken[Side::kRanked * kMaxWorkers];
  __shared__ unsigned long long worst;
  __shared__ int bad, longest;
  // (no loop is unrolled: the kernel runs once per call, and fetching its code
  // takes longer than most of what it does)
  const int tid = threadIdx.x;
  const int B = a.L.B, G = a.G, Hkv = a.Hkv;
  const Plan<Item>& P = a.P;
  const bool near_b = B <= kNearSeqs;
  int* const ustart = near_b ? near_ustart : P.ustart;
  auto seq_of = [&](int b) {
    Seq s;
    if (near_b) {
      s = near_seq[b];
    } else {
      seq_at(a.L, b, s);
    }
    return s;
  };
  if (tid == 0) {
    bad = 0;
    longest = 0;
    worst = 0;
  }
#pragma unroll 1
  for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
#pragma unroll 1
  for (int c = tid; c < G; c += kPlanThreads) {
    P.first[c] = 0x7fffffff;
    P.last[c] = -1;
    P.cuts[c].c1 = -1;
  }
#pragma unroll 1
  for (int c = tid; c < kMaxWorkers; c += kPlanThreads) rank[c] = 0;
  grid_dep_launch();  // the next kernel may start its set-up meanwhile
  __syncthreads();
  // units (low half) and row tiles (high half) of the sequences before each
  long long n_units = 0, sum;
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long n = 0;
    if (b < B) {
      Seq s;
      if (seq_at(a.L, b, s)) {
        n = a.side.units(s) | (static_cast<long long>(a.side.row_tiles(s)) << 32);
      } else {
        bad = 1;
      }
      if (near_b) near_seq[b] = s;
    }
    const long long end = block_scan(n, sums, sum) + n_units;
    if (b < B) {
      ustart[b] = int((end - n) & 0x7fffffff);
      P.tstart[b] = int((end - n) >> 32);
    }
    n_units += sum;
  }
  __syncthreads();
  // lengths that the tensors cannot hold (overlapping sequences among them,
  // by their sum): nothing is computed
  if (bad || (n_units & 0xffffffffll) > P.max_units) {
    if (tid == 0) {
      *P.head = PlanHead{0, 1, 1, 0};
      atomicOr(a.status, kDevBadArg);
    }
    return;
  }
  const int U = int(n_units & 0xffffffffll);
  if (tid == 0) {
    ustart[B] = U;
    P.tstart[B] = int(n_units >> 32);
  }
  long long* const cost = U <= kNearUnits ? near_cost : P.cost;
  int* const order = U <= kNearUnits ? near_order : P.order;
  __syncthreads();
  // n of each unit: running sum, histogram and largest
  long long T = 0;
  int most = 0;
#pragma unroll 1
  for (int u0 = 0; u0 < U; u0 += kPlanThreads) {
    const int u = u0 + tid;
    int n = 0;
    if (u < U) {
      const int b = find_seq(ustart, B, 1, u);
      n = a.side.range(seq_of(b), u - ustart[b]).n;
      most = max(most, n);
      atomicAdd(&hist[kBuckets - 1 - min(n, kBuckets - 1)], 1);
    }
    n = u < U ? n + kItemCost : 0;
    const long long end = block_scan(n, sums, sum) + T;
    if (u < U) cost[u] = end - n;
    T += sum;
  }
  if (tid == 0) cost[U] = T;
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(&longest, most);
  const long long Ttot = T * Hkv;
#pragma unroll 1
  for (int c = tid; c <= G; c += kPlanThreads) share[c] = Ttot * c / G;
  __syncthreads();
  const int width = longest / kBuckets + 1;  // lengths to a bucket
  auto bucket = [&](int u) { return kBuckets - 1 - (int(cost[u + 1] - cost[u]) - kItemCost) / width; };
  if (width > 1) {
#pragma unroll 1
    for (int i = tid; i < kBuckets; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int u = tid; u < U; u += kPlanThreads) atomicAdd(&hist[bucket(u)], 1);
    __syncthreads();
  }
  long long base = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < kBuckets; i0 += kPlanThreads) {
    const int n = hist[i0 + tid];
    const long long end = block_scan(n, sums, sum) + base;
    hist[i0 + tid] = int(end - n);
    base += sum;
  }
  __syncthreads();
  // Sorted order. Units of one length may stand in any order: the workers'
  // loads are the same. Where a bucket holds several lengths they would not be,
  // and neither the choice between the divisions that they lead to (which round
  // differently), so that units then stand in their own order, a warp of them
  // after the other (some 2 us for a thousand).
  if (width == 1) {
#pragma unroll 1
    for (int u = tid; u < U; u += kPlanThreads) order[atomicAdd(&hist[bucket(u)], 1)] = u;
  } else {
    const int lane = tid & 31;
#pragma unroll 1
    for (int u0 = 0; u0 < U; u0 += kPlanThreads) {
      const int u = u0 + tid, key = u < U ? bucket(u) : -1;
#pragma unroll 1
      for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (tid >> 5 == w) {
          const unsigned same = __match_any_sync(0xffffffffu, key);
          const int first = __ffs(same) - 1;
          int at = lane == first && key >= 0 ? atomicAdd(&hist[key], __popc(same)) : 0;
          at = __shfl_sync(0xffffffffu, at, first);
          if (key >= 0) order[at + __popc(same & ((1u << lane) - 1))] = u;
        }
        __syncthreads();
      }
    }
  }
  __syncthreads();
  const int n_items = U * Hkv;
  auto cost_of = [&](int i) {
    const int u = order[i / Hkv];
    return int(cost[u + 1] - cost[u]);
  };
  // Rounds of G items, worker c's at place r * G + c. The last Side::kRanked rounds
  // rank the workers by their load; rounds before them, which leave enough to
  // even out, go back and forth over the workers.
  const int rounds = (n_items + G - 1) / G, early = max(0, rounds - Side::kRanked);
  int mine = tid < G && early > 0 ? tid + (early - 1) * G : -1;  // worker tid's last place
  int own = 0;  // worker tid's load
  auto publish = [&]() {  // as a key that orders equal loads by worker
    load[tid] = tid < G ? (unsigned(min(own, 0x7ffffe)) << 8) | unsigned(tid) : 0xffffffffu;
  };
  if (tid < kMaxWorkers) {
    if (tid < G)
#pragma unroll 1
      for (int r = 0; r < early; ++r) own += cost_of(r * G + ((r & 1) ? G - 1 - tid : tid));
    publish();
  }
  __syncthreads();
  // thread (c, part): how many of the part's workers come before worker c
  const int wide = (G + 31) & ~31, parts = kPlanThreads / wide, per_part = ((G + parts - 1) / parts + 3) & ~3;
  const int c = tid % wide, c0 = tid / wide * per_part, c1 = min(c0 + per_part, kMaxWorkers);
#pragma unroll 1
  for (int r = early; r < rounds; ++r) {
    if (c < G && c0 < G) {
      const unsigned key = load[c];
      int before = 0;
#pragma unroll 1
      for (int x = c0; x < c1; x += 4) {
        const uint4 y = *reinterpret_cast<const uint4*>(&load[x]);
        before += (y.x < key) + (y.y < key) + (y.z < key) + (y.w < key);
      }
      if (before > 0) atomicAdd(&rank[c], before);
    }
    __syncthreads();
    if (tid < G) {
      const int i = r * G + rank[tid];
      rank[tid] = 0;
      taken[(r - early) * kMaxWorkers + tid] = i;
      if (i < n_items) {
        mine = r * G + tid;
        own += cost_of(i);
        publish();
      }
    }
    __syncthreads();
  }
  // The busiest worker against an equal division, which has to win by more
  // than Side::kPartsCost and what CTAs at different places cost (Side::kSplitGain, in
  // eighths).
  if (tid < G) atomicMax(&worst, static_cast<unsigned long long>(own));
  __syncthreads();
  const bool split = static_cast<long long>(worst) > Ttot / G * Side::kSplitGain / 8 + Side::kPartsCost;
  if (tid == 0) *P.head = PlanHead{n_items, split ? 1 : G, 0, 0};
  if (!split) {
    if (tid < G) {
      P.first[tid] = tid;
      P.last[tid] = mine;
    }
#pragma unroll 1
    for (int at = tid; at < rounds * G; at += kPlanThreads) {
      const int r = at / G, c = at - r * G;
      const int i = r < early ? r * G + ((r & 1) ? G - 1 - c : c) : taken[(r - early) * kMaxWorkers + c];
      if (i >= n_items) continue;
      const int u = order[i / Hkv], b = find_seq(ustart, B, 1, u);
      const Seq s = seq_of(b);
      const Range x = a.side.range(s, u - ustart[b]);
      Item it = a.side.item(s, b, u - ustart[b], i % Hkv, P.tstart[b]);
      Side::set_range(it, x.first, x.n);
      P.items[at] = it;
    }
    return;
  }
  const float per_worker = float(G) / float(Ttot);
#pragma unroll 1
  for (int i = tid; i < n_items; i += kPlanThreads) {
    // order (sequence, kv head, unit): the place [x0, x1) of item i's products
    // among all costs; worker c has those in [share(c), share(c + 1))
    const int b = find_seq(ustart, B, Hkv, i);
    const Seq s = seq_of(b);
    const int us = ustart[b], per = ustart[b + 1] - us;
    const int j = i - us * Hkv, kvh = j / per, ju = j - kvh * per;
    const Range r = a.side.range(s, ju);
    const long long of_seq = cost[us + per] - cost[us];
    // (its own cost comes first, and is nobody's)
    const long long x0 = cost[us] * Hkv + kvh * of_seq + (cost[us + ju] - cost[us]) + kItemCost, x1 = x0 + r.n;
    Item it = a.side.item(s, b, ju, kvh, P.tstart[b]);
    const int count = it.count;
    // the worker that has product x0 (fewer products than workers: the last
    // of those whose share begins there), from a guess
    int c = max(0, min(int(float(x0) * per_worker), G - 1));
    while (c > 0 && share[c] > x0) --c;
    while (c + 1 < G && share[c + 1] <= x0) ++c;
    const int c0 = c;
    long long x = x0;
    do {
      const long long e = c + 1 < G ? min(x1, share[c + 1]) : x1;
      const bool part = x > x0 || e < x1;
      it.count = count | (part ? kPart : 0) | (x > x0 ? kCont : 0);
      Side::set_range(it, r.first + int(x - x0), int(e - x));
      // one entry per (item, worker), in order: no two have the same sum, and
      // a worker's entries follow one another
      const int at = i + c;
      P.items[at] = it;
      atomicMin(&P.first[c], at);
      atomicMax(&P.last[c], at);
      x = e;
      if (x < x1)
        do ++c;
        while (c + 1 < G && share[c + 1] <= x);
    } while (x < x1);
    if (c > c0) {
      Cut& k = P.cuts[c0 + 1];
      k.row0 = Side::row0(it);
      k.count = count & 0xffff;
      k.kvh = kvh;
      k.c0 = c0;
      k.c1 = c;
    }
  }
}

// Bounded wait of a whole converged warp on an mbarrier phase: true in every
// lane, or false in every lane when the CTA's abort word is set or limit_ns
// passed (the abort word is then set here). All lanes take the same way, so
// the caller may go on with warp-wide instructions either way. Short, since the
// roles of a kernel, with some fifty waits, share the instruction cache.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint64_t limit_ns) {
  const uint32_t addr = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t n = 1; !__all_sync(0xffffffffu, mbar_try_wait(addr, parity)); ++n) {
    if ((n & 31) != 0) continue;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    const bool late = t - t0 > limit_ns;
    if (late) *abort_flag = 1u;
    if (__any_sync(0xffffffffu, late || *abort_flag != 0)) return false;
  }
  return true;
}

// A worker's walk over its items: i, i + step, ... up to last.
struct Walk {
  int i, step, last;
};
__device__ __forceinline__ Walk walk_begin(const PlanHead* head, const int* first, const int* last) {
  return Walk{first[blockIdx.x], head->step, last[blockIdx.x]};
}
__device__ __forceinline__ void walk_step(Walk& w) { w.i += w.step; }

#endif  // __CUDACC__

}  // namespace seq
}  // namespace fa
