// fa_fwd_paged_fp8: attention of new tokens over a paged cache held in e4m3
// with a scale for each block of 16 keys and head.
//
// The rows of a kv head are (token, query head of the group) pairs, as in
// fa_seq_fwd.cu. With codes k^ and v^ and block scales a and b, the exponent of
// row i, key j is
//   x = scale log2(e) a_j (q_i . k^_j) + log2(b_j),   P' = 2^(x - m),
//   O = sum_j P'_ij v^_j / l, l = sum_j P'_ij / b_j,  LSE = (m + log2 l) ln 2,
// m the running maximum of x: b goes through the exponent, so that P' v^ needs
// no further product and P' is largest where it weighs most. Every e4m3 value
// is an f16 value, so both products are f16 x f16 with 32-bit accumulators.
// Roundings: q to f16 after a division by a power of two of its row (exact
// unless a value is below 2^-28 of the row's largest), P' to f16 (off by at most
// 2^-11 of itself for all P' above 2^-21 of the largest, by 2^-32 of that below), O to bf16.
//
// Few rows to a kv head (single tokens): bound by the cache's bytes. A producer warp
// loads tiles of 128 keys by TMA, and each of 8 warps takes 16 of a tile's keys: their
// codes are turned to f16 in registers and are the A operand of mma.sync.m16n8k16,
// the rows the B operand of 8 columns: S^T = K Q^T, then O^T = V^T P^T. Shared memory
// carries each byte in once and out once, and no warp waits for another before the end
// of a unit. (The tensor-memory pipeline of fa_seq_fwd.cu takes V's codes through
// shared memory as f16 as well and has a softmax of 128 rows for each tile: at half the
// bytes a key it would set the pace.)
//
// Work: a unit is up to 8 NT rows of a sequence and kv head with the tiles of
// 128 keys that they see. All tiles of all units are laid end to end and divided
// evenly between the CTAs, whose producers find their own shares; a unit's warps join
// their results in shared memory, and the parts of a unit that several CTAs share are
// joined by a last kernel, in a fixed order.
//
// Measured (the same calls over a bf16 cache in brackets):
//   64 single tokens over 300 to 32000 keys, 8 kv heads of 128: 0.89 GB in 146 to 160 us
//     (by the GPU), 5.6 to 6.1 TB/s (268 us); two tokens over 116000 and 131000 keys: 90
//     to 98 us (153). A further key costs its bytes at 6.7 TB/s; the rest, 13 to 15 us, is
//     the launch, the CTA's plan (1.6 us), the first lookups (1.5 us), the first tile and
//     the joins.
//   one token over 1000 keys: 11.8 us (13.3), that chain alone. 16 tokens over 8192 keys,
//     0.27 GB: 53 us, of which the bytes are 40.
//   Tried, the 64 tokens (159 us when the first three of these were measured): loads by
//     cp.async, 16 warps a CTA 213 us, four CTAs of 4 warps 194; TMA with 256-byte
//     promotion in L2 201 (a third more is read from memory than is asked for); an L2
//     prefetch of the tile after next 176.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_seq_plan.cuh"
#include "sm103_fp8.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace seq8 {

using seq::Lens;
using seq::Seq;

constexpr int kWarps = 8, kThreads = (kWarps + 1) * 32;  // warp 8: the producer
constexpr int kItems = 4;      // ring of units: the producer is up to three tiles ahead, and each unit has one at least
constexpr int kItemCost = 1;  // of a unit beside its tiles, in tiles (64 single tokens: 158 us; of 2, 4, 6: 159, 162, 166)
// P' is at most 2^15 (f16 holds 65504), and 2^7 where the running maximum is up to date
constexpr float kTop = 15.0f, kShift = 7.0f;
constexpr float kLow = -FLT_MAX;  // a running maximum before any key

// A unit divided between the workers c0 .. c1 (c1 < 0: nothing). The first
// part is in slot 2 c0 + 1, the others in slot 2 c.
struct Cut8 {
  int seq0;      // first packed token of the sequence
  int row0, rows;  // rows of the sequence
  int kvh, c0, c1;
  int pad[2];
};

struct Params8 {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const uint8_t* v_codes;
  const float* scales[2];
  const int* table;
  Lens L;
  int Hq, Hkv, group, total_q;
  long long q_stride;
  int num_pages, page_size, max_pages;
  float scale_log2;
  int wl, wr;
  float* part_o;     // [2 G][8 NT][D]
  float2* part_ml;   // [2 G][8 NT]
  Cut8* cuts;        // [G]
  int* has;          // [G] worker has a share
  int box_rows;      // keys of a TMA box: they lie in one page
  unsigned long long wait_limit_ns;
  int inject;
  unsigned* status;
};

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  // CTAs of an SM: one's units begin and end while the other's keys come in
  // (of 16 rows of 64 too: 64 tokens over 2000 to 8000 keys 139 -> 101 us; of 128 they
  // have no registers for that)
  static constexpr int kPerSm = NT == 1 || D == 64 ? 2 : 1;
  static constexpr int kHalf = 128 * D;            // bytes of a tile's K, or V
  static constexpr int kStages = D == 64 || NT == 2 ? 4 : 2;
  static constexpr int kRing = kStages * 2 * kHalf;
  static constexpr int kJoinLd = D + 4;            // (spreads the rows over the banks)
  static constexpr int kJoin = kWarps * kRows * kJoinLd * 4;
  static constexpr int kSmem = kRing + kJoin + 1024;
};

// A unit, or this CTA's part of it.
struct Item8 {
  int b, q0, qlen, klen;  // the sequence
  int row0, rows;       // the unit's rows of it (token * group + head of the group)
  int head;             // kv head; -1: there are no more items
  int k0, k1;           // keys [k0, k1)
  int slot;             // of a part's results; -1: it is the whole unit
};

template <int D, int NT>
struct Ctl8 {
  Item8 it[kItems];
  uint64_t it_full[kItems], it_empty[kItems];
  uint64_t full[Shape<D, NT>::kStages], empty[Shape<D, NT>::kStages];
  uint64_t join_full, join_empty;
  float sc[Shape<D, NT>::kStages][2][8];  // scales of a tile's blocks of K, V
  float2 ml[kWarps][8 * NT];
  uint32_t nans[kWarps];  // not 0: NaN codes of V were taken as zeros
  long long sums[kWarps + 1];
  struct {
    int b;
    long long before, of_seq;  // costs of the sequences before it, its own for one head
    int bad;
  } start;
  uint32_t abort;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A unit's keys: those that any of its rows sees.
struct Unit {
  int lo, hi;      // [lo, hi)
  int kt, nt;      // tiles of 128 keys
};
__device__ __forceinline__ Unit unit_at(const Params8& p, const Seq& s, int row0, int rows) {
  const int off = s.klen - s.qlen, pos0 = off + row0 / p.group, pos1 = off + (row0 + rows - 1) / p.group;
  Unit u;
  u.lo = p.wl >= 0 ? max(0, pos0 - p.wl) : 0;
  u.hi = p.wr >= 0 ? min(s.klen, pos1 + p.wr + 1) : s.klen;
  if (u.hi <= u.lo) {
    u.lo = u.hi = u.kt = u.nt = 0;
  } else {
    u.kt = u.lo >> 7;
    u.nt = ((u.hi - 1) >> 7) - u.kt + 1;
  }
  return u;
}

// Four columns of V's rows (their place in the first row: codes): a byte of the result is not
// 0 where one of the keys [lo, hi) of sequence b is a NaN code. Not looked at are the blocks
// of 16 keys that lie in [all_lo, all_hi).
__device__ __noinline__ uint32_t hidden_nans(const Params8& p, int b, int lo, int hi, const uint8_t* codes, int d,
                                             int all_lo, int all_hi) {
  const int* const row = p.table + size_t(b) * p.max_pages;
  uint32_t nans = 0;
#pragma unroll 1
  for (int k = lo; k < hi; ++k) {
    const int block = k & ~15;
    if (block >= all_lo && block + 16 <= all_hi) {  // on to the first that does not
      k = (all_hi & ~15) - 1;
      continue;
    }
    const int page = row[k / p.page_size];
    if (page < 0 || page >= p.num_pages) continue;
    const long long token = 1LL * page * p.page_size + k % p.page_size;
    nans |= nan_codes(*reinterpret_cast<const uint32_t*>(codes + token * p.Hkv * d));
  }
  return nans;
}

// A walk over the units in the order (sequence, kv head, rows), with the place
// x of each unit's tiles among all costs.
template <int ROWS>
struct Walk8 {
  int b, kvh, j;   // the unit that follows
  int n;           // units of the sequence and head; 0: the sequence is to be found yet, at b or after
  Seq s;
  long long x;
  // the unit found by next(): what of it is this worker's
  int row0, rows, head, b_of;
  Seq seq;
  int k0, k1;      // keys [k0, k1)
  long long y0, y1;
  bool first, last;  // the unit's first, last part

  // The next sequence with rows, by the whole warp: its lanes look at 32 at a time
  // (a captured call's unused places are empty sequences).
  __device__ __forceinline__ void load(const Params8& p) {
    for (; b < p.L.B; b += 32) {
      Seq t{};
      const int at = b + int(threadIdx.x & 31);
      const bool rows_there = at < p.L.B && seq::seq_at(p.L, at, t) && t.qlen > 0;
      const unsigned found = __ballot_sync(0xffffffffu, rows_there);
      if (found == 0) continue;
      const int of = __ffs(found) - 1;
      b += of;
      s.q0 = __shfl_sync(0xffffffffu, t.q0, of);
      s.qlen = __shfl_sync(0xffffffffu, t.qlen, of);
      s.klen = __shfl_sync(0xffffffffu, t.klen, of);
      n = (s.qlen * p.group + ROWS - 1) / ROWS;
      return;
    }
  }
  // the worker's next part of a unit, if any: lo, hi its share; end: it has what lies at the end too
  __device__ __forceinline__ bool next(const Params8& p, long long lo, long long hi, bool end) {
    for (;;) {
      if (n == 0) {
        if (x + kItemCost >= hi && !end) return false;  // (what follows is others': not looked for)
        load(p);
      }
      if (b >= p.L.B) return false;
      seq = s;
      head = kvh;
      b_of = b;
      row0 = j * ROWS;
      rows = min(ROWS, s.qlen * p.group - row0);
      const Unit u = unit_at(p, s, row0, rows);
      y0 = x + kItemCost;
      y1 = y0 + u.nt;
      if (y0 >= hi && !(end && u.nt == 0)) return false;
      x = y1;
      if (++j == n) {
        j = 0;
        if (++kvh == p.Hkv) {
          kvh = 0;
          ++b;
          n = 0;
        }
      }
      if (u.nt == 0) {
        if (y0 < lo) continue;
        k0 = k1 = 0;
        first = last = true;
        return true;
      }
      if (y1 <= lo) continue;
      first = y0 >= lo;
      last = y1 <= hi;
      k0 = first ? u.lo : (u.kt + int(lo - y0)) << 7;
      k1 = last ? u.hi : (u.kt + int(hi - y0)) << 7;
      return true;
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kPerSm)
    attend8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params8 p) {
  using C = Shape<D, NT>;
  constexpr int R = C::kRows, S = C::kStages;
  constexpr int KS = D / 16;  // products' steps over d, tiles of 16 d of O^T
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl8<D, NT> ctl;
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* const join = reinterpret_cast<float*>(ring + C::kRing);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int G = gridDim.x, me = blockIdx.x;
  const uint64_t LIM = p.wait_limit_ns;
  grid_dep_launch();
  if (tid == 0) {
    ctl.abort = 0;
    ctl.start.b = p.L.B;
    ctl.start.bad = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ctl.it_full[i], 1);
      mbar_init(&ctl.it_empty[i], kWarps);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(&ctl.full[i], 2);  // the codes and the scales
      mbar_init(&ctl.empty[i], kWarps);
    }
    mbar_init(&ctl.join_full, kWarps);
    mbar_init(&ctl.join_empty, kWarps);
    fence_mbar_init();
  }
  __syncthreads();

  // ---- this worker's share: every thread takes some sequences, in order
  const int per = (p.L.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.L.B), b1 = min(b0 + per, p.L.B);
  auto cost_of = [&](int b, bool& ok) {  // of a sequence, for one kv head
    Seq s;
    long long t = 0;
    ok = seq::seq_at(p.L, b, s) && ok;
    if (ok)
      for (int r = 0; r < s.qlen * p.group; r += R) t += unit_at(p, s, r, min(R, s.qlen * p.group - r)).nt + kItemCost;
    return t;
  };
  bool fine = true;
  long long mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += cost_of(b, fine);
  if (!fine) ctl.start.bad = 1;
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += o;
  }
  if (lane == 31) ctl.sums[warp] = upto;
  __syncthreads();
  long long T = 0;
#pragma unroll
  for (int w = 0; w <= kWarps; ++w) {
    if (w < warp) upto += ctl.sums[w];
    T += ctl.sums[w];
  }
  if (ctl.start.bad) {  // lengths that the tensors cannot hold: nothing is computed
    if (tid == 0) {
      p.cuts[me].c1 = -1;
      p.has[me] = 0;
      if (me == 0) atomicOr(p.status, kDevBadArg);
    }
    return;
  }
  const long long all = T * p.Hkv, lo = all * me / G, hi = all * (me + 1) / G;
  // (a unit without keys lies at the end of its cost: lo - 1 is in it, or before it)
  const long long target = lo > 0 ? lo - 1 : 0;
  {
    long long before = (upto - mine) * p.Hkv;
    if (before <= target && target < upto * p.Hkv) {
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const long long t = per == 1 ? mine : cost_of(b, fine);
        if (target < before + t * p.Hkv) {
          ctl.start.b = b;
          ctl.start.before = before;
          ctl.start.of_seq = t;
          break;
        }
        before += t * p.Hkv;
      }
    }
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    Walk8<R> walk;
    walk.b = ctl.start.b;
    walk.kvh = 0;
    walk.j = 0;
    walk.x = 0;
    walk.n = 0;
    if (walk.b < p.L.B) {
      walk.kvh = int((target - ctl.start.before) / ctl.start.of_seq);
      walk.x = ctl.start.before + walk.kvh * ctl.start.of_seq;
    }
    // Tiles three deep: one is loaded, the next one's scales are read, the page of the
    // one after is looked up.
    struct Tile {
      int key;        // first key; -1: there are no more
      int k0, k1;     // of the unit
      int b, head;
      int page;       // of this lane's box, and of its block
      int page_b;
      float scale;    // lanes 0-7: K's, 8-15: V's
    };
    const int n_box = 128 / p.box_rows;
    int n_items = 0;
    bool more = true, ok = true, any = false;
    Cut8 cut;
    cut.c1 = -1;
    int t_key = 0, t_end = 0, t_k0 = 0, t_k1 = 0, t_b = 0, t_head = 0;
    auto next_tile = [&]() -> Tile {  // the tile that follows, with its pages on their way
      while (more && t_key >= t_end) {
        more = walk.next(p, lo, hi, me == G - 1);
        Item8 x;
        x.head = -1;
        if (more) {
          any = true;
          x.b = walk.b_of;
          x.q0 = walk.seq.q0;
          x.qlen = walk.seq.qlen;
          x.klen = walk.seq.klen;
          x.row0 = walk.row0;
          x.rows = walk.rows;
          x.head = walk.head;
          x.k0 = walk.k0;
          x.k1 = walk.k1;
          x.slot = walk.first && walk.last ? -1 : walk.first ? 2 * me + 1 : 2 * me;
          if (walk.first && !walk.last) {
            cut.seq0 = x.q0;
            cut.row0 = x.row0;
            cut.rows = x.rows;
            cut.kvh = x.head;
            cut.c0 = me;
            cut.c1 = int((walk.y1 * G - 1) / all);  // the last whose share begins before y1
          }
          t_k0 = x.k0;
          t_k1 = x.k1;
          t_key = x.k0 & ~127;
          t_end = max(x.k1, 1);  // (a unit without keys has a tile too, an empty one: see kItems)
          t_b = walk.b_of;
          t_head = x.head;
        }
        const int i = n_items++;
        ok = ok && seq::warp_wait(&ctl.it_empty[i % kItems], ((i / kItems) & 1) ^ 1, &ctl.abort, LIM);
        if (!ok) more = false;
        if (lane == 0 && ok) {
          ctl.it[i % kItems] = x;
          mbar_arrive(&ctl.it_full[i % kItems]);
        }
      }
      Tile t;
      t.key = -1;
      t.page = t.page_b = -1;
      t.scale = 1.0f;
      if (!more) return t;
      t.key = t_key;
      t.k0 = t_k0;
      t.k1 = t_k1;
      t.b = t_b;
      t.head = t_head;
      t_key += 128;
      const int* const row = p.table + size_t(t.b) * p.max_pages;
      const int kb = t.key + lane * p.box_rows, kc = t.key + (lane & 7) * kFp8Block;
      // (a box or block that is not wholly outside [k0, k1): the others' pages are not looked up)
      if (lane < n_box && kb < t.k1 && kb + p.box_rows > t.k0) t.page = row[kb / p.page_size];
      if (lane < 16 && kc < t.k1 && kc + kFp8Block > t.k0) t.page_b = row[kc / p.page_size];
      return t;
    };
    auto read_scale = [&](Tile& t) {
      if (t.key >= 0 && t.page_b >= 0 && t.page_b < p.num_pages) {
        const int k = t.key + (lane & 7) * kFp8Block;
        const size_t block = size_t(t.page_b) * (p.page_size / kFp8Block) + k % p.page_size / kFp8Block;
        t.scale = p.scales[lane >> 3 & 1][block * p.Hkv + t.head];
      }
    };
    const uint64_t pol = l2_policy_evict_first();
    bool injected = false;
    auto load = [&](const Tile& t, int slot) {
      const int kb = t.key + lane * p.box_rows;
      const bool wanted = lane < n_box && kb < t.k1 && kb + p.box_rows > t.k0;
      int page = t.page;
      if (wanted && (page < 0 || page >= p.num_pages)) {  // no such page: it reads as zeros, and the caller is told
        atomicOr(p.status, kDevBadArg);
        page = p.num_pages;
      }
      const unsigned boxes = __ballot_sync(0xffffffffu, wanted);
      const int in_page = kb % p.page_size;
      if (p.inject == 1 && !injected) {  // test hook: never deliver this tile
        injected = true;
        return;
      }
      uint8_t* const dst = ring + slot * 2 * C::kHalf;
      if (lane == 0) mbar_arrive_expect_tx(&ctl.full[slot], uint32_t(2 * __popc(boxes) * p.box_rows * D));
      auto issue = [&](auto most) {  // (all pages first: pages of 16, 64 tokens 152 -> 127 us, d = 64 133 -> 97)
        constexpr int N = decltype(most)::value;
        int pg[N], at[N];
#pragma unroll
        for (int x = 0; x < N; ++x) {
          pg[x] = __shfl_sync(0xffffffffu, page, x);
          at[x] = __shfl_sync(0xffffffffu, in_page, x);
        }
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < N; ++x) {
            if (!(boxes >> x & 1)) continue;
            tma_load_4d_hint(dst + x * p.box_rows * D, &tmK, &ctl.full[slot], 0, t.head, at[x], pg[x], pol);
            tma_load_4d_hint(dst + C::kHalf + x * p.box_rows * D, &tmV, &ctl.full[slot], 0, t.head, at[x], pg[x], pol);
          }
        }
        __syncwarp();
      };
      if (n_box <= 2) {
        issue(std::integral_constant<int, 2>{});
      } else {
        issue(std::integral_constant<int, 8>{});
      }
    };
    auto hand_out_scale = [&](const Tile& t, int slot) {
      if (lane < 16) ctl.sc[slot][lane >> 3][lane & 7] = t.scale;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.full[slot]);
    };
    Tile a = next_tile(), b;
    b.key = -1;
    if (a.key >= 0 && ok) {  // the first is loaded before anything else is looked at: a short call is a chain of reads
      load(a, 0);
      read_scale(a);
      hand_out_scale(a, 0);
      a = next_tile();
      b = next_tile();
      read_scale(a);
    }
    for (int n = 1; a.key >= 0 && ok; ++n) {
      const Tile c = next_tile();
      read_scale(b);
      const int slot = n % S;
      ok = ok && seq::warp_wait(&ctl.empty[slot], ((n / S) & 1) ^ 1, &ctl.abort, LIM);
      if (!ok) break;
      hand_out_scale(a, slot);
      load(a, slot);
      a = b;
      b = c;
    }
    if (lane == 0) {
      p.cuts[me] = cut;
      p.has[me] = any ? 1 : 0;
    }
    if (*const_cast<volatile uint32_t*>(&ctl.abort)) {  // let copies in flight land before shared memory is released
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else {
    // ------------------------------------------------------------ a warp's keys
    const int g = lane >> 2, c = lane & 3;
    // Product row g (and g + 8) is key g, of odd g key g ^ 4: the reads of two
    // neighbouring rows' codes then meet in no bank, nor do those of V's rows 2 c.
    const int gk = (g & 1) ? g ^ 4 : g;
    int n = 0;  // tiles so far
    for (int i = 0;; ++i) {
      if (!seq::warp_wait(&ctl.it_full[i % kItems], (i / kItems) & 1, &ctl.abort, LIM)) break;
      const Item8 w = ctl.it[i % kItems];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.it_empty[i % kItems]);
      if (w.head < 0) break;
      // Q^T: rows 8 n + g, of d the 16 at 16 c and (d = 128) 64 + 16 c, as K's; divided by
      // a power of two of the row so that its largest value is in [2^14, 2^15)
      uint32_t qf[NT][KS][2];
      float rf[NT][2];                   // factor of rows 8 n + 2 c, 8 n + 2 c + 1
      int see_lo[NT][2], see_hi[NT][2];  // their keys [see_lo, see_hi)
      int all_lo = 0, all_hi = 0x7fffffff;  // keys that every row sees
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + g;
        uint4 raw[KS / 2];
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) raw[k] = make_uint4(0, 0, 0, 0);
        if (r < w.rows) {
          const int row = w.row0 + r, tok = row / p.group, hd = row - tok * p.group;
          const __nv_bfloat16* src = p.q + (w.q0 + tok) * p.q_stride + (1LL * w.head * p.group + hd) * D + 16 * c;
#pragma unroll
          for (int k = 0; k < KS / 2; ++k) raw[k] = __ldg(reinterpret_cast<const uint4*>(src + (k >> 1) * 64 + (k & 1) * 8));
        }
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          m = max_u16x2(m, max_u16x2(raw[k].x & 0x7fff7fffu, raw[k].y & 0x7fff7fffu));
          m = max_u16x2(m, max_u16x2(raw[k].z & 0x7fff7fffu, raw[k].w & 0x7fff7fffu));
        }
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = max(int(m >> 7) - 127, -100);  // (a row below 2^-100 keeps what f16 has of it)
        const float f = exp2i(14 - e);
#pragma unroll
        for (int k = 0; k < KS / 2; ++k) {
          const uint32_t y[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            qf[t][2 * k + (x >> 1)][x & 1] = f16x2_of(u2f(y[x] << 16) * f, u2f(y[x] & 0xffff0000u) * f);
        }
        // (a row that is not finite gives NaN, also where all its scores are -inf)
        const float back = m < 0x7f80u ? exp2i(e - 14) * p.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          rf[t][x] = __shfl_sync(0xffffffffu, back, (2 * c + x) * 4);
          const int rr = 8 * t + 2 * c + x;
          see_lo[t][x] = 0;
          see_hi[t][x] = w.klen;
          if (rr < w.rows) {
            const int pos = w.klen - w.qlen + (w.row0 + rr) / p.group;
            if (p.wr >= 0) see_hi[t][x] = min(w.klen, pos + p.wr + 1);
            if (p.wl >= 0) see_lo[t][x] = max(0, pos - p.wl);
          }
          all_lo = max(all_lo, see_lo[t][x]);
          all_hi = min(all_hi, see_hi[t][x]);
        }
      }
      all_lo = __reduce_max_sync(0xffffffffu, all_lo);
      all_hi = __reduce_min_sync(0xffffffffu, all_hi);

      float acc[NT][KS][4];
      float mrun[NT][2], l[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[t][k][x] = 0.0f;
        mrun[t][0] = mrun[t][1] = kLow;
        l[t][0] = l[t][1] = 0.0f;
      }
      bool ok = true;
      uint32_t nans = 0;  // not 0: NaN codes were taken as zeros
      for (int key = (w.k0 & ~127) + warp * 16, last = max(w.k1, 1) + warp * 16; key < last; key += 128, ++n) {
        const int slot = n % S;
        ok = seq::warp_wait(&ctl.full[slot], (n / S) & 1, &ctl.abort, LIM);
        if (!ok) break;
        if (key < w.k1 && key + 16 > w.k0) {
          const uint8_t* const kt = ring + slot * 2 * C::kHalf + (warp * 16) * D;
          const uint8_t* const vt = kt + C::kHalf;
          const float ka = ctl.sc[slot][0][warp], vb = ctl.sc[slot][1][warp];
          // S^T, two chains over d
          float sa[NT][4], sb[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) sa[t][x] = sb[t][x] = 0.0f;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            // pieces of 16 bytes, swizzled over 128 bytes (d = 128) or 64
            const int piece = D == 128 ? (4 * h + c) ^ gk : c ^ (gk >> 1 & 3);
            const uint4 x0 = *reinterpret_cast<const uint4*>(kt + gk * D + piece * 16);
            const uint4 x8 = *reinterpret_cast<const uint4*>(kt + (gk + 8) * D + piece * 16);
            const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w8[4] = {x8.x, x8.y, x8.z, x8.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a0 = f16x2_of_e4m3x2(uint16_t(w0[k])), a2 = f16x2_of_e4m3x2(uint16_t(w0[k] >> 16));
              const uint32_t a1 = f16x2_of_e4m3x2(uint16_t(w8[k])), a3 = f16x2_of_e4m3x2(uint16_t(w8[k] >> 16));
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma16816((k & 1) ? sb[t] : sa[t], a0, a1, a2, a3, qf[t][4 * h + k][0], qf[t][4 * h + k][1]);
            }
          }
          // exponents, masked where the block reaches past what some row sees
          const float lb = __log2f(vb), rb = __fdividef(1.0f, vb);
          const bool edge = key < all_lo || key + 16 > all_hi;
          bool over = false;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              sa[t][x] = fmaf(sa[t][x] + sb[t][x], rf[t][x & 1] * ka, lb);
              if (edge) {
                const int kk = key + gk + (x >> 1) * 8;
                if (kk < see_lo[t][x & 1] || kk >= see_hi[t][x & 1]) sa[t][x] = -INFINITY;
              }
              over = over || sa[t][x] - mrun[t][x & 1] > kTop - kShift;
            }
          }
          if (__any_sync(0xffffffffu, over)) {  // a new maximum, rare after the first blocks
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float m = fmaxf(sa[t][x], sa[t][x + 2]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                // (each row for itself, so that no row's roundings depend on its neighbours)
                m = m - mrun[t][x] > kTop - kShift ? m : mrun[t][x];
                const float f = ex2_mufu(mrun[t][x] - m);
                mrun[t][x] = m;
                l[t][x] *= f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                  acc[t][k][x] *= f;
                  acc[t][k][x + 2] *= f;
                }
              }
          }
          uint32_t pf[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int x = 0; x < 4; ++x) sa[t][x] = ex2_mufu(sa[t][x] - (mrun[t][x & 1] - kShift));
            l[t][0] = fmaf(sa[t][0] + sa[t][2], rb, l[t][0]);
            l[t][1] = fmaf(sa[t][1] + sa[t][3], rb, l[t][1]);
            pf[t][0] = transposed8x8(f16x2_of(sa[t][0], sa[t][1]));
            pf[t][1] = transposed8x8(f16x2_of(sa[t][2], sa[t][3]));
          }
          // O^T: lane (g, c) has V's keys of product rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9, and of d the
          // D / 8 at g D / 8, of which 2 t and 2 t + 1 are rows g and g + 8 of tile t
          constexpr int W = D / 32;  // words of a key's D / 8 values
          uint32_t v[4][W];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 2 * c + (k & 1) + (k >> 1) * 8, r = (k & 1) ? row ^ 4 : row;
            if constexpr (D == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(vt + r * 128 + ((g ^ (r & 7)) << 4));
              v[k][0] = y.x;
              v[k][1] = y.y;
              v[k][W - 2] = y.z;
              v[k][W - 1] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(vt + r * 64 + (((g >> 1) ^ (r >> 1 & 3)) << 4) + (g & 1) * 8);
              v[k][0] = y.x;
              v[k][1] = y.y;
            }
            if (key + 16 > w.klen) {  // past the sequence's end: 0 * NaN would stay NaN
#pragma unroll
              for (int x = 0; x < W; ++x) v[k][x] = key + r < w.klen ? v[k][x] : 0;
            }
          }
          // A NaN code of V that some rows do not see would reach them, as 0 * NaN is NaN: a zero here,
          // and the rows that see it are found at the unit's end (hidden_nans)
          if (edge) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int x = 0; x < W; ++x) {
                const uint32_t m = nan_codes(v[k][x]);
                nans |= m;
                v[k][x] &= ~m;
              }
          }
#pragma unroll
          for (int x = 0; x < W; ++x) {
            const uint32_t x0 = __byte_perm(v[0][x], v[1][x], 0x5140), x1 = __byte_perm(v[0][x], v[1][x], 0x7362);
            const uint32_t y0 = __byte_perm(v[2][x], v[3][x], 0x5140), y1 = __byte_perm(v[2][x], v[3][x], 0x7362);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u = k == 0 ? x0 : x1, y = k == 0 ? y0 : y1;
              const uint32_t a0 = f16x2_of_e4m3x2(uint16_t(u)), a1 = f16x2_of_e4m3x2(uint16_t(u >> 16));
              const uint32_t a2 = f16x2_of_e4m3x2(uint16_t(y)), a3 = f16x2_of_e4m3x2(uint16_t(y >> 16));
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(acc[t][2 * x + k], a0, a1, a2, a3, pf[t][0], pf[t][1]);
            }
          }
        }
        __syncwarp();  // every lane has read the tile
        if (lane == 0) mbar_arrive(&ctl.empty[slot]);
      }
      if (!ok) break;

      // ---- the warps' results joined
      if (!seq::warp_wait(&ctl.join_empty, (i & 1) ^ 1, &ctl.abort, LIM)) break;  // the unit's before have been read
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum = l[t][x];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          const int r = 8 * t + 2 * c + x;
          // O and l are 2^kShift of what belongs to mrun
          if (g == 0) ctl.ml[warp][r] = make_float2(mrun[t][x] == kLow ? kLow : mrun[t][x] - kShift, sum);
          float* dst = join + (warp * R + r) * C::kJoinLd + g * (D / 8);
#pragma unroll
          for (int k = 0; k < KS / 2; ++k)
            *reinterpret_cast<float4*>(dst + 4 * k) =
                make_float4(acc[t][2 * k][x], acc[t][2 * k][x + 2], acc[t][2 * k + 1][x], acc[t][2 * k + 1][x + 2]);
        }
      nans = __any_sync(0xffffffffu, nans != 0);
      __syncwarp();
      if (lane == 0) {
        ctl.nans[warp] = nans;
        mbar_arrive(&ctl.join_full);
      }
      if (!seq::warp_wait(&ctl.join_full, i & 1, &ctl.abort, LIM)) break;
      constexpr int Q4 = D / 4;
      nans = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) nans |= ctl.nans[k];
#pragma unroll 1
      for (int at = tid; at < w.rows * Q4; at += kWarps * 32) {
        const int r = at / Q4, d4 = (at - r * Q4) * 4;
        float m = kLow;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) m = fmaxf(m, ctl.ml[k][r].x);
        float lsum = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float2 t = ctl.ml[k][r];
          const float f = ex2_mufu(t.x - m);
          const float4 y = *reinterpret_cast<const float4*>(join + (k * R + r) * C::kJoinLd + d4);
          lsum = fmaf(t.y, f, lsum);
          o.x = fmaf(y.x, f, o.x);
          o.y = fmaf(y.y, f, o.y);
          o.z = fmaf(y.z, f, o.z);
          o.w = fmaf(y.w, f, o.w);
        }
        if (nans != 0) {
          const int pos = w.klen - w.qlen + (w.row0 + r) / p.group;
          const uint32_t x = hidden_nans(p, w.b, p.wl >= 0 ? max(w.k0, pos - p.wl) : w.k0,
                                         p.wr >= 0 ? min(w.k1, pos + p.wr + 1) : w.k1, p.v_codes + 1LL * w.head * D + d4, D,
                                         all_lo, all_hi);
          const float nan = __int_as_float(0x7fffffff);
          if (x & 0xffu) o.x = nan;
          if (x & 0xff00u) o.y = nan;
          if (x & 0xff0000u) o.z = nan;
          if (x & 0xff000000u) o.w = nan;
        }
        if (w.slot >= 0) {
          *reinterpret_cast<float4*>(p.part_o + (size_t(w.slot) * R + r) * D + d4) = o;
          if (d4 == 0) p.part_ml[size_t(w.slot) * R + r] = make_float2(m, lsum);
        } else {
          const int row = w.row0 + r, tok = row / p.group, hd = w.head * p.group + row - tok * p.group;
          const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
          *reinterpret_cast<uint2*>(p.o + (size_t(w.q0 + tok) * p.Hq + hd) * D + d4) =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
          if (d4 == 0)
            p.lse[size_t(hd) * p.total_q + w.q0 + tok] =
                lsum == 0.0f ? -INFINITY : (m + __log2f(lsum)) * 0.69314718055994531f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.join_empty);
    }
  }
  __syncthreads();
  if (tid == 0 && ctl.abort) atomicOr(p.status, kDevTimeout);
}

// The parts of the units that several workers share: O = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i. A block to a unit, 32 warps: several to a row, each of
// which takes every W-th part (one after the other, 19 parts took 5 us), summed
// in the warps' order.
template <int D, int R>
__global__ void __launch_bounds__(1024) join8_kernel(const Params8 p) {
  constexpr int W = 32 / R;  // warps of a row
  constexpr int V = D / 32;  // columns of a lane
  __shared__ float so[32][D];
  grid_dep_wait();
  const Cut8 k = p.cuts[blockIdx.x];
  if (k.c1 < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = warp / W, w = warp % W;
  float m = kLow, l = 0.0f, o[V] = {};
  if (r < k.rows) {
    for (int c0 = k.c0; c0 <= k.c1; c0 += 32) {  // 32 parts at a time; all their (m, l) by each warp
      const int c = c0 + lane;
      float2 t = make_float2(kLow, 0.0f);
      if (c <= k.c1) {  // (a worker without a share has no part: what its slot holds is not used)
        const int has = p.has[c];
        const float2 x = p.part_ml[size_t(c == k.c0 ? 2 * c + 1 : 2 * c) * R + r];
        if (has) t = x;
      }
      float mn = fmaxf(m, t.x);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
      const float wa = ex2_mufu(m - mn), wb = ex2_mufu(t.x - mn);
      float ls = t.y * wb;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      l = l * wa + ls;
      m = mn;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= wa;
      const int n = min(32, k.c1 - c0 + 1);
#pragma unroll 8
      for (int i = w; i < n; i += W) {
        const float wi = __shfl_sync(0xffffffffu, wb, i), li = __shfl_sync(0xffffffffu, t.y, i);
        if (li == 0.0f) continue;  // no part, or no key of it visible to the row
        const int ci = c0 + i;
        const float* src = p.part_o + (size_t(ci == k.c0 ? 2 * ci + 1 : 2 * ci) * R + r) * D + lane * V;
        if constexpr (V == 4) {
          const float4 y = *reinterpret_cast<const float4*>(src);
          o[0] = fmaf(y.x, wi, o[0]);
          o[1] = fmaf(y.y, wi, o[1]);
          o[2] = fmaf(y.z, wi, o[2]);
          o[3] = fmaf(y.w, wi, o[3]);
        } else {
          const float2 y = *reinterpret_cast<const float2*>(src);
          o[0] = fmaf(y.x, wi, o[0]);
          o[1] = fmaf(y.y, wi, o[1]);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) so[warp][lane * V + e] = o[e];
  __syncthreads();
  if (w != 0 || r >= k.rows) return;
#pragma unroll
  for (int x = 1; x < W; ++x)
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] += so[warp + x][lane * V + e];
  const int row = k.row0 + r, tok = row / p.group, hd = k.kvh * p.group + row - tok * p.group;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  __nv_bfloat16* dst = p.o + (size_t(k.seq0 + tok) * p.Hq + hd) * D + lane * V;
  if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  } else {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
  }
  if (lane == 0)
    p.lse[size_t(hd) * p.total_q + k.seq0 + tok] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D, int NT>
cudaError_t launch_t(const SeqProblem& pb, const Fp8Scales& sc, void* o, float* lse, cudaStream_t stream) {
  using C = Shape<D, NT>;
  const int G = num_sms() * C::kPerSm;
  Params8 p{};
  p.q = static_cast<const __nv_bfloat16*>(pb.q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.v_codes = static_cast<const uint8_t*>(pb.v);
  p.scales[0] = sc.k;
  p.scales[1] = sc.v;
  p.table = pb.page_table;
  p.L = Lens{pb.cu_q, nullptr, pb.lens_k, pb.B, pb.total_q, 0, 1LL * pb.max_pages * pb.page_size};
  p.Hq = pb.Hq;
  p.Hkv = pb.Hkv;
  p.group = pb.Hq / pb.Hkv;
  p.total_q = pb.total_q;
  p.q_stride = pb.q_stride;
  p.num_pages = pb.num_pages;
  p.page_size = pb.page_size;
  p.max_pages = pb.max_pages;
  p.scale_log2 = exp_scale_log2(pb.scale);
  p.wl = pb.window_left;
  p.wr = pb.window_right;
  p.status = status_word();
  if (p.status == nullptr) return cudaErrorLaunchFailure;
  const DebugCfg dc = debug_cfg();
  p.wait_limit_ns = dc.wait_limit_ns;
  p.inject = dc.inject;
  CUtensorMap maps[2];
  p.box_rows = 128;
  while (pb.page_size % p.box_rows != 0) p.box_rows /= 2;  // 16 at least
  for (int i = 0; i < 2; ++i)
    if (!encode_codes(&maps[i], i == 0 ? pb.k : pb.v, pb.num_pages, pb.page_size, pb.Hkv, D, p.box_rows,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  auto kern = attend8_kernel<D, NT>;
  static seq::SmemLimit limit;
  cudaError_t e = limit.set(kern, C::kSmem);
  if (e != cudaSuccess) return e;
  auto carve = [&](uint8_t* base) {
    seq::Carver c{base, 0};
    p.cuts = c.take<Cut8>(G);
    p.has = c.take<int>(G);
    p.part_ml = c.take<float2>(size_t(2) * G * C::kRows);
    p.part_o = c.take<float>(size_t(2) * G * C::kRows * D);
    return c.at;
  };
  cudaMemPool_t pool = workspace_pool();
  void* ws = nullptr;
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, carve(nullptr), pool, stream) != cudaSuccess)
    return cudaErrorMemoryAllocation;
  carve(static_cast<uint8_t*>(ws));
  kern<<<G, kThreads, C::kSmem, stream>>>(maps[0], maps[1], p);
  e = cudaGetLastError();
  if (e == cudaSuccess) {  // starts while the kernel before it ends, and waits for it
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(G);
    lc.blockDim = dim3(1024);
    lc.stream = stream;
    lc.attrs = pdl;
    lc.numAttrs = 1;
    e = cudaLaunchKernelEx(&lc, join8_kernel<D, C::kRows>, p);
  }
  const cudaError_t f = cudaFreeAsync(ws, stream);
  return e != cudaSuccess ? e : f;
}

}  // namespace seq8

cudaError_t launch_seq_fwd8(const SeqProblem& pb, const Fp8Scales& sc, void* o, float* lse, cudaStream_t stream) {
  // Few rows or many: by the mean sequence's, as the lengths are on the device.
  // 64 sequences of 2000 to 8000 keys, 8 kv heads, in us here and there, d = 128 (64):
  //   4 rows (single tokens)    125, 181 (84, 149)
  //   16 rows                   155, 184 (101, 151)
  //   24 rows                   294, 187 (185, 151)
  // Of batches that are not alike, over 8000 keys or as above:
  //   63 single tokens and 65 of one sequence (8 rows on the mean)   225, 294 (179, 253)
  //   31 and 96 (16 rows)                                            192, 172 (129, 149)
  //   255 and a chunk of 512 (12 rows)                               964, 740 (631, 602)
  // as the keys of a long one are read anew for each 8 or 16 rows. Empty places count too: 255 of
  // them and a chunk of 512 over 8000 keys (8 rows on the mean) take 578 (492), the chunk by
  // itself, there, 70 (61); 63 and 192 tokens 44 there (118 here, d = 64), by themselves 42 (35).
  // So up to 16 rows come here,
  // but of d = 128 from 9 on only single tokens of wide groups and small batches (4
  // tokens of a group of 4 over 1000 keys: 13.3, 15.5). Above 2^16 rows such a sequence
  // could be very long.
  const long long all = 1LL * pb.total_q * (pb.Hq / pb.Hkv), rows = (all + pb.B - 1) / pb.B;
  const bool few = rows <= 8 || (rows <= 16 && (pb.d == 64 || pb.total_q <= pb.B || all <= 64));
  if (!few || all > (1 << 16)) return launch_seq_fwd_codes(pb, sc, o, lse, stream);
  if (pb.d == 128)
    return rows <= 8 ? seq8::launch_t<128, 1>(pb, sc, o, lse, stream) : seq8::launch_t<128, 2>(pb, sc, o, lse, stream);
  return rows <= 8 ? seq8::launch_t<64, 1>(pb, sc, o, lse, stream) : seq8::launch_t<64, 2>(pb, sc, o, lse, stream);
}

}  // namespace fa
