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
// 2^-12 of itself, for all P' above 2^-21 of the largest), O to bf16.
//
// Few rows to a kv head (single tokens): bound by the cache's bytes. A warp
// takes a block of 16 keys at a time. Its codes come by asynchronous copies into
// the very lanes that use them (16 bytes a lane, a ring of stages per warp), are
// turned to f16 in registers and are the A operand of mma.sync.m16n8k16, the
// rows the B operand of 8 columns: S^T = K Q^T, then O^T = V^T P^T. Shared memory
// carries each byte once in and once out, and no warp waits for another before
// the end of a unit. (The tensor-memory pipeline of fa_seq_fwd.cu would carry
// each code through shared memory six times - in as codes, out, back in as f16,
// to the tensor cores - and that sets its pace below device memory's.)
//
// Work: a unit is up to 8 NT rows of a sequence and kv head with the tiles of
// 128 keys that they see. All tiles of all units are laid end to end and divided
// evenly between the CTAs (one per SM), each of which finds its own share; a
// unit's keys go round its 8 warps by blocks, whose results are joined in shared
// memory, and the parts of a unit that several CTAs share by a last kernel, in a
// fixed order.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kItemCost = 2;  // of a unit beside its tiles, in tiles
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
  const uint8_t* pages[2];  // k, v
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
  unsigned* status;
};

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalf = 16 * D;             // bytes of a block's K, or V
  static constexpr int kStages = NT == 4 && D == 128 ? 2 : 4;
  static constexpr int kRing = kWarps * kStages * 2 * kHalf;
  static constexpr int kJoinLd = D + 4;            // (spreads the rows over the banks)
  static constexpr int kJoin = kWarps * kRows * kJoinLd * 4;
  static constexpr int kSmem = kRing + kJoin;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// A walk over the units in the order (sequence, kv head, rows), with the place
// x of each unit's tiles among all costs.
template <int ROWS>
struct Walk8 {
  int b, kvh, j;   // the unit that follows
  int n;           // units of the sequence and head
  Seq s;
  long long x;
  // the unit found by next(): what of it is this worker's
  int row0, rows, head, b_of;
  Seq seq;
  int k0, k1;      // keys [k0, k1)
  long long y0, y1;
  bool first, last;  // the unit's first, last part

  __device__ __forceinline__ void load(const Params8& p) {
    n = 0;
    while (b < p.L.B) {
      seq::seq_at(p.L, b, s);
      n = (s.qlen * p.group + ROWS - 1) / ROWS;
      if (n > 0) break;
      ++b;
    }
  }
  // the worker's next part of a unit, if any: lo, hi its share; end: it has what lies at the end too
  __device__ __forceinline__ bool next(const Params8& p, long long lo, long long hi, bool end) {
    while (b < p.L.B) {
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
          load(p);
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
    return false;
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attend8_kernel(const Params8 p) {
  using C = Shape<D, NT>;
  constexpr int R = C::kRows, S = C::kStages;
  constexpr int KS = D / 16;  // products' steps over d, tiles of 16 d of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sc[kWarps][S][2];
  __shared__ float2 ml[kWarps][R];
  __shared__ long long sums[kWarps];
  __shared__ struct {
    int b;
    long long before, of_seq;  // costs of the sequences before it, its own for one head
    int bad;
  } start;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int G = gridDim.x, me = blockIdx.x;
  grid_dep_launch();

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
  if (tid == 0) {
    start.b = p.L.B;
    start.bad = 0;
  }
  __syncthreads();
  bool ok = true;
  long long mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += cost_of(b, ok);
  if (!ok) start.bad = 1;
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += o;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  long long T = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sums[w];
    T += sums[w];
  }
  if (start.bad) {  // lengths that the tensors cannot hold: nothing is computed
    if (tid == 0) {
      p.cuts[me].c1 = -1;
      p.has[me] = 0;
      if (me == 0) atomicOr(p.status, kDevBadArg);
    }
    return;
  }
  const long long all = T * p.Hkv, lo = all * me / G, hi = all * (me + 1) / G;
  {
    // (a unit without keys lies at the end of its cost: lo - 1 is in it, or before it)
    const long long target = lo > 0 ? lo - 1 : 0;
    long long before = (upto - mine) * p.Hkv;
    if (before <= target && target < upto * p.Hkv) {
      for (int b = b0; b < b1; ++b) {
        const long long t = cost_of(b, ok);
        if (target < before + t * p.Hkv) {
          start.b = b;
          start.before = before;
          start.of_seq = t;
          break;
        }
        before += t * p.Hkv;
      }
    }
  }
  __syncthreads();
  Walk8<R> fetch;
  fetch.b = start.b;
  fetch.kvh = 0;
  fetch.j = 0;
  fetch.x = 0;
  fetch.load(p);
  if (fetch.b < p.L.B) {
    fetch.kvh = int(((lo > 0 ? lo - 1 : 0) - start.before) / start.of_seq);
    fetch.x = start.before + fetch.kvh * start.of_seq;
  }
  Walk8<R> work = fetch;
  const bool end = me == G - 1;

  // ---- fetching: blocks of 16 keys, this warp's of each unit in turn
  uint8_t* const ring = smem + warp * (S * 2 * C::kHalf);
  const uint32_t ring_at = smem_u32(ring), sc_at = smem_u32(&sc[warp][0][0]);
  int f_blk = 0, f_end = 0, f_page = 0, f_row = 0;  // the block to fetch next, its page, its first row there
  bool f_more = true;
  auto look_up = [&] {  // the page of the block to fetch next
    while (f_more && f_blk >= f_end) {
      f_more = fetch.next(p, lo, hi, end);
      if (f_more) {
        f_blk = (fetch.k0 >> 4) + warp;
        f_end = (fetch.k1 + 15) >> 4;
      }
    }
    if (f_more) {
      const int k = f_blk << 4, pg = k / p.page_size;
      f_row = k - pg * p.page_size;
      f_page = p.table[size_t(fetch.b_of) * p.max_pages + pg];
    }
  };
  auto issue = [&](int stage) {
    if (f_more) {
      int page = f_page;
      const bool there = page >= 0 && page < p.num_pages;
      const uint32_t dst = ring_at + stage * 2 * C::kHalf + lane * 16;
      if (there) {
        const long long row = 1LL * page * p.page_size + f_row;
        const long long tok = 1LL * p.Hkv * D;  // bytes between keys
        const long long at = (row * p.Hkv + fetch.head) * D;
        // K: lane (g, c) has keys g and g + 8, of d the 16 at 16 c and (d = 128) at 64 + 16 c
        const uint8_t* k = p.pages[0] + at + g * tok + c * 16;
        // V: keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9, of d the D / 8 at g D / 8
        const uint8_t* v = p.pages[1] + at + 2 * c * tok + g * (D / 8);
        if constexpr (D == 128) {
          cp16(dst, k);
          cp16(dst + 512, k + 64);
          cp16(dst + 1024, k + 8 * tok);
          cp16(dst + 1536, k + 8 * tok + 64);
          cp16(dst + 2048, v);
          cp16(dst + 2560, v + tok);
          cp16(dst + 3072, v + 8 * tok);
          cp16(dst + 3584, v + 9 * tok);
        } else {
          cp16(dst, k);
          cp16(dst + 512, k + 8 * tok);
          const uint32_t dv = dst + 1024 - lane * 8;
          cp8(dv, v);
          cp8(dv + 256, v + tok);
          cp8(dv + 512, v + 8 * tok);
          cp8(dv + 768, v + 9 * tok);
        }
        if (lane < 2) cp4(sc_at + (stage * 2 + lane) * 4, p.scales[lane] + (row >> 4) * p.Hkv + fetch.head);
      } else {  // no such page: it reads as zeros, and the caller is told
        if (lane == 0) atomicOr(p.status, kDevBadArg);
#pragma unroll
        for (int i = 0; i < 2 * C::kHalf / 512; ++i)
          *reinterpret_cast<uint4*>(ring + stage * 2 * C::kHalf + i * 512 + lane * 16) = make_uint4(0, 0, 0, 0);
        if (lane < 2) sc[warp][stage][lane] = 1.0f;
      }
      f_blk += kWarps;
      look_up();
    }
    cp_commit();
  };
  look_up();
#pragma unroll 1
  for (int s = 0; s < S; ++s) issue(s);

  // ---- the units
  float* const join = reinterpret_cast<float*>(smem + C::kRing);
  int stage = 0;
  Cut8 cut;
  cut.c1 = -1;
  bool any = false;
  while (work.next(p, lo, hi, end)) {
    any = true;
    const Seq s = work.seq;
    // Q^T: rows 8 n + g, of d the 16 at 16 c and (d = 128) 64 + 16 c, as K's; divided by
    // a power of two of the row so that its largest value is in [2^14, 2^15)
    uint32_t qf[NT][KS][2];
    float rf[NT][2];             // factor of rows 8 n + 2 c, 8 n + 2 c + 1
    int see_lo[NT][2], see_hi[NT][2];  // their keys [see_lo, see_hi)
    int all_lo = 0, all_hi = 0x7fffffff;  // keys that every row of this lane sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
      uint4 raw[KS / 2];
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < work.rows) {
        const int row = work.row0 + r, tok = row / p.group, hd = row - tok * p.group;
        const __nv_bfloat16* src = p.q + (s.q0 + tok) * p.q_stride + (1LL * work.head * p.group + hd) * D + 16 * c;
#pragma unroll
        for (int i = 0; i < KS / 2; ++i)
          raw[i] = __ldg(reinterpret_cast<const uint4*>(src + (i >> 1) * 64 + (i & 1) * 8));
      }
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        m = __vmaxu2(m, __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu));
        m = __vmaxu2(m, __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
      }
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = max(int(m >> 7) - 127, -100);  // (a row below 2^-100 keeps what f16 has of it)
      const float f = exp2i(14 - e);
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[i]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qf[n][2 * i + (x >> 1)][x & 1] = f16x2_of(u2f(w[x] << 16) * f, u2f(w[x] & 0xffff0000u) * f);
      }
      const float back = exp2i(e - 14) * p.scale_log2;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        rf[n][x] = __shfl_sync(0xffffffffu, back, (2 * c + x) * 4);
        const int rr = 8 * n + 2 * c + x;
        see_lo[n][x] = 0;
        see_hi[n][x] = s.klen;
        if (rr < work.rows) {
          const int pos = s.klen - s.qlen + (work.row0 + rr) / p.group;
          if (p.wr >= 0) see_hi[n][x] = min(s.klen, pos + p.wr + 1);
          if (p.wl >= 0) see_lo[n][x] = max(0, pos - p.wl);
        }
        all_lo = max(all_lo, see_lo[n][x]);
        all_hi = min(all_hi, see_hi[n][x]);
      }
    }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);

    float acc[NT][KS][4];
    float mrun[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int t = 0; t < KS; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[n][t][x] = 0.0f;
      mrun[n][0] = mrun[n][1] = kLow;
      l[n][0] = l[n][1] = 0.0f;
    }
    const int blk_end = (work.k1 + 15) >> 4;
#pragma unroll 1
    for (int blk = (work.k0 >> 4) + warp; blk < blk_end; blk += kWarps) {
      cp_wait<S - 1>();
      __syncwarp();
      const uint8_t* st = ring + stage * 2 * C::kHalf;
      const float ka = sc[warp][stage][0], vb = sc[warp][stage][1];
      // S^T, two chains over d
      float sa[NT][4], sb[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) sa[n][x] = sb[n][x] = 0.0f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(st + h * 512 + lane * 16);
        const uint4 k8 = *reinterpret_cast<const uint4*>(st + (D / 64 + h) * 512 + lane * 16);
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&k0);
        const uint32_t* w8 = reinterpret_cast<const uint32_t*>(&k8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = f16x2_of_e4m3x2(uint16_t(w0[i])), a2 = f16x2_of_e4m3x2(uint16_t(w0[i] >> 16));
          const uint32_t a1 = f16x2_of_e4m3x2(uint16_t(w8[i])), a3 = f16x2_of_e4m3x2(uint16_t(w8[i] >> 16));
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816((i & 1) ? sb[n] : sa[n], a0, a1, a2, a3, qf[n][4 * h + i][0], qf[n][4 * h + i][1]);
        }
      }
      // exponents, masked where the block reaches past what some row sees
      const float lb = __log2f(vb), rb = __fdividef(1.0f, vb);
      const int key = blk << 4;
      const bool edge = key < all_lo || key + 16 > all_hi;
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sa[n][x] = fmaf(sa[n][x] + sb[n][x], rf[n][x & 1] * ka, lb);
          if (edge) {
            const int kk = key + g + (x >> 1) * 8;
            if (kk < see_lo[n][x & 1] || kk >= see_hi[n][x & 1]) sa[n][x] = -INFINITY;
          }
          over = over || sa[n][x] - mrun[n][x & 1] > kTop - kShift;
        }
      }
      if (__any_sync(0xffffffffu, over)) {  // a new maximum, rare after the first blocks
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float m = fmaxf(sa[n][x], sa[n][x + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            m = fmaxf(m, mrun[n][x]);
            const float f = ex2_mufu(mrun[n][x] - m);
            mrun[n][x] = m;
            l[n][x] *= f;
#pragma unroll
            for (int t = 0; t < KS; ++t) {
              acc[n][t][x] *= f;
              acc[n][t][x + 2] *= f;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sa[n][x] = ex2_mufu(sa[n][x] - (mrun[n][x & 1] - kShift));
        l[n][0] = fmaf(sa[n][0] + sa[n][2], rb, l[n][0]);
        l[n][1] = fmaf(sa[n][1] + sa[n][3], rb, l[n][1]);
        pf[n][0] = transposed8x8(f16x2_of(sa[n][0], sa[n][1]));
        pf[n][1] = transposed8x8(f16x2_of(sa[n][2], sa[n][3]));
      }
      // O^T: the d at g D / 8 + 2 t and + 2 t + 1 are rows g and g + 8 of tile t
      constexpr int W = D / 32;  // words of a key's D / 8 values
      uint32_t v[4][W];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          *reinterpret_cast<uint4*>(v[i]) = *reinterpret_cast<const uint4*>(st + C::kHalf + i * 512 + lane * 16);
        } else {
          *reinterpret_cast<uint2*>(v[i]) = *reinterpret_cast<const uint2*>(st + C::kHalf + i * 256 + lane * 8);
        }
        if (key + 16 > s.klen) {  // past the sequence's end: 0 * NaN would stay NaN
          const bool in = key + 2 * c + (i & 1) + (i >> 1) * 8 < s.klen;
#pragma unroll
          for (int w = 0; w < W; ++w) v[i][w] = in ? v[i][w] : 0;
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = i == 0 ? x0 : x1, y = i == 0 ? y0 : y1;
          const uint32_t a0 = f16x2_of_e4m3x2(uint16_t(x)), a1 = f16x2_of_e4m3x2(uint16_t(x >> 16));
          const uint32_t a2 = f16x2_of_e4m3x2(uint16_t(y)), a3 = f16x2_of_e4m3x2(uint16_t(y >> 16));
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(acc[n][2 * w + i], a0, a1, a2, a3, pf[n][0], pf[n][1]);
        }
      }
      __syncwarp();  // every lane has read the stage
      issue(stage);
      stage = stage + 1 == S ? 0 : stage + 1;
    }

    // ---- the warps' results joined
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float t = l[n][x];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        const int r = 8 * n + 2 * c + x;
        // O and l are 2^kShift of what belongs to mrun
        if (g == 0) ml[warp][r] = make_float2(mrun[n][x] == kLow ? kLow : mrun[n][x] - kShift, t);
        float* dst = join + (warp * R + r) * C::kJoinLd + g * (D / 8);
#pragma unroll
        for (int t4 = 0; t4 < KS / 2; ++t4)
          *reinterpret_cast<float4*>(dst + 4 * t4) =
              make_float4(acc[n][2 * t4][x], acc[n][2 * t4][x + 2], acc[n][2 * t4 + 1][x], acc[n][2 * t4 + 1][x + 2]);
      }
    __syncthreads();
    const bool part = !(work.first && work.last);
    const int slot = work.first ? 2 * me + 1 : 2 * me;
    constexpr int Q4 = D / 4;
    for (int i = tid; i < work.rows * Q4; i += kThreads) {
      const int r = i / Q4, d4 = (i - r * Q4) * 4;
      float m = kLow;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w][r].x);
      float lsum = 0.0f;
      float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 t = ml[w][r];
        const float f = ex2_mufu(t.x - m);
        const float4 y = *reinterpret_cast<const float4*>(join + (w * R + r) * C::kJoinLd + d4);
        lsum = fmaf(t.y, f, lsum);
        o.x = fmaf(y.x, f, o.x);
        o.y = fmaf(y.y, f, o.y);
        o.z = fmaf(y.z, f, o.z);
        o.w = fmaf(y.w, f, o.w);
      }
      if (part) {
        *reinterpret_cast<float4*>(p.part_o + (size_t(slot) * R + r) * D + d4) = o;
        if (d4 == 0) p.part_ml[size_t(slot) * R + r] = make_float2(m, lsum);
      } else {
        const int row = work.row0 + r, tok = row / p.group, hd = work.head * p.group + row - tok * p.group;
        const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
        *reinterpret_cast<uint2*>(p.o + (size_t(s.q0 + tok) * p.Hq + hd) * D + d4) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (d4 == 0)
          p.lse[size_t(hd) * p.total_q + s.q0 + tok] =
              lsum == 0.0f ? -INFINITY : (m + __log2f(lsum)) * 0.69314718055994531f;
      }
    }
    if (work.first && !work.last) {
      cut.seq0 = s.q0;
      cut.row0 = work.row0;
      cut.rows = work.rows;
      cut.kvh = work.head;
      cut.c0 = me;
      cut.c1 = int((work.y1 * G - 1) / all);  // the last whose share begins before y1
    }
    __syncthreads();  // before the next unit's results
  }
  cp_wait<0>();
  if (tid == 0) {
    p.cuts[me] = cut;
    p.has[me] = any ? 1 : 0;
  }
}

// The parts of the units that several workers share: O = sum_i 2^(m_i - m) O_i /
// sum_i 2^(m_i - m) l_i, in the workers' order; a warp per row.
template <int D, int R>
__global__ void __launch_bounds__(R * 32) join8_kernel(const Params8 p) {
  grid_dep_wait();
  const Cut8 k = p.cuts[blockIdx.x];
  const int r = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (k.c1 < 0 || r >= k.rows) return;
  constexpr int V = D / 32;
  float m = kLow, l = 0.0f, o[V] = {};
  for (int c0 = k.c0; c0 <= k.c1; c0 += 32) {
    const int c = c0 + lane;
    float2 t = make_float2(kLow, 0.0f);
    if (c <= k.c1 && p.has[c]) t = p.part_ml[size_t(c == k.c0 ? 2 * c + 1 : 2 * c) * R + r];
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
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
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
  const int G = num_sms();
  Params8 p{};
  p.q = static_cast<const __nv_bfloat16*>(pb.q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.pages[0] = static_cast<const uint8_t*>(pb.k);
  p.pages[1] = static_cast<const uint8_t*>(pb.v);
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
  kern<<<G, kThreads, C::kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) {  // starts while the kernel before it ends, and waits for it
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(G);
    lc.blockDim = dim3(C::kRows * 32);
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
  // rows of a unit: as many as the mean sequence has
  const long long rows = (1LL * pb.total_q + pb.B - 1) / pb.B * (pb.Hq / pb.Hkv);
  if (rows > 32) return launch_seq_fwd_codes(pb, sc, o, lse, stream);
  const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  if (pb.d == 128)
    return nt == 1   ? seq8::launch_t<128, 1>(pb, sc, o, lse, stream)
           : nt == 2 ? seq8::launch_t<128, 2>(pb, sc, o, lse, stream)
                     : seq8::launch_t<128, 4>(pb, sc, o, lse, stream);
  return nt == 1   ? seq8::launch_t<64, 1>(pb, sc, o, lse, stream)
         : nt == 2 ? seq8::launch_t<64, 2>(pb, sc, o, lse, stream)
                   : seq8::launch_t<64, 4>(pb, sc, o, lse, stream);
}

}  // namespace fa
