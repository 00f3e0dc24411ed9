// Backward pass of attention over packed sequences on sm_103a
// (fa_bwd_varlen), bf16 operands, d = 64 or 128.
//
// Method and pipeline are those of the dense backward (fa_bwd.cu): per key
// tile, dK and dV stay in tensor memory while the tiles of query rows that
// see it pass by; P is recomputed from the saved log-sum-exp; dQ is added
// into an fp32 accumulator by TMA reductions:
//   dV = P^T dO, dP = dO V^T, D_i = sum_c dO_ic O_ic, dS = P o (dP - D),
//   dQ = scale dS K, dK = scale dS^T Q.
// What differs:
//   * a tile of 128 query rows holds 128 / group tokens with all query heads
//     of the group (row = token * group + head): a key tile meets every head
//     in the same walk, short sequences fill their tiles, and a causal
//     diagonal wastes 128 / group tokens instead of 128;
//   * work comes from the plan (fa_seq_plan.cuh): units (key tile, kv head)
//     by their row tiles, longest first, or divided evenly, in which case the
//     parts of a unit keep fp32 dK and dV in slots that a last kernel sums in
//     a fixed order (dK, dV are deterministic; dQ's additions are not ordered);
//   * dQ accumulator, LSE and D rows are padded to whole row tiles per
//     sequence, so no tile reaches into another sequence's rows;
//   * tiles read on past a sequence's end: rows past it are zeroed in shared
//     memory by a warp of its own before any product reads them (another
//     sequence's infinities would survive a multiplication by P = 0).
//
// What bounds it: shared memory. A step (a key tile and a tile of 128 rows,
// d = 128) takes 2.2 us, in which the five products' operands, dS and the
// staging of dQ are some 512 KB of shared-memory traffic. Its data pipe is taken
// in 52 % of the cycles by the products and in 48 % by loads and stores; the
// tensor pipe is 58 % busy, DRAM 23 % (2 sequences of 4096 tokens). The 128
// registers of the launch are full: at d = 64 a thread spills 36 bytes (148 of
// reloads in the code), at d = 128 4 (20). One causal sequence of
// 16384 tokens, 32 / 8 heads: 3.9 ms, as the dense backward; 8 of 2048:
// 0.85 ms (dense 1.09, whose diagonals waste more). pre and post move their
// bytes at the memory's rate (85 and 59 us of a step over 16 thousand packed
// tokens of 1.5 ms).
//
// Kernels: plan, pre (D, LSE * log2 e, zeroed accumulator), main, post (dQ to
// bf16, and the parts' sums).
//   main: 512 threads, persistent, one CTA per SM
//     warps 0-7  compute: two warps per lane quarter, a thread per key row
//                and 64 of the tile's 128 query rows
//     warps 8-11 dQ drain, dK/dV epilogue
//     warp 12 TMA producer, warp 13 MMA issuer, warp 14 tail rows
//     TMEM: S^T [0,128) with P^T over columns [0,32) and [64,96)
//           (fa_bwd_layout.h), dP^T / dQ [128,256), dV [256,256+d),
//           dK [256+d, 256+2d)
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "../../include/fa.h"
#include "fa_bwd_layout.h"
#include "fa_internal.h"
#include "fa_seq_plan.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace seqb {

using seq::BwdItem;
using seq::Cut;
using seq::PlanHead;

constexpr int kThreads = 512;

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;  // K, V, Q or dO tile of 128 rows
  static constexpr int kDsBytes = 128 * 128 * 2;
  static constexpr int kStgBytes = 32768;   // dQ staging: 4 warps x 2 boxes of [32 rows][32 d] fp32
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTile;
  static constexpr int kOffQ = 2 * kTile;   // 2 slots
  static constexpr int kOffDO = 4 * kTile;  // 1 slot
  static constexpr int kOffDs = 5 * kTile;
  static constexpr int kOffStg = kOffDs + kDsBytes;
  static constexpr int kOffVec = kOffStg + kStgBytes;  // [2 stages][lse2 128 | delta 128] fp32
  static constexpr int kOffCtl = kOffVec + 2 * 2 * 128 * 4;
  static constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;
};

struct __align__(16) Ctl {
  BwdItem cur[kThreads / 32];  // each warp's current item (the compute and drain warps have no registers for it)
  uint64_t kv_full, kv_seen, kv_empty;
  uint64_t q_full[2], q_seen[2], q_empty[2], do_full, do_seen, do_empty;
  uint64_t vec_full[2], vec_empty[2];
  uint64_t s_full, p_full, dp_full, ds_full, dq_full, dq_empty, acc_full, acc_empty, drain;
  uint32_t tmem_base;
  uint32_t abort;
};

struct OutMaps {
  CUtensorMap acc;     // fp32 dQ accumulator [rows][D], boxes of 32 rows x 32 d (reductions)
  CUtensorMap dk, dv;  // [total_k, Hkv, d], boxes of 32 rows x 64 d (stores)
  CUtensorMap part;    // fp32 parts [2 G][2 (dV, dK)][128][D], boxes of 32 rows x 32 d (stores)
};

struct Params {
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  const float* lse2;   // [Hkv * tiles * 128] LSE * log2(e), +inf for rows that are none or see nothing
  const float* delta;  // D
  const PlanHead* head;
  const int* first;
  const int* last;
  const BwdItem* items;
  int Hkv, group, tok, tile_cap;  // tile_cap: row tiles per kv head in the padded arrays
  int wl, wr;
  float scale, scale_log2;
  unsigned long long wait_limit_ns;
  int inject;
  unsigned* status;
};

// swizzled (128-byte) byte offset of element (row, col) in a [128 rows x 128
// cols] bf16 tile stored as two 64-column atoms
__device__ __forceinline__ uint32_t sw128_off(int row, int col) {
  const int chunk = col >> 6, c = col & 63;
  return chunk * 16384 + (row >> 3) * 1024 + (row & 7) * 128 + ((((c >> 3) ^ (row & 7))) << 4) + ((c & 7) << 1);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// the next item of this CTA into the warp's shared slot; false at the end
__device__ __forceinline__ bool next_item(const Params& p, seq::Walk& w, BwdItem* slot, int lane) {
  if (w.i > w.last) return false;
  __syncwarp();  // the previous item has been read
  if (lane < 3) reinterpret_cast<int4*>(slot)[lane] = reinterpret_cast<const int4*>(p.items + w.i)[lane];
  __syncwarp();
  seq::walk_step(w);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    seq_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const __grid_constant__ OutMaps out, const Params p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + C::kOffCtl);
  // (by a shuffle, so that the compiler knows the warp's index to be uniform)
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int wg = warp >> 2;
  const uint64_t LIM = p.wait_limit_ns;
  volatile uint32_t* abort_flag = &ctl.abort;

  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle atoms need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
    return;
  }
  // rows of the Q and dO tiles past the last whole token are never loaded, but
  // summed over by dK and dV
  for (int i = threadIdx.x; i < 3 * C::kTile / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    ctl.abort = 0;
    mbar_init(&ctl.kv_full, 1);
    mbar_init(&ctl.kv_seen, 1);
    mbar_init(&ctl.kv_empty, 2);  // the products that read it, and the tail warp
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_seen[i], 1);
      mbar_init(&ctl.q_empty[i], 2);
      mbar_init(&ctl.vec_full[i], 1);
      mbar_init(&ctl.vec_empty[i], 8);
    }
    mbar_init(&ctl.do_full, 1);
    mbar_init(&ctl.do_seen, 1);
    mbar_init(&ctl.do_empty, 2);
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.p_full, 8);
    mbar_init(&ctl.dp_full, 1);
    mbar_init(&ctl.ds_full, 8);
    mbar_init(&ctl.dq_full, 1);
    mbar_init(&ctl.dq_empty, 4);
    mbar_init(&ctl.acc_full, 1);
    mbar_init(&ctl.acc_empty, 4);
    mbar_init(&ctl.drain, 1);
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();    // the plan, LSE and D rows, the zeroed accumulator
  grid_dep_launch();  // the last kernel may start (and wait) meanwhile
  const uint32_t tmem = ctl.tmem_base;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sDO = smem + C::kOffDO;
  uint8_t* sDs = smem + C::kOffDs;
  float* sVec = reinterpret_cast<float*>(smem + C::kOffVec);
  seq::Walk wk = seq::walk_begin(p.head, p.first, p.last);
  const BwdItem& I = ctl.cur[warp];

  if (wg <= 1) {
    // ------------------------------------------------------------ compute
    // Registers (launch: 512 threads x 128): compute 8 warps x 136, drain
    // 4 x 144, the others 4 x 96 = the 65536 of the SM.
    setmaxnreg_inc<136>();
    const int row = ((warp & 3) << 5) + lane;  // key row within the tile
    const int c0 = (warp >> 2) * 64;           // first query column of this warp
    const uint32_t t_lane = tmem + (uint32_t(warp & 3) << 21);
    const float sl = p.scale_log2;
    uint32_t ph_s = 0, ph_dp = 0;
    bool ok = true;
    int g = 0;  // step counter across items
    while (ok && next_item(p, wk, &ctl.cur[warp], lane)) {
      const bool kvalid = row < I.nkey();  // keys past the sequence's end: P = 0
      for (int st = 0; st < I.n && ok; ++st, ++g) {
        const int t0 = (I.i0 + st) * p.tok;  // first token of the row tile
        const int vs = g & 1;
        const float* lse2 = sVec + vs * 256 + c0;
        const float* dlt = sVec + vs * 256 + 128 + c0;
        if (!seq::warp_wait(&ctl.vec_full[vs], (g >> 1) & 1, abort_flag, LIM)) { ok = false; break; }
        if (!seq::warp_wait(&ctl.s_full, ph_s, abort_flag, LIM)) { ok = false; break; }
        ph_s ^= 1;
        tc_fence_after();
        float pv[64];
        {
          uint32_t x[64];
          tmem_ld32(t_lane + C::kColS + c0, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
          tmem_ld32(t_lane + C::kColS + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse2 + c);
            const uint64_t y0 = ffma2(pack2(u2f(x[c]), u2f(x[c + 1])), pack2(sl, sl), pack2(-l4.x, -l4.y));
            const uint64_t y1 = ffma2(pack2(u2f(x[c + 2]), u2f(x[c + 3])), pack2(sl, sl), pack2(-l4.z, -l4.w));
            float a0, a1, a2, a3;
            unpack2(y0, a0, a1);
            unpack2(y1, a2, a3);
            pv[c] = ex2_mufu(a0);
            pv[c + 1] = ex2_mufu(a1);
            pv[c + 2] = ex2_mufu(a2);
            pv[c + 3] = ex2_mufu(a3);
          }
        }
        // Token t sees the tile's key `row` iff row - rel - wr <= t <= row -
        // rel + wl, rel the place of token 0 among the tile's keys; a token
        // is `group` columns. Masked in a pass of its own, on tiles that
        // cross a bound and for keys past the end.
        const int rt = I.rel + t0;  // place of the row tile's first token
        const bool need_mask = (p.wr >= 0 && 127 - p.wr > rt) || (p.wl >= 0 && p.wl < rt + p.tok - 1);
        if (need_mask || !kvalid) {
          int lo = 0, hi = 64;  // columns [lo, hi) of this warp see the key
          if (p.wr >= 0) lo = max(0, min(max(row - rt - p.wr, 0), p.tok) * p.group - c0);
          if (p.wl >= 0) hi = min(64, min(max(row - rt + p.wl + 1, 0), p.tok) * p.group - c0);
          // (columns past the last whole token have P = 0 by their LSE)
          const uint32_t span = kvalid ? uint32_t(max(hi - lo, 0)) : 0u;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (uint32_t(c - lo) >= span) pv[c] = 0.0f;
        }
        {
          // P (and dS below) to bf16, nearest even, the type that the products
          // take beside bf16 dO, Q and K: off by at most 2^-8 of each term
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(pv[2 * c], pv[2 * c + 1]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            tmem_st16(t_lane + C::kColS + p_store_col(c0) + c * 16, *reinterpret_cast<uint32_t(*)[16]>(&pk[c * 16]));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full);

        // dS^T = P^T o (dP^T - D), 32 columns per TMEM load
        if (!seq::warp_wait(&ctl.dp_full, ph_dp, abort_flag, LIM)) { ok = false; break; }
        ph_dp ^= 1;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
          uint32_t gg[32];
          tmem_ld32(t_lane + C::kColDP + c0 + h, gg);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 4; ++u) {  // 8 columns = one 16-byte unit
            const int c = h + u * 8;
            const float4 d0 = *reinterpret_cast<const float4*>(dlt + c);
            const float4 d1 = *reinterpret_cast<const float4*>(dlt + c + 4);
            const float dd[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              float s0, s1;
              unpack2(fmul2(pack2(pv[c + e], pv[c + e + 1]),
                            fadd2(pack2(u2f(gg[u * 8 + e]), u2f(gg[u * 8 + e + 1])), pack2(-dd[e], -dd[e + 1]))),
                      s0, s1);
              pk[e >> 1] = pack_bf16x2(s0, s1);
            }
            *reinterpret_cast<uint4*>(sDs + sw128_off(row, c0 + c)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.ds_full);
          mbar_arrive(&ctl.vec_empty[vs]);
        }
      }
    }
  } else if (wg == 2) {
    // ------------------------------------------------ dQ drain + epilogue
    setmaxnreg_inc<144>();
    const int wq = warp & 3;
    const uint32_t t_lane = tmem + (uint32_t(wq) << 21);
    uint8_t* stg = smem + C::kOffStg + wq * 8192;
    uint32_t ph_dq = 0, nacc = 0;
    bool ok = true;
    while (ok && next_item(p, wk, &ctl.cur[warp], lane)) {
      for (int st = 0; st < I.n && ok; ++st) {
        const int arow = (I.kvh * p.tile_cap + I.tiles + I.i0 + st) * 128 + wq * 32;  // this warp's accumulator rows
        if (!seq::warp_wait(&ctl.dq_full, ph_dq, abort_flag, LIM)) { ok = false; break; }
        ph_dq ^= 1;
        tc_fence_after();
        // dQ: lane = query row of the tile, column = d. Staged as
        // 128-byte-swizzled boxes of [32 rows][32 d] fp32, two at a time, and
        // added into the accumulator by TMA reductions; the buffer is
        // rewritten once the previous reductions have read it.
        uint32_t v[D];
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          tmem_ld32(t_lane + C::kColDP + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.dq_empty);
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int b2 = 0; b2 < 2; ++b2) {
            const int db = half * 2 + b2;  // d block of 32
            uint8_t* box = stg + b2 * 4096 + lane * 128;
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(box + ((u ^ (lane & 7)) << 4)) =
                  make_uint4(v[db * 32 + 4 * u], v[db * 32 + 4 * u + 1], v[db * 32 + 4 * u + 2], v[db * 32 + 4 * u + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2)
              tma_reduce_add_4d(&out.acc, stg + b2 * 4096, (half * 2 + b2) * 32, arow, 0, 0);
            bulk_commit();
          }
        }
      }
      if (!ok) break;
      // epilogue: dV, dK rows of the key tile (lane = key row)
      const int nkey = I.nkey();
      const bool mine = wq * 32 + lane < nkey;
      __nv_bfloat16* rows[2] = {p.dv, p.dk};
      const size_t row_off = (size_t(I.krow + wq * 32 + lane) * p.Hkv + I.kvh) * D;
      if (I.n == 0) {  // no row sees the tile (a part has tiles)
        if (mine)
          for (int c = 0; c < 2 * (D / 8); ++c)
            reinterpret_cast<uint4*>(rows[c & 1] + row_off)[c >> 1] = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!seq::warp_wait(&ctl.acc_full, nacc & 1, abort_flag, LIM)) { ok = false; break; }
      ++nacc;
      tc_fence_after();
      const bool part = (I.count & seq::kPart) != 0;
      const int slot = 2 * int(blockIdx.x) + ((I.count & seq::kCont) ? 0 : 1);
      const bool whole = wq * 32 + 32 <= nkey;  // the warp's 32 rows are all keys of the sequence
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {  // dV, then dK
        const uint32_t col = t == 0 ? C::kColDV : C::kColDK;
        const float mul = t == 0 ? 1.0f : p.scale;
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {  // 64 columns at a time
          uint32_t v[64];
          tmem_ld32(t_lane + col + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld32(t_lane + col + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_wait_ld();
          if (t == 1 && h == D / 64 - 1) {  // the next item's products may overwrite the accumulators
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.acc_empty);
          }
          if (lane == 0) bulk_wait_read_all();  // earlier reductions and stores have read the staging
          __syncwarp();
          if (part) {
            // two boxes of [32 rows][32 d] fp32
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2) {
              uint8_t* box = stg + b2 * 4096 + lane * 128;
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const int c = b2 * 32 + 4 * u;
                *reinterpret_cast<uint4*>(box + ((u ^ (lane & 7)) << 4)) =
                    make_uint4(f2u(u2f(v[c]) * mul), f2u(u2f(v[c + 1]) * mul), f2u(u2f(v[c + 2]) * mul),
                               f2u(u2f(v[c + 3]) * mul));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int b2 = 0; b2 < 2; ++b2)
                tma_store_4d(&out.part, stg + b2 * 4096, (h * 2 + b2) * 32, wq * 32, t, slot);
              bulk_commit();
            }
          } else {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(u2f(v[2 * c]) * mul, u2f(v[2 * c + 1]) * mul);
            if (whole) {
              // one box of [32 rows][64 d] bf16
              uint8_t* box = stg + lane * 128;
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<uint4*>(box + ((u ^ (lane & 7)) << 4)) =
                    make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_4d(t == 0 ? &out.dv : &out.dk, stg, h * 64, I.kvh, I.krow + wq * 32, 0);
                bulk_commit();
              }
            } else if (mine) {  // rows of another sequence follow
              uint4* dst = reinterpret_cast<uint4*>(rows[t] + row_off + h * 64);
#pragma unroll
              for (int u = 0; u < 8; ++u) dst[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // everything is written when the kernel ends
  } else {
    setmaxnreg_dec<96>();
  }
  if (warp == 12) {
    // ------------------------------------------------------- TMA producer
    bool ok = true, inject = p.inject == 1;  // test hook: the first Q tile is never delivered
    int g = 0, nkv = 0;
    const uint32_t row_bytes = uint32_t(p.tok * p.group * D * 2);
    while (ok && next_item(p, wk, &ctl.cur[warp], lane)) {
      const int n = I.n;
      if (n == 0) continue;
      ok = seq::warp_wait(&ctl.kv_empty, (nkv & 1) ^ 1, abort_flag, LIM);
      if (!ok) break;
      ++nkv;
      if (elect_one()) {
        mbar_arrive_expect_tx(&ctl.kv_full, 2 * C::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(sK + c * 16384, &tmK, &ctl.kv_full, c * 64, I.kvh, I.krow, 0);
          tma_load_4d(sV + c * 16384, &tmV, &ctl.kv_full, c * 64, I.kvh, I.krow, 0);
        }
      }
      const int kvh = I.kvh, token0 = I.q0 + I.i0 * p.tok;
      const size_t row0 = (size_t(kvh) * p.tile_cap + I.tiles + I.i0) * 128;
      for (int st = 0; st < n; ++st, ++g) {
        const int qs = g & 1, token = token0 + st * p.tok;
        ok = seq::warp_wait(&ctl.q_empty[qs], ((g >> 1) & 1) ^ 1, abort_flag, LIM);
        if (!ok) break;
        if (inject) {
          inject = false;
        } else if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.q_full[qs], row_bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sQ + qs * C::kTile + c * 16384, &tmQ, &ctl.q_full[qs], c * 64, 0, token, kvh);
        }
        // LSE/D rows before dO: the compute warps need them as soon as S is
        // ready, while dO (one slot) waits for the previous dV
        ok = seq::warp_wait(&ctl.vec_empty[qs], ((g >> 1) & 1) ^ 1, abort_flag, LIM);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.vec_full[qs], 1024);
          bulk_load(sVec + qs * 256, p.lse2 + row0 + size_t(st) * 128, 512, &ctl.vec_full[qs]);
          bulk_load(sVec + qs * 256 + 128, p.delta + row0 + size_t(st) * 128, 512, &ctl.vec_full[qs]);
        }
        ok = seq::warp_wait(&ctl.do_empty, (g & 1) ^ 1, abort_flag, LIM);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ctl.do_full, row_bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sDO + c * 16384, &tmDO, &ctl.do_full, c * 64, 0, token, kvh);
        }
      }
    }
    if (*abort_flag) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks the role and an elected lane issues.
    constexpr uint32_t idSS = idesc_bf16_f32(128, 128, 0, 0);  // S^T, dP^T
    constexpr uint32_t idAcc = idesc_bf16_f32(128, D, 0, 1);   // dV, dK
    constexpr uint32_t idDQ = idesc_bf16_f32(128, D, 1, 1);
    const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aQ = smem_u32(sQ), aDO = smem_u32(sDO), aDs = smem_u32(sDs);
    bool ok = true;
    uint32_t ph_p = 0, ph_ds = 0, ph_dqe = 0;
    int g = 0, nkv = 0;
    const uint32_t kK = sdesc_lo(aK, 16), kV = sdesc_lo(aV, 16), kQ = sdesc_lo(aQ, 16);  // K-major
    const uint32_t kDO = sdesc_lo(aDO, 16), kDs = sdesc_lo(aDs, 16);
    const uint32_t mQ = sdesc_lo(aQ, 16384), mDO = sdesc_lo(aDO, 16384);  // MN-major
    const uint32_t mK = sdesc_lo(aK, 16384), mDs = sdesc_lo(aDs, 16384);
    auto wait = [&](uint64_t* bar, uint32_t phase) -> bool { return seq::warp_wait(bar, phase, abort_flag, LIM); };
    // [128 x 128] = A B^T, K = D
    auto issue_kmajor = [&](uint32_t d_col, uint32_t a0, uint32_t b0, uint64_t* done) {
      tc_fence_after();
      if (!elect_one()) return;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
        mma_ss_lo(tmem + d_col, sdesc_step(a0, ko), sdesc_step(b0, ko), idSS, kk > 0);
      }
      mma_commit(done);
    };
    // Q of a step (its rows past the sequence's end zeroed, if it has such)
    auto wait_q = [&](int step, bool tail) -> bool {
      return wait(&ctl.q_full[step & 1], (step >> 1) & 1) && (!tail || wait(&ctl.q_seen[step & 1], (step >> 1) & 1));
    };
    while (ok && next_item(p, wk, &ctl.cur[warp], lane)) {
      const int n = I.n;
      if (n == 0) continue;
      // the step with rows past the sequence's end, if any
      const int tail_st = I.qlen % p.tok != 0 ? I.qlen / p.tok - I.i0 : -1;
      ok = wait(&ctl.kv_full, nkv & 1) && (I.nkey() == 128 || wait(&ctl.kv_seen, nkv & 1));
      if (!ok) break;
      ++nkv;
      // step st issues S^T of step st + 1; the item begins a step early, with its first S^T alone
      for (int st = -1; st < n; ++st) {
        if (st >= 0) {
          ok = wait(&ctl.do_full, g & 1) && (st != tail_st || wait(&ctl.do_seen, g & 1));
          if (ok && g > 0) {
            ok = wait(&ctl.dq_empty, ph_dqe);
            ph_dqe ^= 1;
          }
          if (!ok) break;
          issue_kmajor(C::kColDP, kV, kDO, &ctl.dp_full);  // dP^T = V dO^T
          ok = wait(&ctl.p_full, ph_p);
          ph_p ^= 1;
          // before the first dV of a later item overwrites the accumulators,
          // the previous item's dK/dV must have been read out of TMEM
          if (ok && st == 0 && nkv > 1) ok = wait(&ctl.acc_empty, (nkv - 2) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // dV += P^T dO   (P^T in TMEM, dO MN-major)
              mma_ts_lo(tmem + C::kColDV, tmem + C::kColS + p_operand_col(kk), sdesc_step(mDO, kk * 2048),
                        idAcc, (st > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&ctl.do_empty);
          }
        }
        if (st + 1 < n) {
          const int nx = st < 0 ? g : g + 1;
          ok = wait_q(nx, st + 1 == tail_st);
          if (!ok) break;
          issue_kmajor(C::kColS, kK, sdesc_step(kQ, (nx & 1) * C::kTile), &ctl.s_full);  // S^T = K Q^T
        }
        if (st < 0) continue;
        ok = wait(&ctl.ds_full, ph_ds);
        ph_ds ^= 1;
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t mQcur = sdesc_step(mQ, (g & 1) * C::kTile);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // dK += dS^T Q   (dS^T K-major, Q MN-major)
            const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_ss_lo(tmem + C::kColDK, sdesc_step(kDs, ko), sdesc_step(mQcur, kk * 2048), idAcc,
                      (st > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(&ctl.q_empty[g & 1]);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // dQ = dS K  (both MN-major): lane = query row, column = d
            mma_ss_lo(tmem + C::kColDP, sdesc_step(mDs, kk * 2048), sdesc_step(mK, kk * 2048), idDQ, kk > 0);
          mma_commit(&ctl.dq_full);
          if (st + 1 == n) {
            mma_commit(&ctl.acc_full);  // dK, dV of this item are complete
            mma_commit(&ctl.kv_empty);  // K, V of this item no longer read
          }
        }
        ++g;
      }
    }
    if (*abort_flag) {
      if (elect_one()) mma_commit(&ctl.drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&ctl.drain), 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
    }
  } else if (warp == 14) {
    // ----------------------------------------------------------- tail rows
    // Follows every load, so that it cannot lose count of their phases; zeroes
    // rows [from, 128) of the tiles that need it (a row is 128 bytes of each
    // 64-column chunk; the swizzle stays within it).
    auto zero_rows = [&](uint8_t* tile, int from) {
      for (int i = from * 8 + lane; i < 128 * 8; i += 32)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint4*>(tile + c * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return seq::warp_wait(bar, parity, abort_flag, LIM); };
    auto done = [&](uint64_t* seen, uint64_t* empty) {
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(seen);
        mbar_arrive(empty);
      }
    };
    bool ok = true;
    int g = 0, nkv = 0;
    while (ok && next_item(p, wk, &ctl.cur[warp], lane)) {
      if (I.n == 0) continue;
      ok = wait(&ctl.kv_full, nkv & 1);
      if (!ok) break;
      ++nkv;
      if (I.nkey() < 128) {
        zero_rows(sK, I.nkey());
        zero_rows(sV, I.nkey());
        fence_proxy_async_smem();
      }
      done(&ctl.kv_seen, &ctl.kv_empty);
      for (int st = 0; st < I.n; ++st, ++g) {
        const int left = I.qlen - (I.i0 + st) * p.tok;  // tokens from this row tile on
        const bool tail = left < p.tok;
        ok = wait(&ctl.q_full[g & 1], (g >> 1) & 1);
        if (!ok) break;
        if (tail) {
          zero_rows(sQ + (g & 1) * C::kTile, left * p.group);
          fence_proxy_async_smem();
        }
        done(&ctl.q_seen[g & 1], &ctl.q_empty[g & 1]);
        ok = wait(&ctl.do_full, g & 1);
        if (!ok) break;
        if (tail) {
          zero_rows(sDO, left * p.group);
          fence_proxy_async_smem();
        }
        done(&ctl.do_seen, &ctl.do_empty);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && ctl.abort) atomicOr(p.status, kDevTimeout);
}

// The sequence and row of a padded row: tile index within the kv head's
// tiles, row in the tile. token < 0: no row of a sequence.
struct RowAt {
  int token, head;
};
__device__ __forceinline__ RowAt row_at(const int* cu_q, const int* tstart, int B, int tok, int group, int kvh, int tile,
                                        int r) {
  const int b = seq::find_seq(tstart, B, 1, tile);
  const int t = r / group, i = (tile - tstart[b]) * tok + t;
  const int q0 = cu_q[b];
  RowAt x;
  x.head = kvh * group + (r - t * group);
  x.token = t < tok && i < cu_q[b + 1] - q0 ? q0 + i : -1;
  return x;
}

// D_i = sum_c dO_ic O_ic and LSE * log2(e) of every padded row (+inf and 0
// where a row is none or sees nothing, so that its probabilities recompute to
// 0), and zeroes for the accumulator rows. A warp takes 16 rows of a row tile
// at a time, 16 bytes of O and dO per lane and piece.
// Up to kOwnSeqs sequences, every block finds the sequences' first row tiles by
// itself, and the kernel runs beside the plan (a training step on 2115 tokens
// 47.9 -> 45.3 us); the tiles of larger batches are the plan's.
constexpr int kOwnSeqs = 256;
template <int D>
__global__ void __launch_bounds__(256)
    seq_pre_kernel(const __nv_bfloat16* o, const __nv_bfloat16* dout, const float* lse, const seq::Lens L,
                   const seq::BwdSide side, const int* plan_tstart, const PlanHead* head, float* lse2, float* delta,
                   float* acc, int Hkv, int group, int tile_cap) {
  __shared__ int own[kOwnSeqs + 1];
  __shared__ int sums[8];
  const int B = L.B, tok = side.tok, total_q = L.total_q;
  const int* const cu_q = L.cu_q;
  const int* tstart = own;
  grid_dep_launch();  // the main kernel may start its set-up meanwhile
  if (B <= kOwnSeqs) {
    const int b = threadIdx.x, w = b >> 5;
    seq::Seq s;
    const bool ok = b >= B || seq::seq_at(L, b, s);
    int at = b < B && ok ? side.row_tiles(s) : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, at, m);
      if ((b & 31) >= m) at += x;
    }
    if ((b & 31) == 31) sums[w] = at;
    const bool bad = __syncthreads_or(!ok);
    for (int i = 0; i < w; ++i) at += sums[i];
    own[b + 1] = at;
    if (b == 0) own[0] = 0;
    __syncthreads();
    if (bad) {  // lengths that the tensors cannot hold
      grid_dep_wait();
      return;
    }
  } else {
    grid_dep_wait();  // the plan
    if (head->bad) return;
    tstart = plan_tstart;
  }
  constexpr int TPR = D / 8;          // lanes per row
  constexpr int RPP = 32 / TPR;       // rows per pass of the warp
  constexpr int kPass = 16 / RPP;     // passes per 16 rows
  const int lane = threadIdx.x & 31;
  const int part = lane % TPR, sub = lane / TPR;
  const int Hq = Hkv * group, tiles = tstart[B];
  const long long n_groups = 8LL * Hkv * tiles;
  for (long long grp = (1LL * blockIdx.x * blockDim.x + threadIdx.x) >> 5; grp < n_groups;
       grp += (1LL * gridDim.x * blockDim.x) >> 5) {
    const int tile = int((grp >> 3) % tiles), kvh = int((grp >> 3) / tiles), r0 = int(grp & 7) * 16;
    // lane t < 16: row r0 + t
    const RowAt x = row_at(cu_q, tstart, B, tok, group, kvh, tile, r0 + (lane & 15));
    const long long at = x.token >= 0 ? 1LL * x.token * Hq + x.head : -1;
    uint4 a[kPass], g[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const long long row = __shfl_sync(0xffffffffu, at, i * RPP + sub);
      a[i] = g[i] = make_uint4(0, 0, 0, 0);
      if (row >= 0) {
        a[i] = *reinterpret_cast<const uint4*>(o + row * D + part * 8);
        g[i] = *reinterpret_cast<const uint4*>(dout + row * D + part * 8);
      }
    }
    const size_t arow = (size_t(kvh) * tile_cap + tile) * 128 + r0;
    float4* z = reinterpret_cast<float4*>(acc + arow * D);
#pragma unroll
    for (int i = 0; i < 16 * D / 4 / 32; ++i) z[i * 32 + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float mine = 0.0f;  // lane t < 16: D of row t
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a[i]);
      const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g[i]);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 fa = __bfloat1622float2(a2[e]), fg = __bfloat1622float2(g2[e]);
        s = fmaf(fa.x, fg.x, s);
        s = fmaf(fa.y, fg.y, s);
      }
#pragma unroll
      for (int m = TPR / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      const float v = __shfl_sync(0xffffffffu, s, (lane % RPP) * TPR);
      if (lane / RPP == i) mine = v;
    }
    if (lane < 16) {
      float l = INFINITY;
      if (x.token >= 0) {
        const float y = lse[size_t(x.head) * total_q + x.token];
        if (y != -INFINITY) l = y * 1.4426950408889634f;
      }
      lse2[arow + lane] = l;
      delta[arow + lane] = x.token >= 0 ? mine : 0.0f;
    }
  }
  if (B <= kOwnSeqs) grid_dep_wait();  // the main kernel waits for this one, and needs the plan
}

// dq[token, head, :] = bf16(scale * accumulator row), then the sums of the
// parts' dV and dK (their scale already applied) in the workers' order.
template <int D>
__global__ void __launch_bounds__(256)
    seq_post_kernel(const float* acc, const float* part, const Cut* cuts, const int* last, const int* cu_q,
                    const int* tstart, const PlanHead* head, __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, int B,
                    int Hkv, int group, int tok, int tile_cap, float scale, int G) {
  grid_dep_wait();  // launched while the main kernel may still run
  if (head->bad) return;
  constexpr int TPR = D / 8, RPP = 32 / TPR;  // lanes per row, rows per pass of a warp
  const int lane = threadIdx.x & 31, sub = lane / TPR, c8 = (lane % TPR) * 8;
  const int Hq = Hkv * group, tiles = tstart[B];
  const long long warp = (1LL * blockIdx.x * blockDim.x + threadIdx.x) >> 5, n_warps = (1LL * gridDim.x * blockDim.x) >> 5;
  const long long n_groups = 8LL * Hkv * tiles;
  for (long long grp = warp; grp < n_groups; grp += n_warps) {
    const int tile = int((grp >> 3) % tiles), kvh = int((grp >> 3) / tiles), r0 = int(grp & 7) * 16;
    const RowAt x = row_at(cu_q, tstart, B, tok, group, kvh, tile, r0 + (lane & 15));
    const long long at = x.token >= 0 ? 1LL * x.token * Hq + x.head : -1;
    const float* src = acc + ((size_t(kvh) * tile_cap + tile) * 128 + r0 + sub) * D + c8;
    float4 v[16 / RPP][2];
#pragma unroll
    for (int i = 0; i < 16 / RPP; ++i) {
      v[i][0] = __ldcs(reinterpret_cast<const float4*>(src + i * RPP * D));
      v[i][1] = __ldcs(reinterpret_cast<const float4*>(src + i * RPP * D) + 1);
    }
#pragma unroll
    for (int i = 0; i < 16 / RPP; ++i) {
      const long long row = __shfl_sync(0xffffffffu, at, i * RPP + sub);
      if (row >= 0)
        *reinterpret_cast<uint4*>(dq + row * D + c8) =
            make_uint4(pack_bf16x2(v[i][0].x * scale, v[i][0].y * scale), pack_bf16x2(v[i][0].z * scale, v[i][0].w * scale),
                       pack_bf16x2(v[i][1].x * scale, v[i][1].y * scale), pack_bf16x2(v[i][1].z * scale, v[i][1].w * scale));
    }
  }
  if (head->step != 1) return;  // no unit is divided
  // a warp pass: RPP rows of one cut's dV or dK
  const long long n_pass = 1LL * G * 2 * (128 / RPP);
  for (long long i = warp; i < n_pass; i += n_warps) {
    const int r = int(i % (128 / RPP)) * RPP + sub, t = int(i / (128 / RPP)) & 1;
    const Cut k = cuts[i / (2 * (128 / RPP))];
    if (k.c1 < 0 || r >= k.count) continue;
    float f[8] = {};
    for (int c = k.c0; c <= k.c1; ++c) {
      if (last[c] < 0) continue;  // a worker without a share
      const size_t slot = c == k.c0 ? 2 * c + 1 : 2 * c;
      const float4* src = reinterpret_cast<const float4*>(part + ((slot * 2 + t) * 128 + r) * D + c8);
      const float4 a = src[0], b = src[1];
      f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
      f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
    }
    __nv_bfloat16* dst = (t == 0 ? dv : dk) + (size_t(k.row0 + r) * Hkv + k.kvh) * D + c8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

// the workspace, carved from `base` (null: its size alone)
struct Space {
  seq::Plan<BwdItem> plan;
  float *acc, *lse2, *delta, *part;
  int tile_cap;
  size_t bytes;
};
Space carve(uint8_t* base, const SeqProblem& pb, int G) {
  Space s{};
  seq::Carver c{base, 0};
  long long units = pb.total_k / 128 + pb.B, tiles = seq_row_tiles(pb);
  if (units > pb.total_k) units = pb.total_k;
  if (tiles < 1) tiles = 1;  // (tensor maps need a row)
  s.tile_cap = int(tiles);
  s.plan = seq::carve_plan<BwdItem>(c, pb.B, units, pb.Hkv, G);
  const size_t rows = size_t(pb.Hkv) * tiles * 128;
  s.lse2 = c.take<float>(rows);
  s.delta = c.take<float>(rows);
  s.part = c.take<float>(size_t(2) * G * 2 * 128 * pb.d);
  s.acc = c.take<float>(rows * pb.d);
  s.bytes = c.at;
  return s;
}

template <int D>
cudaError_t launch_t(const SeqProblem& pb, const void* o, const float* lse, const void* dout, void* dq, void* dk,
                     void* dv, cudaStream_t stream) {
  using C = Cfg<D>;
  const int G = std::min(num_sms(), seq::kMaxWorkers);
  const int group = pb.Hq / pb.Hkv, tok = 128 / group;
  unsigned* status = status_word();
  if (status == nullptr) return cudaErrorLaunchFailure;
  auto kern = seq_bwd_kernel<D>;
  constexpr int smem = C::kOffCtl + int(sizeof(Ctl));
  static_assert(smem <= 232448, "shared memory of a CTA");
  static seq::SmemLimit limit;
  cudaError_t e = limit.set(kern, smem);
  if (e != cudaSuccess) return e;
  void* ws = nullptr;
  cudaMemPool_t pool = workspace_pool();
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, carve(nullptr, pb, G).bytes, pool, stream) != cudaSuccess)
    return cudaErrorMemoryAllocation;
  const Space sp = carve(static_cast<uint8_t*>(ws), pb, G);
  CUtensorMap mq, mk, mv, mdo;
  OutMaps out;
  bool ok = true;
  // a tensor without rows: a map over the workspace that no load uses
  auto rows_of = [&](const void* base, int total) { return total > 0 ? base : ws; };
  auto q_map = [&](CUtensorMap* m, const void* base, long long stride) {
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), uint64_t(std::max(pb.total_q, 1)), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(stride) * 2, uint64_t(group) * D * 2};
    const uint32_t box[4] = {64, uint32_t(group), uint32_t(tok), 1};
    ok = ok && encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, rows_of(base, pb.total_q), dims, strides, box,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto k_map = [&](CUtensorMap* m, const void* base, long long stride, uint32_t rows) {
    const uint64_t n = uint64_t(std::max(pb.total_k, 1));
    const uint64_t dims[4] = {uint64_t(D), uint64_t(pb.Hkv), n, 1};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(stride) * 2, uint64_t(stride) * 2 * n};
    const uint32_t box[4] = {64, 1, rows, 1};
    ok = ok && encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, rows_of(base, pb.total_k), dims, strides, box,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  };
  q_map(&mq, pb.q, pb.q_stride);
  q_map(&mdo, dout, 1LL * pb.Hq * D);
  k_map(&mk, pb.k, pb.k_stride, 128);
  k_map(&mv, pb.v, pb.v_stride, 128);
  k_map(&out.dk, dk, 1LL * pb.Hkv * D, 32);
  k_map(&out.dv, dv, 1LL * pb.Hkv * D, 32);
  {
    const uint64_t rows = uint64_t(pb.Hkv) * sp.tile_cap * 128;
    const uint64_t dims[4] = {uint64_t(D), rows, 1, 1};
    const uint64_t strides[3] = {uint64_t(D) * 4, rows * D * 4, rows * D * 4};
    const uint32_t box[4] = {32, 32, 1, 1};
    ok = ok && encode_tiled(&out.acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, sp.acc, dims, strides, box,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  }
  {
    const uint64_t dims[4] = {uint64_t(D), 128, 2, uint64_t(2) * G};
    const uint64_t strides[3] = {uint64_t(D) * 4, uint64_t(D) * 128 * 4, uint64_t(D) * 256 * 4};
    const uint32_t box[4] = {32, 32, 1, 1};
    ok = ok && encode_tiled(&out.part, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, sp.part, dims, strides, box,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  }
  e = ok ? cudaSuccess : cudaErrorInvalidValue;
  seq::PlanArgs<seq::BwdSide> a{};
  a.L = seq::Lens{pb.cu_q, pb.cu_k, nullptr, pb.B, pb.total_q, pb.total_k, 0};
  a.P = sp.plan;
  a.side = seq::BwdSide{tok, pb.window_left, pb.window_right};
  a.Hkv = pb.Hkv;
  a.G = G;
  a.status = status;
  Params p{};
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.lse2 = sp.lse2;
  p.delta = sp.delta;
  p.head = sp.plan.head;
  p.first = sp.plan.first;
  p.last = sp.plan.last;
  p.items = sp.plan.items;
  p.Hkv = pb.Hkv;
  p.group = group;
  p.tok = tok;
  p.tile_cap = sp.tile_cap;
  p.wl = pb.window_left;
  p.wr = pb.window_right;
  p.scale = pb.scale;
  p.scale_log2 = pb.scale * 1.4426950408889634f;
  const DebugCfg dc = debug_cfg();
  p.wait_limit_ns = dc.wait_limit_ns;
  p.inject = dc.inject;
  p.status = status;
  if (e == cudaSuccess) {
    seq::plan_kernel<seq::BwdSide><<<1, seq::kPlanThreads, 0, stream>>>(a);
    e = cudaGetLastError();
  }
  // the kernels after it start while the one before ends, and wait for it
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.stream = stream;
  lc.attrs = pdl;
  lc.numAttrs = 1;
  // 16 rows per warp at a time
  const long long groups = 8LL * pb.Hkv * sp.tile_cap;
  const unsigned wide = unsigned(std::min<long long>((groups + 7) / 8, 8LL * G));
  if (e == cudaSuccess) {
    lc.gridDim = dim3(wide);
    lc.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&lc, seq_pre_kernel<D>, static_cast<const __nv_bfloat16*>(o),
                           static_cast<const __nv_bfloat16*>(dout), lse, a.L, a.side,
                           static_cast<const int*>(sp.plan.tstart), static_cast<const PlanHead*>(sp.plan.head), sp.lse2,
                           sp.delta, sp.acc, pb.Hkv, group, sp.tile_cap);
  }
  if (dc.ev_begin) cudaEventRecord(dc.ev_begin, stream);
  if (e == cudaSuccess) {
    lc.gridDim = dim3(G);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&lc, kern, mq, mk, mv, mdo, out, p);
  }
  if (dc.ev_end) cudaEventRecord(dc.ev_end, stream);
  if (e == cudaSuccess) {
    lc.gridDim = dim3(unsigned(8 * G));  // the parts' sums want warps where there are few rows
    lc.blockDim = dim3(256);
    lc.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&lc, seq_post_kernel<D>, static_cast<const float*>(sp.acc), static_cast<const float*>(sp.part),
                           static_cast<const Cut*>(sp.plan.cuts), static_cast<const int*>(sp.plan.last), pb.cu_q,
                           static_cast<const int*>(sp.plan.tstart), static_cast<const PlanHead*>(sp.plan.head),
                           static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv),
                           pb.B, pb.Hkv, group, tok, sp.tile_cap, pb.scale, G);
  }
  const cudaError_t f = cudaFreeAsync(ws, stream);
  return e != cudaSuccess ? e : f;
}

}  // namespace seqb

cudaError_t launch_seq_bwd(const SeqProblem& pb, const void* o, const float* lse, const void* dout, void* dq, void* dk,
                           void* dv, cudaStream_t stream) {
  return pb.d == 128 ? seqb::launch_t<128>(pb, o, lse, dout, dq, dk, dv, stream)
                     : seqb::launch_t<64>(pb, o, lse, dout, dq, dk, dv, stream);
}

}  // namespace fa
