// Attention over sequences of different lengths on sm_103a, bf16 operands
// (d = 64 or 128): packed sequences (fa_fwd_varlen) and new tokens over a
// paged cache (fa_fwd_paged).
//
// Method: as the dense forward (fa_fwd_pipeline.cuh): tiles of 128 rows meet
// tiles of 128 keys, online softmax with a running maximum and sum, S, P and
// O in tensor memory, tcgen05.mma for both products. What differs is how
// work is cut:
//   * rows are (token, query head of the group) pairs, so a tile of 128 rows
//     holds 128 / group tokens and the query heads of a group share every key
//     tile: one new token of a group of 4 reads its cache once, not 4 times;
//   * the lengths are on the device, so a planning kernel of one block lays
//     out the work there: a list of items sorted by key tiles (longest first)
//     that the CTAs take in snake order, or, where that would leave CTAs idle
//     (few rows over long caches), the same rows' key tiles laid end to end
//     and divided evenly between the CTAs, whose partial results (m, l, O)
//     a last kernel joins in a fixed order;
//   * an item of one row tile (one token, short chunks, a sequence's last
//     rows) has no second row tile to overlap its softmax with: its two
//     stages take alternate key tiles and are joined in the epilogue;
//   * pages: a 128-key tile is 128 / box TMA boxes, each from the page that
//     the table names, box the largest power of two dividing the page size
//     (at most 128); lane i of the producer warp issues box i.
//   * the last key tile of a sequence reads on into what follows it (another
//     sequence, a page's unused rows). Scores are masked by a select; V rows
//     past the end are zeroed in shared memory by a warp of its own before
//     the product reads them, as 0 * NaN would stay NaN.
//
//   CTA = 512 threads, persistent (one per SM):
//     warps 0-3 / 4-7  softmax of stage 0 / 1   (one thread per row)
//     warps 8-11       correction + epilogue
//     warp 12 TMA producer, warp 13 MMA issuer, warp 14 V tail, 15 idle
//   TMEM as in the dense forward: S/P of the stages at columns 0 and 128, O
//   at 256 and 256 + d.
#include <cuda_bf16.h>

#include <cmath>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_seq_plan.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace seq {

constexpr int kThreads = 512;
constexpr uint32_t kOCol0 = 256;
constexpr float kTau = 8.0f;  // rescale threshold (log2 units), as in the dense forward

// --------------------------------------------------------------------------
// main kernel
// --------------------------------------------------------------------------
struct Params {
  __nv_bfloat16* o;
  float* lse;          // [Hq, total_q]
  const PlanHead* head;
  const int* first;
  const int* last;
  const FwdItem* items;
  const Cut* cuts;
  float* part_o;       // [2 G][2 * 128][D] partial O
  float2* part_ml;     // [2 G][2 * 128] their (m, l)
  const int* table;    // paged: [B, max_pages]
  int Hq, group, tok, total_q;
  int num_pages, page_size, box_rows, max_pages;
  float scale_log2;    // |scale| * log2(e)
  uint32_t neg_s;      // 1 for a negative scale
  int wl, wr;
  unsigned long long wait_limit_ns;
  int inject;
  unsigned* status;
};

template <int D>
struct Tiles {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kStgBytes = 16384;  // 4 warps x [32 rows x 64 columns] bf16
  static constexpr int kSmemDyn = (2 + kSlots) * kTileBytes + kStgBytes + 1024;
};
constexpr int kMaxSlots = 8;

struct __align__(8) Ctl {
  uint64_t q_full[2], q_empty;
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  uint64_t s_full[2], p_full[2], alpha_full[2], o_ready[2], o_full[2], stats_full[2], stats_empty[2];
  uint64_t seen[kMaxSlots];  // the tail warp is done with the slot's tile (its rows past the sequence's end are zeroed)
  uint64_t drain;
  float alpha[2][128];
  float stat_l[2][128];
  float stat_m[2][128];
  uint32_t tmem_base;
  uint32_t abort;
};

// An item as the roles see it: key tile t of the item is taken by
//   key mode: stage t & 1, as its step t >> 1;
//   else    : both stages, stage s while a[s] <= t < a[s] + n[s].
struct Work {
  FwdItem it;
  int n[2], a[2];
  int rows[2];  // rows of each stage (key mode: both have the same)
  bool key;
};

// the next item of this CTA, false when there is none
__device__ __forceinline__ bool walk_next(const Params& p, Walk& w, Work& x) {
  if (w.i > w.last) return false;
  const int4* src = reinterpret_cast<const int4*>(p.items + w.i);
  const int4 u = src[0], v = src[1];
  x.it.q0 = u.x;
  x.it.count = u.y;
  x.it.kvh = u.z;
  x.it.kbase = u.w;
  x.it.klen = v.x;
  x.it.pos = v.y;
  x.it.kt = v.z;
  x.it.nt = v.w;
  walk_step(w);
  x.key = (x.it.count & kKeyMode) != 0;
  const int ntok = x.it.ntok(), nt = x.it.nt;
  if (x.key) {
    x.rows[0] = x.rows[1] = ntok * p.group;
    x.n[0] = (nt + 1) >> 1;
    x.n[1] = nt >> 1;
    x.a[0] = x.a[1] = 0;
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int mine = s == 0 ? p.tok : ntok - p.tok;
      x.rows[s] = mine * p.group;
      const int pos = x.it.pos + s * p.tok;
      const int lo = p.wl >= 0 ? max(0, pos - p.wl) : 0;
      const int hi = p.wr >= 0 ? min(x.it.klen - 1, pos + mine - 1 + p.wr) : x.it.klen - 1;
      // this stage's tiles within the item's
      const int t0 = max(lo >> 7, x.it.kt), t1 = min(hi >> 7, x.it.kt + nt - 1);
      x.n[s] = hi < lo || t1 < t0 ? 0 : t1 - t0 + 1;
      x.a[s] = x.n[s] > 0 ? t0 - x.it.kt : 0;
    }
  }
  return true;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Tiles<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::kTileBytes;
  uint8_t* sStg = sKV + C::kSlots * C::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  volatile uint32_t* abort_flag = &ctl.abort;
  const uint64_t LIM = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    ctl.abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.q_full[s], 1);
      mbar_init(&ctl.s_full[s], 1);
      mbar_init(&ctl.p_full[s], 4);
      mbar_init(&ctl.alpha_full[s], 4);
      mbar_init(&ctl.o_ready[s], 4);
      mbar_init(&ctl.o_full[s], 1);
      mbar_init(&ctl.stats_full[s], 4);
      mbar_init(&ctl.stats_empty[s], 4);
    }
    mbar_init(&ctl.q_empty, 1);
    mbar_init(&ctl.drain, 1);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&ctl.kv_full[i], 1);
      mbar_init(&ctl.seen[i], 1);
      mbar_init(&ctl.kv_empty[i], 2);  // the products that read it, and the tail warp
    }
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 12 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();    // the plan
  grid_dep_launch();  // the joining kernel may start (and wait) meanwhile
  const uint32_t tmem = ctl.tmem_base;
  Walk wk = walk_begin(p.head, p.first, p.last);
  Work x;

  if (wg <= 1) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<176>();
    const int s = wg;
    const int row = ((warp & 3) << 5) + lane;
    const uint32_t t_s = tmem + (uint32_t(warp & 3) << 21) + uint32_t(s * 128);
    const float sl = p.scale_log2;
    const int row_tok = row / p.group;
    uint32_t ph_s = 0, ph_se = 0;
    bool ok = true;
    while (ok && walk_next(p, wk, x)) {
      const int n = x.n[s];
      if (n == 0) continue;
      const bool mine = ((warp & 3) << 5) < x.rows[s];  // the warp has rows
      const int stage_pos = x.it.pos + (x.key ? 0 : s * p.tok);
      const int pos = stage_pos + row_tok;  // this row's place among the keys
      const int pos_l = stage_pos + (x.key ? x.it.ntok() : s == 0 ? p.tok : x.it.ntok() - p.tok) - 1;  // the last row's
      const int kt0 = x.it.kt + (x.key ? s : x.a[s]), dkt = x.key ? 2 : 1;
      const int klen = x.it.klen;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = 0; j < n; ++j) {
        if (!mbar_wait_bounded(&ctl.s_full[s], ph_s, abort_flag, LIM)) { ok = false; break; }
        ph_s ^= 1;
        if (!mine) {
          if (lane == 0) {
            mbar_arrive(&ctl.alpha_full[s]);
            mbar_arrive(&ctl.p_full[s]);
          }
          continue;
        }
        tc_fence_after();
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
        tmem_wait_ld();
        const int kb = (kt0 + j * dkt) * 128;
        // masked where the tile reaches past the keys or crosses a bound of some row
        if (kb + 127 >= klen || (p.wr >= 0 && kb + 127 > stage_pos + p.wr) || (p.wl >= 0 && kb < pos_l - p.wl)) {
          int hi = klen - kb;  // columns [lo, hi) are visible
          int lo = 0;
          if (p.wr >= 0) hi = min(hi, pos + p.wr + 1 - kb);
          if (p.wl >= 0) lo = max(lo, pos - p.wl - kb);
          const uint32_t span = uint32_t(max(hi - lo, 0));
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (uint32_t(c - lo) >= span) v[c] = f2u(-INFINITY);
        }
        float mA = -INFINITY, mB = -INFINITY, mC = -INFINITY, mD = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          mA = fmax3(mA, u2f(v[c]), u2f(v[c + 1]));
          mB = fmax3(mB, u2f(v[c + 2]), u2f(v[c + 3]));
          mC = fmax3(mC, u2f(v[c + 4]), u2f(v[c + 5]));
          mD = fmax3(mD, u2f(v[c + 6]), u2f(v[c + 7]));
        }
        const float mx = fmaxf(fmaxf(mA, mB), fmaxf(mC, mD));
        const float m_cand = fmaxf(m_run, mx * sl);
        const float m_new = (m_cand > m_run + kTau) ? m_cand : m_run;
        const float m_use = (m_new == -INFINITY) ? 0.0f : m_new;
        const float alpha = ex2_mufu(m_run - m_use);
        ctl.alpha[s][row] = alpha;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.alpha_full[s]);
        const uint64_t sl2 = pack2(sl, sl);
        const uint64_t nm2 = pack2(-m_use, -m_use);
        uint64_t acc0 = 0, acc1 = 0, acc2 = 0, acc3 = 0;
        uint32_t pk[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const uint64_t y = ffma2(pack2(u2f(v[2 * c]), u2f(v[2 * c + 1])), sl2, nm2);
          float a, b;
          unpack2(y, a, b);
          a = ex2_mufu(a);
          b = ex2_mufu(b);
          const uint64_t pr = pack2(a, b);
          if ((c & 3) == 0) acc0 = c == 0 ? pr : fadd2(acc0, pr);
          if ((c & 3) == 1) acc1 = c == 1 ? pr : fadd2(acc1, pr);
          if ((c & 3) == 2) acc2 = c == 2 ? pr : fadd2(acc2, pr);
          if ((c & 3) == 3) acc3 = c == 3 ? pr : fadd2(acc3, pr);
          // P to bf16 (nearest even), the type the P V product takes beside a
          // bf16 V: off by at most 2^-9 of each probability's binade top; the row sum
          // keeps the 32-bit values
          pk[c] = pack_bf16x2(a, b);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(t_s + c * 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[c * 16]));
        const uint64_t acc = fadd2(fadd2(acc0, acc1), fadd2(acc2, acc3));
        float la, lb;
        unpack2(acc, la, lb);
        l_run = fmaf(l_run, alpha, la + lb);
        m_run = m_new;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[s]);
      }
      if (!ok) break;
      if (!mbar_wait_bounded(&ctl.stats_empty[s], ph_se ^ 1, abort_flag, LIM)) { ok = false; break; }
      ph_se ^= 1;
      ctl.stat_l[s][row] = l_run;
      ctl.stat_m[s][row] = m_run;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.stats_full[s]);
    }
  } else if (wg == 2) {
    // ------------------------------------------------ correction + epilogue
    setmaxnreg_dec<80>();
    const int wq = warp & 3;
    const int row = (wq << 5) + lane;
    const uint32_t t_lane = tmem + (uint32_t(wq) << 21) + kOCol0;
    const int row_tok = row / p.group, row_head = row - row_tok * p.group;
    uint32_t ph_a[2] = {0, 0}, ph_st[2] = {0, 0}, ph_of[2] = {0, 0};
    bool ok = true;
    while (ok && walk_next(p, wk, x)) {
      const int steps = x.key ? x.n[0] : x.it.nt;
      for (int j = 0; j < steps && ok; ++j) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (j < x.a[s] || j >= x.a[s] + x.n[s]) continue;
          if (!mbar_wait_bounded(&ctl.alpha_full[s], ph_a[s], abort_flag, LIM)) { ok = false; break; }
          ph_a[s] ^= 1;
          if ((wq << 5) < x.rows[s] && j > x.a[s]) {
            const float a = ctl.alpha[s][row];
            if (__any_sync(0xffffffffu, a < 1.0f)) {
              tc_fence_after();
              const uint32_t t_o = t_lane + uint32_t(s * D);
              const uint64_t a2 = pack2(a, a);
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(t_o + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float lo, hi;
                  unpack2(fmul2(pack2(u2f(v[i]), u2f(v[i + 1])), a2), lo, hi);
                  v[i] = f2u(lo);
                  v[i + 1] = f2u(hi);
                }
                tmem_st32(t_o + c * 32, v);
              }
              tmem_wait_st();
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.o_ready[s]);
        }
      }
      if (!ok) break;
      // epilogue
      const int ntok = x.it.ntok();
      const bool part = (x.it.count & kPart) != 0;
      const int slot = 2 * int(blockIdx.x) + ((x.it.count & kCont) ? 0 : 1);
      // the stages' rows are the same rows in key mode: one pass over both
      const int passes = x.key || ntok <= p.tok ? 1 : 2;
#pragma unroll 1
      for (int s = 0; s < passes && ok; ++s) {
        const int s1 = x.key ? 1 : s;  // the stages joined by this pass: s and s1
        const bool valid = row < x.rows[s];
        // packed (token, head) row of o, and its place in lse; -1 for none
        const int token = x.it.q0 + s * p.tok + row_tok;
        const int head = x.it.kvh * p.group + row_head;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if ((t != s && t != s1) || x.n[t] == 0) continue;
          if (!mbar_wait_bounded(&ctl.stats_full[t], ph_st[t], abort_flag, LIM)) { ok = false; break; }
          ph_st[t] ^= 1;
          l[t] = ctl.stat_l[t][row];
          m[t] = ctl.stat_m[t][row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.stats_empty[t]);
          if (!mbar_wait_bounded(&ctl.o_full[t], ph_of[t], abort_flag, LIM)) { ok = false; break; }
          ph_of[t] ^= 1;
        }
        if (!ok) break;
        tc_fence_after();
        // join: weights of the two stages' O (a stage without tiles has m = -inf, l = 0)
        const float mj = fmaxf(m[0], m[1]), mu = mj == -INFINITY ? 0.0f : mj;
        const float w0 = m[0] == -INFINITY ? 0.0f : ex2_mufu(m[0] - mu);
        const float w1 = m[1] == -INFINITY ? 0.0f : ex2_mufu(m[1] - mu);
        const float lj = l[0] * w0 + l[1] * w1;
        const float inv = part ? 1.0f : lj == 0.0f ? 0.0f : 1.0f / lj;
        const bool has0 = x.n[0] > 0 && s == 0, has1 = x.n[1] > 0 && s1 == 1;
        const float f0 = w0 * inv, f1 = w1 * inv;
        if ((wq << 5) < x.rows[s]) {
          // columns [16 c, 16 c + 16) of the joined O (inv is 1 for a part)
          auto columns = [&](int c, float (&f)[16]) {
            uint32_t v[16], u[16];
            if (has0) tmem_ld16(t_lane + c * 16, v);
            if (has1) tmem_ld16(t_lane + D + c * 16, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              f[i] = (has0 ? u2f(v[i]) * f0 : 0.0f) + (has1 ? u2f(u[i]) * f1 : 0.0f);
          };
          if (part) {
            const size_t at = size_t(slot) * 256 + s * 128 + row;
            if (valid) p.part_ml[at] = make_float2(mj, lj);
            float* dst = p.part_o + at * D;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float f[16];
              columns(c, f);
              if (valid) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  *reinterpret_cast<float4*>(dst + c * 16 + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
              }
            }
          } else {
            uint8_t* stg = sStg + wq * 4096;
            const int orow = valid ? token * p.Hq + head : -1;
#pragma unroll 1
            for (int hf = 0; hf < D / 64; ++hf) {
              __syncwarp();  // the previous half has been read
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float f[16];
                columns(hf * 4 + c, f);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  *reinterpret_cast<uint4*>(stg + lane * 128 + (((c * 2 + i) ^ (lane & 7)) << 4)) =
                      make_uint4(pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                 pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7]));
              }
              __syncwarp();
              // 8 lanes write a row's 128 bytes, 4 rows at a time
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                const int to = __shfl_sync(0xffffffffu, orow, r);
                const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                if (to >= 0) *reinterpret_cast<uint4*>(p.o + size_t(to) * D + hf * 64 + (lane & 7) * 8) = w;
              }
            }
            if (valid)
              p.lse[size_t(head) * p.total_q + token] = lj == 0.0f ? -INFINITY : (mu + __log2f(lj)) * 0.69314718055994531f;
          }
        }
        tc_fence_before();
      }
    }
  } else {
    setmaxnreg_dec<80>();
  }
  if (warp == 12) {
    // ------------------------------------------------------- TMA producer
    uint32_t kv_it = 0, ph_qe = 0;
    bool first = true, ok = true, injected = false;
    const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
    // paged: lane -> (box of the tile, 64-column chunk)
    const int n_box = PAGED ? 128 / p.box_rows : 1;
    const int box = lane % n_box, chunk = lane / n_box;
    while (ok && walk_next(p, wk, x)) {
      const int nt = x.it.nt;
      if (nt == 0) continue;
      if (!first) {
        ok = mbar_wait_bounded(&ctl.q_empty, ph_qe, abort_flag, LIM);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ph_qe ^= 1;
      }
      first = false;
      if (lane == 0) {
        const uint32_t q_bytes = uint32_t(p.tok * p.group * D * 2);
        for (int s = 0; s < 2; ++s) {
          if (x.n[s] == 0 || (s == 1 && x.key)) continue;
          mbar_arrive_expect_tx(&ctl.q_full[s], q_bytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d_hint(sQ + s * C::kTileBytes + c * 16384, &tmQ, &ctl.q_full[s], c * 64, 0, x.it.q0 + s * p.tok,
                             x.it.kvh, pol_q);
        }
      }
      // K runs d tiles ahead of V: K(0..d-1), then V(t), K(t + d)
      const int d = x.key ? 2 : 1;
      auto load = [&](const CUtensorMap* m, int t) -> bool {
        const uint32_t slot = kv_it % C::kSlots;
        const bool r = __all_sync(0xffffffffu, mbar_wait_bounded(&ctl.kv_empty[slot], ((kv_it / C::kSlots) & 1) ^ 1,
                                                                  abort_flag, LIM));
        if (!r) return false;
        ++kv_it;
        if (p.inject == 1 && !injected) {  // test hook: never deliver this tile
          injected = true;
          return true;
        }
        uint8_t* dst = sKV + slot * C::kTileBytes;
        const int key0 = (x.it.kt + t) * 128;
        if constexpr (PAGED) {
          // boxes that begin before the sequence's end
          const int boxes = min(n_box, (x.it.klen - key0 + p.box_rows - 1) / p.box_rows);
          if (lane == 0) mbar_arrive_expect_tx(&ctl.kv_full[slot], uint32_t(boxes * p.box_rows * D * 2));
          __syncwarp();
          if (chunk < C::kChunks && box < boxes) {
            const int key = key0 + box * p.box_rows;
            const int pg = key / p.page_size;
            int page = p.table[size_t(x.it.kbase) * p.max_pages + pg];
            if (page < 0 || page >= p.num_pages) {  // no such page: its keys read as zeros, and the caller is told
              atomicOr(p.status, kDevBadArg);
              page = p.num_pages;
            }
            tma_load_4d_hint(dst + chunk * 16384 + box * p.box_rows * 128, m, &ctl.kv_full[slot], chunk * 64, x.it.kvh,
                             key - pg * p.page_size, page, pol_kv);
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.kv_full[slot], C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d_hint(dst + c * 16384, m, &ctl.kv_full[slot], c * 64, x.it.kvh, x.it.kbase + key0, 0, pol_kv);
        }
        return true;
      };
      for (int t = 0; t < d && t < nt && ok; ++t) ok = load(&tmK, t);
      for (int t = 0; t < nt && ok; ++t) {
        ok = load(&tmV, t);
        if (ok && t + d < nt) ok = load(&tmK, t + d);
      }
    }
    if (*abort_flag) {
      // let copies already in flight land before shared memory is released
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0) | (p.neg_s << 13);
      constexpr uint32_t idPV = idesc_bf16_f32(128, D, 0, 1);
      const uint32_t dq = sdesc_lo(smem_u32(sQ), 16), dk = sdesc_lo(smem_u32(sKV), 16),
                     dv = sdesc_lo(smem_u32(sKV), 16384);
      uint32_t kv_it = 0, ph_q[2] = {0, 0}, ph_p[2] = {0, 0}, ph_o[2] = {0, 0};
      bool ok = true;
      auto wait_kv = [&](uint32_t& slot) -> bool {
        slot = kv_it % C::kSlots;
        const bool r = mbar_wait_bounded(&ctl.kv_full[slot], (kv_it / C::kSlots) & 1, abort_flag, LIM);
        ++kv_it;
        return r;
      };
      // S of stage s = Q (tile qt) K^T
      auto issue_s = [&](int s, int qt, uint32_t kslot) {
        const uint32_t a0 = sdesc_step(dq, qt * C::kTileBytes), b0 = sdesc_step(dk, kslot * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss_lo(tmem + uint32_t(s * 128), sdesc_step(a0, ko), sdesc_step(b0, ko), idS, kk > 0);
        }
        mma_commit(&ctl.s_full[s]);
      };
      // O of stage s (+)= P V
      auto issue_pv = [&](int s, uint32_t vslot, bool acc) {
        const uint32_t b0 = sdesc_step(dv, vslot * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo(tmem + kOCol0 + uint32_t(s * D), tmem + uint32_t(s * 128) + kk * 8, sdesc_step(b0, kk * 2048), idPV,
                    (acc || kk > 0) ? 1u : 0u);
      };
      auto wait_po = [&](int s) -> bool {
        if (!mbar_wait_bounded(&ctl.p_full[s], ph_p[s], abort_flag, LIM)) return false;
        ph_p[s] ^= 1;
        if (!mbar_wait_bounded(&ctl.o_ready[s], ph_o[s], abort_flag, LIM)) return false;
        ph_o[s] ^= 1;
        tc_fence_after();
        return true;
      };
      while (ok && walk_next(p, wk, x)) {
        const int nt = x.it.nt;
        if (nt == 0) continue;
        // the sequence's last key tile, if partly filled, has V rows to be zeroed first
        const bool tail = (x.it.klen & 127) != 0 && x.it.kt + nt - 1 == (x.it.klen - 1) >> 7;
        uint32_t kslot = 0, vslot = 0, v_phase = 0;
        auto wait_v = [&](int t) -> bool {
          v_phase = (kv_it / C::kSlots) & 1;
          if (!wait_kv(vslot)) return false;
          if (!tail || t != nt - 1) return true;
          // (every tile passes the tail warp, so this slot's count of phases is the ring's)
          return mbar_wait_bounded(&ctl.seen[vslot], v_phase, abort_flag, LIM);
        };
        for (int s = 0; s < 2 && ok; ++s) {
          if (x.n[s] == 0 || (s == 1 && x.key)) continue;
          ok = mbar_wait_bounded(&ctl.q_full[s], ph_q[s], abort_flag, LIM);
          ph_q[s] ^= 1;
        }
        if (!ok) break;
        if (x.key) {
          for (int t = 0; t < 2 && t < nt && ok; ++t) {
            ok = wait_kv(kslot);
            if (!ok) break;
            tc_fence_after();
            issue_s(t, 0, kslot);
            mma_commit(&ctl.kv_empty[kslot]);
          }
          if (nt <= 2) mma_commit(&ctl.q_empty);
          for (int t = 0; t < nt && ok; ++t) {
            const int s = t & 1;
            ok = wait_v(t) && wait_po(s);
            if (!ok) break;
            issue_pv(s, vslot, t > 1);
            if (t + 2 >= nt) mma_commit(&ctl.o_full[s]);
            mma_commit(&ctl.kv_empty[vslot]);
            if (t + 2 < nt) {
              ok = wait_kv(kslot);
              if (!ok) break;
              tc_fence_after();
              issue_s(s, 0, kslot);
              mma_commit(&ctl.kv_empty[kslot]);
              if (t + 3 == nt) mma_commit(&ctl.q_empty);
            }
          }
          continue;
        }
        auto active = [&](int s, int t) { return t >= x.a[s] && t < x.a[s] + x.n[s]; };
        ok = wait_kv(kslot);
        if (!ok) break;
        tc_fence_after();
        for (int s = 0; s < 2; ++s)
          if (active(s, 0)) issue_s(s, s, kslot);
        mma_commit(&ctl.kv_empty[kslot]);
        if (nt == 1) mma_commit(&ctl.q_empty);
        for (int t = 0; t < nt && ok; ++t) {
          const bool nxt = t + 1 < nt;
          ok = wait_v(t) && (!nxt || wait_kv(kslot));
          if (!ok) break;
          const int last_v = active(1, t) ? 1 : 0;  // the last stage that reads V(t)
          for (int s = 0; s < 2; ++s) {
            if (active(s, t)) {
              ok = wait_po(s);
              if (!ok) break;
              issue_pv(s, vslot, t > x.a[s]);
              if (t == x.a[s] + x.n[s] - 1) mma_commit(&ctl.o_full[s]);
              if (s == last_v) mma_commit(&ctl.kv_empty[vslot]);
            }
            if (nxt && active(s, t + 1)) {
              tc_fence_after();
              issue_s(s, s, kslot);
            }
          }
          if (!ok) break;
          if (nxt) mma_commit(&ctl.kv_empty[kslot]);
          if (t + 2 == nt) mma_commit(&ctl.q_empty);
        }
      }
      if (*abort_flag) {
        // drain the tensor pipe before TMEM is released
        mma_commit(&ctl.drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&ctl.drain), 0) && globaltimer_ns() - t0 < 100000000ull) {
        }
      }
    }
  } else if (warp == 14) {
    // ---------------------------------------------------------- V tail rows
    // (follows every ring slot, so that it cannot lose count of their phases)
    uint32_t kv_it = 0;
    bool ok = true;
    while (ok && walk_next(p, wk, x)) {
      const int nt = x.it.nt;
      const int fill = x.it.klen & 127;
      const bool tail = fill != 0 && x.it.kt + nt - 1 == (x.it.klen - 1) >> 7;
      for (int e = 0; e < 2 * nt; ++e, ++kv_it) {
        const uint32_t slot = kv_it % C::kSlots;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&ctl.kv_full[slot], (kv_it / C::kSlots) & 1, abort_flag, LIM));
        if (!ok) break;
        if (tail && e == 2 * nt - 1) {  // an item's last ring entry is its last V tile
          uint8_t* dst = sKV + slot * C::kTileBytes;
          // a row is 128 bytes of each chunk (the swizzle stays within it)
          for (int i = fill * 8 + lane; i < 128 * 8; i += 32)
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              *reinterpret_cast<uint4*>(dst + c * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.seen[slot]);
          mbar_arrive(&ctl.kv_empty[slot]);
        }
      }
    }
  }

  // ------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && ctl.abort) atomicOr(p.status, kDevTimeout);
}

// The parts of the rows whose keys were divided between workers, joined in
// the workers' order: O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
// Block (c, y): cut c, every gridDim.y-th group of rows; a warp per row.
template <int D>
__global__ void __launch_bounds__(256) seq_join_kernel(const Params p) {
  grid_dep_wait();
  if (p.head->n_items == 0 || p.head->split == 0) return;
  const Cut k = p.cuts[blockIdx.x];
  if (k.c1 < 0) return;
  const int lane = threadIdx.x & 31;
  const int ntok = k.count, rows = ntok * p.group;
  const int per_stage = p.tok * p.group;
  constexpr int V = D / 32;  // columns per lane
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 8) {
    const int s = r >= per_stage ? 1 : 0;
    const size_t at = size_t(s) * 128 + (r - s * per_stage);
    float m = -INFINITY, l = 0.0f, o[V] = {};
    for (int c = k.c0; c <= k.c1; ++c) {
      if (p.last[c] < 0) continue;  // a worker without a share (fewer key tiles than workers)
      const size_t i = size_t(c == k.c0 ? 2 * c + 1 : 2 * c) * 256 + at;
      const float2 ml = p.part_ml[i];
      if (ml.y == 0.0f) continue;  // no key of this part is visible to the row: its O was not written
      const float mn = fmaxf(m, ml.x);
      const float wa = m == -INFINITY ? 0.0f : ex2_mufu(m - mn), wb = ex2_mufu(ml.x - mn);
      float f[V];
      if constexpr (V == 4) {
        const float4 t = *reinterpret_cast<const float4*>(p.part_o + i * D + lane * V);
        f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
      } else {
        const float2 t = *reinterpret_cast<const float2*>(p.part_o + i * D + lane * V);
        f[0] = t.x; f[1] = t.y;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = o[e] * wa + f[e] * wb;
      l = l * wa + ml.y * wb;
      m = mn;
    }
    const int tok = r / p.group, head = k.kvh * p.group + (r - tok * p.group), token = k.row0 + tok;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat16* dst = p.o + (size_t(token) * p.Hq + head) * D + lane * V;
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
    }
    if (lane == 0)
      p.lse[size_t(head) * p.total_q + token] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
  }
}

// --------------------------------------------------------------------------
// launch
// --------------------------------------------------------------------------
// the workspace, carved from `base` (null: its size alone)
struct Space {
  Plan<FwdItem> plan;
  float* part_o;
  float2* part_ml;
  size_t bytes;
};
Space carve(uint8_t* base, const SeqProblem& pb, int G, int tok) {
  Space s{};
  Carver c{base, 0};
  // a sequence of n tokens has ceil(n / (2 tok)) units
  long long units = pb.total_q / (2 * tok) + pb.B;
  if (units > pb.total_q) units = pb.total_q;
  s.plan = carve_plan<FwdItem>(c, pb.B, units, pb.Hkv, G);
  s.part_ml = c.take<float2>(size_t(2) * G * 256);
  s.part_o = c.take<float>(size_t(2) * G * 256 * pb.d);
  s.bytes = c.at;
  return s;
}

template <int D, bool PAGED>
cudaError_t launch_t(const SeqProblem& pb, void* o, float* lse, cudaStream_t stream) {
  using C = Tiles<D>;
  const int G = num_sms();
  const int group = pb.Hq / pb.Hkv, tok = 128 / group;
  Params p{};
  // q: rows (token, head of the group), `tok` tokens to a tile
  CUtensorMap mq, mk, mv;
  {
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), uint64_t(pb.total_q), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(pb.q_stride) * 2, uint64_t(group) * D * 2};
    const uint32_t box[4] = {64, uint32_t(group), uint32_t(tok), 1};
    if (!encode_tiled(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pb.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if constexpr (PAGED) {
    p.box_rows = 128;
    while (pb.page_size % p.box_rows != 0) p.box_rows /= 2;  // 16 at least
    if (!make_bshd_map(&mk, pb.k, pb.num_pages, pb.page_size, pb.Hkv, D, p.box_rows) ||
        !make_bshd_map(&mv, pb.v, pb.num_pages, pb.page_size, pb.Hkv, D, p.box_rows))
      return cudaErrorInvalidValue;
  } else {
    // no keys at all: maps over q that no load uses
    const void* kp[2] = {pb.total_k > 0 ? pb.k : pb.q, pb.total_k > 0 ? pb.v : pb.q};
    const long long st[2] = {pb.total_k > 0 ? pb.k_stride : pb.q_stride, pb.total_k > 0 ? pb.v_stride : pb.q_stride};
    const uint64_t rows = pb.total_k > 0 ? uint64_t(pb.total_k) : 1;
    CUtensorMap* maps[2] = {&mk, &mv};
    for (int i = 0; i < 2; ++i) {
      const uint64_t dims[4] = {uint64_t(D), uint64_t(pb.Hkv), rows, 1};
      const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(st[i]) * 2, uint64_t(st[i]) * 2 * rows};
      const uint32_t box[4] = {64, 1, 128, 1};
      if (!encode_tiled(maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, kp[i], dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    }
  }
  p.status = status_word();
  if (p.status == nullptr) return cudaErrorLaunchFailure;
  auto kern = seq_fwd_kernel<D, PAGED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemDyn);
  if (e != cudaSuccess) return e;
  void* ws = nullptr;
  cudaMemPool_t pool = workspace_pool();
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, carve(nullptr, pb, G, tok).bytes, pool, stream) != cudaSuccess)
    return cudaErrorMemoryAllocation;
  const Space sp = carve(static_cast<uint8_t*>(ws), pb, G, tok);
  PlanArgs<FwdSide> a{};
  a.L = Lens{pb.cu_q, pb.cu_k, pb.lens_k, pb.B, pb.total_q, pb.total_k, 1LL * pb.max_pages * pb.page_size};
  a.P = sp.plan;
  a.side = FwdSide{tok, pb.window_left, pb.window_right, pb.page_table != nullptr ? 1 : 0};
  a.Hkv = pb.Hkv;
  a.G = G;
  a.part_cost = 8;
  a.status = p.status;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.head = sp.plan.head;
  p.first = sp.plan.first;
  p.last = sp.plan.last;
  p.items = sp.plan.items;
  p.cuts = sp.plan.cuts;
  p.part_o = sp.part_o;
  p.part_ml = sp.part_ml;
  p.table = pb.page_table;
  p.Hq = pb.Hq;
  p.group = group;
  p.tok = tok;
  p.total_q = pb.total_q;
  p.num_pages = pb.num_pages;
  p.page_size = pb.page_size;
  p.max_pages = pb.max_pages;
  p.scale_log2 = fabsf(exp_scale_log2(pb.scale));
  p.neg_s = pb.scale < 0.0f ? 1u : 0u;
  p.wl = pb.window_left;
  p.wr = pb.window_right;
  const DebugCfg dc = debug_cfg();
  p.wait_limit_ns = dc.wait_limit_ns;
  p.inject = dc.inject;
  plan_kernel<FwdSide><<<1, kPlanThreads, 0, stream>>>(a);
  e = cudaGetLastError();
  // the kernels after it start while the one before ends, and wait for it
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(G);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = C::kSmemDyn;
  lc.stream = stream;
  lc.attrs = pdl;
  lc.numAttrs = 1;
  if (dc.ev_begin) cudaEventRecord(dc.ev_begin, stream);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&lc, kern, mq, mk, mv, p);
  if (dc.ev_end) cudaEventRecord(dc.ev_end, stream);
  if (e == cudaSuccess) {
    lc.gridDim = dim3(G, 8);
    lc.blockDim = dim3(256);
    lc.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&lc, seq_join_kernel<D>, p);
  }
  const cudaError_t f = cudaFreeAsync(ws, stream);
  return e != cudaSuccess ? e : f;
}

}  // namespace seq

cudaError_t launch_seq_fwd(const SeqProblem& pb, void* o, float* lse, cudaStream_t stream) {
  const bool paged = pb.page_table != nullptr;
  if (pb.d == 128)
    return paged ? seq::launch_t<128, true>(pb, o, lse, stream) : seq::launch_t<128, false>(pb, o, lse, stream);
  return paged ? seq::launch_t<64, true>(pb, o, lse, stream) : seq::launch_t<64, false>(pb, o, lse, stream);
}

}  // namespace fa
