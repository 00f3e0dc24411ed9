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
//     that the CTAs take in rounds, or, where that would leave CTAs idle
//     (few rows over long caches), the same rows' key tiles laid end to end
//     and divided evenly between the CTAs, whose partial results (m, l, O)
//     a last kernel joins in a fixed order (fa_seq_plan.cuh);
//   * an item of one row tile (one token, short chunks, a sequence's last
//     rows) has no second row tile to overlap its softmax with: its two
//     stages take alternate key tiles and are joined in the epilogue;
//   * pages: a 128-key tile is 128 / box TMA boxes, each from the page that
//     the table names, box the largest power of two dividing the page size
//     (at most 128); lane i of a producer warp looks box i up.
//   * the last key tile of a sequence reads on into what follows it (another
//     sequence, a page's unused rows). Scores are masked by a select; V rows
//     past the end are zeroed in shared memory, by the warp that loads V,
//     before the product reads them, as 0 * NaN would stay NaN.
//
//   CTA = 512 threads, persistent (one per SM):
//     warps 0-3 / 4-7  softmax of stage 0 / 1 (a thread per row)
//     warps 8-11       correction (O rescaled when a row's maximum grows) and epilogue
//     warps 12 and 14 TMA producers (Q and K, V), 13 MMA issuer, 15 work items
//   TMEM as in the dense forward: S/P of the stages at columns 0 and 128, O
//   at 256 and 256 + d. (At d = 64 there is room for a P apart from its S, so
//   that S is issued a step ahead; measured slower, 16384 causal tokens 1.15
//   -> 1.22 ms: the two stages' softmax then run in step.)
//
// What bounds it, measured:
//   d = 128, long sequences: the tensor pipe. One causal sequence of 16384
//     tokens, 32 query and 8 kv heads: 1.29 ms, 1710 TFLOP/s, 0.89 of the
//     measured bf16 matrix product rate (the dense forward: 1.64 ms).
//   d = 64: the softmax's latency. The same sequence takes 1.15 ms (dense 1.42);
//     the schedulers issue in 47 % of the cycles, tensor pipe 40 %, exponentials
//     41 %. (A thread spills 12 bytes; at d = 128 none.)
//   single tokens: the cache's bytes. 64 sequences of 300 to 32000 keys, 8 kv
//     heads of 128: 1.70 GB in 258 us, 6.6 TB/s, 0.97 of the measured copy.
//   items of few tiles: 1.3 to 2.3 us between two items, most of it instruction
//     fetch (code that runs once per item is not in the cache) and the first
//     S; with a window and one query head per kv head the first and the last
//     of an item's key tiles, which one stage alone sees; the plan before the
//     first item (11 to 15 us); small calls: the launches (77 tokens: 8 us).
#include <cuda_bf16.h>

#include <algorithm>
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
  int* last;
  const FwdItem* items;  // null: few items, every CTA finds its own (self_plan)
  Cut* cuts;
  Lens L;              // for self-planning CTAs
  FwdSide side;
  int Hkv, max_units;
  float* part_o;       // [2 G][2 * 128][D] partial O
  float2* part_ml;     // [2 G][2 * 128] their (m, l)
  const int* table;    // paged: [B, max_pages]
  int Hq, group, tok, total_q;
  int o_box;           // tokens of a warp's 32 rows, if they are whole tokens (tmO's boxes), else 0
  int num_pages, page_size, box_rows, max_pages;
  float scale_log2;    // |scale| * log2(e)
  uint32_t neg_s;      // 1 for a negative scale
  int wl, wr;
  unsigned long long wait_limit_ns;
  int inject;
  unsigned* status;
  unsigned long long* trace;  // optional pipeline trace
};

// Trace points (fa_trace); a step is the CTA's running key-tile counter (in
// key mode two tiles, one of each stage):
//   MMA         0 tiles loaded, 1+s PV of stage s issued, 3 the next S of both issued
//   softmax s   4+3s S ready, 5+3s alpha published, 6+3s P stored
//   correction  10+s O released for PV
//   epilogue s  12+s O written (step of the item's last tile)
constexpr int kItems = 4;  // ring of work items

template <int D>
struct Tiles {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kStgBytes = 16384;  // O staging: 4 warps x [32 rows x 64 columns] bf16
  static constexpr int kSmemDyn = (2 + kSlots) * kTileBytes + kStgBytes + 1024;
};
constexpr int kMaxSlots = 8;

// bits of the MMA issuer's phases: Q loaded, P stored (a pair each)
constexpr int kPhQ = 0, kPhP = 2;

// An item as the roles see it, laid out by warp 15. Its key tile t is taken by
//   key mode: stage t & 1, as its step t >> 1;
//   else    : both stages, stage s while a[s] <= t < a[s] + n[s].
struct Work {
  int q0, ntok, kvh, kbase, klen, pos, kt, nt;
  int n[2], a[2];
  int rows[2];  // rows of each stage (key mode: both have the same)
  int flags;    // kKeyMode | kPart | kCont; -1: there are no more items
  int fill;     // keys of the last tile if the sequence ends inside it, else 0
};

// Few items: the planning kernel would take a good part of the call, so the
// item warp of every CTA lays the work out by itself (77 tokens, 2 heads: 13.7
// -> 10.1 us; one token of 32 heads over 1000 keys: 22 -> 15 us). Few are
// kFewUnits units and no more items than CTAs, or, over a paged cache,
// kFewRounds times as many, which are then always divided: sorting wants the
// planning kernel, and gains where there are many units of as many keys as
// rows (prompts), not where rows are few (64 single tokens, 512 items: 279 us
// planned and sorted, 259 us here). A batch of more sequences than kFewUnits,
// empty ones then, is planned too: a warp reads their lengths 32 at a time (304
// sequences: 36 us either way, 3000: 81 us here, 39 us planned).
constexpr int kFewUnits = 304, kFewRounds = 4;

struct __align__(16) Ctl {
  FwdItem unit[kFewUnits];
  int cost[kFewUnits + 1];  // cost of the units before
  Work it[kItems];
  uint64_t it_full[kItems], it_empty[kItems];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  uint64_t tail_done[kMaxSlots];  // a V tile that the sequence ends in: loaded, its rows past the end zeroed
  // p_full: P stored (4 softmax warps) and O corrected, or read by the epilogue
  // of the stage's item before (4 correction warps)
  uint64_t s_full[2], p_full[2], alpha_full[2], o_full[2];
  uint64_t stats_full[2], stats_empty[2];
  uint64_t drain;
  float alpha[2][128];
  float stat_l[2][128];
  float stat_m[2][128];
  uint32_t tmem_base;
  uint32_t abort;
};

// The laid-out form of an item: key tiles [kt, kt + nt) of the unit at `src`.
__device__ __forceinline__ Work work_of(const Params& p, const FwdItem* src, int kvh, int flags, int kt, int nt) {
  Work x;
  x.q0 = src->q0;
  x.ntok = src->ntok();
  x.flags = flags;
  x.kvh = kvh;
  x.kbase = src->kbase;
  x.klen = src->klen;
  x.pos = src->pos;
  x.kt = kt;
  x.nt = nt;
  const int end = x.klen & 127;
  x.fill = x.nt > 0 && x.kt + x.nt - 1 == (x.klen - 1) >> 7 ? end : 0;
  if (x.flags & kKeyMode) {
    x.rows[0] = x.rows[1] = x.ntok * p.group;
    x.n[0] = (x.nt + 1) >> 1;
    x.n[1] = x.nt >> 1;
    x.a[0] = x.a[1] = 0;
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int mine = s == 0 ? p.tok : x.ntok - p.tok;
      x.rows[s] = mine * p.group;
      const int pos = x.pos + s * p.tok;
      const int lo = p.wl >= 0 ? max(0, pos - p.wl) : 0;
      const int hi = p.wr >= 0 ? min(x.klen - 1, pos + mine - 1 + p.wr) : x.klen - 1;
      // this stage's tiles within the item's
      const int t0 = max(lo >> 7, x.kt), t1 = min(hi >> 7, x.kt + x.nt - 1);
      x.n[s] = hi < lo || t1 < t0 ? 0 : t1 - t0 + 1;
      x.a[s] = x.n[s] > 0 ? t0 - x.kt : 0;
    }
  }
  return x;
}

// A lane's box of a key tile in a paged cache.
struct Place {
  int page, in_page;
  int boxes;    // of the tile
  bool hidden;  // the box ends before the item's first visible key: its page is not looked up
};

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const Params p) {
  using C = Tiles<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::kTileBytes;
  uint8_t* sStg = sKV + C::kSlots * C::kTileBytes;
  // (by a shuffle, so that the compiler knows the warp's index to be uniform)
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, wg = warp >> 2;
  volatile uint32_t* abort_flag = &ctl.abort;
  const uint64_t LIM = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    ctl.abort = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ctl.it_full[i], 1);
      mbar_init(&ctl.it_empty[i], 15);  // every warp but this one's
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl.q_full[s], 1);
      mbar_init(&ctl.q_empty[s], 1);
      mbar_init(&ctl.s_full[s], 1);
      mbar_init(&ctl.p_full[s], 8);
      mbar_init(&ctl.alpha_full[s], 4);
      mbar_init(&ctl.o_full[s], 1);
      mbar_init(&ctl.stats_full[s], 4);
      mbar_init(&ctl.stats_empty[s], 4);
    }
    mbar_init(&ctl.drain, 1);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&ctl.kv_full[i], 1);
      mbar_init(&ctl.kv_empty[i], 1);
      mbar_init(&ctl.tail_done[i], 1);
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
  // item i of this CTA, or null when there is none (or a wait ran out)
  auto item = [&](int i) -> const Work* {
    if (!warp_wait(&ctl.it_full[i % kItems], (i / kItems) & 1, abort_flag, LIM)) return nullptr;
    const Work* x = &ctl.it[i % kItems];
    return x->flags < 0 ? nullptr : x;
  };
  // by each warp once all its lanes have read the item: warp 15 may then write the next one over it
  auto release = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.it_empty[i % kItems]);
  };

  if (wg <= 1) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<168>();
    const int s = wg, wq = warp & 3;
    const int row = (wq << 5) + lane;
    const uint32_t t_s = tmem + (uint32_t(wq) << 21) + uint32_t(s * 128);  // lane quarter + S columns
    const float sl = p.scale_log2;
    const int row_tok = row / p.group;
    uint32_t ph_s = 0, ph_st = 0;
    int step0 = 0;  // running key-tile counter (trace only)
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Work* const w = item(i);
      if (w == nullptr) break;
      const bool key = (w->flags & kKeyMode) != 0;
      const int step = step0 + w->a[s];
      step0 += key ? w->n[0] : w->nt;
      const int n = w->n[s];
      const bool mine = (wq << 5) < w->rows[s];  // the warp has rows
      float m_run = -INFINITY, l_run = 0.0f;
      if (n > 0) {
        const int stage_pos = w->pos + (key ? 0 : s * p.tok);
        const int pos = stage_pos + row_tok;  // this row's place among the keys
        const int pos_l = stage_pos + (key ? w->ntok : s == 0 ? p.tok : w->ntok - p.tok) - 1;  // the last row's
        const int klen = w->klen;
        const int dkb = key ? 256 : 128;
        int kb = (w->kt + (key ? s : w->a[s])) * 128;  // the tile's first key
        for (int j = 0; j < n; ++j, kb += dkb) {
          if (!warp_wait(&ctl.s_full[s], ph_s, abort_flag, LIM)) { ok = false; break; }
          ph_s ^= 1;
          if (row == 0) trace_stamp(p.trace, step + j, 4 + 3 * s);
          if (!mine) {
            if (lane == 0) {
              if (j > 0) mbar_arrive(&ctl.alpha_full[s]);
              mbar_arrive(&ctl.p_full[s]);
            }
            continue;
          }
          tc_fence_after();
          uint32_t v[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
          tmem_wait_ld();
          // masked where the tile reaches past the keys or crosses a bound of some row
          if (kb + 127 >= klen || (p.wr >= 0 && kb + 127 > stage_pos + p.wr) || (p.wl >= 0 && kb < pos_l - p.wl)) {
            int hi = klen - kb;  // columns [lo, hi) are visible
            int lo = 0;
            if (p.wr >= 0) hi = min(hi, pos + p.wr + 1 - kb);
            if (p.wl >= 0) lo = max(lo, pos - p.wl - kb);
            const uint32_t span = uint32_t(max(hi - lo, 0));
            // only the blocks of 32 columns that some row of the warp does not
            // see whole: code that runs once per item is slow to fetch
#pragma unroll
            for (int b = 0; b < 128; b += 32) {
              if (lo <= b && hi >= b + 32) continue;
#pragma unroll
              for (int c = b; c < b + 32; ++c)
                if (uint32_t(c - lo) >= span) v[c] = f2u(-INFINITY);
            }
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
          if (j > 0) {  // (there is no O to correct before the first)
            ctl.alpha[s][row] = alpha;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.alpha_full[s]);
          }
          if (row == 0) trace_stamp(p.trace, step + j, 5 + 3 * s);
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
            // P to bf16 (nearest even), the type that the P V product takes
            // beside a bf16 V: off by at most 2^-8 of each probability; the row
            // sum keeps the 32-bit values
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
          if (row == 0) trace_stamp(p.trace, step + j, 6 + 3 * s);
          if (lane == 0) mbar_arrive(&ctl.p_full[s]);
        }
        if (!ok) break;
      }
      if (n > 0) {  // the rows' statistics for the epilogue
        if (!warp_wait(&ctl.stats_empty[s], ph_st ^ 1, abort_flag, LIM)) { ok = false; break; }
        ph_st ^= 1;
        ctl.stat_l[s][row] = l_run;
        ctl.stat_m[s][row] = m_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.stats_full[s]);
      }
      release(i);
    }
  } else if (wg == 2) {
    // ------------------------------------------------ correction + epilogue
    setmaxnreg_dec<104>();
    const int wq = warp & 3;
    const int row = (wq << 5) + lane;
    const uint32_t t_lane = tmem + (uint32_t(wq) << 21) + kOCol0;
    uint8_t* stg = sStg + wq * 4096;
    const int row_tok = row / p.group, row_head = row - row_tok * p.group;
    uint32_t ph_a = 0, ph_st = 0, ph_of = 0;  // phases, a bit to each stage
    if (lane == 0) {  // O of both stages may be written
      mbar_arrive(&ctl.p_full[0]);
      mbar_arrive(&ctl.p_full[1]);
    }
    int step0 = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Work* const w = item(i);
      if (w == nullptr) break;
      const bool key = (w->flags & kKeyMode) != 0;
      const int steps = key ? w->n[0] : w->nt;
      const int n0 = w->n[0], n1 = w->n[1], a0 = w->a[0], a1 = w->a[1];
      const bool mine0 = (wq << 5) < w->rows[0], mine1 = (wq << 5) < w->rows[1];  // the warp has rows
      for (int j = 0; j < steps && ok; ++j) {
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          const int as = s == 0 ? a0 : a1, es = s == 0 ? a0 + n0 : a1 + n1;
          if (j <= as || j >= es) continue;  // (a stage's first product overwrites O)
          if (!warp_wait(&ctl.alpha_full[s], (ph_a >> s) & 1, abort_flag, LIM)) { ok = false; break; }
          ph_a ^= 1u << s;
          if (s == 0 ? mine0 : mine1) {
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
                for (int e = 0; e < 32; e += 2) {
                  float lo, hi;
                  unpack2(fmul2(pack2(u2f(v[e]), u2f(v[e + 1])), a2), lo, hi);
                  v[e] = f2u(lo);
                  v[e + 1] = f2u(hi);
                }
                tmem_st32(t_o + c * 32, v);
              }
              tmem_wait_st();
            }
          }
          tc_fence_before();
          __syncwarp();
          if (row == 0) trace_stamp(p.trace, step0 + j, 10 + s);
          if (lane == 0) mbar_arrive(&ctl.p_full[s]);
        }
      }
      if (!ok) break;
      step0 += steps;
      // Epilogue: each stage's rows in turn, or in key mode, where both have
      // the same rows, the two joined.
      const bool part = (w->flags & kPart) != 0;
      const int q0 = w->q0, kvh = w->kvh;
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        if (key && s == 1) break;
        const int n = s == 0 ? n0 : n1, nj = key ? n1 : 0;  // nj > 0: stage 1 is joined
        const int rows = w->rows[s] - (wq << 5);            // of the tile, from this warp's first on
        float m = -INFINITY, l = 0.0f, f0 = 1.0f, f1 = 0.0f;
        if (n > 0) {
          if (!warp_wait(&ctl.stats_full[s], (ph_st >> s) & 1, abort_flag, LIM)) { ok = false; break; }
          ph_st ^= 1u << s;
          l = ctl.stat_l[s][row];
          m = ctl.stat_m[s][row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.stats_empty[s]);
        }
        if (nj > 0) {
          if (!warp_wait(&ctl.stats_full[1], (ph_st >> 1) & 1, abort_flag, LIM)) { ok = false; break; }
          ph_st ^= 2u;
          const float l1 = ctl.stat_l[1][row], m1 = ctl.stat_m[1][row];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.stats_empty[1]);
          const float mj = fmaxf(m, m1), mu = mj == -INFINITY ? 0.0f : mj;
          f0 = ex2_mufu(m - mu);  // (0 for a stage that saw no key)
          f1 = ex2_mufu(m1 - mu);
          l = l * f0 + l1 * f1;
          m = mj;
        }
        const float inv = part ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
        f0 *= inv;
        f1 *= inv;
        if (n > 0) {
          if (!warp_wait(&ctl.o_full[s], (ph_of >> s) & 1, abort_flag, LIM)) { ok = false; break; }
          ph_of ^= 1u << s;
          if (nj > 0) {
            if (!warp_wait(&ctl.o_full[1], (ph_of >> 1) & 1, abort_flag, LIM)) { ok = false; break; }
            ph_of ^= 2u;
          }
          tc_fence_after();
        }
        if (rows > 0) {
          const bool valid = lane < rows;
          const int token = q0 + s * p.tok + row_tok, head = kvh * p.group + row_head;
          // 32 columns at a time, the next ones on their way from tensor
          // memory. A part's rows go to its slot as they are. Else 32 rows x
          // 64 columns go through a staging buffer (128-byte swizzle), and out
          // by one TMA store where the warp's rows are whole tokens of the
          // sequence, or by plain stores of whole rows.
          const size_t at = size_t(2 * int(blockIdx.x) + ((w->flags & kCont) ? 0 : 1)) * 256 + s * 128 + row;
          const bool tma = p.o_box != 0 && rows >= 32;
          uint32_t v[32], x[32];
          if (n > 0) tmem_ld32(t_lane + s * D, x);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = n > 0 ? f2u(u2f(x[e]) * f0) : 0u;
            if (nj > 0) {
              tmem_ld32(t_lane + D + c * 32, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = f2u(fmaf(u2f(x[e]), f1, u2f(v[e])));
            }
            if (n > 0 && c + 1 < D / 32) tmem_ld32(t_lane + s * D + (c + 1) * 32, x);
            if (part) {
              if (valid) {
                uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * D + c * 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
              }
              continue;
            }
            if ((c & 1) == 0) {
              if (lane == 0) bulk_wait_read_all();  // the previous store has read the buffer
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t* y = &v[8 * e];
              *reinterpret_cast<uint4*>(stg + lane * 128 + ((((c & 1) * 4 + e) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16x2(u2f(y[0]), u2f(y[1])), pack_bf16x2(u2f(y[2]), u2f(y[3])),
                             pack_bf16x2(u2f(y[4]), u2f(y[5])), pack_bf16x2(u2f(y[6]), u2f(y[7])));
            }
            if ((c & 1) == 0) continue;
            if (tma) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_4d(&tmO, stg, (c >> 1) * 64, 0, q0 + s * p.tok + wq * p.o_box, kvh);
                bulk_commit();
              }
            } else {
              __syncwarp();
              // 8 lanes write a row's 128 bytes, 4 rows at a time
#pragma unroll 1
              for (int e = 0; e < 8; ++e) {
                const int rr = e * 4 + (lane >> 3);
                const int to = __shfl_sync(0xffffffffu, valid ? token * p.Hq + head : -1, rr);
                const uint4 y = *reinterpret_cast<const uint4*>(stg + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                if (to >= 0) *reinterpret_cast<uint4*>(p.o + size_t(to) * D + (c >> 1) * 64 + (lane & 7) * 8) = y;
              }
              __syncwarp();
            }
          }
          if (valid) {
            if (part) {
              p.part_ml[at] = make_float2(m, l);
            } else {
              p.lse[size_t(head) * p.total_q + token] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
            }
          }
        }
        if (n > 0) {  // the next item's products may overwrite O
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ctl.p_full[s]);
            if (nj > 0) mbar_arrive(&ctl.p_full[1]);
          }
        }
        if (row == 0) trace_stamp(p.trace, step0 - 1, 12 + s);
      }
      release(i);
    }
    if (lane == 0) bulk_wait_all();  // stores complete (and staging reads done) before the CTA exits
  } else {
    setmaxnreg_dec<72>();
  }
  if (warp == 12 || warp == 14) {
    // ------------------------------------------------------ TMA producers
    // Warp 12 loads Q and K, warp 14 V: a paged tile takes a warp some 0.5 us
    // to look up and issue, and one warp for both set the pace of single tokens
    // at d = 64 (256 of them over 1000 to 4000 keys, pages of 16: 375 -> 270 us).
    // The ring holds K and V in the order in which the products take them.
    const bool is_v = warp == 14;
    const CUtensorMap* const m = is_v ? &tmV : &tmK;
    uint32_t base = 0, q_uses[2] = {0, 0}, key_items = 0;  // ring entries of the items before
    bool ok = true, injected = false;
    const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
    const uint32_t q_bytes = uint32_t(p.tok * p.group * D * 2);
    const int n_box = PAGED ? 128 / p.box_rows : 1;  // of a tile; lane i looks up box i
    for (int i = 0; ok; ++i) {
      const Work* const w = item(i);
      if (w == nullptr) break;
      const int nt = w->nt, kvh = w->kvh, kt = w->kt, kbase = w->kbase, klen = w->klen;
      const bool key = (w->flags & kKeyMode) != 0;
      // The first key that a row of the item sees. The first tile begins at a
      // multiple of 128 before it, maybe in pages that the window hides whole:
      // a server may have given those to other sequences.
      const int seen = PAGED && p.wl >= 0 ? w->pos - p.wl : 0;
      // Where this lane's box of tile t is. The table is read one tile ahead:
      // read as it was needed, it set the pace (3 chunks of 512 tokens over long
      // caches 228 -> 217 us, a mixed batch with pages of 16 68 -> 63 us).
      auto place = [&](int t) {
        Place at{0, 0, 0, false};
        if constexpr (PAGED) {
          // boxes that begin before the sequence's end
          const int key0 = (kt + t) * 128;
          at.boxes = min(n_box, (klen - key0 + p.box_rows - 1) / p.box_rows);
          if (t < nt && lane < at.boxes) {
            const int k = key0 + lane * p.box_rows, pg = k / p.page_size;
            at.hidden = k + p.box_rows <= seen;
            if (!at.hidden) at.page = p.table[size_t(kbase) * p.max_pages + pg];
            at.in_page = k - pg * p.page_size;
          }
        }
        return at;
      };
      Place next = place(0);
      // Q: key mode takes the two buffers in turn, else stage s takes buffer s
      for (int s = 0; s < 2 && ok && !is_v; ++s) {
        if (w->n[s] == 0 || (key && s == 1)) continue;
        const uint32_t b = key ? (key_items++ & 1) : uint32_t(s);
        ok = warp_wait(&ctl.q_empty[b], (b == 0 ? q_uses[0] : q_uses[1]) & 1 ? 0 : 1, abort_flag, LIM);
        if (!ok) break;
        if (b == 0) {
          ++q_uses[0];
        } else {
          ++q_uses[1];
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.q_full[b], q_bytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d_hint(sQ + b * C::kTileBytes + c * 16384, &tmQ, &ctl.q_full[b], c * 64, 0,
                             w->q0 + (key ? 0 : s * p.tok), kvh, pol_q);
        }
      }
      if (!ok) break;
      // K runs d tiles ahead of V: K(0..d-1), then V(t), K(t + d) in turn, then the last V
      const int d = min(key ? 2 : 1, nt);
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        const uint32_t entry = base + uint32_t(is_v ? (t < nt - d ? d + 2 * t : nt + t) : (t < d ? t : 2 * t - d + 1));
        const uint32_t slot = entry % C::kSlots, use = entry / C::kSlots;
        uint8_t* dst = sKV + slot * C::kTileBytes;
        // (The warp's entry before this one is at most 3 back: what it waited
        // for has been taken, and all before it, so that this wait is for the
        // slot's last use and no earlier one.)
        ok = warp_wait(&ctl.kv_empty[slot], (use & 1) ^ 1, abort_flag, LIM);
        if (!ok) break;
        if (p.inject == 1 && !is_v && !injected) {  // test hook: never deliver this tile
          injected = true;
          continue;
        }
        if constexpr (PAGED) {
          Place at = next;
          next = place(t + 1);
          if (at.hidden) {
            at.page = p.num_pages;  // reads as zeros
          } else if (at.page < 0 || at.page >= p.num_pages) {  // no such page: so too, and the caller is told
            atomicOr(p.status, kDevBadArg);
            at.page = p.num_pages;
          }
          // One lane issues the boxes, unrolled: a copy's operands are uniform
          // registers, which lanes that issue a box each take turns to fill
          // (the mixed batch 62 -> 59 us; in a rolled loop 69 us).
          int page[8], in_page[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            page[x] = __shfl_sync(0xffffffffu, at.page, x);
            in_page[x] = __shfl_sync(0xffffffffu, at.in_page, x);
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(&ctl.kv_full[slot], uint32_t(at.boxes * p.box_rows * D * 2));
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              if (x >= at.boxes) break;
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_4d_hint(dst + c * 16384 + x * p.box_rows * 128, m, &ctl.kv_full[slot], c * 64, kvh, in_page[x],
                                 page[x], pol_kv);
            }
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.kv_full[slot], C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d_hint(dst + c * 16384, m, &ctl.kv_full[slot], c * 64, kvh, kbase + (kt + t) * 128, 0, pol_kv);
        }
        const int fill = w->fill;
        if (is_v && t == nt - 1 && fill != 0) {
          // The sequence ends in this tile: once loaded, its rows past the end
          // are zeroed before the product reads them (a row is 128 bytes of
          // each chunk; the swizzle stays within it).
          __syncwarp();
          ok = warp_wait(&ctl.kv_full[slot], use & 1, abort_flag, LIM);
          if (!ok) break;
          for (int k = fill * 8 + lane; k < 128 * 8; k += 32)
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              *reinterpret_cast<uint4*>(dst + c * 16384 + k * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.tail_done[slot]);
        }
      }
      base += uint32_t(2 * nt);
      release(i);
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks the role and an elected lane issues (with the
    // producer's and all waits, 1.78 -> 1.29 ms on one causal sequence of 16384
    // tokens, against one lane walking: MMA operands are uniform registers).
    {
      const uint32_t idS = idesc_bf16_f32(128, 128, 0, 0) | (p.neg_s << 13);
      constexpr uint32_t idPV = idesc_bf16_f32(128, D, 0, 1);
      const uint32_t dq = sdesc_lo(smem_u32(sQ), 16), dk = sdesc_lo(smem_u32(sKV), 16),
                     dv = sdesc_lo(smem_u32(sKV), 16384);
      // Phases of the barriers of each stage (or slot), a bit each: arrays
      // indexed by the stage would be kept in memory.
      uint32_t phases = 0, tail_phases = 0;
      uint32_t E = 0, key_items = 0;  // ring entry that follows
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
        return warp_wait(bar, phase, abort_flag, LIM);
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(bar);
      };
      auto wait_phase = [&](uint64_t* bar, int bit) -> bool {
        const bool r = wait(bar, (phases >> bit) & 1);
        phases ^= 1u << bit;
        return r;
      };
      // the next ring entry, loaded
      auto wait_kv = [&](uint32_t& slot) -> bool {
        slot = E % C::kSlots;
        const uint32_t phase = (E / C::kSlots) & 1;
        ++E;
        return wait(&ctl.kv_full[slot], phase);
      };
      // rows of a V tile past the sequence's end zeroed
      auto wait_tail = [&](uint32_t slot) -> bool {
        const uint32_t phase = (tail_phases >> slot) & 1;
        tail_phases ^= 1u << slot;
        return wait(&ctl.tail_done[slot], phase);
      };
      // O of stage s (+)= P V; S of stage s = Q (buffer b) K^T
      auto issue_pv = [&](int s, uint32_t slot, bool acc) {
        tc_fence_after();
        if (!elect_one()) return;
        const uint32_t b0 = sdesc_step(dv, slot * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo(tmem + kOCol0 + uint32_t(s * D), tmem + uint32_t(s * 128) + kk * 8, sdesc_step(b0, kk * 2048), idPV,
                    (acc || kk > 0) ? 1u : 0u);
      };
      auto issue_s = [&](int s, uint32_t b, uint32_t slot) {
        tc_fence_after();
        if (!elect_one()) return;
        const uint32_t q0 = sdesc_step(dq, b * C::kTileBytes), b0 = sdesc_step(dk, slot * C::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss_lo(tmem + uint32_t(s * 128), sdesc_step(q0, ko), sdesc_step(b0, ko), idS, kk > 0);
        }
        mma_commit(&ctl.s_full[s]);
      };
      // Both loops begin one step (key mode: two tiles) before the item, with
      // its first S alone: one copy of each product's instructions, since
      // code that runs once per item is not in the instruction cache (a
      // prologue and a general step at the items' ends cost some 5 us each).
      auto trace = [&](unsigned long long* buf, int step, int point) {
        if (lane == 0) trace_stamp(buf, step, point);
      };
      int step0 = 0;
      for (int i = 0; ok; ++i) {
        const Work* const w = item(i);
        if (w == nullptr) break;
        const int nt = w->nt;
        const bool fill = w->fill != 0;
        if (nt > 0 && (w->flags & kKeyMode)) {
          const uint32_t b = key_items++ & 1;
          ok = wait_phase(&ctl.q_full[b], kPhQ + int(b));
          for (int t = -2; t < nt && ok; ++t) {  // V(t) and K(t + 2), of stage t & 1
            const int s = t & 1;
            uint32_t slot;
            if (t >= 0) {
              ok = wait_kv(slot) && (!fill || t < nt - 1 || wait_tail(slot)) && wait_phase(&ctl.p_full[s], kPhP + s);
              if (!ok) break;
              if (s == 0) trace(p.trace, step0 + (t >> 1), 0);
              issue_pv(s, slot, t > 1);
              if (t + 2 >= nt) commit(&ctl.o_full[s]);
              commit(&ctl.kv_empty[slot]);
            }
            if (t + 2 < nt) {
              ok = wait_kv(slot);
              if (!ok) break;
              issue_s(s, b, slot);
              commit(&ctl.kv_empty[slot]);
              if (t + 3 == nt) commit(&ctl.q_empty[b]);
            }
          }
          step0 += (nt + 1) >> 1;
        } else if (nt > 0) {
          const int n0 = w->n[0], n1 = w->n[1], a0 = w->a[0], a1 = w->a[1];
          for (int s = 0; s < 2 && ok; ++s)
            if ((s == 0 ? n0 : n1) > 0) ok = wait_phase(&ctl.q_full[s], kPhQ + s);
          for (int t = -1; t < nt && ok; ++t) {  // V(t) and K(t + 1), of both stages
            const bool v = t >= 0, k = t + 1 < nt;
            // tile t (or t + 1) among a stage's: below n unsigned
            const uint32_t u0 = uint32_t(t - a0), u1 = uint32_t(t - a1);
            uint32_t vs = 0, ks = 0;
            if (v) {
              ok = wait_kv(vs) && (!fill || k || wait_tail(vs));
              if (!ok) break;
              trace(p.trace, step0 + t, 0);
              if (u0 < uint32_t(n0)) {
                ok = wait_phase(&ctl.p_full[0], kPhP);
                if (!ok) break;
                issue_pv(0, vs, u0 > 0);
                trace(p.trace, step0 + t, 1);
                if (u0 + 1 == uint32_t(n0)) commit(&ctl.o_full[0]);
                if (u1 >= uint32_t(n1)) commit(&ctl.kv_empty[vs]);
              }
            }
            if (k) {
              ok = wait_kv(ks);
              if (!ok) break;
              if (u0 + 1 < uint32_t(n0)) {
                issue_s(0, 0, ks);
                if (u0 + 2 == uint32_t(n0)) commit(&ctl.q_empty[0]);
              }
            }
            if (v && u1 < uint32_t(n1)) {
              ok = wait_phase(&ctl.p_full[1], kPhP + 1);
              if (!ok) break;
              issue_pv(1, vs, u1 > 0);
              trace(p.trace, step0 + t, 2);
              if (u1 + 1 == uint32_t(n1)) commit(&ctl.o_full[1]);
              commit(&ctl.kv_empty[vs]);
            }
            if (k) {
              if (u1 + 1 < uint32_t(n1)) {
                issue_s(1, 1, ks);
                if (u1 + 2 == uint32_t(n1)) commit(&ctl.q_empty[1]);
              }
              commit(&ctl.kv_empty[ks]);
            }
            if (v) trace(p.trace, step0 + t, 3);
          }
          step0 += nt;
        }
        if (ok) release(i);
      }
      if (*abort_flag) {
        // drain the tensor pipe before TMEM is released
        if (elect_one()) mma_commit(&ctl.drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&ctl.drain), 0) && globaltimer_ns() - t0 < 100000000ull) {
        }
        __syncwarp();
      }
    }
  } else if (warp == 15) {
    // --------------------------------------------------------- work items
    int n_done = 0;
    // hands an item to the other roles (null: there are no more); false when
    // a wait ran out
    auto hand_out = [&](const FwdItem* src, int kvh, int flags, int kt, int nt) -> bool {
      Work x;
      x.flags = -1;
      if (src != nullptr) {
        x = work_of(p, src, kvh, flags, kt, nt);
        // Its Q and its first K and V tile into L2, a lane to each box: the
        // loads wait for buffers that items before still use, and would then
        // wait for device memory too.
        const int c = lane % C::kChunks * 64, what = lane / C::kChunks;
        if (x.nt > 0) {
          if (what < 2) {
            if ((what == 0 ? x.n[0] : x.n[1]) > 0 && !(what == 1 && (x.flags & kKeyMode)))
              tma_prefetch_l2_4d(&tmQ, c, 0, x.q0 + what * p.tok, x.kvh);
          } else if (!PAGED && what < 4) {
            tma_prefetch_l2_4d(what == 2 ? &tmK : &tmV, c, x.kvh, x.kbase + x.kt * 128, 0);
          }
        }
      }
      const int i = n_done++;
      if (!warp_wait(&ctl.it_empty[i % kItems], ((i / kItems) & 1) ^ 1, abort_flag, LIM)) return false;
      if (lane == 0) {
        ctl.it[i % kItems] = x;
        mbar_arrive(&ctl.it_full[i % kItems]);
      }
      return true;
    };
    bool ok = true;
    if (p.items != nullptr) {
      for (Walk wk = walk_begin(p.head, p.first, p.last); ok && wk.i <= wk.last; walk_step(wk)) {
        const FwdItem* src = p.items + wk.i;
        ok = hand_out(src, src->kvh, src->count & ~0xffff, src->kt, src->nt);
      }
    } else {
      // units, 32 sequences at a time
      int U = 0, bad = 0;
      for (int b0 = 0; b0 < p.L.B; b0 += 32) {
        const int b = b0 + lane;
        Seq q;
        int n = 0;
        if (b < p.L.B) {
          if (seq_at(p.L, b, q)) {
            n = p.side.units(q);
          } else {
            bad = 1;
          }
        }
        int at = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, at, m);
          if (lane >= m) at += o;
        }
        const int sum = __shfl_sync(0xffffffffu, at, 31);
        at += U - n;
        for (int j = 0; j < n && at + j < p.max_units; ++j) {
          const Range r = p.side.range(q, j);
          FwdItem x = p.side.item(q, b, j, 0, 0);
          FwdSide::set_range(x, r.first, r.n);
          ctl.unit[at + j] = x;
        }
        U = min(U + sum, p.max_units + 1);
      }
      bad = __any_sync(0xffffffffu, bad != 0) || U > p.max_units;
      if (bad) U = 0;  // lengths that the tensors cannot hold: nothing is computed
      __syncwarp();
      int T = 0, most = 0;
      for (int u0 = 0; u0 < U; u0 += 32) {
        const int n = u0 + lane < U ? ctl.unit[u0 + lane].nt + kItemCost : 0;
        int at = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, at, m);
          if (lane >= m) at += o;
        }
        if (u0 + lane < U) ctl.cost[u0 + lane] = T + at - n;
        T += __shfl_sync(0xffffffffu, at, 31);
        most = max(most, __reduce_max_sync(0xffffffffu, n));
      }
      __syncwarp();
      // the plan kernel's rule, and its shares, in the order (kv head, unit)
      const int G = int(gridDim.x), me = int(blockIdx.x), n_items = U * p.Hkv;
      const long long all = 1LL * T * p.Hkv;
      const bool split = n_items > G || most > all / G * FwdSide::kSplitGain / 8 + FwdSide::kPartsCost;
      const long long lo = all * me / G, hi = all * (me + 1) / G;
      Cut cut;
      cut.c1 = -1;
      bool any = false;
      for (int i0 = 0; ok && i0 < n_items; i0 += 32) {
        const int i = i0 + lane, kvh = i / U, u = i - kvh * U;
        const long long x0 = i < n_items ? 1LL * kvh * T + ctl.cost[u] + kItemCost : 0, x1 = i < n_items ? x0 + ctl.unit[u].nt : 0;
        const bool mine = i < n_items && (!split ? i == me
                                          : x0 == x1 ? x0 >= lo && (x0 < hi || me == G - 1) : x1 > lo && x0 < hi);
        for (unsigned left = __ballot_sync(0xffffffffu, mine); ok && left != 0; left &= left - 1) {
          const int k = i0 + __ffs(left) - 1, kk = k / U, ku = k - kk * U;
          const FwdItem* src = &ctl.unit[ku];
          int flags = src->count & ~0xffff, kt = src->kt, nt = src->nt;
          if (split && nt > 0) {
            const long long y0 = 1LL * kk * T + ctl.cost[ku] + kItemCost, y1 = y0 + nt;
            const long long z0 = max(y0, lo), z1 = min(y1, hi);
            kt += int(z0 - y0);
            nt = int(z1 - z0);
            if (z0 > y0 || z1 < y1) flags |= kPart;
            if (z0 > y0) flags |= kCont;
            if (z0 == y0 && z1 < y1) {  // the first of a divided unit's parts: its last is in worker c1
              cut.row0 = src->q0;
              cut.count = src->ntok();
              cut.kvh = kk;
              cut.c0 = me;
              cut.c1 = int((y1 * G - 1) / all);  // the last whose share begins before y1
            }
          }
          any = true;
          ok = hand_out(src, kk, flags, kt, nt);
        }
      }
      if (lane == 0) {
        if (p.cuts != nullptr) {  // for the last kernel
          if (me + 1 < G) p.cuts[me + 1] = cut;
          p.last[me] = any ? 0 : -1;
          if (me == 0) p.cuts[0].c1 = -1;
        }
        if (me == 0 && bad) atomicOr(p.status, kDevBadArg);
      }
    }
    if (ok) hand_out(nullptr, 0, 0, 0, 0);
  }

  // ------------------------------------------------------------- teardown
  if ((warp == 12 || warp == 14) && *abort_flag) {
    // let copies already in flight land before shared memory is released
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && ctl.abort) atomicOr(p.status, kDevTimeout);
}

// The parts of the rows whose keys were divided between workers, joined in
// the workers' order: O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i. Block
// (c, y): cut c, every gridDim.y-th group of rows; a warp per row, or several
// that take consecutive parts, where the rows are few and the parts many (the
// parts' reads, one after the other, are what the kernel takes: one token over
// 8000 keys 29 -> 16 us). The lanes read the parts' (m, l) first, so that the
// reads of O are independent.
constexpr int kJoinWarps = 8;  // (of 16 or 32, chunks over a cache took 4 and 10 us longer)
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) seq_join_kernel(const Params p) {
  __shared__ float so[kJoinWarps][D];
  __shared__ float2 sml[kJoinWarps];
  grid_dep_wait();
  const Cut k = p.cuts[blockIdx.x];
  if (k.c1 < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = k.count * p.group, per_stage = p.tok * p.group, parts = k.c1 - k.c0 + 1;
  constexpr int V = D / 32;  // columns per lane
  int per_row = kJoinWarps;  // no more than there are, and four parts to each
  while (per_row > 1 && (per_row * rows > kJoinWarps * int(gridDim.y) || per_row * 4 > parts)) per_row >>= 1;
  const int at_once = kJoinWarps / per_row, share = (parts + per_row - 1) / per_row;
  const int first = k.c0 + warp % per_row * share, last = min(first + share - 1, k.c1);  // this warp's parts
  for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
    const int r = r0 + warp / per_row;
    const int s = r >= per_stage ? 1 : 0;
    const size_t at = size_t(s) * 128 + (r - s * per_stage);
    float m = -INFINITY, l = 0.0f, o[V] = {};
    for (int c0 = first; r < rows && c0 <= last; c0 += 32) {  // 32 parts at a time
      const int c = c0 + lane;
      const size_t mine = size_t(c == k.c0 ? 2 * c + 1 : 2 * c) * 256 + at;
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (c <= last) {
        const bool has = p.last[c] >= 0;  // a worker without a share has no part: what its slot holds is not used
        const float2 x = p.part_ml[mine];
        if (has) ml = x;
      }
      float mn = fmaxf(m, ml.x);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
      const float mu = mn == -INFINITY ? 0.0f : mn;
      const float wa = ex2_mufu(m - mu);  // (0 for m = -inf)
      const float wb = ex2_mufu(ml.x - mu);
      float ls = ml.y * wb;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      l = l * wa + ls;
      m = mn;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= wa;
      const int n = min(32, last - c0 + 1);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wb, i), li = __shfl_sync(0xffffffffu, ml.y, i);
        const int ci = c0 + i;
        if (li == 0.0f) continue;  // no key of this part is visible to the row: its O may not have been written
        const float* src = p.part_o + (size_t(ci == k.c0 ? 2 * ci + 1 : 2 * ci) * 256 + at) * D + lane * V;
        if constexpr (V == 4) {
          const float4 t = *reinterpret_cast<const float4*>(src);
          o[0] = fmaf(t.x, wi, o[0]);
          o[1] = fmaf(t.y, wi, o[1]);
          o[2] = fmaf(t.z, wi, o[2]);
          o[3] = fmaf(t.w, wi, o[3]);
        } else {
          const float2 t = *reinterpret_cast<const float2*>(src);
          o[0] = fmaf(t.x, wi, o[0]);
          o[1] = fmaf(t.y, wi, o[1]);
        }
      }
    }
    if (per_row > 1) {  // the row's warps, in order
      __syncthreads();  // the rows before have been read
#pragma unroll
      for (int e = 0; e < V; ++e) so[warp][lane * V + e] = o[e];
      if (lane == 0) sml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp % per_row != 0) continue;
      for (int i = 1; i < per_row; ++i) m = fmaxf(m, sml[warp + i].x);
      const float mu = m == -INFINITY ? 0.0f : m;
      l = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = 0.0f;
      for (int i = 0; i < per_row; ++i) {
        const float f = ex2_mufu(sml[warp + i].x - mu);
        l = fmaf(sml[warp + i].y, f, l);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(so[warp + i][lane * V + e], f, o[e]);
      }
    }
    if (r >= rows) continue;
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
Space carve(uint8_t* base, const SeqProblem& pb, int G, long long units) {
  Space s{};
  Carver c{base, 0};
  s.plan = carve_plan<FwdItem>(c, pb.B, units, pb.Hkv, G);
  s.part_ml = c.take<float2>(size_t(2) * G * 256);
  s.part_o = c.take<float>(size_t(2) * G * 256 * pb.d);
  s.bytes = c.at;
  return s;
}

template <int D, bool PAGED>
cudaError_t launch_t(const SeqProblem& pb, void* o, float* lse, cudaStream_t stream) {
  using C = Tiles<D>;
  const int G = std::min(num_sms(), seq::kMaxWorkers);
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
  // o: the 32 rows of a warp, where they are whole tokens
  CUtensorMap mo = mq;
  if (32 % group == 0) {
    p.o_box = 32 / group;
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), uint64_t(pb.total_q), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(pb.Hq) * D * 2, uint64_t(group) * D * 2};
    const uint32_t box[4] = {64, uint32_t(group), uint32_t(p.o_box), 1};
    if (!encode_tiled(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, o, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
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
  static SmemLimit limit;
  cudaError_t e = limit.set(kern, C::kSmemDyn);
  if (e != cudaSuccess) return e;
  // a sequence of n tokens has ceil(n / (2 tok)) units
  long long units = pb.total_q / (2 * tok) + pb.B;
  if (units > pb.total_q) units = pb.total_q;
  const bool few = pb.B <= kFewUnits && units <= kFewUnits && units * pb.Hkv <= (PAGED ? kFewRounds : 1) * G;
  // Few items of few key tiles are never divided: no workspace, no last kernel.
  long long keys = pb.page_table != nullptr ? 1LL * pb.max_pages * pb.page_size : pb.total_k;
  if (pb.window_left >= 0 && pb.window_right >= 0)  // and whole tiles around those that a unit sees
    keys = std::min(keys, 2LL * tok + pb.window_left + pb.window_right + 254);
  const bool whole = few && units * pb.Hkv <= G && (keys + 127) / 128 + kItemCost <= FwdSide::kPartsCost;
  void* ws = nullptr;
  Space sp{};
  if (!whole) {
    cudaMemPool_t pool = workspace_pool();
    if (pool == nullptr || cudaMallocFromPoolAsync(&ws, carve(nullptr, pb, G, units).bytes, pool, stream) != cudaSuccess)
      return cudaErrorMemoryAllocation;
    sp = carve(static_cast<uint8_t*>(ws), pb, G, units);
  }
  PlanArgs<FwdSide> a{};
  a.L = Lens{pb.cu_q, pb.cu_k, pb.lens_k, pb.B, pb.total_q, pb.total_k, 1LL * pb.max_pages * pb.page_size};
  a.P = sp.plan;
  a.side = FwdSide{tok, pb.window_left, pb.window_right, pb.page_table != nullptr ? 1 : 0};
  a.Hkv = pb.Hkv;
  a.G = G;
  a.status = p.status;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.head = sp.plan.head;
  p.first = sp.plan.first;
  p.last = sp.plan.last;
  p.L = a.L;
  p.side = a.side;
  p.Hkv = pb.Hkv;
  p.max_units = int(units);
  p.items = few ? nullptr : sp.plan.items;
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
  p.trace = dc.trace;
  if (!few) {
    plan_kernel<FwdSide><<<1, kPlanThreads, 0, stream>>>(a);
    e = cudaGetLastError();
  }
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
  lc.numAttrs = few ? 0 : 1;
  if (dc.ev_begin) cudaEventRecord(dc.ev_begin, stream);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&lc, kern, mq, mk, mv, mo, p);
  if (dc.ev_end) cudaEventRecord(dc.ev_end, stream);
  if (e == cudaSuccess && !whole) {
    lc.numAttrs = 1;
    // 256 rows of a cut at most. Units of some parts get a warp per row at once
    // (64 tokens over 4000 keys 43 -> 32 us); of many units none has more than
    // a few, if any are divided, and half as many blocks start 1 us sooner.
    const long long high = (units * pb.Hkv * 4 < G ? 256 : 128) / kJoinWarps;
    lc.gridDim = dim3(G, unsigned(std::min(high, 1LL * pb.total_q * group)));
    lc.blockDim = dim3(kJoinWarps * 32);
    lc.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&lc, seq_join_kernel<D>, p);
  }
  const cudaError_t f = whole ? cudaSuccess : cudaFreeAsync(ws, stream);
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
