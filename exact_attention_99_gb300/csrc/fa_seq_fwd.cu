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
// Over a cache of e4m3 codes (fa_fwd_paged_fp8, many rows to a kv head) the same
// pipeline with other softmax warps and converters; see Codes below.
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
//   codes, 3 chunks of 512 tokens over 6000 to 16384 keys, 32 query and 8 kv heads of
//     128: 230 us (bf16 205 to 217), 1.6 us a tile of two stages, of which a stage's
//     softmax takes 0.95 (the converters issue beside it, and 16 keys at a time have
//     scales of their own), the products behind it 0.65; 3 us at an item's end, where
//     the softmax warps write O. (Of d = 128 a thread spills 16 bytes, of d = 64 none.)
//   items of few tiles: 1.3 to 2.3 us between two items, most of it instruction
//     fetch (code that runs once per item is not in the cache) and the first
//     S; with a window and one query head per kv head the first and the last
//     of an item's key tiles, which one stage alone sees; the plan before the
//     first item (11 to 15 us); small calls: the launches (77 tokens: 8 us).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_seq_plan.cuh"
#include "sm103_fp8.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace seq {

// what the keys are: packed sequences, a paged cache, a paged cache of codes
enum Kind { kPacked, kPaged, kCodes };
constexpr int kThreads = 512;
constexpr uint32_t kOCol0 = 256;
constexpr float kTau = 8.0f;  // rescale threshold (log2 units), as in the dense forward

// --------------------------------------------------------------------------
// main kernel
// --------------------------------------------------------------------------
struct Params {
  __nv_bfloat16* o;
  const float* q_factor;   // codes: [total_q, Hq] what a row of Q was divided by
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
  const float* scales[2];  // codes: of K, V, [num_pages, page_size / 16, Hkv]
  const uint8_t* v_codes;
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
//   codes       15 a V tile's codes turned to f16
constexpr int kItems = 4;  // ring of work items

template <int D>
struct Tiles {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  // Over codes the same memory is two rings, as a K tile has half as many bytes as a V
  // tile's f16 values (one ring of slots for either, as above: 3 chunks of 512 tokens
  // over 6000 to 16384 keys 245 us, with K's tiles further ahead 236).
  static constexpr int kKSlots = 4, kVSlots = D == 128 ? 2 : 6, kKBytes = kTileBytes / 2, kVRing = kKSlots * kKBytes;
  static_assert(kVRing + kVSlots * kTileBytes == kSlots * kTileBytes, "the same memory");
  static constexpr int kStgBytes = 16384;  // O staging: 4 warps x [32 rows x 64 columns] bf16
  static constexpr int kSmemDyn = (2 + kSlots) * kTileBytes + kStgBytes + 1024;
};
constexpr int kMaxSlots = 8;

// bits of the MMA issuer's phases: Q loaded, P stored, of codes its second half (a pair each)
constexpr int kPhQ = 0, kPhP = 2, kPhP2 = 4;

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

// Over a cache of codes (kCodes) the products take K as it is: S = (Q_hi + Q_lo) K^T
// in e4m3, where a row of Q, divided by a power of two, is the sum of two e4m3
// values, each off by at most half a step: exact for what is 2^-9 of the row's largest
// value or more (bf16 has 8 bits, two e4m3 significands 4 each), and off by at most
// 2^-17 of that largest below. The rate is twice that of 16 bits, so S takes as long.
// P V wants P's 11 bits: V's codes land in the lower half of their ring slot, and the
// warps that elsewhere correct O and write it turn those of 32 rows each to f16 in
// place (every e4m3 value is one). The scales of the tile's blocks of 16 keys go to
// the softmax: with a of K and b of V,
//   x = scale log2(e) a (q . k^) + log2(b), P' = 2^(x - m + kShift), l = sum P' / b:
// b in the exponent leaves the P V product without a further factor, and P' largest
// where it weighs most. P' is at most 2^(kShift + kTau) = 2^15, which f16 holds.
constexpr float kShift = 7.0f;
constexpr float kLow = -3.4028235e38f;  // the running maximum before any key
// Ring of scales. A tile's go out when V of the tile three before has landed, so that V of
// kVSlots tiles before that has been taken, and with it all S up to there but one.
constexpr int kScaleTiles = 16;
struct Codes {
  uint64_t k_full[kMaxSlots], k_empty[kMaxSlots];  // K's tiles; V's are the other rings' (kv_full, ...)
  uint64_t sc_full[kScaleTiles];
  float4 sc[kScaleTiles][8];       // of each block: a scale log2(e), log2(b), 1 / b
  uint32_t nans[kItems];           // not 0: NaN codes of V were taken as zeros (see Seen)
};
static_assert(kScaleTiles >= Tiles<128>::kVSlots + 4 && kScaleTiles >= Tiles<64>::kVSlots + 4, "see there");
struct NoCodes {};

template <Kind KIND>
struct __align__(16) Ctl {
  static constexpr int kUnits = KIND == kCodes ? 240 : kFewUnits;  // (the codes' share of shared memory)
  FwdItem unit[kUnits];
  int cost[kUnits + 1];  // cost of the units before
  std::conditional_t<KIND == kCodes, Codes, NoCodes> codes;
  Work it[kItems];
  uint64_t it_full[kItems], it_empty[kItems];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  // a V tile that the sequence ends in: loaded, its rows past the end zeroed; of codes any V tile, turned to f16
  uint64_t tail_done[kMaxSlots];
  // p_full: P stored (4 softmax warps) and O corrected, or read by the epilogue
  // of the stage's item before (4 correction warps; over codes the 4 softmax warps
  // again, those of stage 0 for both where they join them)
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

// item i of this CTA, or null when there is none (or a wait ran out)
template <Kind KIND>
__device__ __forceinline__ const Work* next_item(Ctl<KIND>& ctl, int i, uint64_t LIM) {
  if (!warp_wait(&ctl.it_full[i % kItems], (i / kItems) & 1, &ctl.abort, LIM)) return nullptr;
  const Work* x = &ctl.it[i % kItems];
  return x->flags < 0 ? nullptr : x;
}
// by each warp once all its lanes have read the item: warp 15 may then write the next one over it
template <Kind KIND>
__device__ __forceinline__ void release_item(Ctl<KIND>& ctl, int i) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (lane == 0) mbar_arrive(&ctl.it_empty[i % kItems]);
}

// Codes: the keys [lo, hi) that every row of an item sees. A NaN code of V would reach the
// rows that do not see it, as 0 * NaN is NaN: among 32 keys that not all rows see it becomes
// zero, and the rows that see it are found at the item's end (hidden_nans). Elsewhere
// the products do that.
struct Seen {
  int lo, hi;
  // the 32 keys from k on, of klen
  __device__ __forceinline__ bool hides(int k, int klen) const { return k < lo || min(k + 32, klen) > hi; }
};
__device__ __forceinline__ Seen seen_by_all(const Params& p, int pos, int ntok) {
  return Seen{p.wl >= 0 ? pos + ntok - 1 - p.wl : 0, p.wr >= 0 ? pos + p.wr + 1 : 0x7fffffff};
}
// A bit for each of 16 columns of V's rows (their place in the first row: codes) in which one
// of the keys [lo, hi) of sequence b, in 32 that hide some, is a NaN code.
__device__ __forceinline__ uint32_t hidden_nans(const Params& p, int b, int lo, int hi, int klen, Seen seen,
                                                 const uint8_t* codes, int d) {
  const int* const row = p.table + size_t(b) * p.max_pages;
  uint4 nans = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int k = lo; k < hi; ++k) {
    if (!seen.hides(k & ~31, klen)) {  // on to the next 32
      k |= 31;
      continue;
    }
    const int page = row[k / p.page_size];
    if (page < 0 || page >= p.num_pages) continue;
    const long long token = 1LL * page * p.page_size + k % p.page_size;
    const uint4 x = *reinterpret_cast<const uint4*>(codes + token * p.Hkv * d);
    nans.x |= nan_codes(x.x);
    nans.y |= nan_codes(x.y);
    nans.z |= nan_codes(x.z);
    nans.w |= nan_codes(x.w);
  }
  auto bits = [](uint32_t x) { return (x & 1u) | (x >> 7 & 2u) | (x >> 14 & 4u) | (x >> 21 & 8u); };
  return bits(nans.x) | bits(nans.y) << 4 | bits(nans.z) << 8 | bits(nans.w) << 12;
}

// Codes: rows [32 cw, 32 cw + 32) of every V tile turned to f16; the tiles' scales.
template <int D>
__device__ __forceinline__ void codes_convert(const Params& p, Ctl<kCodes>& ctl, uint8_t* sKV, int cw, int lane,
                                              uint64_t LIM) {
  using C = Tiles<D>;
  uint32_t tiles0 = 0;  // tiles of the items before
  bool ok = true;
  // A lane reads 16 codes of a row and writes them as two pieces of 8 values.
  // Four lanes have half a row (d = 128); the rows of neighbouring fours differ in
  // bits 0 and 2, so that neither the reads of codes (128-byte swizzle, or rows of 64
  // bytes) nor the writes meet in a bank.
  const int in8 = (0x63724150u >> (4 * (lane >> 2))) & 7, quarter = lane & 3;
  for (int i = 0; ok; ++i) {
    const Work* const w = next_item(ctl, i, LIM);
    if (w == nullptr) break;
    const int nt = w->nt, kvh = w->kvh, kt = w->kt, klen = w->klen, fill = w->fill;
    const int seen = p.wl >= 0 ? w->pos - p.wl : 0;  // the first key that a row of the item sees
    const Seen by_all = seen_by_all(p, w->pos, w->ntok);
    const int* const row_of_table = p.table + size_t(w->kbase) * p.max_pages;
    // This lane's block of a tile, 2 cw + lane (lanes 0, 1): its page looked up two tiles ahead
    // (-1: not used), its scales read one ahead.
    auto block_key = [&](int t) { return ((kt + t) * 8 + 2 * cw + lane) * kFp8Block; };
    auto look_up = [&](int t) {
      const int k = block_key(t);
      return t < nt && lane < 2 && k < klen && k + kFp8Block > seen ? row_of_table[k / p.page_size] : -1;
    };
    auto read = [&](int t, int page) {
      float2 r = make_float2(1.0f, 1.0f);
      if (page >= 0 && page < p.num_pages) {
        const int k = block_key(t);
        const size_t at = (size_t(page) * (p.page_size / kFp8Block) + k % p.page_size / kFp8Block) * p.Hkv + kvh;
        r.x = p.scales[0][at];
        r.y = p.scales[1][at];
      }
      return r;
    };
    int page0 = look_up(0);
    int page1 = look_up(1);
    float2 next = read(0, page0);
    int published = 0;  // tiles whose scales are out
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      // S runs up to two tiles ahead of V
      for (; published < min(nt, t + 3); ++published) {
        float4* const sc = ctl.codes.sc[(tiles0 + published) % kScaleTiles];
        if (lane < 2) sc[2 * cw + lane] = make_float4(next.x * p.scale_log2, __log2f(next.y), __fdividef(1.0f, next.y), 0.0f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.codes.sc_full[(tiles0 + published) % kScaleTiles]);
        next = read(published + 1, page1);
        page1 = look_up(published + 2);
      }
      const uint32_t slot = (tiles0 + t) % C::kVSlots;
      ok = warp_wait(&ctl.kv_full[slot], ((tiles0 + t) / C::kVSlots) & 1, &ctl.abort, LIM);
      if (!ok) break;
      uint8_t* const tile = sKV + C::kVRing + slot * C::kTileBytes;
      uint8_t* const mine = tile + cw * 4096;
      if (by_all.hides((kt + t) * 128 + cw * 32, klen)) {
        uint32_t nans = 0;
        const int end = t == nt - 1 && fill != 0 ? max(0, min(32, fill - cw * 32)) * (D / 16) : 2 * D;
#pragma unroll 1
        for (int g = lane; g < end; g += 32) {
          uint4* const at = reinterpret_cast<uint4*>(mine) + g;
          const uint4 z = *at, m = make_uint4(nan_codes(z.x), nan_codes(z.y), nan_codes(z.z), nan_codes(z.w));
          if ((m.x | m.y | m.z | m.w) != 0) {
            nans = 1;
            *at = make_uint4(z.x & ~m.x, z.y & ~m.y, z.z & ~m.z, z.w & ~m.w);
          }
        }
        if (nans != 0) ctl.codes.nans[i % kItems] = 1;
        __syncwarp();
      }
      constexpr int kHalves = D / 64;
      uint4 c[4][kHalves];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          c[g][h] = *reinterpret_cast<const uint4*>(
              mine + (g * 8 + in8) * D + (D == 128 ? ((h * 4 + quarter) ^ in8) << 4 : quarter << 4));
      if (t == nt - 1 && fill != 0) {  // rows past the sequence's end, whatever they hold
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (cw * 32 + g * 8 + in8 >= fill)
#pragma unroll
            for (int h = 0; h < kHalves; ++h) c[g][h] = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();  // the warp's codes have been read: its rows may be written over them
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const uint32_t z[4] = {c[g][h].x, c[g][h].y, c[g][h].z, c[g][h].w};
          uint32_t f[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[2 * k] = f16x2_of_e4m3x2(uint16_t(z[k]));
            f[2 * k + 1] = f16x2_of_e4m3x2(uint16_t(z[k] >> 16));
          }
          uint8_t* const to = tile + h * 16384 + (cw * 32 + g * 8 + in8) * 128;
          *reinterpret_cast<uint4*>(to + (((2 * quarter) ^ in8) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<uint4*>(to + (((2 * quarter + 1) ^ in8) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (threadIdx.x == 256) trace_stamp(p.trace, int(tiles0) + t, 15);
      if (lane == 0) mbar_arrive(&ctl.tail_done[slot]);
    }
    tiles0 += uint32_t(nt);
    if (ok) release_item(ctl, i);
  }
}

// The scales of a tile's block b. Reads that the compiler may move over the stores to
// tensor memory, though not over the wait before scales_at (as it may with no plain
// read): every second block waited for its own.
__device__ __forceinline__ uint32_t scales_at(const float4* sc) {
  uint32_t r;
  asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(smem_u32(sc)) : "memory");
  return r;
}
__device__ __forceinline__ float4 scales_of(uint32_t sc, int b) {
  float4 r;
  asm("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(sc + 16 * b));
  return r;
}

// O's columns of a warp's rows times alpha
template <int D>
__device__ __forceinline__ void codes_rescale(uint32_t t_o, float alpha) {
  const uint64_t a2 = pack2(alpha, alpha);
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t x[16];
    tmem_ld16(t_o + c, x);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float a, b;
      unpack2(fmul2(pack2(u2f(x[e]), u2f(x[e + 1])), a2), a, b);
      x[e] = f2u(a);
      x[e + 1] = f2u(b);
    }
    tmem_st16(t_o + c, x);
  }
}

// Codes: softmax of stage s, rows [32 wq, 32 wq + 32), with O's corrections and the epilogue.
template <int D>
__device__ __forceinline__ void codes_softmax(const Params& p, Ctl<kCodes>& ctl, uint32_t tmem, uint8_t* stg, int s, int wq,
                                              int lane, uint64_t LIM) {
  const int row = (wq << 5) + lane;
  const uint32_t t_lane = tmem + (uint32_t(wq) << 21), t_s = t_lane + uint32_t(s * 128), t_o = t_lane + kOCol0 + uint32_t(s * D);
  const int row_tok = row / p.group, row_head = row - row_tok * p.group;
  // ph_of: phases of o_full, bit 0 of this stage's, bit 1 of stage 1's for stage 0. A
  // stage's phase ends with each item that it has tiles of, also where the other's
  // warps wait for it: the bit then turns without a wait (the next wait for it comes
  // after an S that was issued behind those products).
  uint32_t ph_s = 0, ph_st = 0, ph_of = 0;
  int step0 = 0;        // running key-tile counter (trace only)
  uint32_t tiles0 = 0;  // key tiles of the items before
  bool ok = true;
  if (lane == 0) mbar_arrive(&ctl.p_full[s]);  // O may be written
  for (int i = 0; ok; ++i) {
    const Work* const w = next_item(ctl, i, LIM);
    if (w == nullptr) break;
    const bool key = (w->flags & kKeyMode) != 0;
    const int step = step0 + w->a[s];
    step0 += key ? w->n[0] : w->nt;
    const int n = w->n[s];
    const bool mine = (wq << 5) < w->rows[s];  // the warp has rows
    uint32_t tile = tiles0 + uint32_t(key ? s : w->a[s]);
    tiles0 += uint32_t(w->nt);
    float m_run = kLow, l_run = 0.0f;
    // the row's factor (rows past the last: those of other tokens, as Q's are)
    const int f_token = min(w->q0 + (key ? 0 : s * p.tok) + row_tok, p.total_q - 1);
    const float rf = mine ? __ldg(p.q_factor + size_t(f_token) * p.Hq + w->kvh * p.group + row_head) : 0.0f;
    if (n > 0) {
      const int stage_pos = w->pos + (key ? 0 : s * p.tok);
      const int pos = stage_pos + row_tok;  // this row's place among the keys
      const int pos_l = stage_pos + (key ? w->ntok : s == 0 ? p.tok : w->ntok - p.tok) - 1;  // the last row's
      const int klen = w->klen;
      int kb = (w->kt + (key ? s : w->a[s])) * 128;  // the tile's first key
      for (int j = 0; j < n; ++j, kb += key ? 256 : 128, tile += key ? 2 : 1) {
        // the scales of the tile's blocks, there before S is
        const uint32_t ring = tile % kScaleTiles, use = tile / kScaleTiles;
        // (a product of scales that underflows would make -inf * 0 of a masked score)
        auto factor = [&](float a) { return fmaxf(a * rf, 1.1754944e-38f); };
        float f[8], lb[8];
        if (mine) {
          if (!warp_wait(&ctl.codes.sc_full[ring], use & 1, &ctl.abort, LIM)) { ok = false; break; }
          const uint32_t sc = scales_at(ctl.codes.sc[ring]);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const float4 t = scales_of(sc, b);
            f[b] = factor(t.x);
            lb[b] = t.y;
          }
        }
        if (!warp_wait(&ctl.s_full[s], ph_s, &ctl.abort, LIM)) { ok = false; break; }
        ph_s ^= 1;
        if (row == 0) trace_stamp(p.trace, step + j, 4 + 3 * s);
        if (mine) {
          tc_fence_after();
          const bool edge = kb + 127 >= klen || (p.wr >= 0 && kb + 127 > stage_pos + p.wr) || (p.wl >= 0 && kb < pos_l - p.wl);
          int hi = klen - kb, lo = 0;  // columns [lo, hi) are visible
          if (p.wr >= 0) hi = min(hi, pos + p.wr + 1 - kb);
          if (p.wl >= 0) lo = max(lo, pos - p.wl - kb);
          const uint32_t span = uint32_t(max(hi - lo, 0));
          uint32_t v[128];
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (uint32_t(c - lo) >= span) v[c] = f2u(-INFINITY);
          }
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t* z = &v[16 * b];
            float ma = fmax3(u2f(z[0]), u2f(z[1]), u2f(z[2])), mb = fmax3(u2f(z[3]), u2f(z[4]), u2f(z[5]));
#pragma unroll
            for (int c = 6; c < 14; c += 4) {
              ma = fmax3(ma, u2f(z[c]), u2f(z[c + 1]));
              mb = fmax3(mb, u2f(z[c + 2]), u2f(z[c + 3]));
            }
            ma = fmaxf(fmax3(ma, u2f(z[14]), u2f(z[15])), mb);
            mx = fmaxf(mx, fmaf(ma, f[b], lb[b]));
          }
          // A maximum that passes the one held by more than kTau is rare after an item's
          // first tile. (Each row for itself, so that no row's roundings depend on its
          // neighbours.)
          const bool over = mx > m_run + kTau;
          if (__any_sync(0xffffffffu, over)) {
            const float m_new = over ? mx : m_run;
            const float alpha = ex2_mufu(m_run - m_new);  // (0 for the first)
            m_run = m_new;
            l_run *= alpha;
            if (j > 0) codes_rescale<D>(t_o, alpha);  // S is there, so the product before it is done
          }
          const float base = kShift - m_run;
          const uint32_t sc2 = scales_at(ctl.codes.sc[ring]);  // (read again: no registers to keep them in)
          if (row == 0) trace_stamp(p.trace, step + j, 5 + 3 * s);
          uint32_t pk[16];
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const float x = lb[b] + base;
            const uint64_t f2 = pack2(f[b], f[b]), x2 = pack2(x, x);
            uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float a, e;
              unpack2(ffma2(pack2(u2f(v[16 * b + 2 * c]), u2f(v[16 * b + 2 * c + 1])), f2, x2), a, e);
              a = ex2_mufu(a);
              e = ex2_mufu(e);
              const uint64_t pr = pack2(a, e);
              if ((c & 1) == 0) acc0 = c == 0 ? pr : fadd2(acc0, pr);
              if ((c & 1) == 1) acc1 = c == 1 ? pr : fadd2(acc1, pr);
              // P' to f16 (nearest even), the type of the products: off by at most
              // 2^-11 of each that is 2^-21 of the largest; the row sum keeps 32 bits
              pk[8 * (b & 1) + c] = f16x2_of(a, e);
            }
            float la, lb2;
            unpack2(fadd2(acc0, acc1), la, lb2);
            l_run = fmaf(la + lb2, scales_of(sc2, b).z, l_run);
            if (b == 5) {  // the first 64 keys' P' are there: their product may begin
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&ctl.p_full[s]);
                if (j > 0) mbar_arrive(&ctl.p_full[s]);  // for O
              }
            }
            if (b & 1) tmem_st16(t_s + (b >> 1) * 16, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.alpha_full[s]);
          if (row == 0) trace_stamp(p.trace, step + j, 6 + 3 * s);
        } else if (lane == 0) {
          mbar_arrive(&ctl.p_full[s]);
          if (j > 0) mbar_arrive(&ctl.p_full[s]);
          mbar_arrive(&ctl.alpha_full[s]);
        }
      }
      if (!ok) break;
    }
    // ---- epilogue: O and l are 2^kShift of what belongs to m
    float m = m_run == kLow ? -INFINITY : m_run - kShift, l = l_run;
    if (key && s == 1) {  // joined by stage 0's warps
      if (n > 0) {
        if (!warp_wait(&ctl.stats_empty[1], ph_st ^ 1, &ctl.abort, LIM)) break;
        ph_st ^= 1;
        ctl.stat_l[1][row] = l;
        ctl.stat_m[1][row] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.stats_full[1]);
        ph_of ^= 1;
      }
      release_item(ctl, i);
      continue;
    }
    const int nj = key ? w->n[1] : 0;  // > 0: stage 1 is joined
    if (s == 0 && !key && w->n[1] > 0) ph_of ^= 2;
    float f0 = 1.0f, f1 = 0.0f;
    if (nj > 0) {
      if (!warp_wait(&ctl.stats_full[1], ph_st, &ctl.abort, LIM)) break;
      ph_st ^= 1;
      const float l1 = ctl.stat_l[1][row], m1 = ctl.stat_m[1][row];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.stats_empty[1]);
      const float mj = fmaxf(m, m1), mu = mj == -INFINITY ? 0.0f : mj;
      f0 = ex2_mufu(m - mu);  // (0 for a stage that saw no key)
      f1 = ex2_mufu(m1 - mu);
      l = l * f0 + l1 * f1;
      m = mj;
    }
    const bool part = (w->flags & kPart) != 0;
    const float inv = part ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
    f0 *= inv;
    f1 *= inv;
    if (n > 0) {
      if (!warp_wait(&ctl.o_full[s], ph_of & 1, &ctl.abort, LIM)) break;
      ph_of ^= 1;
      if (nj > 0) {
        if (!warp_wait(&ctl.o_full[1], (ph_of >> 1) & 1, &ctl.abort, LIM)) break;
        ph_of ^= 2;
      }
      tc_fence_after();
      if (row == 0) trace_stamp(p.trace, step0 - 1, 10 + s);
    }
    if (mine) {
      // 16 columns of each row at a time go through a staging buffer, so that a store
      // writes 8 rows' whole sectors and not 32 rows' halves. Loops that are not
      // unrolled: code that runs once per item is slow to fetch (32 columns at a time,
      // unrolled: 4 us an item).
      const bool valid = row < w->rows[s];
      const int token = w->q0 + s * p.tok + row_tok, head = w->kvh * p.group + row_head;
      const size_t at = size_t(2 * int(blockIdx.x) + ((w->flags & kCont) ? 0 : 1)) * 256 + s * 128 + row;
      const int dst_row = !valid ? -1 : part ? int(at) : token * p.Hq + head;  // (below 2^31 both)
      const int turn = (lane >> 1) & 3, quarter = lane & 3;  // neighbouring rows' pieces in other banks
      uint8_t* dst[4];  // of this lane's quarter of rows 8 e + lane / 4
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int to = __shfl_sync(0xffffffffu, dst_row, 8 * e + (lane >> 2));
        dst[e] = to < 0 ? nullptr
                        : (part ? reinterpret_cast<uint8_t*>(p.part_o + size_t(to) * D + 4 * quarter)
                                : reinterpret_cast<uint8_t*>(p.o + size_t(to) * D + 4 * quarter));
      }
      // (the converters' word, from before the products that o_full told of)
      const bool nans = n > 0 && valid && *const_cast<volatile uint32_t*>(&ctl.codes.nans[i % kItems]) != 0;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t x[16];
        tmem_ld16(t_o + c, x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = n > 0 ? f2u(u2f(x[e]) * f0) : 0u;
        if (nj > 0) {
          uint32_t y[16];
          tmem_ld16(t_o + D + c, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = f2u(fmaf(u2f(y[e]), f1, u2f(x[e])));
        }
        if (nans) {
          const int pos = w->pos + (key ? 0 : s * p.tok) + row_tok, k0 = w->kt * 128, k1 = min(w->klen, k0 + w->nt * 128);
          const uint32_t bits = hidden_nans(p, w->kbase, p.wl >= 0 ? max(k0, pos - p.wl) : k0,
                                            p.wr >= 0 ? min(k1, pos + p.wr + 1) : k1, w->klen,
                                            seen_by_all(p, w->pos, w->ntok), p.v_codes + 1LL * w->kvh * D + c, D);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (bits >> e & 1) x[e] = 0x7fffffffu;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(stg + lane * 64 + ((e ^ turn) << 4)) =
              make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = 8 * e + (lane >> 2);
          const float4 y = *reinterpret_cast<const float4*>(stg + rr * 64 + ((quarter ^ ((rr >> 1) & 3)) << 4));
          if (part) {
            if (dst[e] != nullptr) *reinterpret_cast<float4*>(dst[e] + c * 4) = y;
          } else {
            if (dst[e] != nullptr)
              *reinterpret_cast<uint2*>(dst[e] + c * 2) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
          }
        }
        __syncwarp();  // (the next read of tensor memory is one of the whole warp)
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
    release_item(ctl, i);
  }
}

template <int D, Kind KIND>
__global__ void __launch_bounds__(kThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const Params p) {
  using C = Tiles<D>;
  constexpr bool PAGED = KIND != kPacked, CODES = KIND == kCodes;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl<KIND> ctl;
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
      mbar_init(&ctl.tail_done[i], CODES ? 4 : 1);
    }
    if constexpr (CODES) {
      for (int i = 0; i < C::kKSlots; ++i) {
        mbar_init(&ctl.codes.k_full[i], 1);
        mbar_init(&ctl.codes.k_empty[i], 1);
      }
      for (int i = 0; i < kScaleTiles; ++i) mbar_init(&ctl.codes.sc_full[i], 4);
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
  // The plan; of codes also Q's parts, for which only Q's producer and the softmax warps
  // (their rows' factors) wait where there is no plan: the lengths are a caller's, there
  // before the kernel that makes the parts began.
  if (!CODES || p.items != nullptr || wg <= 1 || warp == 12) grid_dep_wait();
  grid_dep_launch();  // the joining kernel may start (and wait) meanwhile
  const uint32_t tmem = ctl.tmem_base;
  auto item = [&](int i) { return next_item(ctl, i, LIM); };
  auto release = [&](int i) { release_item(ctl, i); };

  if (CODES && wg <= 2) {
    if constexpr (CODES) {
      if (wg <= 1) {
        setmaxnreg_inc<168>();
        codes_softmax<D>(p, ctl, tmem, sStg + warp * 2048, wg, warp & 3, lane, LIM);
      } else {
        setmaxnreg_dec<104>();
        codes_convert<D>(p, ctl, sKV, warp & 3, lane, LIM);
      }
    }
  } else if (wg <= 1) {
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
          if (CODES) {  // its high and its low parts
            for (int c = 0; c < 2; ++c)
              tma_load_4d_hint(sQ + b * C::kTileBytes + c * (C::kTileBytes / 2), &tmQ, &ctl.q_full[b], 0, 0,
                               c * p.total_q + w->q0 + (key ? 0 : s * p.tok), kvh, pol_q);
          } else
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
        const uint32_t entry =
            CODES ? base + uint32_t(t) : base + uint32_t(is_v ? (t < nt - d ? d + 2 * t : nt + t) : (t < d ? t : 2 * t - d + 1));
        const uint32_t slots = !CODES ? C::kSlots : is_v ? C::kVSlots : C::kKSlots, slot = entry % slots, use = entry / slots;
        uint8_t* dst = sKV + (!CODES ? slot * C::kTileBytes : is_v ? C::kVRing + slot * C::kTileBytes : slot * C::kKBytes);
        uint64_t *full = &ctl.kv_full[slot], *empty = &ctl.kv_empty[slot];
        if constexpr (CODES) {
          if (!is_v) {
            full = &ctl.codes.k_full[slot];
            empty = &ctl.codes.k_empty[slot];
          }
        }
        // (The warp's entry before this one is at most 3 back: what it waited
        // for has been taken, and all before it, so that this wait is for the
        // slot's last use and no earlier one.)
        ok = warp_wait(empty, (use & 1) ^ 1, abort_flag, LIM);
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
          if (CODES) {
            if (elect_one()) {
              mbar_arrive_expect_tx(full, uint32_t(at.boxes * p.box_rows * D));
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                if (x >= at.boxes) break;
                // K's rows of codes follow one another, 32 of V's stand where those of 64 values will
                const int r = x * p.box_rows;
                tma_load_4d_hint(dst + (is_v ? (r >> 5) * 4096 + (r & 31) * D : r * D), m, full, 0, kvh,
                                 in_page[x], page[x], pol_kv);
              }
            }
          } else if (elect_one()) {
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
        if (!CODES && is_v && t == nt - 1 && fill != 0) {
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
      base += uint32_t(CODES ? nt : 2 * nt);
      release(i);
    }
  } else if (warp == 13) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks the role and an elected lane issues (with the
    // producer's and all waits, 1.78 -> 1.29 ms on one causal sequence of 16384
    // tokens, against one lane walking: MMA operands are uniform registers).
    {
      const uint32_t idS = (CODES ? idesc_codes_f32(128, 128) : idesc_bf16_f32(128, 128, 0, 0)) | (p.neg_s << 13);
      constexpr uint32_t idPV = CODES ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
      const uint32_t dq = sdesc_lo(smem_u32(sQ), 16), dk = sdesc_lo(smem_u32(sKV), 16),
                     dv = sdesc_lo(smem_u32(sKV) + (CODES ? C::kVRing : 0), 16384);
      // Phases of the barriers of each stage (or slot), a bit each: arrays
      // indexed by the stage would be kept in memory.
      uint32_t phases = 0, tail_phases = 0;
      uint32_t E = 0, EK = 0, key_items = 0;  // ring entry that follows (over codes V's, K's)
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
        constexpr int kSlots = CODES ? C::kVSlots : C::kSlots;
        slot = E % kSlots;
        const uint32_t phase = (E / kSlots) & 1;
        ++E;
        return wait(&ctl.kv_full[slot], phase);
      };
      // the next K tile of codes
      auto wait_k = [&](uint32_t& slot) -> bool {
        if constexpr (CODES) {
          slot = EK % C::kKSlots;
          const uint32_t phase = (EK / C::kKSlots) & 1;
          ++EK;
          return wait(&ctl.codes.k_full[slot], phase);
        } else {
          return wait_kv(slot);
        }
      };
      auto k_empty = [&](uint32_t slot) -> uint64_t* {
        if constexpr (CODES) {
          return &ctl.codes.k_empty[slot];
        } else {
          return &ctl.kv_empty[slot];
        }
      };
      // rows of a V tile past the sequence's end zeroed
      auto wait_tail = [&](uint32_t slot) -> bool {
        const uint32_t phase = (tail_phases >> slot) & 1;
        tail_phases ^= 1u << slot;
        return wait(&ctl.tail_done[slot], phase);
      };
      // O of stage s (+)= P V; S of stage s = Q (buffer b) K^T
      // (over codes, where the softmax has more to do for a tile, the product of its
      // first 64 keys does not wait for the others' P)
      auto issue_pv = [&](int s, uint32_t slot, bool acc) {
        const uint32_t b0 = sdesc_step(dv, slot * C::kTileBytes);
        if constexpr (CODES) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts_lo(tmem + kOCol0 + uint32_t(s * D), tmem + uint32_t(s * 128) + kk * 8, sdesc_step(b0, kk * 2048), idPV,
                        (acc || kk > 0) ? 1u : 0u);
          }
          __syncwarp();
          if (!wait_phase(&ctl.alpha_full[s], kPhP2 + s)) {
            ok = false;
            return;
          }
        }
        tc_fence_after();
        if (!elect_one()) return;
#pragma unroll
        for (int kk = CODES ? 4 : 0; kk < 8; ++kk)
          mma_ts_lo(tmem + kOCol0 + uint32_t(s * D), tmem + uint32_t(s * 128) + kk * 8, sdesc_step(b0, kk * 2048), idPV,
                    (acc || kk > 0) ? 1u : 0u);
      };
      auto issue_s = [&](int s, uint32_t b, uint32_t slot) {
        tc_fence_after();
        if (!elect_one()) return;
        const uint32_t q0 = sdesc_step(dq, b * C::kTileBytes), b0 = sdesc_step(dk, slot * (CODES ? C::kKBytes : C::kTileBytes));
        if constexpr (CODES) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // 32 of d at a time, Q's high and then its low parts
            const uint32_t ko = kk % (D / 32) * 32;
            const uint32_t qo = kk / (D / 32) * (C::kTileBytes / 2) + ko;
            mma_codes_lo<D == 128 ? kSdescHi : kSdescHi64>(tmem + uint32_t(s * 128), sdesc_step(q0, qo), sdesc_step(b0, ko), idS,
                                                        kk > 0);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_ss_lo(tmem + uint32_t(s * 128), sdesc_step(q0, ko), sdesc_step(b0, ko), idS, kk > 0);
          }
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
              ok = wait_kv(slot) && ((!CODES && (!fill || t < nt - 1)) || wait_tail(slot)) && wait_phase(&ctl.p_full[s], kPhP + s);
              if (!ok) break;
              if (s == 0) trace(p.trace, step0 + (t >> 1), 0);
              issue_pv(s, slot, t > 1);
              if (t + 2 >= nt) commit(&ctl.o_full[s]);
              commit(&ctl.kv_empty[slot]);
            }
            if (t + 2 < nt) {
              ok = wait_k(slot);
              if (!ok) break;
              issue_s(s, b, slot);
              commit(k_empty(slot));
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
              ok = wait_kv(vs) && ((!CODES && (!fill || k)) || wait_tail(vs));
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
              ok = wait_k(ks);
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
              commit(k_empty(ks));
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
        constexpr int kParts = CODES ? 2 : C::kChunks;
        const int c = CODES ? 0 : lane % kParts * 64, what = lane / kParts, t0 = CODES ? lane % kParts * p.total_q : 0;
        if (x.nt > 0) {
          if (what < 2) {
            if ((what == 0 ? x.n[0] : x.n[1]) > 0 && !(what == 1 && (x.flags & kKeyMode)))
              tma_prefetch_l2_4d(&tmQ, c, 0, t0 + x.q0 + what * p.tok, x.kvh);
          } else if (!PAGED && what < 4) {
            tma_prefetch_l2_4d(what == 2 ? &tmK : &tmV, c, x.kvh, x.kbase + x.kt * 128, 0);
          }
        }
      }
      const int i = n_done++;
      if (!warp_wait(&ctl.it_empty[i % kItems], ((i / kItems) & 1) ^ 1, abort_flag, LIM)) return false;
      if (lane == 0) {
        ctl.it[i % kItems] = x;
        if constexpr (CODES) ctl.codes.nans[i % kItems] = 0;
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

// Codes: Q's rows, divided by a power of two, as sums of two e4m3 values (see Codes),
// high parts [total_q, Hq, D] and then the low ones, and what each row was divided by.
// A pass of its own, over as many bytes as Q has twice: done by the warps of the main
// kernel that wait for it, it took 15 us of each item of two row tiles.
template <int D>
__global__ void __launch_bounds__(256) codes_q_kernel(const __nv_bfloat16* q, long long q_stride, int rows, int Hq,
                                                      uint8_t* hi_out, uint8_t* lo_out, float* factor) {
  constexpr int kLanes = D / 8, kAtOnce = 256 / kLanes, kBatch = 4;
  grid_dep_launch();
  const int col = threadIdx.x % kLanes, r0 = blockIdx.x * (kAtOnce * kBatch) + threadIdx.x / kLanes;
  uint4 x[kBatch];
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    const int r = r0 + e * kAtOnce, tok = r / Hq;
    x[e] = make_uint4(0, 0, 0, 0);
    if (r < rows) x[e] = __ldg(reinterpret_cast<const uint4*>(q + tok * q_stride + 1LL * (r - tok * Hq) * D + col * 8));
  }
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    const int r = r0 + e * kAtOnce;
    uint32_t m = max_u16x2(max_u16x2(x[e].x & 0x7fff7fffu, x[e].y & 0x7fff7fffu),
                          max_u16x2(x[e].z & 0x7fff7fffu, x[e].w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (r >= rows) continue;
    // the row's largest value into [2^7, 2^8); a row that is not finite becomes NaN
    const int ex = max(int(m >> 7) - 127, -100) - 7;
    const float f = m < 0x7f80u ? exp2i(-ex) : __int_as_float(0x7fffffff);
    const uint32_t y[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = u2f(y[k] << 16) * f, c = u2f(y[k] & 0xffff0000u) * f;
      const uint32_t h = e4m3x2_of(a, c), back = f16x2_of_e4m3x2(uint16_t(h));
      const uint32_t l = e4m3x2_of(a - f16_lo(back), c - f16_hi(back));
      hi[k >> 1] |= h << (16 * (k & 1));
      lo[k >> 1] |= l << (16 * (k & 1));
    }
    *reinterpret_cast<uint2*>(hi_out + size_t(r) * D + col * 8) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(lo_out + size_t(r) * D + col * 8) = make_uint2(lo[0], lo[1]);
    if (col == 0) factor[r] = exp2i(ex);
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
  uint8_t* q_parts;  // codes: Q's high and low parts
  float* q_factor;
  size_t bytes;
};
Space carve(uint8_t* base, const SeqProblem& pb, int G, long long units, bool codes) {
  Space s{};
  Carver c{base, 0};
  s.plan = carve_plan<FwdItem>(c, pb.B, units, pb.Hkv, G);
  s.part_ml = c.take<float2>(size_t(2) * G * 256);
  s.part_o = c.take<float>(size_t(2) * G * 256 * pb.d);
  if (codes) {
    s.q_parts = c.take<uint8_t>(size_t(2) * pb.total_q * pb.Hq * pb.d);
    s.q_factor = c.take<float>(size_t(pb.total_q) * pb.Hq);
  }
  s.bytes = c.at;
  return s;
}

template <int D, Kind KIND>
cudaError_t launch_t(const SeqProblem& pb, const Fp8Scales* sc, void* o, float* lse, cudaStream_t stream) {
  using C = Tiles<D>;
  constexpr bool PAGED = KIND != kPacked;
  constexpr int few_units = Ctl<KIND>::kUnits;
  const int G = std::min(num_sms(), seq::kMaxWorkers);
  const int group = pb.Hq / pb.Hkv, tok = 128 / group;
  Params p{};
  // q: rows (token, head of the group), `tok` tokens to a tile
  CUtensorMap mq{}, mk, mv;
  if constexpr (KIND != kCodes) {
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), uint64_t(pb.total_q), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(pb.q_stride) * 2, uint64_t(group) * D * 2};
    const uint32_t box[4] = {64, uint32_t(group), uint32_t(tok), 1};
    if (!encode_tiled(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pb.q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  // o: the 32 rows of a warp, where they are whole tokens
  CUtensorMap mo = mq;
  if (KIND != kCodes && 32 % group == 0) {
    p.o_box = 32 / group;
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), uint64_t(pb.total_q), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D) * 2, uint64_t(pb.Hq) * D * 2, uint64_t(group) * D * 2};
    const uint32_t box[4] = {64, uint32_t(group), uint32_t(p.o_box), 1};
    if (!encode_tiled(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, o, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if constexpr (KIND == kCodes) {
    // rows of D bytes; 32 of 64 bytes go together (see the producers)
    p.box_rows = D == 128 ? 128 : 32;
    while (pb.page_size % p.box_rows != 0) p.box_rows /= 2;  // 16 at least
    if (!encode_codes(&mk, pb.k, pb.num_pages, pb.page_size, pb.Hkv, D, p.box_rows,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_codes(&mv, pb.v, pb.num_pages, pb.page_size, pb.Hkv, D, p.box_rows,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
    p.scales[0] = sc->k;
    p.scales[1] = sc->v;
    p.v_codes = static_cast<const uint8_t*>(pb.v);
  } else if constexpr (PAGED) {
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
  auto kern = seq_fwd_kernel<D, KIND>;
  static SmemLimit limit;
  cudaError_t e = limit.set(kern, C::kSmemDyn);
  if (e != cudaSuccess) return e;
  // a sequence of n tokens has ceil(n / (2 tok)) units
  long long units = pb.total_q / (2 * tok) + pb.B;
  if (units > pb.total_q) units = pb.total_q;
  const bool few = pb.B <= few_units && units <= few_units && units * pb.Hkv <= (PAGED ? kFewRounds : 1) * G;
  // Few items of few key tiles are never divided: no workspace, no last kernel.
  long long keys = pb.page_table != nullptr ? 1LL * pb.max_pages * pb.page_size : pb.total_k;
  if (pb.window_left >= 0 && pb.window_right >= 0)  // and whole tiles around those that a unit sees
    keys = std::min(keys, 2LL * tok + pb.window_left + pb.window_right + 254);
  const bool whole = KIND != kCodes && few && units * pb.Hkv <= G && (keys + 127) / 128 + kItemCost <= FwdSide::kPartsCost;
  void* ws = nullptr;
  Space sp{};
  if (!whole) {
    cudaMemPool_t pool = workspace_pool();
    if (pool == nullptr || cudaMallocFromPoolAsync(&ws, carve(nullptr, pb, G, units, KIND == kCodes).bytes, pool, stream) != cudaSuccess)
      return cudaErrorMemoryAllocation;
    sp = carve(static_cast<uint8_t*>(ws), pb, G, units, KIND == kCodes);
  }
  if constexpr (KIND == kCodes) {
    const uint64_t row = uint64_t(pb.Hq) * D;
    const uint64_t dims[4] = {uint64_t(D), uint64_t(group), 2 * uint64_t(pb.total_q), uint64_t(pb.Hkv)};
    const uint64_t strides[3] = {uint64_t(D), row, uint64_t(group) * D};
    const uint32_t box[4] = {uint32_t(D), uint32_t(group), uint32_t(tok), 1};
    if (!encode_tiled(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, sp.q_parts, dims, strides, box,
                      D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)) {
      cudaFreeAsync(ws, stream);
      return cudaErrorInvalidValue;
    }
    mo = mq;  // (not used)
    p.q_factor = sp.q_factor;
    const int rows = pb.total_q * pb.Hq, per_block = 256 / (D / 8) * 4;
    codes_q_kernel<D><<<unsigned((rows + per_block - 1LL) / per_block), 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(pb.q), pb.q_stride, rows, pb.Hq, sp.q_parts, sp.q_parts + size_t(pb.total_q) * row,
        sp.q_factor);
    e = cudaGetLastError();
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
  if (!few && e == cudaSuccess) {
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
  lc.numAttrs = few && KIND != kCodes ? 0 : 1;
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
    return paged ? seq::launch_t<128, seq::kPaged>(pb, nullptr, o, lse, stream)
                 : seq::launch_t<128, seq::kPacked>(pb, nullptr, o, lse, stream);
  return paged ? seq::launch_t<64, seq::kPaged>(pb, nullptr, o, lse, stream)
               : seq::launch_t<64, seq::kPacked>(pb, nullptr, o, lse, stream);
}

cudaError_t launch_seq_fwd_codes(const SeqProblem& pb, const Fp8Scales& sc, void* o, float* lse, cudaStream_t stream) {
  return pb.d == 128 ? seq::launch_t<128, seq::kCodes>(pb, &sc, o, lse, stream)
                     : seq::launch_t<64, seq::kCodes>(pb, &sc, o, lse, stream);
}

}  // namespace fa
