// Host-side declarations shared by the translation units of libfa.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// Status bits written by kernels into the per-device status word.
constexpr unsigned kDevTimeout = 1u;
constexpr unsigned kDevBadArg = 2u;  // lengths or pages on the device that the tensors cannot hold

struct Problem {
  const void* q;
  const void* k;
  const void* v;
  int B, Hq, Hkv, Nq, Nk, d;
  float scale;
  int causal;
  // sliding window: key j visible to query i iff i + off - window_left <= j
  // <= i + off + window_right (off = Nk - Nq); -1 = no limit on that side
  int window_left = -1, window_right = -1;
  // backward: largest workspace the call may use (0: any); the tail pieces
  // fall back to whole single tiles when their slots would not fit
  size_t ws_cap = 0;
  bool masked() const { return causal || window_left >= 0 || window_right >= 0; }
  // the causal mask and nothing else (window bounds already normalised)
  bool plain_causal() const { return window_left < 0 && (causal || window_right == 0); }
};

struct DebugCfg {
  unsigned long long wait_limit_ns;
  int inject;
  cudaEvent_t ev_begin;  // recorded around the main kernel when set
  cudaEvent_t ev_end;
  unsigned long long* trace;  // optional device trace buffer
  int poly_every;             // forward exp2 split (fa_tune FA_TUNE_EXP2_SPLIT)
  int cta_pairs;              // forward on CTA pairs (fa_tune FA_TUNE_CTA_PAIRS)
  int bwd_split;              // causal backward split count, -1 = model (fa_tune FA_TUNE_BWD_SPLIT)
};
DebugCfg debug_cfg();

// Per-device stream-ordered pool for the backward workspace (nullptr if it
// could not be created).
cudaMemPool_t workspace_pool();

// Device properties cached per device.
int num_sms();

// The calling thread's current context by its id (no two have the same, also
// after one was destroyed); 0 if it has none.
unsigned long long context_id();

// Status word of the current context (device pointer).
unsigned* status_word();

// 4-D bf16 tensor map over a BSHD tensor [B, N, H, d]: dims {d, H, N, B},
// box {64, 1, box_rows, 1}, 128-byte swizzle, zero fill out of range.
bool make_bshd_map(CUtensorMap* m, const void* base, int B, int N, int H, int d, int box_rows);

// Any tiled tensor map: rank <= 5, dims innermost first, strides (bytes) of
// dims 1..rank-1, zero fill out of range; promotion: what L2 fetches at least.
bool encode_tiled(CUtensorMap* m, CUtensorMapDataType dtype, int rank, const void* base, const uint64_t* dims,
                  const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle,
                  CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
// A tensor map over pages of codes [num_pages, page_size, Hkv, d]: boxes of box_rows
// rows of one head. L2 fetches no more than the row's own bytes: the next head's, of
// which 256 bytes would have some too, are gone before their turn (two single tokens
// over 116000 and 131000 keys read 668 MB and not 506).
inline bool encode_codes(CUtensorMap* m, const void* pages, int num_pages, int page_size, int Hkv, int d, int box_rows,
                         CUtensorMapSwizzle swizzle) {
  const uint64_t row = uint64_t(Hkv) * d;
  const uint64_t dims[4] = {uint64_t(d), uint64_t(Hkv), uint64_t(page_size), uint64_t(num_pages)};
  const uint64_t strides[3] = {uint64_t(d), row, row * page_size};
  const uint32_t box[4] = {uint32_t(d), 1, uint32_t(box_rows), 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pages, dims, strides, box, swizzle,
                      d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
}

// Window bounds as the kernels take them: negative -> -1 (no limit); a
// bound that reaches past every key (>= Nq + Nk) is no limit either.
int normalize_window(int w, int Nq, int Nk);

// The forward's exponent scale, scale * log2(e). A zero scale (every visible
// key equally weighted) becomes 2^-100: the scaled scores are then 0 to
// within fp32 rounding while a masked score (-inf) still gives probability 0,
// which 0 * -inf would not.
inline float exp_scale_log2(float scale) {
  return scale == 0.0f ? 7.888609052210118e-31f : scale * 1.4426950408889634f;
}

// Launchers. Return a cudaError_t (cudaSuccess on success).
cudaError_t launch_fwd(const Problem& p, void* o, float* lse, cudaStream_t stream);
// FP8 (e4m3) forward, d = 128 only; incoherent != 0 applies the Hadamard
// transform to Q and K before quantisation. Workspace from the pool.
cudaError_t launch_fwd8(const Problem& p, void* o, float* lse, int incoherent, cudaStream_t stream);
// The host-side checks fa_bwd performs (pointers, sizes, device), as one call.
int check_bwd_args(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                   void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                   int causal);

// Backward workspace (fp32 dQ accumulator, padded LSE*log2e and D rows).
size_t bwd_workspace_bytes(const Problem& p);
// kernels fa_bwd launches for p
int bwd_launch_count(const Problem& p);
cudaError_t launch_bwd(const Problem& p, const void* o, const float* lse, const void* dout, void* dq, void* dk,
                       void* dv, float* ws, cudaStream_t stream);

// Sequences of different lengths (fa_fwd_varlen, fa_fwd_paged): lengths and
// pages are device arrays. Strides are elements between tokens.
struct SeqProblem {
  const void* q;
  const void* k;  // packed [total_k, Hkv, d], or pages [num_pages, page_size, Hkv, d]
  const void* v;
  const int* cu_q;        // [B + 1]
  const int* cu_k;        // packed: [B + 1]
  const int* lens_k;      // paged: [B]
  const int* page_table;  // paged: [B, max_pages]; null: packed
  int B, Hq, Hkv, total_q, total_k, d;
  int num_pages, page_size, max_pages;
  long long q_stride, k_stride, v_stride;
  float scale;
  int window_left, window_right;  // -1: no limit
};
// Tiles of 128 / group tokens that B sequences of total_q tokens fill at most,
// each its last one in part.
inline long long seq_row_tiles(const SeqProblem& p) {
  const long long tiles = p.total_q / (128 / (p.Hq / p.Hkv)) + 1LL * p.B;
  return tiles < p.total_q ? tiles : p.total_q;
}
// cudaErrorMemoryAllocation: the workspace could not be allocated
cudaError_t launch_seq_fwd(const SeqProblem& p, void* o, float* lse, cudaStream_t stream);
cudaError_t launch_seq_bwd(const SeqProblem& p, const void* o, const float* lse, const void* dout, void* dq, void* dk,
                           void* dv, cudaStream_t stream);

// Rows of k and v (row strides in elements) into the pages.
struct AppendProblem {
  const void* k;
  const void* v;
  void* k_pages;
  void* v_pages;
  const int* cu_q;
  const int* lens_k;
  const int* page_table;
  int B, Hkv, total_q, d;
  int num_pages, page_size, max_pages;
  long long k_stride, v_stride;
};
cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t stream);

// A cache in e4m3: the pages of SeqProblem and AppendProblem hold codes, and
// these their scales, [num_pages, page_size / 16, Hkv].
struct Fp8Scales {
  const float* k;
  const float* v;
};
cudaError_t launch_cache_append8(const AppendProblem& p, float* k_scales, float* v_scales, cudaStream_t stream);
// as the packed and paged forward (any rows), and for few rows to a kv head
cudaError_t launch_seq_fwd_codes(const SeqProblem& p, const Fp8Scales& sc, void* o, float* lse, cudaStream_t stream);
cudaError_t launch_seq_fwd8(const SeqProblem& p, const Fp8Scales& sc, void* o, float* lse, cudaStream_t stream);

// q and k turned by their places (strides in elements; Hq or Hk 0: none).
struct RotaryProblem {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const float* inv_freq;  // [rot / 2]
  const int* cu_q;
  const int* lens;        // [B], or null: sequences begin at place 0
  int B, Hq, Hk, total, d, rot;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  float mscale;
  int interleaved, transposed;
};
cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream);

cudaError_t launch_debug_exp2(const float* x, float* y, int n, int mode, cudaStream_t stream);

}  // namespace fa
