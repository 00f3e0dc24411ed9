/*
 * fa.h — C ABI of the exact-attention library for one NVIDIA GB300 (sm_103a).
 *
 * What is computed. Exact scaled-dot-product attention
 *     O = softmax(scale * Q K^T [+ causal mask]) V
 * (the post "FlashAttention v1", deep_school #630, section "Проблема
 * базового attention"), evaluated tile by tile with online softmax so the
 * Nq x Nk score matrix never reaches device memory (same post, sections
 * "Тайлинг (Tiling)" and "Онлайн-Softmax"). The result equals the classical
 * softmax up to floating-point rounding. The backward pass recomputes the
 * probabilities from the saved log-sum-exp instead of storing them (the
 * FlashAttention-3 summary on news.hada.io, section "Resumo do
 * FlashAttention": tiling and recomputation).
 *
 * Conventions shared by every call.
 *   Layout   : contiguous, head dimension innermost ("BSHD").
 *              q, o, dout, dq : [B, Nq, Hq, d]   bf16
 *              k, v, dk, dv   : [B, Nk, Hkv, d]  bf16
 *              lse            : [B, Hq, Nq]      fp32, natural log:
 *                               lse[b,h,i] = ln sum_j exp(scale * q_i . k_j)
 *                               over the keys j visible to row i.
 *   GQA      : query head h reads kv head h / (Hq / Hkv); Hq % Hkv == 0.
 *   Causal   : causal = 1 hides key j from query i when j > i + (Nk - Nq)
 *              (bottom-right alignment; with Nq == Nk this is j > i). A row
 *              that sees no key gets o = 0 and lse = -inf.
 *   Sizes    : B, Hq, Hkv, Nq, Nk >= 1; d in {64, 128}; scale any finite
 *              value (negative: the softmax of the negated scores; zero:
 *              every visible key weighted equally); every element count
 *              and B*Hq*Nq*d fit in int32 indices per the limits checked
 *              below.
 *   Pointers : device pointers owned by the caller, 16-byte aligned. The
 *              library keeps no pointer after a call returns.
 *   Stream   : `stream` is a cudaStream_t (NULL = legacy default stream).
 *              Calls only enqueue work; outputs are valid once the stream
 *              has been synchronised. The calls are not re-entrant on one
 *              stream from several host threads.
 *   Errors   : argument errors are detected on the host before anything is
 *              enqueued and return FA_ERR_INVALID_ARG / FA_ERR_UNSUPPORTED.
 *              A failed launch returns FA_ERR_LAUNCH. Every wait inside the
 *              kernels is bounded; a wait that runs out stops the kernel and
 *              records FA_ERR_TIMEOUT in a status word of the device (one per
 *              context, where a caller uses several) that fa_get_status()
 *              returns.
 */
#ifndef FA_H_
#define FA_H_

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad scale or flag */
  FA_ERR_UNSUPPORTED = 2, /* valid request this build does not serve (e.g. d not in {64,128}) */
  FA_ERR_ALLOC = 3,       /* device workspace allocation failed */
  FA_ERR_LAUNCH = 4,      /* a CUDA call or kernel launch failed */
  FA_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (reported by fa_get_status) */
  FA_ERR_NO_DEVICE = 6    /* no usable sm_103 device is current */
} fa_status;

/*
 * fa_fwd — forward pass.
 *   in : q [B,Nq,Hq,d], k [B,Nk,Hkv,d], v [B,Nk,Hkv,d]   (bf16, device)
 *   out: o [B,Nq,Hq,d] (bf16), lse [B,Hq,Nq] (fp32)        (device)
 * Needs no device workspace. All outputs are fully written.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int Nk,
           int d, float scale, int causal, void* stream);

/*
 * fa_fwd_window — the forward pass with a sliding-window (local) mask (the
 *   FlashAttention-4 article on smntcn.com names variable and local masks;
 *   the pages do not define them, so this is the causal mask's bottom-right
 *   alignment with two bounds).
 *   Key j is visible to query row i iff
 *       i + off - window_left <= j <= i + off + window_right,  off = Nk - Nq
 *   (the bottom-right alignment of the causal mask); a negative bound, or one
 *   of at least Nq + Nk, means no limit on that side. window_right = 0 with
 *   window_left < 0 is the causal mask; both negative is fa_fwd non-causal.
 *   Rows that see no key get O = 0 and LSE = -inf. Key tiles outside every
 *   row's window are skipped, so the work scales with the window.
 *   Arguments, layouts, ownership and errors otherwise as fa_fwd.
 */
int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                  int Nk, int d, float scale, int window_left, int window_right, void* stream);

/*
 * fa_fwd_fp8 — the forward pass with e4m3 (FP8) tensor-core GEMMs, d = 128.
 *   Inputs, outputs, layouts and the causal flag as fa_fwd (bf16 q, k, v in,
 *   bf16 o and fp32 lse out). incoherent = 1 first multiplies Q and K along
 *   d by diag(signs) H_128 / sqrt(128) (H the Sylvester-Hadamard matrix;
 *   sign_i = -1 where bit 31 of 2654435769 * (i + 1) mod 2^32 is set), which
 *   leaves Q K^T unchanged and spreads outlier channels; incoherent = 0
 *   skips it. Q (transformed), K (transformed) and V are then divided per
 *   (batch, head) by the smallest power of two that brings their largest
 *   magnitude to at most 448 (into (224, 448]) and rounded to e4m3 (nearest,
 *   ties to even; a division by a power of two is exact, so each code is the
 *   rounding of the exact quotient); P is rounded to e4m3 for the P V GEMM.
 *   The result approximates fa_fwd's: O is the attention of the dequantised
 *   tensors up to the rounding of P. (The FlashAttention-3 summary on
 *   news.hada.io, sections on FP8 and incoherent processing: e4m3 GEMMs,
 *   and a random orthogonal transform that spreads outliers before
 *   quantisation.)
 *   Workspace: the e4m3 copies (B*(Nq*Hq + Nk*Hkv)*128 bytes plus
 *   B*Hkv*128*ceil(Nk/128)*128 for V transposed) and per-head maxima, from
 *   the per-device pool fa_bwd uses, on `stream`.
 *   Errors as fa_fwd; d != 128 returns FA_ERR_UNSUPPORTED; incoherent other
 *   than 0/1 returns FA_ERR_INVALID_ARG.
 */
int fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
               int Nk, int d, float scale, int causal, int incoherent, void* stream);

/*
 * fa_bwd — backward pass for L = sum(dout * o).
 *   in : q, k, v, o (bf16), lse (fp32, as written by fa_fwd for the same
 *        inputs), dout [B,Nq,Hq,d] (bf16)
 *   out: dq [B,Nq,Hq,d], dk [B,Nk,Hkv,d], dv [B,Nk,Hkv,d] (bf16), fully written.
 * Allocates its fp32 workspace (dq accumulator, row terms D_i) with the
 * stream-ordered allocator on `stream`, from a memory pool the library keeps
 * per device, and frees it on the same stream; the pool keeps freed memory
 * (up to the largest workspace used so far) for later calls until the
 * process exits. Returns FA_ERR_ALLOC if the allocation fails. GQA gradients of dk/dv are summed over
 * the query heads of each group inside the kernel.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout, void* dq,
           void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
           void* stream);

/*
 * fa_bwd_window — the backward pass of fa_fwd_window: the same window
 *   bounds (and the o, lse that fa_fwd_window wrote); key tiles and query
 *   tiles outside every window are skipped. Arguments, layouts, workspace
 *   and errors otherwise as fa_bwd.
 */
int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                  int window_left, int window_right, void* stream);

/*
 * fa_step_host — one forward and backward pass on HOST buffers: the
 * end-to-end call for a caller whose tensors live in host memory. The
 * operations are those of fa_fwd followed by fa_bwd (same arguments, layouts
 * and results), with every pointer a host address:
 *   in : q [B,Nq,Hq,d], k, v [B,Nk,Hkv,d], dout [B,Nq,Hq,d] (bf16)
 *   out: o [B,Nq,Hq,d] (bf16), lse [B,Hq,Nq] (fp32), dq, dk, dv (bf16).
 * The batch is processed in chunks and pipelined over library-owned
 * streams (one copy stream each way, one compute stream): a chunk is one
 * batch element, or, for a batch of one element with an even Hkv, one half
 * of its kv heads with their query heads (copied as 2-D slices of the head
 * dimension). The forward runs as two launches over halves of the chunks:
 * the first starts once its half's q, k, v are in, and its O and LSE go
 * out while the second runs; dout is copied in meanwhile. The backward runs
 * as one launch over all chunks, and dq, dk, dv go out after it.
 * The call only enqueues; `stream` is ordered after all of it, so
 * synchronise `stream` before reading the outputs, and keep every host
 * buffer alive (and the inputs unchanged) until then. Nothing of the
 * call waits for earlier work on `stream` (the copies and kernels touch only
 * the host buffers and the library's device buffers): the host inputs must
 * hold their values when the call is made. Consecutive calls therefore
 * overlap: the inputs of one call are copied in while the previous call
 * computes, and its kernels start while the previous call's last results
 * are still being copied out.
 * Page-locked host memory gives asynchronous, full-speed copies; pageable
 * memory works but the copies are staged by the driver.
 * Device memory: two library-owned buffers per device, each a copy of every
 * tensor of the batch (about the size of all inputs and outputs), used by
 * alternate calls and kept (grown to the largest call) until the process
 * exits; a call waits only for the call two before it to release its
 * buffer. Calls from several host threads on one device are serialised
 * while they enqueue. Plus the backward's own workspace from its pool.
 * Errors: a null pointer or a bad size gives FA_ERR_INVALID_ARG /
 * FA_ERR_UNSUPPORTED before anything is enqueued; FA_ERR_ALLOC if the device
 * copy cannot be allocated; FA_ERR_LAUNCH if a copy, launch or event call
 * fails (work already enqueued still completes in order on `stream`).
 */
int fa_step_host(const void* q, const void* k, const void* v, const void* dout, void* o, float* lse, void* dq,
                 void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                 void* stream);

/*
 * fa_bwd_noalloc — the same backward pass as fa_bwd, for callers that may
 * not allocate device memory during the call: serving loops that fix their
 * memory plan at start-up, and code that runs where the CUDA allocator must
 * not be entered. The pages have no counterpart of this call; it only
 * changes where the workspace lives.
 *   Arguments, layouts, results and argument errors are those of fa_bwd.
 *   Workspace: a file-scope device array of FA_BWD_NOALLOC_SCRATCH_BYTES
 *     (64 MiB) inside the library. Every device that loads the library holds
 *     it until the process exits. The call needs
 *       4 * B*Hq*ceil(Nq/128)*128 * (d + 2) bytes of it and returns
 *     FA_ERR_UNSUPPORTED, without enqueuing anything, when that exceeds the
 *     array. The causal GQA backward at d = 128 splits its last round per
 *     query head only where the pieces' fp32 slots (4 * 2 * 128 * d bytes
 *     each) fit in the rest of the array; otherwise that round runs whole
 *     single tiles (same results up to the order of fp32 additions).
 *   No cudaMalloc, cudaFree or other allocating routine is called.
 *   Set-up: the first call on each device looks up the array's device
 *     address on that device (cudaGetSymbolAddress); make that first call
 *     before any stream capture. A failed look-up returns FA_ERR_LAUNCH.
 *   Sharing: all calls on a device share the one array, and it keeps the
 *     last call's contents (the call re-initialises what it reads). Calls
 *     whose work overlaps on the GPU (different streams, no ordering between
 *     them) race on the array and give wrong results; order them.
 */
#define FA_BWD_NOALLOC_SCRATCH_BYTES (64ull << 20)
/*
 * fa_bwd_launches — how many kernels fa_bwd launches for this problem
 *   (fa_bwd_noalloc: the same, or one fewer where the tail slots would not
 *   fit its array): the pre-pass, the main kernel and the dQ conversion,
 *   plus, for the causal GQA backward at d = 128 whose last round is split
 *   per query head, the pass that sums the pieces' dK/dV. With the split
 *   count of the current fa_tune setting and this GPU's SM count. For
 *   profiling and accounting; returns the count, or minus an fa_status for
 *   sizes fa_bwd would reject.
 */
int fa_bwd_launches(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal);
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                   void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale,
                   int causal, void* stream);

/*
 * Sequences of different lengths.
 *
 * The calls below take a batch whose sequences differ in length, as language
 * models have them: packed one behind the other for training and prompts
 * (fa_fwd_varlen), or new tokens over a cache that is kept in pages
 * (fa_cache_append, fa_fwd_paged). Shared conventions:
 *   Tokens   : q, o [total_q, Hq, d], k, v [total_k, Hkv, d] (bf16), the heads
 *              of a token contiguous; consecutive tokens of q, k and v lie
 *              q_stride, k_stride and v_stride elements apart (multiples of 8,
 *              at least heads * d), so that they may be slices of one fused
 *              projection. o is contiguous; lse is [Hq, total_q] fp32.
 *   Lengths  : device arrays of 32-bit integers, read when the kernels run (a
 *              captured graph reads those of each replay). Sequence b has the
 *              rows cu_q[b] .. cu_q[b + 1] - 1 of q and o (0 <= cu_q[0] <= ...
 *              <= cu_q[B] <= total_q), n_b in number, and m_b keys. Either may
 *              be 0. Rows before cu_q[0] and from cu_q[B] on are left as
 *              they are.
 *   Mask     : key j of the sequence is visible to its row i iff
 *                i + off - window_left <= j <= i + off + window_right,
 *              off = m_b - n_b; a negative bound is no limit. Causal is
 *              window_left = -1, window_right = 0. A row that sees no key gets
 *              o = 0 and lse = -inf. What lies past a sequence's keys (other
 *              sequences, unused rows of a page) is never used, whatever its
 *              bits; v rows that only the window hides must be finite.
 *   Sizes    : B >= 1, total_q, total_k >= 0 (0: nothing, or no keys at all),
 *              Hq % Hkv == 0, Hq / Hkv <= 128, d in {64, 128}, any finite scale;
 *              counts are held in 32 bits (total * Hq below 2^31, (total + B) *
 *              Hkv below 2^30; fa_cache_append: Hkv * d below 2^30), tensors
 *              below 2^40 bytes, max_pages * page_size at most 2^28, else
 *              FA_ERR_UNSUPPORTED.
 *   Workspace: from the per-device pool that fa_bwd uses, on `stream`: 40 MB
 *              at d = 128 and 20 MB at d = 64 for the parts of divided work, and
 *              about 40 bytes per block of 128 rows and kv head for the plan.
 *              The smallest calls need none.
 *   Errors   : as above for what the host can see. Lengths or pages on the
 *              device that the tensors cannot hold set FA_ERR_INVALID_ARG in the
 *              status word (fa_get_status); bad lengths: the outputs stay as
 *              they are (fa_cache_append: see there); a bad page: it reads as
 *              zeros, or is not written. Without rows (total_q = 0; the
 *              backward: nor keys) nothing is launched and no length read.
 */

/*
 * fa_fwd_varlen — the forward pass over packed sequences.
 *   in : q, k, v, cu_q [B + 1], cu_k [B + 1] (sequence b has the rows
 *        cu_k[b] .. cu_k[b + 1] - 1 of k and v; cu_k may be cu_q)
 *   out: o, lse
 */
int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int* cu_q, const int* cu_k,
                  int B, int Hq, int Hkv, int total_q, int total_k, int d, long long q_stride, long long k_stride,
                  long long v_stride, float scale, int window_left, int window_right, void* stream);

/*
 * fa_bwd_varlen — the backward pass of fa_fwd_varlen for L = sum(dout * o).
 *   in : q, k, v, cu_q, cu_k and the strides as the forward had them; o, lse as
 *        it wrote them; dout [total_q, Hq, d] (contiguous)
 *   out: dq [total_q, Hq, d], dk, dv [total_k, Hkv, d] (bf16, contiguous): the
 *        rows of every sequence; other rows are left as they are.
 * dk and dv are sums over the query heads of a group, taken in a fixed order;
 * the additions into dq are not ordered (as in fa_bwd). q, k, v and dout of a
 * sequence's rows must be finite, also where only the window hides them
 * (a hidden probability is 0, and 0 times them is added). Workspace: the parts
 * and the plan (of key tiles here) as above, and an fp32 dQ that is padded to
 * whole tiles of 128 rows for every sequence and kv head, with T = 128 / (Hq /
 * Hkv) tokens to a tile:
 *   512 * (d + 2) * Hkv * min(total_q / T + B, total_q) bytes.
 * That is about 4 * total_q * Hq * d where sequences are long beside T, and up
 * to T times as much where they are a token each (4000 of them, 32 query and 8
 * kv heads, d = 128: 2.1 GB); the time of the passes that clear and read it
 * grows alike. 128 * Hkv * min(...) below 2^31, else FA_ERR_UNSUPPORTED.
 */
int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, const int* cu_q, const int* cu_k, int B, int Hq, int Hkv, int total_q,
                  int total_k, int d, long long q_stride, long long k_stride, long long v_stride, float scale,
                  int window_left, int window_right, void* stream);

/*
 * fa_fwd_paged — the forward pass of new tokens over a paged cache: one token
 *   per sequence, a chunk, a whole prompt, or any mixture in one call.
 *   in : q, cu_q [B + 1]
 *        k_pages, v_pages [num_pages, page_size, Hkv, d] (bf16, contiguous),
 *        page_size a multiple of 16
 *        lens_k [B]: keys of each sequence (with its new tokens, if those are
 *        in the cache), at most max_pages * page_size
 *        page_table [B, max_pages]: key j of sequence b is row j % page_size of
 *        page page_table[b][j / page_size]. Entries past its last page are
 *        not read, nor are those of pages that a window hides whole from all
 *        of its new tokens (they may hold anything; v rows that the window
 *        hides in the other pages must be finite)
 *   out: o, lse
 */
int fa_fwd_paged(const void* q, const void* k_pages, const void* v_pages, void* o, float* lse, const int* cu_q,
                 const int* lens_k, const int* page_table, int B, int Hq, int Hkv, int total_q, int num_pages,
                 int page_size, int max_pages, int d, long long q_stride, float scale, int window_left,
                 int window_right, void* stream);

/*
 * fa_cache_append — the new tokens' k and v into the pages: row i of sequence
 *   b goes to place lens_k[b] - n_b + i of the sequence (lens_k: the lengths
 *   with the new tokens, as fa_fwd_paged takes them next; n_b <= lens_k[b]).
 *   Every other row of the pages stays as it is. Two rows that the table
 *   sends to one place leave a mixture (every 16 bytes are one's or the
 *   other's). Needs no workspace.
 *   Wrong lengths, also those of a sequence without new tokens, set
 *   FA_ERR_INVALID_ARG in the status word. Unlike the other calls this one then
 *   still writes the sequences whose own lengths are right; where offsets are
 *   not in order and two such sequences claim a row, it goes to one of them.
 */
int fa_cache_append(const void* k, const void* v, void* k_pages, void* v_pages, const int* cu_q, const int* lens_k,
                    const int* page_table, int B, int Hkv, int total_q, int num_pages, int page_size, int max_pages,
                    int d, long long k_stride, long long v_stride, void* stream);

/*
 * A cache in 8 bits.
 *
 * k_pages and v_pages hold e4m3 codes (a byte each) in the layout of
 * fa_fwd_paged's, and k_scales and v_scales [num_pages, page_size / 16, Hkv]
 * (fp32) a scale for each block of 16 tokens and head: row r of a page stands
 * for scale[page][r / 16][head] * code[page][r][head][...]. A scale that is used
 * must lie between 2^-90 and 2^120, and V's scales of one sequence and head within
 * a factor of 2^100 of each other: farther apart, keys of the smaller scales that have
 * less than 2^-33 of the largest weight are lost, and in the end all of them.
 * Conventions, limits and errors are those of the bf16 calls; scales are aligned to
 * 4 bytes.
 */

/*
 * fa_cache_append_fp8 — the new tokens' k and v (bf16) into the pages of such a
 *   cache, at the places that fa_cache_append gives them. The scale of a block
 *   is 2^e with the smallest whole e, -64 at least, for which every finite value
 *   of its rows is at most 448 * 2^e. New rows of a block that holds rows of the
 *   sequence before them leave its scale or raise it; raised, the rows held are
 *   rounded again in the new scale (exactly, but where a code becomes subnormal or
 *   the old scale, of something else that filled the block, is no power of two).
 *   Rows behind the new ones keep their codes, whose meaning goes with the
 *   block's scale. Codes are the nearest, ties to even; infinities and NaN are
 *   held as NaN, and a block of nothing else has the smallest scale. Two
 *   sequences whose new rows the table sends to one block leave it undefined.
 *   Lengths and errors as fa_cache_append. Needs no workspace.
 */
int fa_cache_append_fp8(const void* k, const void* v, void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                        const int* cu_q, const int* lens_k, const int* page_table, int B, int Hkv, int total_q,
                        int num_pages, int page_size, int max_pages, int d, long long k_stride, long long v_stride,
                        void* stream);

/*
 * fa_fwd_paged_fp8 — fa_fwd_paged over such a cache: the attention of the
 *   values that it stands for. Of those nothing is rounded; P times V's scale is
 *   rounded to f16 for the product with V's codes (off by at most 2^-11 of itself, or
 *   2^-32 of the row's largest where that is more; the row sum keeps 32 bits), and q
 *   to f16 after a division by a power of two of its row where
 *   the batch's sequences have few rows (new tokens * query heads of a group: on the
 *   mean 8 or fewer, or 16 where d = 64 or there are no more tokens than sequences or 64
 *   rows in all; 2^16 in all), to the sum of two e4m3 values where they have many: exact
 *   for what is 2^-9 of the row's largest value or more, off by at most 2^-17 of that
 *   below. A row of q that is not finite gives NaN.
 *   Rows past a sequence's end are not used, whatever their codes; their block's
 *   scale is that of the rows before them. NaN codes of v, of rows that some tokens'
 *   mask hides too, reach the tokens that see them and no others (a call that meets
 *   any among keys that only some see looks them up again, which takes longer). A row's result does not depend on what
 *   else is in the call but for this rounding of q and how its keys are divided
 *   (the order of fp32 sums).
 *   Workspace, from the pool: few rows, 2.6 MB; many, as fa_fwd_paged and
 *   (2 * d + 4) * total_q * Hq bytes for q.
 */
int fa_fwd_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                     const float* v_scales, void* o, float* lse, const int* cu_q, const int* lens_k,
                     const int* page_table, int B, int Hq, int Hkv, int total_q, int num_pages, int page_size,
                     int max_pages, int d, long long q_stride, float scale, int window_left, int window_right,
                     void* stream);

/*
 * fa_rotary — q and k of packed tokens turned by their places.
 *   in : q [total, Hq, d], k [total, Hk, d] (bf16, strided as above; Hq or Hk
 *        may be 0, their pointers then are not used), inv_freq [rot / 2] (fp32,
 *        device, finite), cu_q [B + 1], lens [B] or null
 *   out: q_out, k_out (same shapes, strides of their own), or q and k
 *        themselves, in place
 *   Row i of sequence b is at place p = lens[b] - n_b + i, the place that
 *   fa_cache_append gives it, or i where lens is null. The first rot values of
 *   each head are pairs, (x[j], x[j + rot / 2]), or with interleaved = 1
 *   (x[2 j], x[2 j + 1]), j < rot / 2; pair (a, b) becomes
 *     mscale * (a cos t - b sin t), mscale * (b cos t + a sin t), t = p * inv_freq[j],
 *   with transposed = 1 the same with -t: the gradient of the call's inputs
 *   from that of its outputs. The other values of a head are copied. Angles
 *   are off by less than 2^-24 of a half turn, whatever the place and the frequency;
 *   cos and sin are rounded to fp32 and the results to bf16.
 *   rot is a multiple of 16, 16 <= rot <= d, d in {64, 128}; (Hq + Hk) * d below
 *   2^30, total * (Hq + Hk) below 2^31. Outputs may not overlap other rows of
 *   the inputs. Rows outside every sequence are left as they are. Needs no
 *   workspace. Wrong lengths as in fa_cache_append (n_b <= lens[b]).
 */
int fa_rotary(const void* q, const void* k, void* q_out, void* k_out, const float* inv_freq, const int* cu_q,
              const int* lens, int B, int Hq, int Hk, int total, int d, int rot, long long q_stride,
              long long k_stride, long long q_out_stride, long long k_out_stride, float mscale, int interleaved,
              int transposed, void* stream);

/*
 * fa_get_status — synchronises `stream`, then returns and clears the
 * current device's status word: FA_OK, or FA_ERR_TIMEOUT if any kernel of
 * this library gave up on a bounded wait since the last call, or else
 * FA_ERR_INVALID_ARG if one found lengths or pages on the device that its
 * tensors cannot hold. A CUDA error seen while synchronising is returned as
 * FA_ERR_LAUNCH.
 */
int fa_get_status(void* stream);

/* fa_status_string — static, human-readable name of a status code. */
const char* fa_status_string(int status);

/*
 * Test hooks (not for production use).
 * fa_debug_set — wait_limit_ns: per-wait time limit of every kernel (0
 *   restores the default of 2 s). inject: 0 = off; 1 = the forward's producer
 *   never issues its first K-tile load (that of fa_bwd_varlen its first Q
 *   tile), so the consumer's bounded wait must run out and the kernel must
 *   report FA_ERR_TIMEOUT and exit cleanly. Process-wide; not thread-safe.
 * fa_debug_exp2 — y[i] = 2^x[i] for n device floats, evaluated by the
 *   kernels' own device routine: mode 0 = ex2.approx on the special-function
 *   unit, mode 1 = the fitted polynomial on the FMA pipes.
 */
int fa_debug_set(unsigned long long wait_limit_ns, int inject);

int fa_debug_exp2(const float* x, float* y, int n, int mode, void* stream);

/*
 * fa_tune — process-wide tuning knob, read by every later launch (not
 *   thread-safe). Returns FA_ERR_INVALID_ARG for an unknown knob or value.
 *   FA_TUNE_EXP2_SPLIT: how the forward softmax evaluates its exponentials
 *     (the FlashAttention-4 article on smntcn.com: part of the exponentials
 *     are emulated in software on the FMA pipes because the special-function
 *     unit does not keep up with the tensor cores). value 0 (the default):
 *     every exponential by ex2.approx on the special-function unit; value N
 *     in {1, 2, 4, 8}: one column pair in every N by the fitted degree-3
 *     polynomial on the FMA pipes (relative error below 7.5e-5; N = 1: all
 *     of them), the rest as before. Applies to fa_fwd (both head dims,
 *     causal or not) and fa_fwd_fp8; fa_fwd_window and the backward always
 *     use the special-function unit. Results differ from the default only
 *     by the polynomial's rounding.
 */
#define FA_TUNE_EXP2_SPLIT 1
/*
 *   FA_TUNE_CTA_PAIRS: value 1 runs fa_fwd (d = 128, causal or not; not
 *     fa_fwd_window) on pairs of CTAs: a cluster of two CTAs takes 512
 *     query rows at a time and the even one issues tcgen05.mma with
 *     cta_group::2 (M = 256 over both CTAs' tensor memory), each CTA loading
 *     half of every K and V tile (the FlashAttention-4 article on smntcn.com:
 *     fifth-generation tensor cores and 256 KB of tensor memory per SM; the
 *     pair form halves the MMA instructions and the K/V shared-memory
 *     traffic per flop). value 0 (the default): one CTA per SM. The exp2
 *     split does not apply to the paired kernel. Results are the same up to
 *     the order of floating-point additions.
 */
#define FA_TUNE_CTA_PAIRS 2
/*
 *   FA_TUNE_BWD_SPLIT: the causal backward (no left window bound) runs key
 *     tiles in pairs (j, n-1-j) of equal work; of each kv head's pairs, the
 *     m nearest the middle run as single tiles to fill the last round of
 *     the persistent CTAs, and with grouped-query heads at d = 128 each such
 *     single is split further into one unit per query head, whose dK/dV are
 *     partial sums kept in fp32 and summed in a fixed order by a last pass
 *     (dK, dV stay deterministic). value -1
 *     (the default): m from a model of the round-robin schedule on this
 *     GPU's SM count; value m >= 0: that m (at most n/2). For tests of the
 *     split paths on small shapes; results differ only in the order of
 *     floating-point additions.
 */
#define FA_TUNE_BWD_SPLIT 3
int fa_tune(int knob, int value);

/*
 * fa_profile_events — begin/end are cudaEvent_t handles (or NULL to stop).
 *   While set, fa_fwd records `begin` on its stream right before its kernel
 *   and `end` right after it; fa_bwd does the same around its main
 *   (five-GEMM) kernel, leaving out the preprocess and dQ-convert kernels.
 *   The events are owned by the caller. Process-wide; not thread-safe.
 */
int fa_profile_events(void* begin, void* end);

/*
 * fa_trace — buf: device buffer of FA_TRACE_WORDS uint64 words (or NULL to
 *   stop). While set, the first FA_TRACE_CTAS CTAs of each main kernel write
 *   %globaltimer stamps (ns) at their pipeline hand-off points into
 *   buf[(cta * FA_TRACE_STEPS + step) * FA_TRACE_POINTS + point], for the
 *   first FA_TRACE_STEPS steps of that CTA; a step is one key tile of one
 *   unit (forward) or one query tile (backward). The points are listed in the
 *   kernels' sources. The buffer is owned by the caller; the library only
 *   writes it. Process-wide; not thread-safe. Available only in a library
 *   built with -DFA_ENABLE_TRACE (the build's FA_BUILD_TRACE=1); otherwise a
 *   non-NULL buffer returns FA_ERR_UNSUPPORTED.
 */
#define FA_TRACE_CTAS 4
#define FA_TRACE_STEPS 64
#define FA_TRACE_POINTS 16
#define FA_TRACE_WORDS (FA_TRACE_CTAS * FA_TRACE_STEPS * FA_TRACE_POINTS)
int fa_trace(void* buf);

#ifdef __cplusplus
}
#endif
#endif /* FA_H_ */
