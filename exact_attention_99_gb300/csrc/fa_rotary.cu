// fa_rotary: q and k of packed tokens turned by their places (rotary
// positions), and back, for the gradients.
//
// Pair (a, b) of a token at place p, with frequency f:
//   a' = m (a cos pf - b sin pf), b' = m (b cos pf + a sin pf),
// transposed (the gradient's way) with -sin. The angle of a far place would
// lose its fraction of a turn in 32 bits, and 64-bit floating point is slow
// here; so f / 2 pi is held as a 64-bit fraction of a turn, made from f's
// significand by wide integer products, and p times that, modulo 2^64, is
// p f modulo one turn, off by less than 1.5 p 2^-64 turns. What sine and cosine get of
// it are its first 32 bits, as a float: off by less than 2^-24 half turns.
//
// Each value is read once and written once and the rest is little, so memory
// bound: 21000 tokens of 32 + 8 heads of 128 take 70 us, 6.2 TB/s (the measured copy
// 6.8); one token 3.5 us, the launch. A block takes a few tokens; a thread's loads are issued before the
// block looks up its tokens' sequences and makes the tokens' cosines and sines,
// which all heads share.
#include <cuda_bf16.h>

#include <algorithm>

#include "fa_internal.h"
#include "fa_seq.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxRows = kWarps;  // tokens of a block: a warp looks each up
constexpr int kBatch = 4;         // pieces of 2 x 16 bytes that a thread has in flight
constexpr int kItems = kBatch * kThreads;

struct RotaryArgs {
  const uint4* x[2];  // q, k (16-byte pieces)
  uint4* y[2];
  long long xs[2], ys[2];  // pieces between tokens
  const float* inv_freq;
  seq::Lens L;
  int heads, hq;     // of both, of q
  int turned;        // of a head's pairs of pieces the first rot / 16 are turned
  int rows;          // tokens of a block
  int copy_rest;     // the part of a head that is not turned: copied, or left alone in place
  float mscale, sign;
  unsigned* status;
};

// f / 2 pi as a fraction of a turn in units of 2^-64 (modulo one turn), f finite, off by less
// than 1.5 of them. |f| = m 2^(e - 23), and 1 / 2 pi in units of 2^-194 is the 192 bits
// c2 c1 c0, so that the bits from 153 - e on of m times those are wanted; of |f| < 2 the
// first word has enough.
__device__ __forceinline__ unsigned long long turn_of(float f) {
  constexpr unsigned long long c2 = 0xa2f9836e4e441529ull, c1 = 0xfc2757d1f534ddc0ull, c0 = 0xdb6295993c439041ull;
  const unsigned bits = __float_as_uint(f);
  const int field = int(bits >> 23) & 0xff;
  const unsigned long long m = field == 0 ? (bits & 0x7fffff) : (bits & 0x7fffff) | 0x800000;
  const int e = max(field, 1) - 127;
  unsigned long long u;
  if (e <= 0) {
    const unsigned long long lo = m * c2, hi = __umul64hi(m, c2);
    const int s = 25 - e;
    u = s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : (hi << (64 - s)) | (lo >> s);
  } else {
    const unsigned long long w0 = m * c0, h0 = __umul64hi(m, c0), l1 = m * c1, w1 = l1 + h0;
    const unsigned long long h1 = __umul64hi(m, c1) + (w1 < l1 ? 1 : 0), l2 = m * c2, w2 = l2 + h1;
    const unsigned long long w3 = __umul64hi(m, c2) + (w2 < l2 ? 1 : 0);
    const int s = 153 - e, off = s & 63;  // (25 to 152)
    const unsigned long long lo = s >= 128 ? w2 : s >= 64 ? w1 : w0, hi = s >= 128 ? w3 : s >= 64 ? w2 : w1;
    u = off == 0 ? lo : (lo >> off) | (hi << (64 - off));
  }
  return (bits >> 31) ? 0 - u : u;
}

// A thread's piece: 16 values of a head, the two 16-byte pieces of which are
// c and c + rot / 16 of the head (halves) or 2 c and 2 c + 1 (neighbours, and what is
// not turned).
template <int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryArgs a) {
  constexpr int kPerHead = D / 16;  // pairs of pieces
  __shared__ __align__(16) float cosines[kMaxRows][D / 2], sines[kMaxRows][D / 2];
  __shared__ int place[kMaxRows];  // of each token in its sequence, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.rows;
  const int rows = min(a.rows, a.L.total_q - t0);
  // pieces of this block: (token, head, pair of pieces), all heads of a token together; blockIdx.y takes a share
  const int per_token = a.heads * kPerHead, n = rows * per_token;
  const int per_block = (n + gridDim.y - 1) / gridDim.y;
  const int first = int(blockIdx.y) * per_block, last = min(first + per_block, n);
  const int c = (first + tid) % kPerHead;  // (the same for all of a thread's pieces: first + tid moves by 256)
  const bool turn = c < a.turned, idle = !turn && !a.copy_rest;
  const int one = turn && !NEIGHBOURS ? c : 2 * c, second = turn && !NEIGHBOURS ? a.turned : 1;

  bool ready = false;
  for (int base = first; base < last || !ready; base += kItems) {
    uint4 va[kBatch], vb[kBatch];
    uint4* to[kBatch];
    int row_of[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kThreads + tid;
      row_of[k] = -1;
      if (i >= last || idle) continue;
      const int head = i / kPerHead, row = head / a.heads, h = head - row * a.heads;
      const int which = h < a.hq ? 0 : 1;
      const long long off = 1LL * (which == 0 ? h : h - a.hq) * (2 * kPerHead) + one;
      const uint4* const p = a.x[which] + ((t0 + row) * a.xs[which] + off);
      to[k] = a.y[which] + ((t0 + row) * a.ys[which] + off);
      row_of[k] = row;
      va[k] = __ldcs(p);
      vb[k] = __ldcs(p + second);
    }
    if (!ready) {
      ready = true;
      if (warp < rows) {
        const int t = t0 + warp;
        const int b = seq::find_token(a.L.cu_q, a.L.B, t);
        seq::Seq s;
        const bool ok = seq::seq_at(a.L, b, s) && s.qlen <= s.klen;
        const int at = t - s.q0;
        if (lane == 0) place[warp] = ok && at >= 0 && at < s.qlen ? s.klen - s.qlen + at : -1;
      }
      __syncthreads();
      const int half = a.turned * 8;  // pairs of a head
      for (int i = tid; i < rows * half; i += kThreads) {
        const int r = i / half, j = i - r * half;
        // the top 32 bits of p f's fraction of a turn, in [-1/2, 1/2) turns
        const unsigned long long fraction = turn_of(a.inv_freq[j]) * static_cast<unsigned long long>(max(place[r], 0));
        float sn, cn;
        sincospif(float(int(fraction >> 32)) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: in half turns
        cosines[r][j] = a.mscale * cn;
        sines[r][j] = a.sign * a.mscale * sn;
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int row = row_of[k];
      if (row < 0 || place[row] < 0) continue;
      uint32_t x[4] = {va[k].x, va[k].y, va[k].z, va[k].w}, y[4] = {vb[k].x, vb[k].y, vb[k].z, vb[k].w};
      if (turn) {
        auto lo = [](uint32_t w) { return u2f(w << 16); };
        auto hi = [](uint32_t w) { return u2f(w & 0xffff0000u); };
        const float4* const fc = reinterpret_cast<const float4*>(&cosines[row][c * 8]);
        const float4* const fs = reinterpret_cast<const float4*>(&sines[row][c * 8]);
        // two pairs (a, b) at a time
        auto turned2 = [](uint64_t p, uint64_t q, float c0, float c1, float s0, float s1, float* out) {
          const uint64_t co = pack2(c0, c1), si = pack2(s0, s1);
          unpack2(ffma2(q, si ^ 0x8000000080000000ull, fmul2(p, co)), out[0], out[1]);
          unpack2(ffma2(p, si, fmul2(q, co)), out[2], out[3]);
        };
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // pairs 4 e .. 4 e + 3
          const float4 co = fc[e], si = fs[e];
          float r[8];
          if constexpr (!NEIGHBOURS) {
            const uint32_t x0 = x[2 * e], x1 = x[2 * e + 1], y0 = y[2 * e], y1 = y[2 * e + 1];
            turned2(pack2(lo(x0), hi(x0)), pack2(lo(y0), hi(y0)), co.x, co.y, si.x, si.y, r);
            turned2(pack2(lo(x1), hi(x1)), pack2(lo(y1), hi(y1)), co.z, co.w, si.z, si.w, r + 4);
            x[2 * e] = pack_bf16x2(r[0], r[1]);
            y[2 * e] = pack_bf16x2(r[2], r[3]);
            x[2 * e + 1] = pack_bf16x2(r[4], r[5]);
            y[2 * e + 1] = pack_bf16x2(r[6], r[7]);
          } else {
            uint32_t* const w = e == 0 ? x : y;
            turned2(pack2(lo(w[0]), lo(w[1])), pack2(hi(w[0]), hi(w[1])), co.x, co.y, si.x, si.y, r);
            turned2(pack2(lo(w[2]), lo(w[3])), pack2(hi(w[2]), hi(w[3])), co.z, co.w, si.z, si.w, r + 4);
            w[0] = pack_bf16x2(r[0], r[2]);
            w[1] = pack_bf16x2(r[1], r[3]);
            w[2] = pack_bf16x2(r[4], r[6]);
            w[3] = pack_bf16x2(r[5], r[7]);
          }
        }
      }
      to[k][0] = make_uint4(x[0], x[1], x[2], x[3]);
      to[k][second] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  // every wrong length is told, also where no token leads to it
  bool ok = true;
  const long long blocks = 1LL * gridDim.x * gridDim.y, me = 1LL * blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll 1
  for (long long b = me * kThreads + tid; b < a.L.B; b += blocks * kThreads) {
    seq::Seq s;
    ok = seq::seq_at(a.L, int(b), s) && s.qlen <= s.klen && ok;
  }
  if (!ok) atomicOr(a.status, kDevBadArg);
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem& pb, cudaStream_t stream) {
  RotaryArgs a{};
  const void* x[2] = {pb.q, pb.k};
  void* y[2] = {pb.q_out, pb.k_out};
  const long long xs[2] = {pb.q_stride, pb.k_stride}, ys[2] = {pb.q_out_stride, pb.k_out_stride};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint4*>(x[i]);
    a.y[i] = static_cast<uint4*>(y[i]);
    a.xs[i] = xs[i] / 8;
    a.ys[i] = ys[i] / 8;
    if ((i == 0 ? pb.Hq : pb.Hk) > 0 && x[i] != y[i]) a.copy_rest = 1;
  }
  a.inv_freq = pb.inv_freq;
  // without lengths a sequence's tokens are all it has: their own offsets in the keys' place
  a.L = seq::Lens{pb.cu_q, pb.lens != nullptr ? nullptr : pb.cu_q, pb.lens, pb.B, pb.total, pb.total, 0x7fffffff};
  a.heads = pb.Hq + pb.Hk;
  a.hq = pb.Hq;
  a.turned = pb.rot / 16;
  // A block's pieces are a thread's one batch or a little less, while that
  // gives each SM several blocks; a token of very many heads is shared by
  // several blocks, and so is the only token of a call.
  const int per_token = a.heads * (pb.d / 16);
  a.rows = std::max(1, std::min({kMaxRows, kItems / per_token, pb.total / (4 * num_sms())}));
  const long long share = 1LL * a.rows * per_token / kThreads;
  const long long blocks = (1LL * pb.total + a.rows - 1) / a.rows;
  const unsigned split = unsigned(std::max(1LL, std::min({share, 64LL, 2LL * num_sms() / std::max(1LL, blocks)})));
  a.mscale = pb.mscale;
  a.sign = pb.transposed ? -1.0f : 1.0f;
  a.status = status_word();
  if (a.status == nullptr) return cudaErrorLaunchFailure;
  const dim3 grid{unsigned(blocks), split};
  if (pb.d == 128) {
    if (pb.interleaved) {
      rotary_kernel<128, true><<<grid, kThreads, 0, stream>>>(a);
    } else {
      rotary_kernel<128, false><<<grid, kThreads, 0, stream>>>(a);
    }
  } else if (pb.interleaved) {
    rotary_kernel<64, true><<<grid, kThreads, 0, stream>>>(a);
  } else {
    rotary_kernel<64, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fa
