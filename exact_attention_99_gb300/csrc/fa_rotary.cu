// fa_rotary: q and k of packed tokens turned by their places (rotary
// positions), and back, for the gradients.
//
// Pair (a, b) of a token at place p, with frequency f:
//   a' = m (a cos pf - b sin pf), b' = m (b cos pf + a sin pf),
// transposed (the gradient's way) with -sin. The angle of a far place would
// lose its fraction of a turn in 32 bits, and 64-bit floating point is slow
// here; so f / 2 pi is held as a 64-bit fraction of a turn, made from f's
// significand by one wide integer product, and p times that, modulo 2^64, is
// p f modulo one turn, off by less than p 2^-64 turns.
//
// Each value is read once and written once and the rest is little, so memory
// bound. A block takes a few tokens; a thread's loads are issued before the
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
  int per_head;      // d / 16 pairs of pieces
  int turned;        // of those the first rot / 16 are turned
  int rows;          // tokens of a block
  int interleaved;
  int copy_rest;     // the part of a head that is not turned: copied, or left alone in place
  float mscale, sign;
  unsigned* status;
};

// f / 2 pi as a fraction of a turn in units of 2^-64 (modulo one turn), f finite
__device__ __forceinline__ unsigned long long turn_of(float f) {
  const unsigned bits = __float_as_uint(f);
  const int field = int(bits >> 23) & 0xff;
  // |f| = m 2^(e - 23); 0xa2f9836e4e441529 = floor(2^66 / 2 pi), so f / 2 pi 2^64 = m * that * 2^(e - 25)
  const unsigned long long m = field == 0 ? (bits & 0x7fffff) : (bits & 0x7fffff) | 0x800000;
  const int e = max(field, 1) - 127;
  const unsigned long long c = 0xa2f9836e4e441529ull, lo = m * c, hi = __umul64hi(m, c);
  const int s = 25 - e;
  unsigned long long u;
  if (s >= 128) {
    u = 0;
  } else if (s >= 64) {
    u = hi >> (s - 64);
  } else if (s > 0) {
    u = (hi << (64 - s)) | (lo >> s);
  } else {
    u = s > -64 ? lo << -s : 0;  // (frequencies of 2^25 and more)
  }
  return (bits >> 31) ? 0 - u : u;
}

__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  __shared__ float2 cs[kMaxRows][64];
  __shared__ int place[kMaxRows];  // of each token in its sequence, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.rows;
  const int rows = min(a.rows, a.L.total_q - t0);
  // pieces of this block: (token, head, pair of pieces), all heads of a token together; blockIdx.y takes a share
  const int per_token = a.heads * a.per_head, n = max(rows, 0) * per_token;
  const int per_block = (n + gridDim.y - 1) / gridDim.y;
  const int first = int(blockIdx.y) * per_block, last = min(first + per_block, n);

  uint4 va[kBatch], vb[kBatch];
  long long to[kBatch];
  // of piece i: its place in x and y, its pair of pieces within the head
  auto locate = [&](int i, int& row, int& c, int& which, long long& in, long long& out, int& second) {
    row = i / per_token;
    const int r = i - row * per_token, h = r / a.per_head;
    c = r - h * a.per_head;
    which = h < a.hq ? 0 : 1;
    const int head = which == 0 ? h : h - a.hq;
    // pieces of the pair: half layout c and c + rot / 16, neighbours 2 c and 2 c + 1 (as the rest's)
    const int one = c < a.turned && !a.interleaved ? c : 2 * c;
    second = c < a.turned && !a.interleaved ? a.turned : 1;
    const long long off = 1LL * head * (2 * a.per_head) + one;
    in = (t0 + row) * a.xs[which] + off;
    out = (t0 + row) * a.ys[which] + off;
  };
  bool ready = false;
  for (int base = first; base < last || !ready; base += kItems) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kThreads + tid;
      if (i >= last) continue;
      int row, c, which, second;
      long long in;
      locate(i, row, c, which, in, to[k], second);
      if (c >= a.turned && !a.copy_rest) continue;
      const uint4* p = a.x[which] + in;
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
        const unsigned long long turn = turn_of(a.inv_freq[j]) * static_cast<unsigned long long>(max(place[r], 0));
        float sn, cn;
        sincospif(float(int(turn >> 32)) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: in half turns
        cs[r][j] = make_float2(a.mscale * cn, a.sign * a.mscale * sn);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * kThreads + tid;
      if (i >= last) continue;
      int row, c, which, second;
      long long in, out;
      locate(i, row, c, which, in, out, second);
      if (place[row] < 0 || (c >= a.turned && !a.copy_rest)) continue;
      uint4 x = va[k], y = vb[k];
      if (c < a.turned) {
        const float4* f = reinterpret_cast<const float4*>(&cs[row][c * 8]);  // two pairs each
        uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
        auto lo = [](uint32_t w) { return u2f(w << 16); };
        auto hi = [](uint32_t w) { return u2f(w & 0xffff0000u); };
        if (!a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 t = f[e];
            const float a0 = lo(xw[e]), a1 = hi(xw[e]), b0 = lo(yw[e]), b1 = hi(yw[e]);
            xw[e] = pack_bf16x2(a0 * t.x - b0 * t.y, a1 * t.z - b1 * t.w);
            yw[e] = pack_bf16x2(b0 * t.x + a0 * t.y, b1 * t.z + a1 * t.w);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 t = f[e >> 1], u = f[2 + (e >> 1)];
            const float xc = (e & 1) ? t.z : t.x, xs = (e & 1) ? t.w : t.y;
            const float yc = (e & 1) ? u.z : u.x, ys = (e & 1) ? u.w : u.y;
            const float a0 = lo(xw[e]), b0 = hi(xw[e]), a1 = lo(yw[e]), b1 = hi(yw[e]);
            xw[e] = pack_bf16x2(a0 * xc - b0 * xs, b0 * xc + a0 * xs);
            yw[e] = pack_bf16x2(a1 * yc - b1 * ys, b1 * yc + a1 * ys);
          }
        }
      }
      uint4* q = a.y[which] + out;
      q[0] = x;
      q[second] = y;
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
  a.per_head = pb.d / 16;
  a.turned = pb.rot / 16;
  // A block's pieces are a thread's one batch or a little less, while that
  // gives each SM several blocks; a token of very many heads is shared by
  // several blocks, and so is the only token of a call.
  const int per_token = a.heads * a.per_head;
  a.rows = std::max(1, std::min({kMaxRows, kItems / per_token, pb.total / (4 * num_sms())}));
  const long long share = 1LL * a.rows * per_token / kThreads;
  const long long blocks = (1LL * pb.total + a.rows - 1) / a.rows;
  const unsigned split = unsigned(std::max(1LL, std::min({share, 64LL, 2LL * num_sms() / std::max(1LL, blocks)})));
  a.interleaved = pb.interleaved;
  a.mscale = pb.mscale;
  a.sign = pb.transposed ? -1.0f : 1.0f;
  a.status = status_word();
  if (a.status == nullptr) return cudaErrorLaunchFailure;
  rotary_kernel<<<dim3(unsigned(blocks), split), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
