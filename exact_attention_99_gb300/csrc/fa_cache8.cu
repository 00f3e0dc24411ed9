// fa_cache_append_fp8: K and V rows of new tokens into the pages of a cache
// held in e4m3, with a scale for each block of 16 tokens and head.
//
// A block's scale is the smallest power of two, 2^-64 at least, for which the
// largest finite value of its rows is at most 448 (e4m3's largest) times it.
// A division by a power of two is exact, so a code is the rounding of the exact
// value, and a block that later rows make coarser loses bits only where a code
// becomes subnormal. In a block with a scale of another kind (something else filled it)
// quotients and products are cut with their last bit set before they become codes, so
// that these too are the roundings of the exact values. (The scale amax / 448 would use the range up to a factor
// of two further, which a floating type does not need: its relative error is
// the same over all its normal values.)
//
// Each value is read once (2 bytes) and written once (1 byte), so memory bound:
// 51000 tokens of 8 heads of 128 in prompts take 53 us, 5.9 TB/s (the measured copy
// 6.8); 100 single tokens 3.8 us, the launch and a chain of four loads.
// The first new token of a block speaks for it: a warp takes the block's new
// rows of one head of K or V, all 16 rows' loads in flight, finds their largest
// magnitude by packed 16-bit integer maxima (of bf16's bits without the sign),
// and writes codes and scale.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "fa_internal.h"
#include "fa_seq.cuh"
#include "sm103_fp8.cuh"
#include "sm103_math.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = kFp8Block;
constexpr int kMaxTokens = 16;  // packed tokens that a thread block looks through

struct Append8Args {
  const uint16_t* x[2];     // k, v
  long long stride[2];      // values between tokens
  uint8_t* pages[2];
  float* scales[2];
  const int* table;
  seq::Lens L;
  int Hkv, num_pages, page_size, max_pages;
  int tokens;               // packed tokens of a thread block
  unsigned* status;
};

// the new rows of a block: packed tokens t .. t + n - 1 to the pool's rows row .. row + n - 1
struct Part {
  long long row;
  int t, n;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 4) append8_kernel(const Append8Args a) {
  __shared__ Part parts[kMaxTokens];
  __shared__ int n_parts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * a.tokens;
  if (tid == 0) n_parts = 0;
  __syncthreads();
  for (int i = warp; i < a.tokens; i += kWarps) {
    const int t = t0 + i;
    Part p{-1, t, 0};
    if (t < a.L.total_q) {
      const int b = seq::find_token(a.L.cu_q, a.L.B, t);
      seq::Seq s;
      if (seq::seq_at(a.L, b, s) && s.qlen <= s.klen && t >= s.q0 && t < s.q0 + s.qlen) {
        const int place = s.klen - s.qlen + (t - s.q0);
        if (t == s.q0 || place % kBlock == 0) {  // the first of its block
          const int pg = place / a.page_size, page = a.table[size_t(b) * a.max_pages + pg];
          if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, kDevBadArg);
          } else {
            p.row = 1LL * page * a.page_size + (place - pg * a.page_size);
            p.n = min(kBlock - place % kBlock, s.q0 + s.qlen - t);
          }
        }
      }
    }
    if (lane == 0 && p.n > 0) parts[atomicAdd(&n_parts, 1)] = p;  // (in any order: no two have a block in common)
  }
  __syncthreads();
  constexpr int kLanes = D / 8;         // lanes of a row, 8 values each
  constexpr int kAtOnce = 32 / kLanes;  // rows of an access
  constexpr int kSteps = kBlock / kAtOnce;
  const int r0 = lane / kLanes, c = lane % kLanes * 8;
  const int tasks = n_parts * 2 * a.Hkv;
  // A block's new rows of one head of K or V, in kN accesses. A single token has one:
  // the instructions of seven idle ones took longer than its memory (256 tokens of 8
  // heads of 128 5.3 -> 4.3 us, 4096 35 -> 27 us).
  auto write = [&](auto steps, const Part& p, int head, int kv) {
    constexpr int kN = decltype(steps)::value;
    const int held = int(p.row % kBlock);  // rows of the block before the new ones
    float* const scale_at = a.scales[kv] + p.row / kBlock * a.Hkv + head;
    const float before = held > 0 ? *scale_at : 0.0f;
    const uint16_t* src = a.x[kv] + p.t * a.stride[kv] + 1LL * head * D + c;
    uint4 v[kN];
    {
      const uint16_t* at = src + r0 * a.stride[kv];
      const long long step = kAtOnce * a.stride[kv];
#pragma unroll
      for (int s = 0; s < kN; ++s, at += step)
        v[s] = s * kAtOnce + r0 < p.n ? __ldcs(reinterpret_cast<const uint4*>(at)) : make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < kN; ++s) {
      m = max_u16x2(m, max_u16x2(v[s].x & 0x7fff7fffu, v[s].y & 0x7fff7fffu));
      m = max_u16x2(m, max_u16x2(v[s].z & 0x7fff7fffu, v[s].w & 0x7fff7fffu));
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if (top >= 0x7f80u) {  // infinities and NaN, held as NaN, are no part of the scale
      uint32_t fin = 0;
#pragma unroll
      for (int s = 0; s < kN; ++s) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[s]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
          if (lo < 0x7f80u) fin = max(fin, lo);
          if (hi < 0x7f80u) fin = max(fin, hi);
          if (lo >= 0x7f80u) w[e] |= 0x7fffu;
          if (hi >= 0x7f80u) w[e] |= 0x7fff0000u;
        }
      }
      top = __reduce_max_sync(0xffffffffu, fin);
    }
    // 448 = 1.75 2^8; top = (1 + f / 128) 2^E: e = E - 8, one more where 1 + f / 128 > 1.75
    const int e = max(-64, int(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0));
    float scale = exp2i(e);
    float inv = exp2i(-e);
    // a block that something else filled may have a scale that is no power of two
    const bool odd = held > 0 && (f2u(before) & 0x7fffffu) != 0;
    if (held > 0) {
      const float ratio = before * inv;
      if (before >= scale) {
        scale = before;
        inv = 1.0f / before;
      } else {
        // the rows held, rounded again in the coarser scale
        uint8_t* dst = a.pages[kv] + ((p.row - held) * a.Hkv + head) * D + c;
#pragma unroll 1
        for (int r = r0; r < held; r += kAtOnce) {
          uint2* at = reinterpret_cast<uint2*>(dst + 1LL * r * a.Hkv * D);
          const uint2 x = *at;
          *at = odd ? make_uint2(e4m3x4_odd_times(x.x, ratio), e4m3x4_odd_times(x.y, ratio))
                    : make_uint2(e4m3x4_times(x.x, ratio), e4m3x4_times(x.y, ratio));
        }
      }
    }
    const int row_bytes = a.Hkv * D;
    uint8_t* dst = a.pages[kv] + ((p.row + r0) * a.Hkv + head) * D + c;
    if (odd && scale == before) {
#pragma unroll
      for (int s = 0; s < kN; ++s, dst += kAtOnce * row_bytes)
        if (s * kAtOnce + r0 < p.n)
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(e4m3x4_of_bf16_over(v[s].x, v[s].y, scale), e4m3x4_of_bf16_over(v[s].z, v[s].w, scale));
    } else {
#pragma unroll
      for (int s = 0; s < kN; ++s, dst += kAtOnce * row_bytes)
        if (s * kAtOnce + r0 < p.n)
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(e4m3x4_of_bf16(v[s].x, v[s].y, inv), e4m3x4_of_bf16(v[s].z, v[s].w, inv));
    }
    if (lane == 0) *scale_at = scale;
  };
  for (int task = blockIdx.y * kWarps + warp; task < tasks; task += gridDim.y * kWarps) {
    const int i = task / (2 * a.Hkv), what = task - i * 2 * a.Hkv, head = what >> 1, kv = what & 1;
    const Part p = parts[i];
    if (p.n <= kAtOnce) {
      write(std::integral_constant<int, 1>{}, p, head, kv);
    } else {
      write(std::integral_constant<int, kSteps>{}, p, head, kv);
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

cudaError_t launch_cache_append8(const AppendProblem& pb, float* k_scales, float* v_scales, cudaStream_t stream) {
  Append8Args a{};
  a.x[0] = static_cast<const uint16_t*>(pb.k);
  a.x[1] = static_cast<const uint16_t*>(pb.v);
  a.stride[0] = pb.k_stride;
  a.stride[1] = pb.v_stride;
  a.pages[0] = static_cast<uint8_t*>(pb.k_pages);
  a.pages[1] = static_cast<uint8_t*>(pb.v_pages);
  a.scales[0] = k_scales;
  a.scales[1] = v_scales;
  a.table = pb.page_table;
  a.L = seq::Lens{pb.cu_q, nullptr, pb.lens_k, pb.B, pb.total_q, 0, 1LL * pb.max_pages * pb.page_size};
  a.Hkv = pb.Hkv;
  a.num_pages = pb.num_pages;
  a.page_size = pb.page_size;
  a.max_pages = pb.max_pages;
  a.status = status_word();
  if (a.status == nullptr) return cudaErrorLaunchFailure;
  // Of a long prompt one token in 16 speaks for a block, of single tokens
  // each does: fewer tokens to a thread block where that leaves SMs without one,
  // and the heads of a token shared by several.
  a.tokens = std::max(1, std::min(kMaxTokens, pb.total_q / (4 * num_sms())));
  const long long blocks = (1LL * pb.total_q + a.tokens - 1) / a.tokens;
  const long long rounds = (2LL * a.tokens * pb.Hkv + kWarps - 1) / kWarps;
  const unsigned split = unsigned(std::max(1LL, std::min({rounds, 64LL, 4LL * num_sms() / blocks})));
  const dim3 grid{unsigned(blocks), split};
  if (pb.d == 128) {
    append8_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  } else {
    append8_kernel<64><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fa
