// Sequences of different lengths: their lengths as the packed and paged
// attention calls get them (device arrays).
#pragma once
#include <cstddef>
#include <cstdint>

#include "fa_internal.h"

namespace fa {
namespace seq {

// Packed keys: cu_k holds the B + 1 row offsets of k and v. Paged keys:
// lens_k holds the B lengths, at most max_len each.
struct Lens {
  const int* cu_q;
  const int* cu_k;    // packed, else null
  const int* lens_k;  // paged, else null
  int B, total_q, total_k;
  long long max_len;
};

// A sequence: its first packed query row, its query and key counts, its first
// packed key row (0 for paged keys).
struct Seq {
  int q0, qlen, k0, klen;
};
// False if the arrays say something that the tensors cannot hold.
__device__ __forceinline__ bool seq_at(const Lens& L, int b, Seq& s) {
  s.q0 = L.cu_q[b];
  const int q1 = L.cu_q[b + 1];
  s.qlen = q1 - s.q0;
  bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= L.total_q;
  if (L.cu_k != nullptr) {
    s.k0 = L.cu_k[b];
    const int k1 = L.cu_k[b + 1];
    s.klen = k1 - s.k0;
    ok = ok && s.k0 >= 0 && k1 >= s.k0 && k1 <= L.total_k;
  } else {
    s.k0 = 0;
    s.klen = L.lens_k[b];
    ok = ok && s.klen >= 0 && s.klen <= L.max_len;
  }
  return ok;
}

// The last sequence that begins at or before token t, by a whole warp: its
// lanes look at 32 places at a time, so that 1000 sequences take two reads one
// after the other and not ten.
__device__ __forceinline__ int find_token(const int* cu_q, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool before = at < n && (lane == 0 || cu_q[lo + at] <= t);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

}  // namespace seq
}  // namespace fa
