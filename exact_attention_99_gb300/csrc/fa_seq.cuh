// Sequences of different lengths: what the packed and paged attention calls
// share between their host code, the planning kernels and the main kernels.
#pragma once
#include <cstddef>
#include <cstdint>

#include "fa_internal.h"

namespace fa {
namespace seq {

// The lengths, as the calls get them (device arrays). Packed keys: cu_k
// holds the B + 1 row offsets of k and v. Paged keys: lens_k holds the B
// lengths, at most max_len each.
struct Lens {
  const int* cu_q;
  const int* cu_k;    // packed, else null
  const int* lens_k;  // paged, else null
  int B, total_q, total_k;
  long long max_len;
};

// Sequence b: its first packed query row, its query and key counts, its first
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

// A piece of the forward's work: up to two tiles of query rows of one
// (sequence, kv head) against the key tiles [kt, kt + nt) of 128 keys each.
// A tile of rows holds `tok` = 128 / group tokens with all query heads of
// the group (row = token * group + head), so that they share the key tiles.
struct __align__(16) Item {
  int q0;          // first packed token
  int ntok_flags;  // tokens (at most 2 * tok, in the low 16 bits) and the flags below
  int kvh;
  int kbase;       // packed: the sequence's first key row; paged: the sequence
  int klen;
  int pos;         // place of the first token among the keys (klen - qlen + its place in the sequence)
  int kt, nt;
  __device__ __forceinline__ int ntok() const { return ntok_flags & 0xffff; }
};
static_assert(sizeof(Item) == 32, "two 16-byte loads");
// At most `tok` tokens (one tile of rows): the two stages of the pipeline
// take alternate key tiles of the same rows; else each has rows of its own.
constexpr int kKeyMode = 1 << 16;
// The item sees only part of its rows' keys: (m, l, O) go to a slot, to be
// joined with the other parts. kCont: not the rows' first keys.
constexpr int kPart = 1 << 17;
constexpr int kCont = 1 << 18;

// Rows whose keys were divided at the start of worker c's share (and not at
// an earlier share's start): parts in slot 2 * c0 + 1 and 2 * c for c in (c0, c1].
struct Cut {
  int q0, ntok_flags, kvh, c0, c1, pad[3];  // c1 < 0: nothing
};

struct PlanHead {
  int n_items;  // sorted order: worker c takes items c, 2G-1-c, 2G+c, ...
  int split;    // 1: worker c takes items [first[c], last[c]] instead
  int pad[2];
};

// The forward plan in device memory, made by plan_kernel for every call.
struct Plan {
  PlanHead* head;
  int* first;   // [G]
  int* last;    // [G]
  Cut* cuts;    // [G]
  int* ustart;  // [B + 1] first unit of each sequence
  long long* cost;  // [units + 1] key tiles of the units before
  int* order;   // [units] by key tiles, most first
  Item* items;  // [units * Hkv + G]
  int max_units;
};

}  // namespace seq
}  // namespace fa
