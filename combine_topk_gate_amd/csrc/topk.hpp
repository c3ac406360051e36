// Top-k selection of one token's gate logits by a group of 16 lanes, shared by
// the route kernel and the decode layer's plan (the scheme is described in
// route.hip).
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kLanesPerToken = 16;

// a ahead of b: larger value, or equal value and lower index
__device__ __forceinline__ bool route_before(float va, int ia, float vb, int ib) {
  return va > vb || (va == vb && ia < ib);
}

template <int KMAX>
__device__ __forceinline__ void topk_insert(float (&vals)[KMAX], int (&ids)[KMAX], float v, int e) {
  // e exceeds every index kept so far, so v enters only if strictly larger
  // than the last kept value, behind every kept value it does not exceed
  if (!(v > vals[KMAX - 1])) return;
#pragma unroll
  for (int i = KMAX - 1; i >= 0; --i) {
    if (vals[i] >= v) continue;
    const bool above_ge = (i == 0) ? true : (vals[i - 1] >= v);
    if (above_ge) {
      vals[i] = v;
      ids[i] = e;
    } else {
      vals[i] = vals[i - 1];
      ids[i] = ids[i - 1];
    }
  }
}

// Keep the KMAX best of two sorted lists (own and the partner lane's):
// pairing own[i] with partner[KMAX-1-i] and keeping the better of each pair
// leaves the KMAX best as a bitonic sequence, which a bitonic merger sorts.
template <int KMAX>
__device__ __forceinline__ void topk_merge_partner(float (&vals)[KMAX], int (&ids)[KMAX], int off) {
  float pv[KMAX];
  int pi[KMAX];
#pragma unroll
  for (int i = 0; i < KMAX; ++i) {
    pv[i] = __shfl_xor(vals[i], off);
    pi[i] = __shfl_xor(ids[i], off);
  }
#pragma unroll
  for (int i = 0; i < KMAX; ++i) {
    const float bv = pv[KMAX - 1 - i];
    const int bi = pi[KMAX - 1 - i];
    if (!route_before(vals[i], ids[i], bv, bi)) {
      vals[i] = bv;
      ids[i] = bi;
    }
  }
#pragma unroll
  for (int half = KMAX / 2; half >= 1; half >>= 1) {
#pragma unroll
    for (int i = 0; i < KMAX; ++i) {
      if (i & half) continue;
      const int j = i + half;
      if (!route_before(vals[i], ids[i], vals[j], ids[j])) {
        const float tv = vals[i];
        const int ti = ids[i];
        vals[i] = vals[j];
        ids[i] = ids[j];
        vals[j] = tv;
        ids[j] = ti;
      }
    }
  }
}

// The KMAX best (value, index) pairs of row[0 .. E), in every lane of the
// token's 16 (q = the lane's place among them); a place that no logit above
// -inf fills keeps -inf and index 0x7fffffff.  valid: the group has a token.
template <int KMAX>
__device__ __forceinline__ void topk_row(const float* __restrict__ row, int E, int q, bool valid, float (&vals)[KMAX],
                                         int (&ids)[KMAX]) {
#pragma unroll
  for (int i = 0; i < KMAX; ++i) {
    vals[i] = -__builtin_inff();
    ids[i] = 0x7fffffff;  // behind every real expert
  }
  if (valid) {
    // 4 loads in flight per lane, then insertion in increasing expert order
    int e = q;
    for (; e + 3 * kLanesPerToken < E; e += 4 * kLanesPerToken) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = row[e + u * kLanesPerToken];
#pragma unroll
      for (int u = 0; u < 4; ++u) topk_insert<KMAX>(vals, ids, v[u], e + u * kLanesPerToken);
    }
    for (; e < E; e += kLanesPerToken) topk_insert<KMAX>(vals, ids, row[e], e);
  }
#pragma unroll
  for (int off = 1; off < kLanesPerToken; off <<= 1) topk_merge_partner<KMAX>(vals, ids, off);
}

}  // namespace moe
