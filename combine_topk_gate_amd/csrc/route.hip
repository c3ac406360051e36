// Top-k routing with renormalised softmax weights.
//
// COMET paper review §4.1.1 (Top-K reduction couples a token's expert
// outputs) and the PTO MoE article's seven serial stages (top-K weighted
// accumulation): each token keeps its k largest gate logits, and the
// weights are the softmax over the k chosen logits.
//
// Sixteen lanes handle one token (a 256-thread block: 16 tokens).  Lane q
// reads experts q, q + 16, q + 32, ... (the 16 lanes of a token read 64
// consecutive bytes at a time) and keeps its KMAX best (value, index) pairs
// sorted in registers.  The lanes' lists are then merged in four butterfly
// steps: partners exchange their lists and both keep the KMAX best of the
// union.  "Best" is the total order value descending, then index ascending,
// which is the order the selection defines (equal logits keep the lower
// expert index first), so the merged list is unique and every lane of the
// token ends with the same one.
#include "common.hpp"
#include "launch.hpp"
#include "topk.hpp"

namespace moe {

constexpr int kRouteThreads = 256;

// Words the caller needs zero before the kernels that follow (the layer
// call's status word and the fused kernel's ready counters): block 0 clears
// them, which saves a launch per range.
struct ClearRanges {
  int32_t* p0 = nullptr;
  int n0 = 0;
  int32_t* p1 = nullptr;
  int n1 = 0;
};

template <int KMAX>
__global__ __launch_bounds__(kRouteThreads) void route_topk_kernel(const float* __restrict__ logits, int64_t M, int E,
                                                                   int k, int32_t* __restrict__ topk_idx,
                                                                   float* __restrict__ topk_w, ClearRanges clr) {
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < clr.n0; i += kRouteThreads) clr.p0[i] = 0;
    for (int i = threadIdx.x; i < clr.n1; i += kRouteThreads) clr.p1[i] = 0;
  }
  const int q = threadIdx.x % kLanesPerToken;
  const int64_t t = (int64_t)blockIdx.x * (kRouteThreads / kLanesPerToken) + threadIdx.x / kLanesPerToken;
  const bool valid = t < M;  // whole 16-lane groups share `valid`
  float vals[KMAX];
  int ids[KMAX];
  topk_row<KMAX>(logits + (valid ? t : 0) * (int64_t)E, E, q, valid, vals, ids);
  if (!valid) return;

  // weights: softmax over the k chosen logits, shifted by the largest,
  // summed in slot order; lane j < k writes slot j
  const float l0 = vals[0];
  float denom = 0.0f;
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < k) denom += expf(vals[j] - l0);
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j < k && j == q) {
      topk_idx[t * k + j] = ids[j];
      topk_w[t * k + j] = expf(vals[j] - l0) / denom;
    }
  }
}

hipError_t launch_route(const float* logits, int64_t M, int E, int k, int32_t* topk_idx, float* topk_w,
                        hipStream_t s, int32_t* clear0, int n0, int32_t* clear1, int n1) {
  if (M == 0) return hipSuccess;
  ClearRanges clr;
  clr.p0 = clear0;
  clr.n0 = clear0 ? n0 : 0;
  clr.p1 = clear1;
  clr.n1 = clear1 ? n1 : 0;
  const int64_t per_block = kRouteThreads / kLanesPerToken;
  const dim3 grid((unsigned)((M + per_block - 1) / per_block)), block(kRouteThreads);
  if (k <= 1)
    route_topk_kernel<1><<<grid, block, 0, s>>>(logits, M, E, k, topk_idx, topk_w, clr);
  else if (k <= 2)
    route_topk_kernel<2><<<grid, block, 0, s>>>(logits, M, E, k, topk_idx, topk_w, clr);
  else if (k <= 4)
    route_topk_kernel<4><<<grid, block, 0, s>>>(logits, M, E, k, topk_idx, topk_w, clr);
  else if (k <= 8)
    route_topk_kernel<8><<<grid, block, 0, s>>>(logits, M, E, k, topk_idx, topk_w, clr);
  else
    route_topk_kernel<16><<<grid, block, 0, s>>>(logits, M, E, k, topk_idx, topk_w, clr);
  return hipGetLastError();
}

}  // namespace moe
