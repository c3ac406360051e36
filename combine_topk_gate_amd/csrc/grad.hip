// Gradients of the layer's memory-bound steps: router, dispatch, combine.
//
// COMET paper review §4.1.1 (Top-K reduction) and the PTO MoE article (local
// reorder, top-K weighted accumulation) give the forward steps; these are
// their transposes.  With pair f = t k + j, its row r = flat_to_sorted[f] (-1:
// not held) and its weight w[f]:
//   combine   out[t] = drop(sum_j w[f] Y[r])  ->  g[t] = drop(dout[t]),
//             dY[r] = w[f] g[t],  dw[f] = sum_n g[t,n] Y[r,n]
//   dispatch  X_perm[r] = x[t]  ->  dx[t] = sum_j dX_perm[r]  (+ residual)
//   route     w = softmax of the chosen logits  ->
//             dlogits[t, idx_j] = w_j (dw_j - sum_i w_i dw_i), the rest 0
// All are bound by HBM traffic.  Nothing is added by atomics: a token's rows
// are read (or written) by the lanes that own the token.
#include "common.hpp"
#include "launch.hpp"
#include "philox.hpp"

namespace moe {

constexpr int kGradThreads = 256;

__device__ __forceinline__ bool pair_held(int32_t row, int64_t R) { return (uint64_t)(int64_t)row < (uint64_t)R; }

__device__ __forceinline__ float4 load4(const void* p, int bf16, int64_t i) {
  if (bf16) {
    const bf16x4_t b = *reinterpret_cast<const bf16x4_t*>(reinterpret_cast<const __bf16*>(p) + i);
    return make_float4((float)b[0], (float)b[1], (float)b[2], (float)b[3]);
  }
  return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
}

__device__ __forceinline__ void store4(void* p, int bf16, int64_t i, float4 v) {
  if (bf16) {
    bf16x4_t o;
    o[0] = (__bf16)v.x;
    o[1] = (__bf16)v.y;
    o[2] = (__bf16)v.z;
    o[3] = (__bf16)v.w;
    *reinterpret_cast<bf16x4_t*>(reinterpret_cast<__bf16*>(p) + i) = o;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = v;
  }
}

// ---------------------------------------------------------------- combine ---
// TPT threads own a token (256 / TPT tokens a block) and walk its columns, 4
// a thread and step; g is formed once for all k pairs, the k sums of dw stay
// in registers (KMAX >= k of them) and are added across the token's threads
// in a fixed order.
template <int TPT, int KMAX, bool DROP>
__global__ __launch_bounds__(kGradThreads) void combine_backward_kernel(CombineBackwardArgs a) {
  constexpr int TOK = kGradThreads / TPT;  // tokens per block
  __shared__ float part[kGradThreads / kWave][KMAX];
  const int q0 = threadIdx.x % TPT;
  const int groups = a.H / 4;
  const int64_t R = a.M * a.k;
  for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.M; t0 += (int64_t)gridDim.x * TOK) {
    const int64_t t = t0 + threadIdx.x / TPT;
    const bool valid = t < a.M;
    int32_t row[KMAX];
    float w[KMAX], s[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const bool in = valid && j < a.k;
      row[j] = in ? a.f2s[t * a.k + j] : -1;
      w[j] = in ? a.topk_w[t * a.k + j] : 0.f;
      if (!pair_held(row[j], R)) row[j] = -1;
      s[j] = 0.f;
    }
    for (int q = q0; valid && q < groups; q += TPT) {
      float4 g = load4(a.dout, a.dout_bf16, t * a.H + (int64_t)q * 4);
      float4 y[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        y[j] = row[j] >= 0 ? *reinterpret_cast<const float4*>(a.y + (int64_t)row[j] * a.H + (int64_t)q * 4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      if constexpr (DROP) {
        // what is dropped adds nothing to dw, whatever y holds there
        const Kept keep = kept(Philox(a.drop.rng), a.drop, (uint64_t)t * groups + q);
        g = dropped(keep, a.drop.scale, g);
#pragma unroll
        for (int j = 0; j < KMAX; ++j) y[j] = dropped(keep, 1.f, y[j]);
      }
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (row[j] < 0) continue;
        s[j] = fmaf(g.x, y[j].x, fmaf(g.y, y[j].y, fmaf(g.z, y[j].z, fmaf(g.w, y[j].w, s[j]))));
        store4(a.dy, a.dy_bf16, (int64_t)row[j] * a.H + (int64_t)q * 4,
               make_float4(w[j] * g.x, w[j] * g.y, w[j] * g.z, w[j] * g.w));
      }
    }
    // across the token's lanes, then (TPT > a wave) across its waves
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
      for (int off = (TPT < kWave ? TPT : kWave) / 2; off > 0; off >>= 1) s[j] += __shfl_xor(s[j], off);
    }
    if constexpr (TPT > kWave) {
      if (threadIdx.x % kWave == 0) {
#pragma unroll
        for (int j = 0; j < KMAX; ++j) part[threadIdx.x / kWave][j] = s[j];
      }
      __syncthreads();
      if (threadIdx.x < a.k) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < kGradThreads / kWave; ++v) sum += part[v][threadIdx.x];
        a.dtopk_w[t * a.k + threadIdx.x] = sum;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (valid && j < a.k && j % TPT == q0) a.dtopk_w[t * a.k + j] = s[j];
    }
  }
}

template <int TPT, int KMAX>
hipError_t combine_backward_launch(const CombineBackwardArgs& a, hipStream_t s) {
  const int64_t blocks = (a.M + kGradThreads / TPT - 1) / (kGradThreads / TPT);
  const unsigned grid = (unsigned)(blocks < 16384 ? blocks : 16384);
  if (a.drop.rng)
    combine_backward_kernel<TPT, KMAX, true><<<grid, kGradThreads, 0, s>>>(a);
  else
    combine_backward_kernel<TPT, KMAX, false><<<grid, kGradThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <int KMAX>
hipError_t combine_backward_k(const CombineBackwardArgs& a, hipStream_t s) {
  // threads per token: no more than the 4-column groups of a row
  if (a.H <= 128) return combine_backward_launch<16, KMAX>(a, s);
  if (a.H <= 512) return combine_backward_launch<64, KMAX>(a, s);
  return combine_backward_launch<256, KMAX>(a, s);
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  if (a.k <= 1) return combine_backward_k<1>(a, s);
  if (a.k <= 2) return combine_backward_k<2>(a, s);
  if (a.k <= 4) return combine_backward_k<4>(a, s);
  if (a.k <= 8) return combine_backward_k<8>(a, s);
  return combine_backward_k<16>(a, s);
}

// --------------------------------------------------------------- dispatch ---
// dx[t] = sum over the token's held pairs of their rows, f32 from zero in slot
// order, then the output epilogue.
template <int TPT>
__global__ __launch_bounds__(kGradThreads) void dispatch_backward_kernel(const void* __restrict__ dxp, int bf16,
                                                                         const int32_t* __restrict__ f2s, int64_t M,
                                                                         int H, int k, OutEpilogue ep) {
  constexpr int TOK = kGradThreads / TPT;
  const int q0 = threadIdx.x % TPT;
  const int groups = H / 4;
  for (int64_t t = (int64_t)blockIdx.x * TOK + threadIdx.x / TPT; t < M; t += (int64_t)gridDim.x * TOK) {
    for (int q = q0; q < groups; q += TPT) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j = 0; j < k; ++j) {
        const int32_t row = f2s[t * k + j];
        if (!pair_held(row, M * k)) continue;
        const float4 v = load4(dxp, bf16, (int64_t)row * H + (int64_t)q * 4);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      store_out(ep, t * H + (int64_t)q * 4, acc);
    }
  }
}

template <int TPT>
hipError_t dispatch_backward_launch(const void* dxp, int bf16, const int32_t* f2s, int64_t M, int H, int k,
                                    const OutEpilogue& ep, hipStream_t s) {
  const int64_t blocks = (M + kGradThreads / TPT - 1) / (kGradThreads / TPT);
  dispatch_backward_kernel<TPT><<<(unsigned)(blocks < 16384 ? blocks : 16384), kGradThreads, 0, s>>>(dxp, bf16, f2s, M,
                                                                                                      H, k, ep);
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const void* dxp, bool bf16, const int32_t* f2s, int64_t M, int H, int k,
                                    const OutEpilogue& ep, hipStream_t s) {
  if (M == 0) return hipSuccess;
  if (H <= 128) return dispatch_backward_launch<16>(dxp, bf16, f2s, M, H, k, ep, s);
  if (H <= 512) return dispatch_backward_launch<64>(dxp, bf16, f2s, M, H, k, ep, s);
  return dispatch_backward_launch<256>(dxp, bf16, f2s, M, H, k, ep, s);
}

// ----------------------------------------------------------------- router ---
// A block builds the rows of `tokens` tokens in LDS (zeros, then the k values
// of each) and stores them as one contiguous range, 16 bytes a lane.  A thread
// per pair adds the pairs of its token that name the same expert in slot order
// (moe_route never repeats one), so equal ones all write the same sum.
constexpr int kRouteGradFloats = 8192;  // row values a block holds: 32 KiB
constexpr int kRouteGradPairs = 1024;

__global__ __launch_bounds__(kGradThreads) void route_backward_kernel(const int32_t* __restrict__ idx,
                                                                      const float* __restrict__ w,
                                                                      const float* __restrict__ dw, int64_t M, int E,
                                                                      int k, int tokens, float* __restrict__ dlogits) {
  __shared__ __attribute__((aligned(16))) float rows[kRouteGradFloats];
  __shared__ int se[kRouteGradPairs];
  __shared__ float sw[kRouteGradPairs], sd[kRouteGradPairs];
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int n = (int)(M - t0 < tokens ? M - t0 : tokens);
  for (int i = threadIdx.x; i < n * k; i += kGradThreads) {
    se[i] = idx[t0 * k + i];
    sw[i] = w[t0 * k + i];
    sd[i] = dw[t0 * k + i];
  }
  const int values = n * E;
  for (int i = threadIdx.x * 4; i < values; i += kGradThreads * 4)
    *reinterpret_cast<float4*>(rows + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  for (int i = threadIdx.x; i < n * k; i += kGradThreads) {
    const int t = i / k, p0 = t * k, e = se[i];
    float mean = 0.f;
    for (int j = 0; j < k; ++j) mean = fmaf(sw[p0 + j], sd[p0 + j], mean);
    float v = 0.f;
    for (int j = 0; j < k; ++j)
      if (se[p0 + j] == e) v += sw[p0 + j] * (sd[p0 + j] - mean);
    if ((unsigned)e < (unsigned)E) rows[t * E + e] = v;
  }
  __syncthreads();
  float* dst = dlogits + t0 * E;  // 16-byte aligned: tokens * E is a multiple of 4 for every block but the last
  for (int i = threadIdx.x * 4; i + 3 < values; i += kGradThreads * 4)
    *reinterpret_cast<float4*>(dst + i) = *reinterpret_cast<const float4*>(rows + i);
  if (threadIdx.x < values % 4) dst[values / 4 * 4 + threadIdx.x] = rows[values / 4 * 4 + threadIdx.x];
}

hipError_t launch_route_backward(const int32_t* idx, const float* w, const float* dw, int64_t M, int E, int k,
                                 float* dlogits, hipStream_t s) {
  if (M == 0) return hipSuccess;
  // a multiple of 4 tokens, so that every block's range starts 16-byte aligned
  int tokens = kRouteGradFloats / E < kRouteGradPairs / k ? kRouteGradFloats / E : kRouteGradPairs / k;
  tokens = tokens < 64 ? tokens / 4 * 4 : 64;  // E <= 512: at least 16
  const int64_t blocks = (M + tokens - 1) / tokens;
  route_backward_kernel<<<(unsigned)blocks, kGradThreads, 0, s>>>(idx, w, dw, M, E, k, tokens, dlogits);
  return hipGetLastError();
}

}  // namespace moe
