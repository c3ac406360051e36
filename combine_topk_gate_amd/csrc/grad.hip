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
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "philox.hpp"

namespace moe {

constexpr int kGradThreads = 256;

__device__ __forceinline__ bool pair_held(int32_t row, int64_t R) { return (uint64_t)(int64_t)row < (uint64_t)R; }

// Outputs are stored as used once ("nt"), so that they do not wait for the L2 to
// make room, though the next call of a training step reads dY and dX_perm (whole
// steps, kept and so: 1024 tokens, 16 experts 2048 x 1408, top 4: 533, 526 us; 8192,
// 16 of them, top 2: 1212, 1201; 1024, 8 of 1024 x 512: 186, 186).  f32 rows of a
// large call are loaded so too (ONCE): from about 96 MiB on they have left the
// last-level cache (256 MB) since they were written, and loading them there again
// only pushes out the rest.  Measured with inputs that change from call to call,
// plain loads and once, tokens of 4096, top 2: combine with dropout of 2048 tokens
// (64 MiB) 17.5, 19.5 us; 4096: 41, 35; 8192: 77, 65; its gradient 22, 27; 51, 43; 94,
// 78.  bf16 rows are loaded plainly (4096 tokens of 2048, top 4: 16.4 us, once 29).
template <bool ONCE>
__device__ __forceinline__ float4 load4(const float* p) {
  f32x4_t v;
  if constexpr (ONCE)
    v = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
  else
    v = *reinterpret_cast<const f32x4_t*>(p);
  return make_float4(v[0], v[1], v[2], v[3]);
}
template <bool>
__device__ __forceinline__ float4 load4(const __bf16* p) {
  const bf16x4_t b = *reinterpret_cast<const bf16x4_t*>(p);
  return make_float4((float)b[0], (float)b[1], (float)b[2], (float)b[3]);
}
template <bool ONCE>
__device__ __forceinline__ float4 load4(const void* p, int bf16, int64_t i) {
  return bf16 ? load4<ONCE>(reinterpret_cast<const __bf16*>(p) + i) : load4<ONCE>(reinterpret_cast<const float*>(p) + i);
}
constexpr int64_t kOnceBytes = 96ll << 20;
__device__ __forceinline__ void store4(void* p, int bf16, int64_t i, float4 v) {
  if (bf16) {
    bf16x4_t o;
    o[0] = (__bf16)v.x;
    o[1] = (__bf16)v.y;
    o[2] = (__bf16)v.z;
    o[3] = (__bf16)v.w;
    __builtin_nontemporal_store(o, reinterpret_cast<bf16x4_t*>(reinterpret_cast<__bf16*>(p) + i));
  } else {
    const f32x4_t o{v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(o, reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(p) + i));
  }
}
// The values of out from element i on: acc and the residual's, one f32 addition, then the cast (as store_out).
__device__ __forceinline__ void finish4(const OutEpilogue& ep, int64_t i, float4 acc) {
  if (ep.residual) {
    const float4 r = load4<false>(ep.residual, ep.res_bf16, i);
    acc.x += r.x;
    acc.y += r.y;
    acc.z += r.z;
    acc.w += r.w;
  }
  store4(ep.out, ep.out_bf16, i, acc);
}

// All kernels here: TPT threads own a token (256 / TPT tokens a block) and walk
// its columns, 4 a thread and U such groups at a time, all of whose loads are
// issued before any is used.  Threads per token by the row's length, so that
// each has one to four groups where it can.
// f(TPT, ONCE); f32_bytes: the f32 rows read; wave_h: the longest row that a wave
// takes alone.
template <typename F>
hipError_t by_size(int H, int64_t f32_bytes, int wave_h, F&& f) {
  const bool once = f32_bytes >= kOnceBytes;
  if (H <= 128) return f(std::integral_constant<int, 16>{}, std::false_type{});
  if (H <= wave_h) {
    if (once) return f(std::integral_constant<int, 64>{}, std::true_type{});
    return f(std::integral_constant<int, 64>{}, std::false_type{});
  }
  if (once) return f(std::integral_constant<int, 256>{}, std::true_type{});
  return f(std::integral_constant<int, 256>{}, std::false_type{});
}
// Measured (256 threads, a wave): combine with dropout of 16384 tokens of 1024, top
// 2: 37.6, 40.5 us; its gradient, whose waves else meet for every token: 53, 41;
// 15712 of 960, 3 of 14 held: 86, 50; 8192 of 2048, top 4: 85, 102.
constexpr int kWaveSums = 512, kWaveGrad = 1024;
inline unsigned token_blocks(int64_t M, int tpt) {
  const int64_t n = (M + kGradThreads / tpt - 1) / (kGradThreads / tpt);
  return (unsigned)(n < 16384 ? n : 16384);
}

// A token's pairs, for waves that own one token each: lane j has pair j's row and
// weight, and only those held are gone through, in slot order (a share of an
// expert-parallel layer holds few: 16 of 128 experts, 4096 tokens of 7168, 8 pairs
// each, all gone through and so: combine with dropout 76, 52 us, its gradient 78,
// 50, the dispatch's 41, 32).  A wave reads other lanes' pairs while some of its lanes
// are past the row's end; the lanes that hold pairs (at most 16) never are, as a row
// has a multiple of 16 groups of four columns.
struct TokenPairs {
  int32_t row;  // of lane j
  float w;
  uint32_t held;  // bit j

  __device__ __forceinline__ TokenPairs(const int32_t* f2s, const float* weights, int64_t t, int k, int64_t R) {
    const int lane = threadIdx.x % kWave;
    row = lane < k ? f2s[t * k + lane] : -1;
    w = weights && lane < k ? weights[t * k + lane] : 1.f;
    held = (uint32_t)__ballot(pair_held(row, R));
  }
  __device__ __forceinline__ int32_t row_of(int j) const { return __builtin_amdgcn_readlane(row, j); }
  __device__ __forceinline__ float w_of(int j) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), j));
  }
};

// ---------------------------------------------------------- rows to tokens ---
// Forward combine with dropout (SRC f32, weights w, DROP) and the dispatch's
// gradient (SRC the problem's type): the sum over the token's held pairs of
// their rows (times w), f32 from zero in slot order, two slots' loads together.
template <int TPT, bool ONCE, typename SRC, bool DROP>
__global__ __launch_bounds__(kGradThreads) void rows_to_tokens_kernel(const SRC* __restrict__ src,
                                                                      const float* __restrict__ w,
                                                                      const int32_t* __restrict__ f2s, int64_t M, int H,
                                                                      int k, OutEpilogue ep, Dropout drop) {
  constexpr int TOK = kGradThreads / TPT, U = 2;
  const int q0 = threadIdx.x % TPT, groups = H / 4;
  for (int64_t t = (int64_t)blockIdx.x * TOK + threadIdx.x / TPT; t < M; t += (int64_t)gridDim.x * TOK) {
    // short rows, several tokens a wave: all k pairs are gone through
    constexpr bool ONE = TPT >= kWave;
    const TokenPairs pairs(f2s, w, ONE ? t : 0, ONE ? k : 0, M * k);
    for (int q = q0; q < groups; q += U * TPT) {
      float4 acc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      uint32_t left = ONE ? pairs.held : (1u << k) - 1;
      while (left) {
        float4 v[2][U];
        bool held[2];
        float wj[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = left ? __builtin_ctz(left) : -1;
          left &= left - 1;
          int32_t row = -1;
          if (j >= 0) row = ONE ? pairs.row_of(j) : f2s[t * k + j];
          held[h] = pair_held(row, M * k);
          wj[h] = 1.f;
          if (DROP && held[h]) wj[h] = ONE ? pairs.w_of(j) : w[t * k + j];
          const SRC* p = src + (int64_t)(held[h] ? row : 0) * H;
#pragma unroll
          for (int u = 0; u < U; ++u)
            v[h][u] = held[h] && q + u * TPT < groups ? load4<ONCE>(p + (int64_t)(q + u * TPT) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!held[h]) continue;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            acc[u].x = fmaf(wj[h], v[h][u].x, acc[u].x);
            acc[u].y = fmaf(wj[h], v[h][u].y, acc[u].y);
            acc[u].z = fmaf(wj[h], v[h][u].z, acc[u].z);
            acc[u].w = fmaf(wj[h], v[h][u].w, acc[u].w);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int qu = q + u * TPT;
        if (qu >= groups) continue;
        if constexpr (DROP) acc[u] = dropped(kept(Philox(drop.rng), drop, (uint64_t)t * groups + qu), drop.scale, acc[u]);
        finish4(ep, t * H + (int64_t)qu * 4, acc[u]);
      }
    }
  }
}

hipError_t launch_combine_dropout(const float* y, const float* topk_w, const int32_t* f2s, int64_t M, int64_t rows, int H,
                                  int k, const OutEpilogue& ep, const Dropout& drop, hipStream_t s) {
  if (M == 0) return hipSuccess;
  return by_size(H, rows * H * 4, kWaveSums, [&](auto tpt, auto once) {
    rows_to_tokens_kernel<tpt.value, once.value, float, true>
        <<<token_blocks(M, tpt.value), kGradThreads, 0, s>>>(y, topk_w, f2s, M, H, k, ep, drop);
    return hipGetLastError();
  });
}

hipError_t launch_dispatch_backward(const void* dxp, bool bf16, const int32_t* f2s, int64_t M, int64_t rows, int H,
                                    int k, const OutEpilogue& ep, hipStream_t s) {
  if (M == 0) return hipSuccess;
  return by_size(H, bf16 ? 0 : rows * H * 4, kWaveSums, [&](auto tpt, auto once) {
    const unsigned grid = token_blocks(M, tpt.value);
    if (bf16)
      rows_to_tokens_kernel<tpt.value, false, __bf16, false>
          <<<grid, kGradThreads, 0, s>>>((const __bf16*)dxp, nullptr, f2s, M, H, k, ep, Dropout{});
    else
      rows_to_tokens_kernel<tpt.value, once.value, float, false>
          <<<grid, kGradThreads, 0, s>>>((const float*)dxp, nullptr, f2s, M, H, k, ep, Dropout{});
    return hipGetLastError();
  });
}

// ------------------------------------------------------- combine's gradient ---
// g is formed once for all k pairs; the k sums of dw stay in registers (KMAX >=
// k of them) and are added across the token's threads in a fixed order.
template <int TPT, bool ONCE, int KMAX, bool DROP>
__global__ __launch_bounds__(kGradThreads) void combine_backward_kernel(CombineBackwardArgs a) {
  constexpr int TOK = kGradThreads / TPT;
  constexpr int U = 2, JG = KMAX < 4 ? KMAX : 4;  // pairs whose loads are issued together
  __shared__ float part[kGradThreads / kWave][KMAX];
  const int q0 = threadIdx.x % TPT, groups = a.H / 4;
  const int64_t R = a.M * a.k;
  for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.M; t0 += (int64_t)gridDim.x * TOK) {
    const int64_t t = t0 + threadIdx.x / TPT;
    const bool valid = t < a.M;
    // the pairs gone through, and how many: of a wave that owns one token those held, else all k
    constexpr bool ONE = TPT >= kWave;
    const TokenPairs pairs(a.f2s, a.topk_w, ONE && valid ? t : 0, ONE && valid ? a.k : 0, R);
    const int n = ONE ? __builtin_popcount(pairs.held) : KMAX;
    int32_t row[KMAX];
    float w[KMAX], s[KMAX];
    uint32_t left = pairs.held;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      row[j] = -1;
      w[j] = s[j] = 0.f;
      if (ONE && j < n) {
        const int from = __builtin_ctz(left);
        left &= left - 1;
        row[j] = pairs.row_of(from);
        w[j] = pairs.w_of(from);
      } else if (!ONE && valid && j < a.k) {
        row[j] = a.f2s[t * a.k + j];
        w[j] = a.topk_w[t * a.k + j];
        if (!pair_held(row[j], R)) row[j] = -1;
      }
    }
    for (int q = q0; n > 0 && valid && q < groups; q += U * TPT) {  // (no pair held: dout is not read)
      float4 g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = q + u * TPT < groups ? load4<false>(a.dout, a.dout_bf16, t * a.H + (int64_t)(q + u * TPT) * 4)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      Kept keep[U];
#pragma unroll
      for (int j0 = 0; j0 < KMAX; j0 += JG) {
        if (j0 >= n) continue;
        float4 y[JG][U];
#pragma unroll
        for (int h = 0; h < JG; ++h) {
          if (row[j0 + h] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u)
            y[h][u] = q + u * TPT < groups ? load4<ONCE>(a.y + (int64_t)row[j0 + h] * a.H + (int64_t)(q + u * TPT) * 4)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if constexpr (DROP) {
          if (j0 == 0) {  // behind the first loads
#pragma unroll
            for (int u = 0; u < U; ++u) {
              keep[u] = kept(Philox(a.drop.rng), a.drop, (uint64_t)t * groups + q + u * TPT);
              g[u] = dropped(keep[u], a.drop.scale, g[u]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int qu = q + u * TPT;
          if (qu >= groups) continue;
#pragma unroll
          for (int h = 0; h < JG; ++h) {
            const int j = j0 + h;
            if (row[j] < 0) continue;
            // what is dropped adds nothing to dw, whatever y holds there
            const float4 v = DROP ? dropped(keep[u], 1.f, y[h][u]) : y[h][u];
            s[j] = fmaf(g[u].x, v.x, fmaf(g[u].y, v.y, fmaf(g[u].z, v.z, fmaf(g[u].w, v.w, s[j]))));
            store4(a.dy, a.dy_bf16, (int64_t)row[j] * a.H + (int64_t)qu * 4,
                   make_float4(w[j] * g[u].x, w[j] * g[u].y, w[j] * g[u].z, w[j] * g[u].w));
          }
        }
      }
    }
    // across the token's lanes, then (TPT > a wave) across its waves
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (j >= n) continue;
#pragma unroll
      for (int off = (TPT < kWave ? TPT : kWave) / 2; off > 0; off >>= 1) s[j] += __shfl_xor(s[j], off);
    }
    // slot j's place among the pairs gone through
    const uint32_t lane = threadIdx.x % kWave, at = __builtin_popcount(pairs.held & ((1u << (lane & 31)) - 1));
    const bool held = lane < 32 && (pairs.held >> (lane & 31) & 1);
    if constexpr (TPT > kWave) {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KMAX; ++j) part[threadIdx.x / kWave][j] = s[j];
      }
      __syncthreads();
      if (threadIdx.x < a.k) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < kGradThreads / kWave; ++v) sum += held ? part[v][at] : 0.f;
        a.dtopk_w[t * a.k + threadIdx.x] = sum;
      }
      __syncthreads();
    } else if constexpr (ONE) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < KMAX; ++j) sum = held && at == j ? s[j] : sum;
      if (valid && lane < a.k) a.dtopk_w[t * a.k + lane] = sum;
    } else {
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (valid && j < a.k && j % TPT == q0) a.dtopk_w[t * a.k + j] = s[j];
    }
  }
}

template <int KMAX>
hipError_t combine_backward_k(const CombineBackwardArgs& a, hipStream_t s) {
  return by_size(a.H, a.rows * a.H * 4, kWaveGrad, [&](auto tpt, auto once) {
    const unsigned grid = token_blocks(a.M, tpt.value);
    if (a.drop.rng)
      combine_backward_kernel<tpt.value, once.value, KMAX, true><<<grid, kGradThreads, 0, s>>>(a);
    else
      combine_backward_kernel<tpt.value, once.value, KMAX, false><<<grid, kGradThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  if (a.k <= 1) return combine_backward_k<1>(a, s);
  if (a.k <= 2) return combine_backward_k<2>(a, s);
  if (a.k <= 4) return combine_backward_k<4>(a, s);
  if (a.k <= 8) return combine_backward_k<8>(a, s);
  return combine_backward_k<16>(a, s);
}

// ----------------------------------------------------------------- router ---
// A block builds the rows of `tokens` tokens in LDS (zeros, then the k values
// of each) and stores them as one contiguous range, 16 bytes a lane.  A thread
// per pair adds the pairs of its token that name the same expert in slot order
// (moe_route never repeats one), so equal ones all write the same sum.
constexpr int kRouteGradFloats = 2048;  // row values a block holds
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
  tokens = tokens < 64 ? tokens / 4 * 4 : 64;  // E <= 512: at least 4
  const int64_t blocks = (M + tokens - 1) / tokens;
  route_backward_kernel<<<(unsigned)blocks, kGradThreads, 0, s>>>(idx, w, dw, M, E, k, tokens, dlogits);
  return hipGetLastError();
}

}  // namespace moe
