// Gradients of the experts' products (grouped GEMM), rows and weights.
//
// "Grouped GEMM 为什么适合 MoE" (C_i = A_i B_i per expert) transposed: with the
// forward g = X Wg^T, u = X Wu^T, h = silu(g) u, Y = h Wd^T per expert,
//   rows, layer 1     dh = dY Wd;  s = 1 / (1 + e^-g);
//                     dg = dh u s (1 + g (1 - s)),  du = dh g s
//   rows, layer 0     dX = dg Wg + du Wu
//   weights, layer 1  dWd = dY^T h
//   weights, layer 0  dWg = dg^T X,  dWu = du^T X   (the sums run over rows)
// A static tile queue as in the forward grouped GEMM; each output element is
// formed by one workgroup in a fixed order, so nothing depends on scheduling.
#include "common.hpp"
#include "gemm_grad_bf16.hpp"
#include "gemm_grad_f32.hpp"
#include "launch.hpp"
#include "tiles.hpp"

namespace moe {

// as swiglu_grad_fast, for f32 outputs
__device__ __forceinline__ SwigluGrad swiglu_grad(float dh, float g, float u) {
  const float s = 1.0f / (1.0f + expf(-g));
  return {dh * u * (s * fmaf(g, 1.0f - s, 1.0f)), dh * (g * s)};
}

// ------------------------------------------------------------------- bf16 ---
// Rows: the experts' rows (over all source blocks) in tiles of 256, or of 128
// where an expert has no more and in a last round that would leave half the
// workgroups idle, in the forward queue's order.
template <GradKind KIND>
__global__ __launch_bounds__(kGemmThreads) void grad_rows_bf16_kernel(GradGemmArgs a, int xcd_slots) {
  __shared__ __attribute__((aligned(16))) char lds[kGemmLdsBytes];
  __shared__ TileLds tl;
  __shared__ int rowpos[2][kTileRows];  // of this tile and of the next
  const int K = KIND == kGradRows0 ? a.F : a.H, N = KIND == kGradRows0 ? a.H : a.F, S = a.G / a.E;
  const int NT = (N + 255) / 256;
  const int T = build_expert_tile_table(a.offsets, a.G, a.E, kTileRows, tl) * NT;
  const int64_t panel = (int64_t)kTileRows * K * (KIND == kGradRows0 ? 4 : 2);
  const int grid = gridDim.x;
  const int r = T % grid;
  const int half = (r > 0 && 2 * r <= grid && T > grid) ? r : 0;  // tiles of the last round to halve
  const int entries = T + half;
  const Shuffle sm = make_shuffle(a.shuffle, T - half), sh = make_shuffle(a.shuffle, half);
  GradTile t{0, 0, 0, 0};
  bool low = false;  // 128 rows
  // Entry v or the next one of this workgroup that has rows; its rows' positions into rowpos[b].
  auto find = [&](int v, int b) {
    for (; v < entries; v += grid) {
      const bool is_half = v >= T - half;
      const int j = v - (T - half);
      const TileCoord c = tile_coord(is_half ? T - half + shuffled(sh, j / 2) : shuffled(sm, v), a.E, NT, kTileRows,
                                     xcd_slots, panel, tl);
      const int m0 = is_half ? c.m0 + (j & 1) * (kTileRows / 2) : c.m0;
      const int n = tl.expert_rows[c.g];
      if (m0 >= n) continue;
      rowpos[b][threadIdx.x] = expert_row(tl, c.g, a.E, S, m0, threadIdx.x);
      t = {c.g, 0, c.nt * 256, 0};
      low = is_half || n <= kTileRows / 2;
      break;
    }
    return v;
  };
  int b = 0;
  int v = find(xcd_slot(blockIdx.x, grid), b);
  // Tiles as long as they are of one height; the first loads of each but the first are issued before the epilogue of
  // the one before.
  auto run = [&]<int TM>() {
    GradWave<KIND, TM> wave(a, lds, nullptr);
    __syncthreads();  // rowpos[b]
    wave.begin(t, rowpos[b]);
    bool more;
    do {
      const GradTile now = t;
      wave.multiply();
      v = find(v + grid, b ^ 1);
      more = v < entries && low == (TM < kTileRows);
      if (more) {
        __syncthreads();
        wave.begin(t, rowpos[b ^ 1]);
      }
      wave.epilogue(now, rowpos[b]);
      b ^= 1;
    } while (more);
  };
  while (v < entries) {
    if (low)
      run.template operator()<kTileRows / 2>();
    else
      run.template operator()<kTileRows>();
  }
}

// Weights: 256 x 256 tiles of dW, expert by expert; the row tiles (layer 0:
// of both matrices, which share x's panels) in blocks of 8, so that the 32
// tiles an XCD runs at once share 8 + 4 panels in its L2.
__global__ __launch_bounds__(kGemmThreads) void grad_weights_bf16_kernel(GradGemmArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[kGemmLdsBytes];
  __shared__ int offsets[kMaxTileSegs + 1];
  for (int i = threadIdx.x; i <= a.G; i += kGemmThreads) offsets[i] = a.offsets[i];
  const bool l0 = a.layer == 0;
  const int N = l0 ? a.F : a.H, C = l0 ? a.H : a.F;
  const int NR = (N + 255) / 256, NC = (C + 255) / 256, rows = (l0 ? 2 : 1) * NR;
  const int T = a.E * rows * NC, grid = gridDim.x;
  const Shuffle sm = make_shuffle(a.shuffle, T);
  auto tile = [&](int v) {
    const int s = shuffled(sm, v), e = s / (rows * NC), l = s - e * rows * NC;
    const int nb = (rows + 7) / 8, b = min((int)((int64_t)(l / NC) * nb / rows), nb - 1);
    auto first = [&](int i) { return (int)((int64_t)i * rows / nb); };
    const int bb = first(b + 1) <= l / NC ? b + 1 : b;
    const int r0 = first(bb), rb = first(bb + 1) - r0, lb = l - r0 * NC;
    const int row = r0 + lb % rb, second = row >= NR;
    return GradTile{e, (row - second * NR) * 256, lb / rb * 256, second};
  };
  GradWave<kGradWeights, kTileRows> wave(a, lds, offsets);
  int v = xcd_slot(blockIdx.x, grid);
  if (v >= T) return;
  __syncthreads();
  GradTile t = tile(v);
  wave.begin(t, nullptr);
  while (true) {
    wave.multiply();
    v += grid;
    const GradTile now = t;
    if (v < T) {
      t = tile(v);
      wave.begin(t, nullptr);
    }
    wave.epilogue(now, nullptr);
    if (v >= T) break;
  }
}

// -------------------------------------------------------------------- f32 ---
template <int LAYER, int TS>
__global__ __launch_bounds__(kGfThreads) void grad_rows_f32_kernel(GradGemmArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[gf_lds_floats<TS>];
  __shared__ TileLds tl;
  __shared__ int rowpos[TS];
  const int K = LAYER == 0 ? a.F : a.H, N = LAYER == 0 ? a.H : a.F;  // reduction and columns of a product
  const int NT = (N + TS - 1) / TS, S = a.G / a.E;
  const int total = build_expert_tile_table(a.offsets, a.G, a.E, TS, tl) * NT;
  const Shuffle sm = make_shuffle(a.shuffle, total);
  constexpr int kBuf = kGfK * gf_pitch<TS>;
  for (int v = blockIdx.x; v < total; v += gridDim.x) {
    const TileCoord c = tile_coord(shuffled(sm, v), a.E, NT, TS, 1, 0, tl);
    const int e = c.g, col0 = c.nt * TS;
    for (int i = threadIdx.x; i < TS; i += kGfThreads) rowpos[i] = expert_row(tl, e, a.E, S, c.m0, i);
    __syncthreads();
    const float* rows0[TS / 32];
    const float* rows1[TS / 32];
#pragma unroll
    for (int i = 0; i < TS / 32; ++i) {
      const int r = rowpos[(threadIdx.x >> 3) + 32 * i];
      rows0[i] = r >= 0 ? (const float*)a.d0 + (int64_t)r * K : nullptr;
      rows1[i] = LAYER == 0 && r >= 0 ? (const float*)a.d1 + (int64_t)r * K : nullptr;
    }
    const float* w0 = (const float*)a.w0 + (int64_t)e * K * N;
    const float* w1 = LAYER == 0 ? (const float*)a.w1 + (int64_t)e * K * N : nullptr;
    const int per = K / kGfK, steps = LAYER == 0 ? 2 * per : per;
    GfPart<TS> pw, px;
    auto load = [&](int s) {
      const bool second = LAYER == 0 && s >= per;
      const int k = (second ? s - per : s) * kGfK;
      gf_load_k<TS>(px, second ? rows1 : rows0, k);
      gf_load_c<TS>(pw, (second ? w1 : w0) + (int64_t)k * N, N, kGfK, col0, N);
    };
    auto store = [&](int b) {
      gf_store_c<TS>(lds + b * 2 * kBuf, pw);
      gf_store_k<TS>(lds + b * 2 * kBuf + kBuf, px);
    };
    GfAcc<TS> acc;
    gf_zero(acc);
    load(0);
    store(0);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
      if (s + 1 < steps) load(s + 1);
      gf_mul<TS>(acc, lds + (s & 1) * 2 * kBuf, lds + (s & 1) * 2 * kBuf + kBuf);
      if (s + 1 < steps) store((s + 1) & 1);
      __syncthreads();
    }
    gf_each<TS>(acc, [&](int t, int n, f32x4_t o) {
      const int r = rowpos[t];
      if (r < 0 || col0 + n >= N) return;
      const int64_t at = (int64_t)r * N + col0 + n;
      if constexpr (LAYER == 0) {
        gf_store4((float*)a.o0 + at, o);
      } else {
        const f32x4_t g = gf_load4((const float*)a.gate + at), u = gf_load4((const float*)a.up + at);
        f32x4_t dg, du;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const SwigluGrad d = swiglu_grad(o[i], g[i], u[i]);
          dg[i] = d.dg;
          du[i] = d.du;
        }
        gf_store4((float*)a.o0 + at, dg);
        gf_store4((float*)a.o1 + at, du);
      }
    });
    __syncthreads();  // rowpos and the LDS buffers are free for the next tile
  }
}

// Tile of dW[e]: TS of the first operand's columns (its rows) x TS of x's.
// The K steps run over the expert's segments one after the other, the last
// step of each filled up with zero rows.
template <int LAYER, int TS>
__global__ __launch_bounds__(kGfThreads) void grad_weights_f32_kernel(GradGemmArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[gf_lds_floats<TS>];
  const int N = LAYER == 0 ? a.F : a.H, C = LAYER == 0 ? a.H : a.F;  // rows and columns of dW
  const int NR = (N + TS - 1) / TS, NC = (C + TS - 1) / TS, S = a.G / a.E;
  const int mats = LAYER == 0 ? 2 : 1;
  const int64_t total = (int64_t)a.E * mats * NR * NC;
  constexpr int kBuf = kGfK * gf_pitch<TS>;
  for (int64_t v = blockIdx.x; v < total; v += gridDim.x) {
    const int e = (int)(v / ((int64_t)mats * NR * NC));
    int l = (int)(v - (int64_t)e * mats * NR * NC);
    const int m = l / (NR * NC);
    l -= m * NR * NC;
    const int row0 = l % NR * TS, col0 = l / NR * TS;
    const float* d = (const float*)(m ? a.d1 : a.d0);
    int s = 0, r = 0, end = 0;  // the segment being read, its next row and its end
    auto next_segment = [&] {  // to the first unread row; false: none left
      while (r >= end && s < S) {
        r = a.offsets[s * a.E + e];
        end = a.offsets[s * a.E + e + 1];
        ++s;
      }
      return r < end;
    };
    GfPart<TS> pw, px;
    auto load = [&] {
      const int n = end - r;
      gf_load_c<TS>(pw, (const float*)a.x + (int64_t)r * C, C, n, col0, C);
      gf_load_c<TS>(px, d + (int64_t)r * N, N, n, row0, N);
      r += kGfK;
    };
    auto store = [&](int b) {
      gf_store_c<TS>(lds + b * 2 * kBuf, pw);
      gf_store_c<TS>(lds + b * 2 * kBuf + kBuf, px);
    };
    GfAcc<TS> acc;
    gf_zero(acc);
    bool more = next_segment();
    if (more) {
      load();
      store(0);
    }
    __syncthreads();
    for (int b = 0; more; b ^= 1) {
      more = next_segment();
      if (more) load();
      gf_mul<TS>(acc, lds + b * 2 * kBuf, lds + b * 2 * kBuf + kBuf);
      if (more) store(b ^ 1);
      __syncthreads();
    }
    void* out = m ? a.o1 : a.o0;
    gf_each<TS>(acc, [&](int t, int n, f32x4_t o) {
      if (row0 + t >= N || col0 + n >= C) return;
      const int64_t at = ((int64_t)e * N + row0 + t) * C + col0 + n;
      if (a.out_bf16) {
        gf_store4((__bf16*)out + at, o);
      } else {
        float* p = (float*)out + at;
        gf_store4(p, a.accumulate ? *(const f32x4_t*)p + o : o);
      }
    });
  }
}

template <int LAYER>
hipError_t grad_rows_launch(const GradGemmArgs& a, hipStream_t s) {
  grad_rows_f32_kernel<LAYER, 64><<<2 * device_cu_count(), kGfThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_rows(const GradGemmArgs& a, bool bf16, hipStream_t s) {
  if (a.R == 0) return hipSuccess;
  const int grid = device_cu_count(), xcd_slots = grid / kXcds > 0 ? grid / kXcds : 1;
  if (bf16) {
    if (a.layer == 0)
      grad_rows_bf16_kernel<kGradRows0><<<grid, kGemmThreads, 0, s>>>(a, xcd_slots);
    else
      grad_rows_bf16_kernel<kGradRows1><<<grid, kGemmThreads, 0, s>>>(a, xcd_slots);
    return hipGetLastError();
  }
  return a.layer == 0 ? grad_rows_launch<0>(a, s) : grad_rows_launch<1>(a, s);
}

template <int LAYER>
hipError_t grad_weights_launch(const GradGemmArgs& a, hipStream_t s) {
  grad_weights_f32_kernel<LAYER, 64><<<2 * device_cu_count(), kGfThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_weights(const GradGemmArgs& a, bool bf16, hipStream_t s) {
  if (bf16) {
    grad_weights_bf16_kernel<<<device_cu_count(), kGemmThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  return a.layer == 0 ? grad_weights_launch<0>(a, s) : grad_weights_launch<1>(a, s);
}

}  // namespace moe
