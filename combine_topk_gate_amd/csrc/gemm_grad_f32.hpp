// f32 tiles of the grouped GEMM's gradients, on the f32 matrix instruction
// v_mfma_f32_32x32x2_f32 (each product and sum in f32).
//
// A tile is TS rows x TS columns of the output (TS = 128, or 64 where there
// are few tiles), 4 waves of TS/2 x TS/2.  The columns are the instruction's
// first operand, so a lane holds 4 consecutive columns of one row.  The K
// index is stepped by 32 through LDS, [k][TS] per operand, double-buffered,
// the next step's loads in registers while the current one is multiplied.
// An operand whose memory is contiguous along k (the token rows of a rows'
// gradient) is turned while it is stored to LDS; all others (weights there,
// both operands of a weights' gradient) lie as LDS has them.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "tiles.hpp"

namespace moe {

constexpr int kGfThreads = 256;
constexpr int kGfK = 32;

__device__ __forceinline__ f32x4_t gf_load4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }

template <typename T>
__device__ __forceinline__ void gf_store4(T* p, f32x4_t v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f32x4_t*>(p) = v;
  } else {
    bf16x4_t b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = (__bf16)v[i];
    *reinterpret_cast<bf16x4_t*>(p) = b;
  }
}

// One operand's part of a K step: TS x 32 values as TS / 32 groups of 4 a thread.
template <int TS>
struct GfPart {
  f32x4_t v[TS / 32];
};

template <int TS>
constexpr int gf_pitch = TS + 4;  // LDS floats per k: 16-byte aligned, 4 k apart on other banks
template <int TS>
constexpr int gf_lds_floats = 4 * kGfK * gf_pitch<TS>;

// k contiguous: row i of the tile at rows[i] (null: zeros), values k .. k + 31
template <int TS>
__device__ __forceinline__ void gf_load_k(GfPart<TS>& o, const float* const (&rows)[TS / 32], int k) {
#pragma unroll
  for (int i = 0; i < TS / 32; ++i)
    o.v[i] = rows[i] ? gf_load4(rows[i] + k + 4 * (threadIdx.x & 7)) : f32x4_t{0.f, 0.f, 0.f, 0.f};
}
template <int TS>
__device__ __forceinline__ void gf_store_k(float* lds, const GfPart<TS>& o) {
#pragma unroll
  for (int i = 0; i < TS / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) lds[(4 * (threadIdx.x & 7) + j) * gf_pitch<TS> + (threadIdx.x >> 3) + 32 * i] = o.v[i][j];
}

// columns contiguous: k rows base + kk * pitch, kk < valid, columns col0 .. col0 + TS (those from cols on: zeros)
template <int TS>
__device__ __forceinline__ void gf_load_c(GfPart<TS>& o, const float* base, int64_t pitch, int valid, int col0, int cols) {
  constexpr int per = TS / 4, step = kGfThreads / per;
  const int c = col0 + 4 * (threadIdx.x % per);
#pragma unroll
  for (int i = 0; i < TS / 32; ++i) {
    const int kk = threadIdx.x / per + step * i;
    o.v[i] = kk < valid && c < cols ? gf_load4(base + kk * pitch + c) : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}
template <int TS>
__device__ __forceinline__ void gf_store_c(float* lds, const GfPart<TS>& o) {
  constexpr int per = TS / 4, step = kGfThreads / per;
#pragma unroll
  for (int i = 0; i < TS / 32; ++i)
    *reinterpret_cast<f32x4_t*>(lds + (threadIdx.x / per + step * i) * gf_pitch<TS> + 4 * (threadIdx.x % per)) = o.v[i];
}

// The wave's fragments: rows 32 j + (lane & 31) of its half, columns 32 i + 8 (v / 4) + 4 (lane >> 5) + v % 4.
template <int TS>
struct GfAcc {
  f32x16_t v[TS / 64][TS / 64];  // [column fragment][row fragment]
};

template <int TS>
__device__ __forceinline__ void gf_zero(GfAcc<TS>& a) {
#pragma unroll
  for (int i = 0; i < TS / 64; ++i)
#pragma unroll
    for (int j = 0; j < TS / 64; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) a.v[i][j][v] = 0.f;
}

template <int TS>
__device__ __forceinline__ void gf_mul(GfAcc<TS>& a, const float* wlds, const float* xlds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = (lane >> 5) * gf_pitch<TS> + (lane & 31);
  const float* wp = wlds + at + (wave & 1) * (TS / 2);
  const float* xp = xlds + at + (wave >> 1) * (TS / 2);
#pragma unroll
  for (int k = 0; k < kGfK; k += 2) {
    float fw[TS / 64], fx[TS / 64];
#pragma unroll
    for (int i = 0; i < TS / 64; ++i) {
      fw[i] = wp[k * gf_pitch<TS> + 32 * i];
      fx[i] = xp[k * gf_pitch<TS> + 32 * i];
    }
#pragma unroll
    for (int i = 0; i < TS / 64; ++i)
#pragma unroll
      for (int j = 0; j < TS / 64; ++j)
        a.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fw[i], fx[j], a.v[i][j], 0, 0, 0);
  }
}

// f(row of the tile, first of 4 columns of the tile, values)
template <int TS, typename F>
__device__ __forceinline__ void gf_each(const GfAcc<TS>& a, F&& f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < TS / 64; ++j)
#pragma unroll
    for (int i = 0; i < TS / 64; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4_t o;
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = a.v[i][j][4 * q + v];
        f((wave >> 1) * (TS / 2) + 32 * j + (lane & 31), (wave & 1) * (TS / 2) + 32 * i + 8 * q + 4 * (lane >> 5), o);
      }
}

}  // namespace moe
