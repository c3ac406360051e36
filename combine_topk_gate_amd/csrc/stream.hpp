// Weight-streaming product tile for few token rows (gfx950): the decode
// layer's two products and the adapter projection's short batches.
//
//   acc[i][j] = sum_k W[i, k] X[j, k]    i: 16 NW weight rows, j: 16 NT token rows
//
// With few token rows every weight is used once per call, so the tile has no
// LDS staging: the weight rows are the MFMA "A" operand and go from HBM
// straight into registers, 16 bytes per lane and load (a 16-row x 64-byte
// block per wave), and the token rows, the "B" operand, come from the L2 the
// same way.  The block's waves split the reduction: wave w takes chunks
// w, w + waves, ... of U steps, so one weight row is read as a contiguous run
// by the waves together, and the partial accumulators are added in LDS in
// wave order at the end (a fixed order: the bits do not depend on timing).
// Two chunks are in flight per wave (one computing, one loading).
//
// Token rows that do not exist (row offset kNoRow) and steps past the
// reduction read zeros through the buffer range check, without touching
// memory.
#pragma once

#include "common.hpp"
#include "gemm_bf16.hpp"

namespace moe {

constexpr int kStreamThreads = 256;
constexpr int kStreamWaves = kStreamThreads / 64;
constexpr uint32_t kNoRow = 0x80000000u;  // row offset past every buffer range

// f32 value as NP bf16 values whose sum is the value (NP = 3: exactly, but
// for magnitudes below 2^-110; NP = 2: to 2^-17 of it).
template <int NP>
__device__ __forceinline__ void split_bf16(float v, __bf16 (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    p[i] = (__bf16)v;
    v -= (float)p[i];
  }
}

// ---- operand kinds: kStep reduction elements a step; a weight row takes 64
// bytes of every step, 16 of them per lane group q = lane / 16; a token row
// takes kX loads of 16 bytes per lane at kXBytes a step.

// bf16 weights, token rows in NP bf16 planes (their sum is the row's value).
template <int NP>
struct StreamBf16 {
  static constexpr int kStep = 32, kX = NP, kXBytes = 64, kXLane = 16;
  static __device__ __forceinline__ void load_x(i32x4_t (&x)[kX], __amdgpu_buffer_rsrc_t r, uint32_t off,
                                                uint32_t soff, uint32_t plane) {
#pragma unroll
    for (int p = 0; p < NP; ++p) x[p] = buf_load16(r, off + (uint32_t)p * plane, soff);
  }
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, uint32_t, int,
                                             const i32x4_t (&x)[NT][kX]) {
    const bf16x8_t a = __builtin_bit_cast(bf16x8_t, w);
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[j][p]), acc[j], 0, 0, 0);
  }
};

// f32 weights and token rows: a lane's 4 consecutive elements feed 4 MFMAs
// of K = 4 (both operands in the same permuted order of k).
struct StreamF32 {
  static constexpr int kStep = 16, kX = 1, kXBytes = 64, kXLane = 16;
  static __device__ __forceinline__ void load_x(i32x4_t (&x)[kX], __amdgpu_buffer_rsrc_t r, uint32_t off,
                                                uint32_t soff, uint32_t) {
    x[0] = buf_load16(r, off, soff);
  }
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, uint32_t, int,
                                             const i32x4_t (&x)[NT][kX]) {
    const f32x4_t a = __builtin_bit_cast(f32x4_t, w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], __builtin_bit_cast(f32x4_t, x[j][0])[i], acc[j], 0, 0, 0);
  }
};

// MXFP8 weights (e4m3 codes, one scale byte per 32), token rows in NP bf16
// planes.  A lane's 16 codes are two bf16 fragments: the conversion applies
// the block's power-of-two scale, and every e4m3 value times it is a bf16
// value (3 bits of mantissa), so nothing is rounded.  Fragment s takes the
// codes 8 s .. 8 s + 7 of every lane group; the token loads follow.
template <int NP>
struct StreamMx {
  static constexpr int kStep = 64, kX = 2 * NP, kXBytes = 128, kXLane = 32;
  static __device__ __forceinline__ void load_x(i32x4_t (&x)[kX], __amdgpu_buffer_rsrc_t r, uint32_t off,
                                                uint32_t soff, uint32_t plane) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int s = 0; s < 2; ++s) x[2 * p + s] = buf_load16(r, off + (uint32_t)p * plane + 16u * s, soff);
  }
  // scales: the 4 scale bytes of the lane's row for the 128 columns the step
  // lies in; byte: which of them holds the lane's block
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, uint32_t scales, int byte,
                                             const i32x4_t (&x)[NT][kX]) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const uint32_t e = (scales >> (8 * byte)) & 0xFFu;
    const float sc = __builtin_bit_cast(float, e << 23);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t a;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = (uint32_t)w[2 * s + h];
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, false);
        const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, true);
        a[4 * h] = lo[0];
        a[4 * h + 1] = lo[1];
        a[4 * h + 2] = hi[0];
        a[4 * h + 3] = hi[1];
      }
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[j][2 * p + s]), acc[j], 0,
                                                           0, 0);
    }
  }
};

template <class Op>
struct StreamTraits {
  static constexpr bool kMx = Op::kXLane == 32;
};

// The rows a tile reads.
struct StreamArgs {
  const void* w0;        // first weight row of groups 0 .. NW0 - 1 (16 rows each)
  const void* w1;        // first weight row of groups NW0 .. NW - 1
  uint32_t w_bytes;      // bytes of the weight rows that exist at w0 and at w1
  uint32_t row_bytes;    // bytes of a weight row
  const void* x;         // base of the token rows
  uint32_t x_bytes;      // bytes that exist there (at most 2^31)
  uint32_t plane;        // bytes between the planes of a token row
  int steps;             // K / Op::kStep
  const uint8_t* scale;  // MXFP8: scale bytes of the 32-row group that holds weight row 0
  uint32_t scale_bytes;
  int scale_row;         // row of that group which is weight row 0 (0 or 16)
  uint32_t scale_pitch;  // bytes of a 32-row group (= K)
};

// The wave's share of the tile.  xoff[j]: byte offset of this lane's token
// row (row 16 j + lane % 16 of the tile) from a.x, or kNoRow.
template <class Op, int NW, int NW0, int NT, int U>
__device__ __forceinline__ void stream_tile(const StreamArgs& a, const uint32_t (&xoff)[NT], f32x4_t (&acc)[NW][NT]) {
  constexpr bool MX = StreamTraits<Op>::kMx;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  uint32_t woff[NW], xo[NT], so[NW];
#pragma unroll
  for (int g = 0; g < NW; ++g) {
    const int row = (g < NW0 ? g : g - NW0) * 16 + r;
    woff[g] = (uint32_t)row * a.row_bytes + 16u * q;
    if (MX) {
      const int sr = a.scale_row + row;
      so[g] = (uint32_t)(sr >> 5) * a.scale_pitch + 4u * (sr & 31);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    xo[j] = xoff[j] + (uint32_t)Op::kXLane * q;
#pragma unroll
    for (int g = 0; g < NW; ++g) acc[g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  struct Chunk {
    i32x4_t w[U][NW];
    i32x4_t x[U][NT][Op::kX];
    uint32_t s[MX ? U : 1][NW];
  };
  auto load = [&](Chunk& c, int chunk) {
    const int s0 = chunk * U;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // steps past the reduction read zeros: an empty range, at offset 0 (the
      // range check may subtract the scalar offset from the range)
      const bool live = s0 + u < a.steps;
      const uint32_t soff = live ? (uint32_t)(s0 + u) * 64u : 0u;
      const __amdgpu_buffer_rsrc_t r0 = make_rsrc(a.w0, live ? a.w_bytes : 0u);
      const __amdgpu_buffer_rsrc_t r1 = make_rsrc(a.w1, live ? a.w_bytes : 0u);
#pragma unroll
      for (int g = 0; g < NW; ++g) c.w[u][g] = buf_load16(g < NW0 ? r0 : r1, woff[g], soff);
      if constexpr (MX) {
        // 4 scale bytes of a row per 128 columns, i.e. per two steps
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.scale, live ? a.scale_bytes : 0u);
#pragma unroll
        for (int g = 0; g < NW; ++g)
          c.s[u][g] = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)so[g], live ? ((s0 + u) >> 1) * 128 : 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = s0 + u < a.steps;
      const uint32_t soff = live ? (uint32_t)(s0 + u) * (uint32_t)Op::kXBytes : 0u;
      const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, live ? a.x_bytes : 0u);
#pragma unroll
      for (int j = 0; j < NT; ++j) Op::load_x(c.x[u][j], rx, xo[j], soff, a.plane);
    }
  };
  auto compute = [&](const Chunk& c, int chunk) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < NW; ++g)
        Op::template mma<NT>(acc[g], c.w[u][g], MX ? c.s[u][g] : 0u, 2 * ((chunk * U + u) & 1) + (q >> 1), c.x[u]);
  };
  const int chunks = (a.steps + U - 1) / U;
  Chunk ca, cb;
  load(ca, wave);
  for (int c = wave; c < chunks; c += 2 * kStreamWaves) {
    load(cb, c + kStreamWaves);
    __builtin_amdgcn_sched_barrier(0);
    compute(ca, c);
    __builtin_amdgcn_sched_barrier(0);
    load(ca, c + 2 * kStreamWaves);
    __builtin_amdgcn_sched_barrier(0);
    compute(cb, c + kStreamWaves);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The waves' accumulators, added in wave order in LDS: stream_put (all
// threads, then a barrier), then stream_sum(t) for tile t = g * NT + j gives
// the lane weight rows 16 g + 4 (lane / 16) + 0..3 of token row 16 j + lane
// % 16.  lds: kStreamWaves * NW * NT KiB.
template <int NW, int NT>
__device__ __forceinline__ void stream_put(const f32x4_t (&acc)[NW][NT], f32x4_t* __restrict__ lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int g = 0; g < NW; ++g)
#pragma unroll
    for (int j = 0; j < NT; ++j) lds[((g * NT + j) * kStreamWaves + wave) * 64 + lane] = acc[g][j];
  __syncthreads();
}

__device__ __forceinline__ f32x4_t stream_sum(const f32x4_t* __restrict__ lds, int t) {
  const int lane = threadIdx.x & 63;
  f32x4_t s = lds[(t * kStreamWaves) * 64 + lane];
#pragma unroll
  for (int w = 1; w < kStreamWaves; ++w) s += lds[(t * kStreamWaves + w) * 64 + lane];
  return s;
}

}  // namespace moe
