// Weight-streaming product tile for few token rows (gfx950): the decode
// layer's two products and the adapter projection's short batches.
//
//   acc[i][j] = sum_k W[i, k] X[j, k]    i: 16 NW weight rows, j: 16 NT token rows
//
// With few token rows every weight is used once per call, so what counts is
// that the loads never pause.  The block's waves split the reduction: a line
// is 128 bytes of every row, wave w takes lines w, w + waves, ...; the partial
// accumulators are added in LDS in wave order at the end (a fixed order: the
// bits do not depend on timing).  A wave loads a line of 8 rows with one
// instruction, 8 lanes of 16 bytes beside each other in a row, keeps one to
// four lines in flight in registers, and turns each to the matrix cores' layout
// (lane = row, then 16-byte chunk) through a place in LDS of its own, without
// a barrier.
//   Loading straight in the matrix cores' layout, where neighbouring lanes
// are different rows, needs no LDS but gives 38 bytes per ns and CU from the
// L2; 8 lanes to a row give 124 (measured; HBM gives 27).  With weights and
// token rows on that path, 200 rows x 4096 x 4096 took 33 us.
// Weight rows that do not exist read the last one that does (their sums are not
// used).
#pragma once

#include "common.hpp"
#include "gemm_bf16.hpp"

namespace moe {

constexpr uint32_t kNoRow = 0x80000000u;  // offset past every buffer range

// A weight load: NT marks it as used once, so that it does not push the token
// rows out of the caches (2 experts of 4096 x 14336, one token: 78 + 43 us
// instead of 84 + 46; not for weights that the caches may keep between calls).
template <bool NT>
__device__ __forceinline__ i32x4_t load_weight(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, NT ? 2 : 0));
}

// f32 value as NP bf16 values whose sum is the value (NP = 3: exactly, but
// for magnitudes below 2^-110; NP = 2: to 2^-16 of it).  An infinity or NaN is
// its first plane alone; a finite value that would round to infinity is cut
// off instead of rounded there.  (No contraction: where v is a product, the
// compiler made v - f an fma of the unrounded one in some copies of the code and
// not in others, so that a row's bits depended on its place in a tile.)
template <int NP>
__device__ __forceinline__ void split_bf16(float v, __bf16 (&p)[NP]) {
#pragma clang fp contract(off)
  p[0] = (__bf16)v;
  float f = (float)p[0];
  if (__builtin_isinf(f)) {
    f = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u);
    p[0] = (__bf16)f;
  }
  float rest = __builtin_isfinite(f) ? v - f : 0.0f;
#pragma unroll
  for (int i = 1; i < NP; ++i) {
    p[i] = (__bf16)rest;
    rest -= (float)p[i];
  }
}

// ---- operand kinds.  A line of a weight row is kW = 8 chunks of 16 bytes;
// kLine elements.  A line of a token row is kXC chunks per plane, kP planes.
// mma: half h (0, 1) of a line; w: the lane's chunk 4 h + q (q = lane / 16)
// of its weight row; x(c): chunk c of plane p of its token row.

// bf16 weights, token rows in NP bf16 planes (their sum is the row's value).
template <int NP>
struct StreamBf16 {
  static constexpr int kLine = 64, kP = NP, kXC = 8;
  static constexpr bool kMx = false;
  // element k of a weight row
  static __device__ __forceinline__ float weight(const char* row, const uint8_t*, int k) {
    return (float)reinterpret_cast<const __bf16*>(row)[k];
  }
  // x chunks that go with half h: one per plane
  static constexpr int kXH = 1;
  static __device__ __forceinline__ int x_chunk(int h, int q, int) { return 4 * h + q; }
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, float, const i32x4_t (&x)[NT][NP]) {
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
  static constexpr int kLine = 32, kP = 1, kXC = 8;
  static constexpr bool kMx = false;
  static constexpr int kXH = 1;
  static __device__ __forceinline__ int x_chunk(int h, int q, int) { return 4 * h + q; }
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, float, const i32x4_t (&x)[NT][1]) {
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
// value (3 bits of mantissa), so nothing is rounded.
template <int NP>
struct StreamMx {
  static constexpr int kLine = 128, kP = NP, kXC = 16;
  static constexpr bool kMx = true;
  // scale: the row's bytes of the first line (those of the next: 128 bytes on)
  static __device__ __forceinline__ float weight(const char* row, const uint8_t* scale, int k) {
    const int s = scale[k / 128 * 128 + k / 32 % 4];
    const float v = __builtin_amdgcn_cvt_f32_fp8((uint8_t)row[k], 0);
    return s == 255 ? __builtin_nanf("") : ldexpf(v, s - 127);
  }
  static constexpr int kXH = 2;
  static __device__ __forceinline__ int x_chunk(int h, int q, int s) { return 2 * (4 * h + q) + s; }
  template <int NT>
  static __device__ __forceinline__ void mma(f32x4_t (&acc)[NT], const i32x4_t& w, float scale,
                                             const i32x4_t (&x)[NT][2 * NP]) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t a;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = (uint32_t)w[2 * s + h];
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, false);
        const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, true);
        a[4 * h] = lo[0];
        a[4 * h + 1] = lo[1];
        a[4 * h + 2] = hi[0];
        a[4 * h + 3] = hi[1];
      }
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[j][p * 2 + s]), acc[j], 0,
                                                           0, 0);
    }
  }
};

// The rows a tile reads.
struct StreamArgs {
  const void* w0;        // first weight row (of kPaired: of the even groups of 16)
  const void* w1;        // first weight row of the other groups (kPaired, kFirst)
  int w_rows;            // weight rows that exist there (>= 1)
  int w1_rows;           // kFirst: ... at w1
  uint32_t row_bytes;    // bytes of a weight row
  const void* x;         // base of the token rows
  uint32_t x_bytes;      // bytes that exist there (below 2^31)
  uint32_t plane;        // bytes between the planes of a token row
  int lines;             // K / Op::kLine
  int line0;             // first line of the tile (stream_wide), usually 0
  const uint8_t* scale;  // MXFP8: scale bytes of the 32-row group that holds weight row 0
  int scale_row;         // row of that group which is weight row 0 (0 or 16)
  uint32_t scale_pitch;  // bytes of a 32-row group (= K)
};

// Bytes of LDS of one wave: a line of the weight rows and of the token rows.
// XG: token rows of a group that are loaded, 16, or 8 where there are no more.
template <class Op, int NW, int NT, int XG = 16>
constexpr int stream_line_bytes() {
  return 16 * NW * 128 + XG * NT * Op::kP * Op::kXC * 16;
}

// The rows of weight group g: kOne, rows 16 g .. of w0; kPaired, rows 16 (g / 2)
// .. of w0 (g even) or w1 (g odd); kFirst, rows 0 .. of w0 (g = 0) or 16 (g - 1)
// .. of w1.
constexpr int kOne = 0, kPaired = 1, kFirst = 2;

// One wave's share of the tile: lines first, first + stride, ....  row_off(i): byte offset from a.x of token row i (0 <= i <
// 16 NT), any row for one that does not exist.  lds: stream_line_bytes() of
// the wave's own.  DEPTH: lines in flight, fewer where about 96 registers hold
// fewer (stream_depth; a line of 64 weight and 64 token rows takes 64: one is in
// flight): 4 where the weights come from HBM for long (decode, 2 experts of
// 4096 x 14336: 81 us for Layer0 instead of 84), 2 for short streams, where
// filling and draining the pipe costs more (333 x 2048 x 1408: 13 us, 17).
// ONCE: the weights are not used again soon (load_weight).
template <class Op, int NW, int NT, int DEPTH, int XG>
constexpr int stream_depth() {
  constexpr int regs = 4 * (2 * NW + Op::kP * (Op::kXC / 4) * NT * XG / 16), d = 96 / regs;
  return d > DEPTH ? DEPTH : d < 1 ? 1 : d;
}

template <class Op, int NW, int GROUPS, int NT, int DEPTH, int XG, bool ONCE, class RowOff>
__device__ __forceinline__ void stream_share(const StreamArgs& a, int first, int stride, RowOff row_off,
                                             char* __restrict__ lds, f32x4_t (&acc)[NW][NT]) {
  constexpr bool MX = Op::kMx;
  constexpr int XC = Op::kXC, XR = 64 / XC;            // chunks of a token row; token rows per load
  constexpr int XL = XG / XR;                          // loads per group of token rows and plane
  constexpr int XPITCH = XC * 16;
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4, rx16 = r % XG;
  // Chunk c of row i sits at place c ^ swz(i): 16 rows read at one chunk, and
  // 8 (or 4) whole rows written, hit every bank once.
  auto swz_w = [](int i) { return (i >> 1) & 7; };
  auto swz_x = [](int i) { return XC == 8 ? (i >> 1) & 7 : i & 15; };
  uint32_t woff[2 * NW], xo[XL * NT];
#pragma unroll
  for (int l = 0; l < 2 * NW; ++l) {
    const int i = 8 * (l & 1) + (lane >> 3), g = l >> 1;
    const int grp = GROUPS == kPaired ? g >> 1 : GROUPS == kFirst && g > 0 ? g - 1 : g;
    const int last = (GROUPS == kFirst && g > 0 ? a.w1_rows : a.w_rows) - 1;
    woff[l] = (uint32_t)min(16 * grp + i, last) * a.row_bytes + 16u * ((lane & 7) ^ swz_w(i));
  }
#pragma unroll
  for (int l = 0; l < XL * NT; ++l) {
    const int i = XR * (l % XL) + lane / XC;
    xo[l] = row_off(XG * (l / XL) + i) + 16u * ((lane % XC) ^ swz_x(i));
  }
  uint32_t so[NW];
#pragma unroll
  for (int g = 0; g < NW; ++g) {
    if (MX) {
      const int sr = a.scale_row + min(16 * g + r, a.w_rows - 1);
      so[g] = (uint32_t)(sr >> 5) * a.scale_pitch + 4u * (sr & 31);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  const uint32_t w_bytes = (uint32_t)a.w_rows * a.row_bytes;
  struct Line {
    i32x4_t w[2 * NW];
    i32x4_t x[Op::kP][XL * NT];
    uint32_t s[MX ? NW : 1];
  };
  auto load = [&](Line& c, int line) {
    // past the last line: nothing is read (an empty range, at offset 0: the
    // range check may take the scalar offset from the range)
    const bool live = line < a.lines;
    const uint32_t at = live ? (uint32_t)line : 0u;
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(a.w0, live ? w_bytes : 0u);
    const __amdgpu_buffer_rsrc_t r1 =
        make_rsrc(GROUPS == kOne ? a.w0 : a.w1, live ? GROUPS == kFirst ? (uint32_t)a.w1_rows * a.row_bytes : w_bytes : 0u);
    auto second = [](int l) { return GROUPS == kPaired ? (l & 2) != 0 : GROUPS == kFirst && l >= 2; };
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, live ? a.x_bytes : 0u);
#pragma unroll
    for (int l = 0; l < 2 * NW; ++l) c.w[l] = load_weight<ONCE>(second(l) ? r1 : r0, woff[l], at * 128u);
    if constexpr (MX) {
#pragma unroll
      for (int g = 0; g < NW; ++g)
        c.s[g] = *reinterpret_cast<const uint32_t*>(a.scale + so[g] + at * 128u);  // the row's 4 blocks of the line
    }
#pragma unroll
    for (int p = 0; p < Op::kP; ++p)
#pragma unroll
      for (int l = 0; l < XL * NT; ++l) c.x[p][l] = buf_load16(rx, xo[l] + (uint32_t)p * a.plane, at * (uint32_t)XPITCH);
  };
  char* const ldx = lds + NW * 2048;
  constexpr int D = stream_depth<Op, NW, NT, DEPTH, XG>();
  Line ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(ring[d], first + d * stride);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int c = first; c < a.lines; c += D * stride) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Line& n = ring[d];
#pragma unroll
      for (int l = 0; l < 2 * NW; ++l) *reinterpret_cast<i32x4_t*>(lds + l * 1024 + lane * 16) = n.w[l];
#pragma unroll
      for (int p = 0; p < Op::kP; ++p)
#pragma unroll
        for (int l = 0; l < XL * NT; ++l)
          *reinterpret_cast<i32x4_t*>(ldx + (p * XL * NT + l) * 1024 + lane * 16) = n.x[p][l];
      uint32_t scales[MX ? NW : 1];
      if constexpr (MX) {
#pragma unroll
        for (int g = 0; g < NW; ++g) scales[g] = n.s[g];
      }
      __builtin_amdgcn_sched_barrier(0);
      load(n, c + (d + D) * stride);
      __builtin_amdgcn_sched_barrier(0);
      // (a line past the last one is zeros: it adds nothing)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4_t x[NT][Op::kXH * Op::kP];
#pragma unroll
        for (int p = 0; p < Op::kP; ++p)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int t = 0; t < Op::kXH; ++t)
              x[j][p * Op::kXH + t] = *reinterpret_cast<const i32x4_t*>(
                  ldx + ((p * NT + j) * XG + rx16) * XPITCH + ((Op::x_chunk(h, q, t) ^ swz_x(rx16)) << 4));
#pragma unroll
        for (int g = 0; g < NW; ++g) {
          const i32x4_t w =
              *reinterpret_cast<const i32x4_t*>(lds + (16 * g + r) * 128 + (((4 * h + q) ^ swz_w(r)) << 4));
          // MXFP8: the scale byte of the lane's block of 32, as a power of two
          const float sc =
              MX ? __builtin_bit_cast(float, ((scales[MX ? g : 0] >> (8 * (2 * h + (q >> 1)))) & 0xFFu) << 23) : 0.f;
          Op::template mma<NT>(acc[g], w, sc, x);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The whole tile by the WAVES waves of a block.
template <class Op, int WAVES, int NW, int GROUPS, int NT, int DEPTH, bool ONCE, class RowOff>
__device__ __forceinline__ void stream_tile(const StreamArgs& a, RowOff row_off, char* __restrict__ lds,
                                            f32x4_t (&acc)[NW][NT]) {
  stream_share<Op, NW, GROUPS, NT, DEPTH, 16, ONCE>(a, uniform(threadIdx.x >> 6), WAVES, row_off, lds, acc);
}

constexpr int imax(int a, int b) { return a > b ? a : b; }

// The same product with the weight rows, not the reduction, split over the
// block's WAVES waves (16 NW rows each: group g of wave w is weight group w NW
// + g), which share the lines of the token rows: every wave loads its part of
// a line, and one barrier per line, over two places for it, hands them round.
// For many or wide (several planes) token rows, whose lines would otherwise be
// as much traffic as the weights'.  lds: stream_wide_bytes().  The sums are
// complete: acc as in stream_share.
template <class Op, int WAVES, int NW, int NT>
constexpr int stream_wide_bytes() {
  return WAVES * NW * 2048 + 2 * 16 * NT * Op::kP * Op::kXC * 16;
}

template <class Op, int WAVES, int NW, int GROUPS, int NT, int DEPTH, bool ONCE, class RowOff>
__device__ __forceinline__ void stream_wide(const StreamArgs& a, RowOff row_off, char* __restrict__ lds,
                                            f32x4_t (&acc)[NW][NT]) {
  constexpr bool MX = Op::kMx;
  constexpr int XC = Op::kXC, XR = 64 / XC, XL = 16 / XR, XPITCH = XC * 16;
  constexpr int kLoads = XL * NT * Op::kP, XW = (kLoads + WAVES - 1) / WAVES;  // a line's token loads; of one wave
  constexpr int kX = 16 * NT * Op::kP * XPITCH;                              // bytes of a token line
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  auto swz_w = [](int i) { return (i >> 1) & 7; };
  auto swz_x = [](int i) { return XC == 8 ? (i >> 1) & 7 : i & 15; };
  uint32_t woff[2 * NW], xo[XW], so[NW];
#pragma unroll
  for (int l = 0; l < 2 * NW; ++l) {
    const int i = 8 * (l & 1) + (lane >> 3), grp = wave * NW + (l >> 1);
    woff[l] = (uint32_t)min(16 * (GROUPS == kPaired ? grp >> 1 : grp) + i, a.w_rows - 1) * a.row_bytes +
              16u * ((lane & 7) ^ swz_w(i));
  }
  // token load l of a line: plane l / (XL NT), rows XR (l % (XL NT)) ..
#pragma unroll
  for (int v = 0; v < XW; ++v) {
    const int l = min(wave + v * WAVES, kLoads - 1), p = l / (XL * NT), i = XR * (l % (XL * NT)) + lane / XC;
    xo[v] = row_off(i) + (uint32_t)p * a.plane + 16u * ((lane % XC) ^ swz_x(i & 15));
  }
#pragma unroll
  for (int g = 0; g < NW; ++g) {
    if (MX) {
      const int sr = a.scale_row + min(16 * (wave * NW + g) + r, a.w_rows - 1);
      so[g] = (uint32_t)(sr >> 5) * a.scale_pitch + 4u * (sr & 31);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  const uint32_t w_bytes = (uint32_t)a.w_rows * a.row_bytes;
  struct Line {
    i32x4_t w[2 * NW];
    i32x4_t x[XW];
    uint32_t s[MX ? NW : 1];
  };
  static_assert(GROUPS == kOne || (GROUPS == kPaired && NW % 2 == 0), "a wave's pairs are its own");
  auto load = [&](Line& c, int line) {
    const bool live = line < a.lines;  // else nothing is read (see stream_share)
    const uint32_t at = live ? (uint32_t)(a.line0 + line) : 0u;
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(a.w0, live ? w_bytes : 0u);
    const __amdgpu_buffer_rsrc_t r1 = make_rsrc(GROUPS == kPaired ? a.w1 : a.w0, live ? w_bytes : 0u);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, live ? a.x_bytes : 0u);
#pragma unroll
    for (int l = 0; l < 2 * NW; ++l) c.w[l] = load_weight<ONCE>(GROUPS == kPaired && (l & 2) ? r1 : r0, woff[l], at * 128u);
    if constexpr (MX) {
#pragma unroll
      for (int g = 0; g < NW; ++g) c.s[g] = *reinterpret_cast<const uint32_t*>(a.scale + so[g] + at * 128u);
    }
#pragma unroll
    for (int v = 0; v < XW; ++v) c.x[v] = buf_load16(rx, xo[v], at * (uint32_t)XPITCH);
  };
  char* const ldw = lds + wave * NW * 2048;
  char* const ldx = lds + WAVES * NW * 2048;
  constexpr int D = DEPTH;
  Line ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(ring[d], d);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int c = 0; c < a.lines; c += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      Line& n = ring[d];
      char* const xb = ldx + ((D % 2 == 0 ? d : c + d) & 1) * kX;
#pragma unroll
      for (int l = 0; l < 2 * NW; ++l) *reinterpret_cast<i32x4_t*>(ldw + l * 1024 + lane * 16) = n.w[l];
#pragma unroll
      for (int v = 0; v < XW; ++v)
        if (kLoads % WAVES == 0 || wave + v * WAVES < kLoads)
          *reinterpret_cast<i32x4_t*>(xb + (wave + v * WAVES) * 1024 + lane * 16) = n.x[v];
      uint32_t scales[MX ? NW : 1];
      if constexpr (MX) {
#pragma unroll
        for (int g = 0; g < NW; ++g) scales[g] = n.s[g];
      }
      __builtin_amdgcn_sched_barrier(0);
      load(n, c + d + D);
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4_t w[NW];
#pragma unroll
        for (int g = 0; g < NW; ++g)
          w[g] = *reinterpret_cast<const i32x4_t*>(ldw + (16 * g + r) * 128 + (((4 * h + q) ^ swz_w(r)) << 4));
        // up to 4 groups of 16 token rows at a time, so that their fragments fit
        constexpr int NS = NT == 6 ? 3 : NT > 4 ? 4 : NT;
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += NS) {
          i32x4_t x[NS][Op::kXH * Op::kP];
#pragma unroll
          for (int p = 0; p < Op::kP; ++p)
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
              for (int t = 0; t < Op::kXH; ++t)
                x[j][p * Op::kXH + t] = *reinterpret_cast<const i32x4_t*>(
                    xb + ((p * NT + j0 + j) * 16 + r) * XPITCH + ((Op::x_chunk(h, q, t) ^ swz_x(r)) << 4));
#pragma unroll
          for (int g = 0; g < NW; ++g) {
            const float sc =
                MX ? __builtin_bit_cast(float, ((scales[MX ? g : 0] >> (8 * (2 * h + (q >> 1)))) & 0xFFu) << 23) : 0.f;
            Op::template mma<NS>(*reinterpret_cast<f32x4_t(*)[NS]>(&acc[g][j0]), w[g], sc, x);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The planes of a token value are multiplied one by one, and where a weight is
// infinite, or a product past the range, they give NaN (inf * 0, inf - inf)
// for what is an infinity: a plane may be zero or of the other sign.  No sum
// that is not NaN is wrong in this way (its infinities have one sign, that of
// the first planes').  So a NaN is summed again from the whole values, in f32,
// by the wave, until each is known to be one (a NaN among the values or
// weights ends it at once).
//   v: the lane's sums of weight rows row .. row + 3 of a.w0 (kOne) and the
// token row at byte x_off; live: they are used.  The whole wave calls it, for
// the tile's lines line0 .. line0 + lines - 1.
template <class Op>
__device__ __forceinline__ void stream_resum(const StreamArgs& a, int row, uint32_t x_off, bool live, f32x4_t& v) {
  if constexpr (Op::kP > 1) {
    int nan = 0;  // bit c: v[c]
#pragma unroll
    for (int c = 0; c < 4; ++c) nan |= __builtin_isnan(v[c]) ? 1 << c : 0;
    const int lane = threadIdx.x & 63;
    const int k0 = a.line0 * Op::kLine, k1 = k0 + a.lines * Op::kLine;
#pragma unroll 1
    for (uint64_t left = __ballot(live && nan); left; left &= left - 1) {
      const int src = __ffsll((unsigned long long)left) - 1, r0 = __builtin_amdgcn_readlane(row, src);
      const char* x = reinterpret_cast<const char*>(a.x) + (uint32_t)__builtin_amdgcn_readlane((int)x_off, src);
      const char* w = reinterpret_cast<const char*>(a.w0) + (int64_t)r0 * a.row_bytes;
      const int sr = a.scale_row + r0;
      const uint8_t* scale = Op::kMx ? a.scale + (int64_t)(sr >> 5) * a.scale_pitch + 4 * (sr & 31) : nullptr;
      f32x4_t s = {0.f, 0.f, 0.f, 0.f};
      int open = __builtin_amdgcn_readlane(nan, src);  // the sums that may yet be infinite
#pragma unroll 1
      for (int k = k0 + lane; k < k1 && open; k += 64) {  // (lines are whole 64s: the waves' lanes stay together)
        float h = 0.0f;
#pragma unroll
        for (int p = Op::kP - 1; p >= 0; --p) h += (float)reinterpret_cast<const __bf16*>(x + p * (int64_t)a.plane)[k];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[c] = fmaf(Op::weight(w + c * (int64_t)a.row_bytes, scale + 4 * c, k), h, s[c]);
          if (__any(__builtin_isnan(s[c]))) open &= ~(1 << c);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        for (int off = 1; off < 64; off <<= 1) s[c] += __shfl_xor(s[c], off);
        if (lane == src && (open >> c & 1)) v[c] = s[c];
      }
    }
  }
}

// Adds the WAVES partial accumulators in wave order through LDS, G groups of
// 16 weight rows at a time (lds: WAVES * G * NT KiB), and hands the sums out:
// visit(g, j, s) with s[0 .. V - 1] the sums of groups g .. g + V - 1 (V = 2:
// a gate group and its up group; lds may hold the waves' lines: a barrier
// comes first), lane: weight rows 4 (lane / 16) + 0..3 of
// the group, token row 16 j + lane % 16.  All threads of the block call it.
template <int WAVES, int NW, int NT, int G, int V, class F>
__device__ __forceinline__ void stream_reduce(const f32x4_t (&acc)[NW][NT], f32x4_t* __restrict__ lds, F visit) {
  static_assert(NW % G == 0 && G % V == 0, "whole rounds");
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
#pragma unroll
  for (int g0 = 0; g0 < NW; g0 += G) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < NT; ++j) lds[((g * NT + j) * WAVES + wave) * 64 + lane] = acc[g0 + g][j];
    __syncthreads();
    for (int t = wave; t < G / V * NT; t += WAVES) {
      const int g = t / NT * V, j = t % NT;
      f32x4_t s[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const f32x4_t* at = lds + ((g + v) * NT + j) * WAVES * 64 + lane;
        s[v] = at[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s[v] += at[w * 64];
      }
      visit(g0 + g, j, s);
    }
  }
}

}  // namespace moe
