// f32 tiles of the grouped GEMM's training products, on the f32 matrix
// instruction v_mfma_f32_32x32x2_f32 (each product and sum in f32).
//
// A tile is TX rows x TW columns of the output, computed by KG groups of 4
// waves (2 x 2, TX/2 x TW/2 each) that take a share of the K steps each: small
// problems have few tiles with long reductions, and 4 waves a SIMD hide each
// other's latency (layer 0's rows, 512 of 8 experts 256 x 512: 35 us with one
// group of 4 waves a tile, 21 with four).  The columns are the
// instruction's first operand, so a lane holds 4 consecutive columns of one
// row.  K is stepped by 32 through LDS, [k][T] per operand, double-buffered per
// group, the next step's loads in registers while the current one is
// multiplied.  An operand whose memory is contiguous along k is turned while it
// is stored to LDS; all others (weights in a rows' gradient, both operands of
// a weights' gradient) lie as LDS has them.
//
// A sum is held in two levels: the matrix cores' accumulators are added to the
// lane's own every 128 terms and start again, so the rounding error grows with
// sqrt(128) + sqrt(K / 128) instead of sqrt(K).
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "tiles.hpp"

namespace moe {

constexpr int kGfK = 32;
constexpr int kGfFlush = 4;  // K steps between two flushes of the accumulators

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

// One operand's part of a K step, T x 32 values: T / 32 groups of 4 a thread of the group's 256 (i: its number there).
template <int T>
struct GfPart {
  static constexpr int kPitch = T + 4;  // LDS floats per k: 16-byte aligned, 4 k apart on other banks
  f32x4_t v[T / 32];

  // k contiguous: row j of the thread at rows[j] (null: zeros), values k .. k + 31
  __device__ __forceinline__ void load_k(const float* const (&rows)[T / 32], int k, int i) {
#pragma unroll
    for (int j = 0; j < T / 32; ++j)
      v[j] = rows[j] ? *reinterpret_cast<const f32x4_t*>(rows[j] + k + 4 * (i & 7)) : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void store_k(float* lds, int i) const {
#pragma unroll
    for (int j = 0; j < T / 32; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) lds[(4 * (i & 7) + u) * kPitch + (i >> 3) + 32 * j] = v[j][u];
  }
  // columns contiguous: k rows at base + kk * pitch, kk < valid, columns col0 .. col0 + T (those from cols on: zeros)
  __device__ __forceinline__ void load_c(const float* base, int64_t pitch, int valid, int col0, int cols, int i) {
    constexpr int per = T / 4, step = 256 / per;
    const int c = col0 + 4 * (i % per);
#pragma unroll
    for (int j = 0; j < T / 32; ++j) {
      const int kk = i / per + step * j;
      v[j] = kk < valid && c < cols ? *reinterpret_cast<const f32x4_t*>(base + kk * pitch + c) : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }
  __device__ __forceinline__ void store_c(float* lds, int i) const {
    constexpr int per = T / 4, step = 256 / per;
#pragma unroll
    for (int j = 0; j < T / 32; ++j)
      *reinterpret_cast<f32x4_t*>(lds + (i / per + step * j) * kPitch + 4 * (i % per)) = v[j];
  }
};

// A tile's geometry and sums.  Fragment (i, j) of a wave: rows (wave / 2) TX/2 + 32 j + lane % 32, columns (wave % 2)
// TW/2 + 32 i + 8 q + 4 (lane / 32) + 0..3.
template <int TX, int TW, int KG>
struct GfTile {
  static constexpr int MI = TW / 64, NJ = TX / 64, kThreads = 256 * KG;
  static constexpr int kBuf = kGfK * (GfPart<TW>::kPitch + GfPart<TX>::kPitch);  // floats of one step's operands
  static constexpr int kLds = 2 * kBuf * KG;
  static_assert(MI * NJ * 4 * 4 * 64 * 4 <= 2 * kBuf, "a group's sums fit its buffers");

  f32x16_t acc[MI][NJ], sum[MI][NJ];

  __device__ __forceinline__ static void clear(f32x16_t (&a)[MI][NJ]) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) a[i][j][v] = 0.f;
  }
  __device__ __forceinline__ void step(const float* wl, const float* xl, int i) {
    const int lane = i & 63, wave = i >> 6;
    const float* wp = wl + (lane >> 5) * GfPart<TW>::kPitch + (lane & 31) + (wave & 1) * (TW / 2);
    const float* xp = xl + (lane >> 5) * GfPart<TX>::kPitch + (lane & 31) + (wave >> 1) * (TX / 2);
    // the fragments of k + 2 are read while k's are multiplied
    float fw[2][MI], fx[2][NJ];
    auto read = [&](int k) {
#pragma unroll
      for (int u = 0; u < MI; ++u) fw[k / 2 & 1][u] = wp[k * GfPart<TW>::kPitch + 32 * u];
#pragma unroll
      for (int u = 0; u < NJ; ++u) fx[k / 2 & 1][u] = xp[k * GfPart<TX>::kPitch + 32 * u];
    };
    read(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kGfK; k += 2) {
      if (k + 2 < kGfK) read(k + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < MI; ++u)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[u][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fw[k / 2 & 1][u], fx[k / 2 & 1][j], acc[u][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __device__ __forceinline__ void flush() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) sum[i][j] += acc[i][j];
    clear(acc);
  }

  // The K loop over this group's n steps (the groups' largest: most).  load(): the next step's parts; `lds` the
  // block's buffers.
  template <typename Load, typename StoreX, typename StoreW>
  __device__ __forceinline__ void run(float* lds, int n, int most, Load&& load, StoreX&& store_x, StoreW&& store_w) {
    const int i = threadIdx.x & 255;
    float* mine = lds + (threadIdx.x >> 8) * 2 * kBuf;
    constexpr int kX = kGfK * GfPart<TW>::kPitch;  // x behind w
    clear(acc);
    clear(sum);
    __syncthreads();  // the buffers are free
    if (n > 0) {
      load(0);
      store_w(mine);
      store_x(mine + kX);
    }
    __syncthreads();
    for (int s = 0; s < most; ++s) {
      if (s + 1 < n) load(s + 1);
      if (s < n) {
        step(mine + (s & 1) * kBuf, mine + (s & 1) * kBuf + kX, i);
        if (s % kGfFlush == kGfFlush - 1) flush();
      }
      if (s + 1 < n) {
        store_w(mine + ((s + 1) & 1) * kBuf);
        store_x(mine + ((s + 1) & 1) * kBuf + kX);
      }
      __syncthreads();
    }
    flush();
    if constexpr (KG > 1) {
      // every group's sums into its buffers, fragment by fragment as the lanes hold them
#pragma unroll
      for (int u = 0; u < MI; ++u)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) *reinterpret_cast<f32x4_t*>(mine + at(i, u, j, q)) = quad(sum[u][j], q);
      __syncthreads();
    }
  }
  __device__ __forceinline__ static f32x4_t quad(const f32x16_t& v, int q) {
    return f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  }
  __device__ __forceinline__ static int at(int i, int u, int j, int q) {
    return ((((i >> 6) * MI * NJ + u * NJ + j) * 4 + q) * 64 + (i & 63)) * 4;
  }
  // f(u, j, q, values of column fragments u = 0 .. MI - 1) for the quads that this group finishes: its share of the 4
  template <typename F>
  __device__ __forceinline__ void each(const float* lds, F&& f) {
    const int i = threadIdx.x & 255, g = threadIdx.x >> 8;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int qq = 0; qq < 4 / KG; ++qq) {
        const int q = g * (4 / KG) + qq;
        f32x4_t v[MI];
#pragma unroll
        for (int u = 0; u < MI; ++u) {
          if constexpr (KG > 1) {
            v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < KG; ++h) v[u] += *reinterpret_cast<const f32x4_t*>(lds + h * 2 * kBuf + at(i, u, j, q));
          } else {
            v[u] = quad(sum[u][j], qq);
          }
        }
        f(j, q, v);
      }
  }
  // the thread's row of fragment j and first of 4 columns of fragment u, quad q
  __device__ __forceinline__ static int row(int j) {
    const int i = threadIdx.x & 255;
    return (i >> 7) * (TX / 2) + 32 * j + (i & 31);
  }
  __device__ __forceinline__ static int col(int u, int q) {
    const int i = threadIdx.x & 255;
    return ((i >> 6) & 1) * (TW / 2) + 32 * u + 8 * q + 4 * ((i & 63) >> 5);
  }
};

}  // namespace moe
