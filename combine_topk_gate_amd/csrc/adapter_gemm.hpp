// Matrix-core tile of the adapter projection for long batches (gfx950, bf16):
//   out[m, n] = cast(x[m] . W[n] + t[m] . B[a_m, n] + residual[m, n])
//
// A tile is 256 columns (W rows, the MFMA "A" operand) x TM rows of x (256, or
// 128 where 256-row tiles would leave CUs idle), K stepped by 64, 4 waves of
// 128 x TM/2 in 32x32x16 MFMAs, operands HBM -> VGPR -> LDS double-buffered:
// the schedule of the grouped GEMM's tile (gemm_bf16.hpp), whose measurements
// hold here too.  What is different is that the reduction does not end with
// H: the adapters that rows of the tile use follow as further K steps of the
// same pipeline: for each of the tile's distinct adapters its planes times
// its rank (t in bf16 planes whose sum is the f32 value, one after the other;
// B repeated beside them), in whole steps; a token row of another adapter
// holds zeros.  Only the buffers and offsets that a step's loads go to
// change, so the loop is one and the same.
// Zeros only cancel finite values, so an element of B that is infinite or NaN
// is left out of the product (staged as zero) and added in the epilogue, to
// the rows of its adapter alone; rows where that, or t's planes, may have made a
// NaN of an infinity are formed again there (mend_sum).
#pragma once

#include "gemm_bf16.hpp"
#include "launch.hpp"
#include "stream.hpp"

namespace moe {

// 4 values at any element's address (rows need not be whole 8-byte units): one
// access still, where each element by itself took 205 us instead of 107 for
// 7060 x 384 x 5789 with a residual.
typedef bf16x4_t bf16x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

__device__ __forceinline__ bf16x4_t load_any(const __bf16* p) { return *reinterpret_cast<const bf16x4_any_t*>(p); }
__device__ __forceinline__ void store_any(const AdapterArgs& a, int64_t i, f32x4_t v) {
  if (a.out.out_bf16) {
    const bf16x4_t o = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    *reinterpret_cast<bf16x4_any_t*>(reinterpret_cast<__bf16*>(a.out.out) + i) = o;
  } else {
    *reinterpret_cast<f32x4_any_t*>(reinterpret_cast<float*>(a.out.out) + i) = v;
  }
}

// Element i of the output: residual, cast.
__device__ __forceinline__ void store_one(const AdapterArgs& a, int64_t i, float v) {
  if (a.out.residual)
    v += a.out.res_bf16 ? (float)reinterpret_cast<const __bf16*>(a.out.residual)[i]
                        : reinterpret_cast<const float*>(a.out.residual)[i];
  if (a.out.out_bf16)
    reinterpret_cast<__bf16*>(a.out.out)[i] = (__bf16)v;
  else
    reinterpret_cast<float*>(a.out.out)[i] = v;
}

// Stores 4 columns (those below N) of row m: residual, cast.
__device__ __forceinline__ void adapter_store(const AdapterArgs& a, int64_t m, int n, f32x4_t acc) {
  const int64_t i = m * a.N + n;
  if (n + 4 <= a.N) {
    if (a.out.residual) {
      if (a.out.res_bf16) {
        const bf16x4_t r = load_any(reinterpret_cast<const __bf16*>(a.out.residual) + i);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] += (float)r[c];
      } else {
        acc += *reinterpret_cast<const f32x4_any_t*>(reinterpret_cast<const float*>(a.out.residual) + i);
      }
    }
    store_any(a, i, acc);
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (n + c >= a.N) break;
    store_one(a, i + c, acc[c]);
  }
}

// Grid of a kernel whose blocks take `tiles` tiles by xcd_tile: a multiple of 8
// wide, and high where the work items of one dimension would pass 32 bits.
inline dim3 tile_grid(int64_t tiles) {
  constexpr int64_t kWide = 1 << 20;
  const int64_t n = (tiles + 7) / 8 * 8;
  return n <= kWide ? dim3((unsigned)n) : dim3((unsigned)kWide, (unsigned)((n + kWide - 1) / kWide));
}

// This block's tile, -1 for none: the workgroups go to the 8 XCDs in turn, and
// each XCD's take a contiguous run of tiles, so that neighbouring tiles share
// operands in its L2.
__device__ __forceinline__ int64_t xcd_tile(int64_t tiles) {
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, per = (tiles + 7) / 8;
  const int64_t v = (b & 7) * per + (b >> 3);
  return (b >> 3) < per && v < tiles ? v : -1;
}

struct AdapterTileLds {
  int id[256];    // adapter of each row, -1: none
  int list[256];  // the tile's distinct adapters
  int wsum[4];
  int n;          // how many
  int nonfinite;  // an element of B was left out
};

// Fills id, list and n for rows m0 .. m0 + rows - 1 of a tile of TM (TM <=
// threads).  All threads call it; barriers inside.
template <int TM>
__device__ __forceinline__ void list_adapters(const AdapterArgs& p, int64_t m0, int rows, AdapterTileLds& t) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int id = -1;
  if (tid < rows) id = p.idx[m0 + tid];
  if ((uint32_t)id >= (uint32_t)p.P) id = -1;
  if (tid < TM) t.id[tid] = id;
  if (tid == 0) t.nonfinite = 0;
  __syncthreads();
  // appends the threads' values with `keep` to t.list, in thread order
  auto compact = [&](bool keep, int value) {
    const uint64_t m = __ballot(keep);
    if (lane == 0) t.wsum[wave] = __popcll(m);
    __syncthreads();
    int at = __popcll(m & lanemask_lt()), n = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += t.wsum[w];
      n += t.wsum[w];
    }
    if (keep) t.list[at] = value;
    __syncthreads();
    return n;
  };
  // the rows where a run of one adapter begins, then the first run of each
  const int runs = compact(tid < TM && id >= 0 && (tid == 0 || t.id[tid - 1] != id), id);
  const int run = tid < runs ? t.list[tid] : -1;
  bool first = tid < runs;
  for (int j = 0; j < runs - 1; ++j)
    if (j < tid && t.list[j] == run) first = false;
  __syncthreads();
  const int n = compact(first, run);
  if (tid == 0) t.n = n;
  __syncthreads();
}

// Non-finite elements among 32 bits of B (f32, or two bf16), as a mask of
// their bits.
template <class T>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t d) {
  if (sizeof(T) == 4) return (d & 0x7F800000u) == 0x7F800000u ? ~0u : 0u;
  return ((d & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((d & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// Sets the non-finite elements of 16 bytes of B to zero; whether there were any.
template <class T>
__device__ __forceinline__ bool drop_nonfinite(i32x4_t& v) {
  uint32_t bad[4], any = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) any |= bad[e] = nonfinite_bits<T>((uint32_t)v[e]);
  if (any) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (int)((uint32_t)v[e] & ~bad[e]);
  }
  return any != 0;
}

// Value j of t[m] (p.planes parts).
template <class T>
__device__ __forceinline__ float t_value(const AdapterArgs& p, int64_t m, int j) {
  const T* t = reinterpret_cast<const T*>(p.t) + m * p.planes * p.r + j;
  float v = 0.0f;
  for (int q = p.planes - 1; q >= 0; --q) v += (float)t[q * p.r];
  return v;
}

// What the elements of B that a tile left out add to out[m, n].
template <class T>
__device__ __forceinline__ float nonfinite_part(const AdapterArgs& p, int64_t m, int id, int n) {
  const T* b = reinterpret_cast<const T*>(p.b) + ((int64_t)id * p.N + n) * p.r;
  float s = 0.0f;
  for (int j = 0; j < p.r; ++j) {
    const float v = (float)b[j];
    if (__builtin_isfinite(v)) continue;
    s += t_value<T>(p, m, j) * v;
  }
  return s;
}

// A tile's sum v for out[m, n] (before the residual) of a row with adapter id,
// with what the tile left out of it.  A NaN may stand for an infinity: an
// infinite t times the zero of an element left out, or products of t's planes
// past the range with opposite signs.  Then t . B is formed again from whole
// values, and, if that is infinite, x . W as well.
template <class T>
__device__ __forceinline__ float mend_sum(const AdapterArgs& p, int64_t m, int id, int n, bool left_out, float v) {
  if (left_out) v += nonfinite_part<T>(p, m, id, n);
  if (!__builtin_isnan(v)) return v;
  const T* b = reinterpret_cast<const T*>(p.b) + ((int64_t)id * p.N + n) * p.r;
  float tb = 0.0f;
#pragma unroll 1
  for (int j = 0; j < p.r; ++j) tb = fmaf(t_value<T>(p, m, j), (float)b[j], tb);
  if (!__builtin_isinf(tb)) return v;
  const T* x = reinterpret_cast<const T*>(p.x) + m * p.H;
  const T* w = reinterpret_cast<const T*>(p.w) + (int64_t)n * p.H;
  float xw = 0.0f;
#pragma unroll 1
  for (int h = 0; h < p.H; ++h) xw = fmaf((float)x[h], (float)w[h], xw);
  return xw + tb;
}

// The same for 4 columns n .. n + 3 (those below N).
template <class T>
__device__ __forceinline__ void mend_sums(const AdapterArgs& p, int64_t m, int id, int n, bool left_out, f32x4_t& v) {
  const bool nan = __builtin_isnan(v[0]) | __builtin_isnan(v[1]) | __builtin_isnan(v[2]) | __builtin_isnan(v[3]);
  if ((!left_out && !nan) || (uint32_t)id >= (uint32_t)p.P) return;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (n + c < p.N) v[c] = mend_sum<T>(p, m, id, n + c, left_out, v[c]);
}

template <int TM>
__device__ __forceinline__ void adapter_gemm_tile(const AdapterArgs& p, int64_t m0, int n0, char* __restrict__ lds,
                                                  AdapterTileLds& tl) {
  constexpr int NJ = TM / 64;  // token fragments per wave
  constexpr int XI = TM / 32;  // token-row loads per thread per K step
  constexpr int XQ = XI / 4;   // ... per sub-step
  constexpr int NR = 4 + NJ, NW = 2 + XQ, NM = 4 * NJ;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wm = wave >> 1;
  const uint32_t row_bytes = p.row_bytes;
  const int rows = (int)min((int64_t)TM, p.M - m0), cols = min(p.N - n0, 256);

  // thread: 16-byte chunk lc of rows lr + 32 i of both operands
  const int lc = tid & 7, lr = tid >> 3;
  // where the loads of a step go: row lr + 32 i of an operand is at vw + i
  // (or vx + i) times a step of 32 rows; bit i of xdead: the token row reads
  // zeros (past the range)
  __amdgpu_buffer_rsrc_t rw =
      make_rsrc(reinterpret_cast<const char*>(p.w) + (int64_t)n0 * row_bytes, (uint32_t)cols * row_bytes);
  __amdgpu_buffer_rsrc_t rx =
      make_rsrc(reinterpret_cast<const char*>(p.x) + m0 * row_bytes, (uint32_t)rows * row_bytes);
  uint32_t vw = (uint32_t)lr * row_bytes + (uint32_t)lc * 16u, vx = vw;
  uint32_t wstep = 32u * row_bytes, xstep = wstep;
  uint32_t xdead = 0;
  const uint32_t st_off = (uint32_t)lr * 128u + ((uint32_t)(lc ^ (lr & 7) ^ ((lr >> 3) & 1)) << 4);

  i32x4_t wreg[8], xreg[XI];
  auto gload_one = [&](uint32_t soff, int q, int j) {
    if (j < 2) {
      wreg[2 * q + j] = buf_load16(rw, vw + (uint32_t)(2 * q + j) * wstep, soff);
    } else {
      const int i = q * XQ + j - 2;
      xreg[i] = buf_load16(rx, (vx + (uint32_t)i * xstep) | ((xdead << (31 - i)) & kNoRow), soff);
    }
  };
  auto lstore_one = [&](int stage, int q, int j) {
    char* dst = lds + stage * kStageBytes + st_off;
    if (j < 2)
      *reinterpret_cast<i32x4_t*>(dst + (2 * q + j) * 4096) = wreg[2 * q + j];
    else
      *reinterpret_cast<i32x4_t*>(dst + kOperandBytes + (q * XQ + j - 2) * 4096) = xreg[q * XQ + j - 2];
  };
  // the extension's step s: slice s % slices of adapter list[s / slices]
  const int kx = p.planes * p.r, slices = (kx + kBK - 1) / kBK;
  int ext = 0;  // its steps
  auto ext_step = [&](int s) {
    const int ai = s / slices, kk = (s - ai * slices) * kBK + 8 * lc;
    const int id = uniform(tl.list[ai]);
    const int plane = kk / p.r, j = kk - plane * p.r;
    rw = make_rsrc(reinterpret_cast<const __bf16*>(p.b) + ((int64_t)id * p.N + n0) * p.r, (uint32_t)(cols * p.r) * 2u);
    rx = make_rsrc(reinterpret_cast<const __bf16*>(p.t) + m0 * kx, (uint32_t)(rows * kx) * 2u);
    const uint32_t dead = kk < kx ? 0u : kNoRow;
    vw = (uint32_t)(lr * p.r + j) * 2u | dead;
    vx = (uint32_t)(lr * kx + kk) * 2u | dead;
    wstep = 64u * p.r;
    xstep = 64u * kx;
    xdead = 0;
#pragma unroll
    for (int i = 0; i < XI; ++i) xdead |= (tl.id[lr + 32 * i] != id ? 1u : 0u) << i;
  };
  auto drop_step = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (drop_nonfinite<__bf16>(wreg[i])) tl.nonfinite = 1;
  };

  // fragments
  const int lrow = lane & 31, lk = lane >> 5;
  const uint32_t wrow_off = (uint32_t)(wn * 128 + lrow) * 128u;
  const uint32_t xrow_off = (uint32_t)(kOperandBytes + (wm * (TM / 2) + lrow) * 128);
  uint32_t kswz[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) kswz[ks] = (uint32_t)(((2 * ks + lk) ^ (lrow & 7) ^ ((lrow >> 3) & 1)) << 4);
  bf16x8_t fa[2][4], fb[2][NJ];
  // fragment j of sub-step ks in the order the MFMAs use them: weight 0, the
  // token fragments, weights 1..3
  auto read_one = [&](int set, int stage, int ks, int j) {
    const char* base = lds + stage * kStageBytes;
    if (j == 0)
      fa[set][0] = *reinterpret_cast<const bf16x8_t*>(base + wrow_off + kswz[ks]);
    else if (j <= NJ)
      fb[set][j - 1] = *reinterpret_cast<const bf16x8_t*>(base + xrow_off + (j - 1) * 4096 + kswz[ks]);
    else
      fa[set][j - NJ] = *reinterpret_cast<const bf16x8_t*>(base + wrow_off + (j - NJ) * 4096 + kswz[ks]);
  };
  auto read_frags = [&](int set, int stage, int ks) {
#pragma unroll
    for (int j = 0; j < NR; ++j) read_one(set, stage, ks, j);
  };
  f32x16_t acc[4][NJ];
#pragma unroll
  for (int mi = 0; mi < 4; ++mi)
#pragma unroll
    for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[mi][nj][v] = 0.0f;
  auto mfma_rows = [&](int set, int mi0, int mi1) {
#pragma unroll
    for (int mi = mi0; mi < mi1; ++mi)
#pragma unroll
      for (int nj = 0; nj < NJ; ++nj)
        acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][mi], fb[set][nj], acc[mi][nj], 0, 0, 0);
  };

  const int nk = p.H / kBK;  // at least 2
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < NW; ++j) gload_one(0, q, j);
  if (p.P > 0) {
    list_adapters<TM>(p, m0, rows, tl);
    ext = uniform(tl.n) * slices;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < NW; ++j) lstore_one(0, q, j);
  // (fenced one by one: the loop's loads must be issued in the same order)
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      gload_one(kBK * 2, q, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  __syncthreads();
  read_frags(0, 0, 0);
  // step kt computes LDS stage kt & 1 while the registers (stage kt + 1) drain
  // into the other one and refill with stage kt + 2, a quarter per sub-step;
  // the last steps' stores, loads and reads go to idle places.  (The loop is
  // one copy, entered from one place: with a second copy, or a second way
  // in, it waits for its own loads in every step, 239 instead of 211 us at
  // 8192 x 4096 x 4096 without adapters.)
  const int steps = nk + ext;
  for (int kt = 0; kt < steps; ++kt) {
    const int cur = kt & 1, nxt = cur ^ 1;
    uint32_t soff = (uint32_t)min(kt + 2, nk - 1) * (kBK * 2);
    if (kt + 2 >= nk && ext > 0) {
      soff = 0;
      if (kt + 2 < steps) ext_step(kt + 2 - nk);
      if (kt + 1 >= nk) drop_step();
    }
    auto load_one = [&](int q, int j) { gload_one(soff, q, j); };
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
      if constexpr (TM == 256) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          read_one((ks + 1) & 1, cur, ks + 1, 2 * j);
          lstore_one(nxt, ks, j);
          read_one((ks + 1) & 1, cur, ks + 1, 2 * j + 1);
          load_one(ks, j);
        }
      } else {
        read_frags((ks + 1) & 1, cur, ks + 1);
#pragma unroll
        for (int j = 0; j < NW; ++j) lstore_one(nxt, ks, j);
#pragma unroll
        for (int j = 0; j < NW; ++j) load_one(ks, j);
      }
      mfma_rows(ks & 1, 0, 4);
      if constexpr (TM == 256) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // DS read
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // DS write
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
        }
      } else {
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 3, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < NW; ++j) lstore_one(nxt, 3, j);
#pragma unroll
    for (int j = 0; j < NW; ++j) load_one(3, j);
    mfma_rows(1, 0, 2);
    if constexpr (TM == 256) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NM / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x220, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x220, 2 * NW - NM / 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    read_frags(0, nxt, 0);
    mfma_rows(1, 2, 4);
#pragma unroll
    for (int i = 0; i < NM / 2; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (NR > NM / 2) __builtin_amdgcn_sched_group_barrier(0x100, NR - NM / 2, 0);
    __builtin_amdgcn_sched_barrier(0);
  }

  // ---- epilogue, through LDS: passes of 128 rows, 1 KiB per staged row (256
  // f32 columns; 16-byte unit u of staged row t at unit u ^ (t & 15)), so each
  // wave stores whole row segments: 4 columns of a row per thread, 32 rows a
  // pass.  A bf16 residual is loaded for all
  // of them before the staging (loaded row by row it cost 67 us of 279 at
  // 8192 x 4096 x 4096).  (8 columns per thread, i.e. wider stores but two
  // lanes per LDS bank, took 7 us more per tile.)
  const bool left_out = ext > 0 && uniform(tl.nonfinite) != 0;
  const int c = tid & 63, n = n0 + 4 * c, wv = uniform(wave);
  const bool whole = n + 4 <= p.N;  // all of the thread's columns exist
  const bool pre = p.out.residual && whole;
#pragma unroll
  for (int P = 0; P < NJ / 2; ++P) {
    auto tile_row = [&](int i) {  // of the thread's i-th staged row of the pass
      const int ts = wv + 4 * i;
      return (ts >> 6) * (TM / 2) + 64 * P + (ts & 63);
    };
    bf16x4_t res[32];
    if (pre) {
      const __bf16* r0 = reinterpret_cast<const __bf16*>(p.out.residual) + m0 * p.N + n;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        res[i] = load_any(r0 + (int64_t)min(tile_row(i), rows - 1) * p.N);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nj = 2 * P + j, ts = wm * 64 + j * 32 + lrow;
#pragma unroll
      for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t o;
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = acc[mi][nj][4 * q + v];
          const int u = wn * 32 + mi * 8 + 2 * q + lk;
          *reinterpret_cast<f32x4_t*>(lds + ts * 1024 + ((u ^ (ts & 15)) << 4)) = o;
        }
    }
    __syncthreads();
    auto staged = [&](int i) {
      const int ts = wv + 4 * i;
      return reinterpret_cast<f32x4_t*>(lds + ts * 1024 + ((c ^ (ts & 15)) << 4));
    };
    // 8 rows at a time, so that the look at the sums costs nothing (in a pass of
    // its own 1.7 us of 267 at 8192 x 4096 x 4096; with all 32 rows in registers,
    // or before the staging, they spill).
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += 8) {
      f32x4_t v[8];
      float bad = 0.0f;  // NaN once a sum is not finite
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = *staged(i0 + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) bad = fmaf(v[i][e], 0.0f, bad);
      }
      if (ext > 0 && (left_out || __builtin_isnan(bad))) {
#pragma unroll 1
        for (int i = i0; i < i0 + 8; ++i) {
          const int row = tile_row(i);
          if (row >= rows || tl.id[row] < 0) continue;
#pragma unroll 1
          for (int e = 0; e < 4 && n + e < p.N; ++e) {
            float* at = reinterpret_cast<float*>(staged(i)) + e;
            *at = mend_sum<__bf16>(p, m0 + row, tl.id[row], n + e, left_out, *at);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *staged(i0 + i);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = tile_row(i0 + i);
        if (pre) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] += (float)res[i0 + i][e];
        }
        if (row >= rows || !whole) continue;
        store_any(p, (m0 + row) * p.N + n, v[i]);
      }
    }
    if (n < p.N && !whole) {  // the last columns of a row
#pragma unroll 1
      for (int i = 0; i < 32; ++i) {
        const int row = tile_row(i);
        for (int e = 0; row < rows && n + e < p.N; ++e) store_one(p, (m0 + row) * p.N + n + e, (*staged(i))[e]);
      }
    }
    __syncthreads();
  }
}

// Tiles of the grid, in an order that lets the workgroups of one XCD share
// operand panels in its L2: 8 row tiles x all column tiles at a time, the row
// tiles fastest, a contiguous run of that order per XCD.
template <int TM>
__global__ __launch_bounds__(kGemmThreads) void adapter_gemm_kernel(AdapterArgs p, int mt, int nt) {
  __shared__ __attribute__((aligned(16))) char lds[kGemmLdsBytes];
  __shared__ AdapterTileLds tl;
  const int64_t v = xcd_tile((int64_t)mt * nt);
  if (v < 0) return;
  const int64_t band = v / (8ll * nt);
  const int rb = min(8, mt - (int)band * 8);
  const int64_t in = v - band * 8ll * nt;
  const int64_t m = band * 8 + in % rb;
  adapter_gemm_tile<TM>(p, m * TM, (int)(in / rb) * 256, lds, tl);
}

}  // namespace moe
