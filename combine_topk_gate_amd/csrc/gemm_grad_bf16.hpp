// bf16 MFMA tiles of the grouped GEMM's training products (gfx950).
//
// The forward tile (gemm_bf16.hpp) has both operands contiguous along the
// reduction, and so have the forward products that are kept (keep: gate and up,
// each tile 128 columns of both).  In the gradients that holds for the token
// rows of a rows' gradient alone:
//   rows     C[r, n] = sum_k D[r, k] W[k, n]: W's stored rows are the k index;
//   weights  C[f, h] = sum_r D[r, f] X[r, h]: so are the rows of both operands.
// An operand that lies [k][columns] in memory is staged the same way in LDS
// and turned on the way to the registers by ds_read_b64_tr_b16: the 16 lanes
// of a group read 4 k rows x 16 columns, and each ends with the 4 k values of
// one column, half of what v_mfma_f32_32x32x16_bf16 takes.  No copy of the
// weights or the activations is turned in memory (for 8 experts of 4096 x
// 14336 that alone would move 2.8 GB each way, 1.2 ms).
//
// Otherwise the schedule is the forward tile's: 256 columns x TM rows (TM =
// 256, or 128 for rows of short segments), 4 waves of 128 x TM/2, K steps of
// 64 through two LDS buffers, the loads two steps ahead in registers, one
// memory operation after every matrix instruction.  The columns are the
// instruction's first operand, so a lane holds 4 consecutive columns of a row.
//
// LDS of an operand [64 k][256 columns]: rows of 512 B; the 32-byte piece s of
// row k is stored at s ^ 2 (k & 3), so the 4 rows x 2 pieces that 32 lanes
// read lie in different banks (all 64 once).  The [rows][64 k] operand lies as
// in the forward tile.
//
// Rows past the end are never read from memory: the buffers' ranges end with
// the rows of the expert's segment (weights), and a row that a tile does not
// have lies past the range (rows).  Columns past the end read the next row or
// zeros; they only reach outputs that are not stored.
#pragma once

#include <utility>

#include "common.hpp"
#include "gemm_bf16.hpp"
#include "launch.hpp"
#include "tiles.hpp"

namespace moe {

typedef __attribute__((address_space(3))) char lds_byte;
typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4;

enum GradKind { kGradRows0, kGradRows1, kGradWeights, kKeep };

// d silu(g) u / dg and / du times dh, with the hardware exponential and
// reciprocal (about 1 ulp each), as the forward epilogue's silu_mul_fast: the
// outputs round to bf16.  With s = 1 / (1 + e^-g) (0 where e^-g overflows):
//   dg = dh u (s + g s (1 - s)),  du = dh g s
struct SwigluGrad {
  float dg, du;
};
__device__ __forceinline__ SwigluGrad swiglu_grad_fast(float dh, float g, float u) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
  const float a = g * s;
  return {dh * u * fmaf(a, 1.0f - s, s), dh * a};
}

typedef int i32x2_t __attribute__((ext_vector_type(2)));

// Results are stored, and gate and up loaded, as used once ("nt"): kept like
// other lines they push the operands' panels, which the tiles of an XCD share,
// out of its L2 (weights of 64 experts 2048 x 1408, 256 rows each: 466 us, as
// used once 366; 16 experts 4096 x 6400: 3065, 3047).  The next call of a training
// step reads most of them, but whole steps gain too (bf16, dropout, kept, as used
// once): 1024 tokens, 16 experts 2048 x 1408, top 4: 563, 526 us; 4096, 64 of them:
// 1809, 1748; 2048, 8 of 1024 x 1024, top 2: 270, 270; 8192, 8 of 4096 x 14336:
// 15.54, 15.48 ms.
constexpr int kOnce = 2;

__device__ __forceinline__ void buf_store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, i32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)voff, 0, kOnce);
}
__device__ __forceinline__ i32x4_t buf_load16_once(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, 0, kOnce));
}

// Byte offset of column n of row pos in a bf16 buffer of N columns; past any
// range (of at most 2^32 - 128 bytes) for a row that the tile lacks (-1) or a
// column that the buffer lacks.
__device__ __forceinline__ uint32_t grad_offset(int pos, int n, int N) {
  return pos >= 0 && n < N ? ((uint32_t)pos * (uint32_t)N + (uint32_t)n) * 2u : 0xFFFFFFF0u;
}

struct GradTile {
  int e;        // weight slot
  int row0;     // weights: first row of dW (column of D)
  int col0;     // first column
  int second;   // weights: the second pair of matrices (d1, o1)
  int part, parts;  // which of the parts of the K steps (0 of 1: all)
};

__device__ __forceinline__ const __bf16* uniform_ptr(const __bf16* p) {
  const uint64_t v = (uint64_t)p;
  return (const __bf16*)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// First step of part i of n of nk K steps.
__device__ __forceinline__ int part_begin(int nk, int i, int n) { return (int)((int64_t)nk * i / n); }

// K steps of expert e's weights' gradient: each segment's last one is filled up with zero rows.
__device__ __forceinline__ int weight_steps(const GradGemmArgs& p, const int* offsets, int e) {
  int nk = 0;
  const int S = p.G / p.E;
  for (int s = 0; s < S; ++s) nk += (offsets[s * p.E + e + 1] - offsets[s * p.E + e] + kBK - 1) / kBK;
  return uniform(nk);
}

// What a wave does for one tile after the other:
//   begin(t)     addresses, and the loads of the first K step into registers
//   multiply()   the K loop
//   epilogue(t)  from the accumulators to memory, or store_part(u): a split
//                tile's sums over its part of the K steps, as they are
// The kernels call begin of the next tile before the epilogue of this one, so
// the first loads' latency is not waited for.
template <GradKind KIND, int TM>
struct GradWave {
  static constexpr bool XKC = KIND != kGradWeights;  // x operand contiguous along k
  static constexpr bool WKC = KIND == kKeep;         // w operand too
  static_assert(TM == 256 || (TM == 128 && XKC), "tile height");
  static constexpr int NJ = TM / 64;             // row fragments per wave
  static constexpr int XI = XKC ? TM / 32 : 8;   // x loads per thread per K step
  static constexpr int XQ = XI / 4;              // ... per sub-step
  static constexpr int NRX = XKC ? NJ : 2 * NJ;  // LDS reads of x per sub-step
  static constexpr int WH = WKC ? 1 : 2;         // LDS reads of a w fragment
  static constexpr int NR = 4 * WH + NRX;        // LDS reads per sub-step
  static constexpr int NW = 2 + XQ;              // LDS stores (and loads) per sub-step
  static constexpr int NM = 4 * NJ;              // matrix instructions per sub-step

  const GradGemmArgs& p;
  char* __restrict__ const lds;
  const int* const offsets;  // weights: the offsets, in LDS
  const int tid = threadIdx.x, lane = tid & 63, wn = (tid >> 6) & 1, wm = tid >> 7;
  const int lrow = lane & 31, lk = lane >> 5;
  // a product's reduction length (rows), the columns of D and of the output
  const bool l0 = KIND == kGradRows0 || (KIND == kGradWeights && p.layer == 0);
  const int K = KIND == kGradRows0 ? p.F : p.H;
  const int N = KIND == kGradRows1 || KIND == kKeep ? p.F : KIND == kGradRows0 ? p.H : (l0 ? p.H : p.F);
  const int DN = KIND == kGradWeights ? (l0 ? p.F : p.H) : K;
  const uint32_t wpitch = (uint32_t)N * 2u, xpitch = (uint32_t)DN * 2u;
  const int cr = tid >> 5, cc = tid & 31;
  const uint32_t wvoff = (uint32_t)cr * wpitch + (uint32_t)cc * 16u;
  __amdgpu_buffer_rsrc_t rw1;  // keep: W_up's rows (rw: W_gate's)

  // the K step to load next: its buffers, and (weights) where they begin and how long they are
  __amdgpu_buffer_rsrc_t rw, rx;
  const __bf16 *wbase = nullptr, *xbase = nullptr;
  uint32_t wbytes = 0, xbytes = 0;
  uint32_t xs = 0;
  int e = 0, col0 = 0, row0 = 0, k0 = 0, nk = 0;  // K steps k0 .. k0 + nk
  const __bf16* d = nullptr;
  int r = 0, rend = 0, sb = 0;  // weights: the segment's row and end, the next source block
  uint32_t xvoff[XKC ? XI : 1];

  i32x4_t wreg[8], xreg[XI];
  f32x16_t acc[4][NJ];

  __device__ __forceinline__ GradWave(const GradGemmArgs& p, char* lds, const int* offsets)
      : p(p), lds(lds), offsets(offsets) {}

  // Steps are asked for in order, once each; past the last one the buffers stay.
  __device__ __forceinline__ void source(int kt) {
    if constexpr (KIND == kGradWeights) {
      if (kt < nk) {
        r += kBK;
        while (r >= rend && sb < p.G / p.E) {
          r = uniform(offsets[sb * p.E + e]);
          rend = uniform(offsets[sb * p.E + e + 1]);
          ++sb;
        }
        const uint32_t n = (uint32_t)min(rend - r, kBK);
        wbase = (const __bf16*)p.x + (int64_t)r * N + col0;
        xbase = d + (int64_t)r * DN + row0;
        wbytes = n * wpitch - (uint32_t)col0 * 2u;
        xbytes = n * xpitch - (uint32_t)row0 * 2u;
      }
      // (made uniform here, in every step: a descriptor that the compiler cannot tell to be is loaded through lane by lane)
      rw = make_rsrc(uniform_ptr(wbase), (uint32_t)uniform((int)wbytes));
      rx = make_rsrc(uniform_ptr(xbase), (uint32_t)uniform((int)xbytes));
    } else if constexpr (KIND == kKeep) {
      xs = (uint32_t)min(kt, nk - 1) * (kBK * 2);
    } else {
      const int per = K / kBK;
      kt = k0 + min(kt, nk - 1);
      const bool second = KIND == kGradRows0 && kt >= per;
      const int kk = second ? kt - per : kt;
      const __bf16* w = (const __bf16*)(second ? p.w1 : p.w0) + (int64_t)e * K * N;
      rw = make_rsrc(w + (int64_t)kk * kBK * N + col0, (uint32_t)kBK * wpitch - (uint32_t)col0 * 2u);
      rx = make_rsrc(second ? p.d1 : p.d0, (uint32_t)(p.R * (int64_t)xpitch));
      xs = (uint32_t)kk * (kBK * 2);
    }
  }

  // Global -> register loads.  [k][columns]: thread owns 16-byte chunk tid & 31
  // of k rows (tid >> 5) + 8 i; [rows][k]: chunk tid & 7 of rows (tid >> 3) + 32 i
  // (keep's weights: 128 of gate, then 128 of up).
  __device__ __forceinline__ void gload_one(int q, int j) {
    if (j < 2) {
      const int i = 2 * q + j;
      if constexpr (WKC)
        wreg[i] = buf_load16(i < 4 ? rw : rw1, (uint32_t)((tid >> 3) + 32 * (i & 3)) * xpitch + (uint32_t)(tid & 7) * 16u, xs);
      else
        wreg[i] = buf_load16(rw, wvoff + (uint32_t)i * (8u * wpitch), 0);
    } else {
      const int i = q * XQ + j - 2;
      if constexpr (XKC)
        xreg[i] = buf_load16(rx, xvoff[i], xs);
      else
        xreg[i] = buf_load16(rx, xvoff[0] + (uint32_t)i * (8u * xpitch), 0);
    }
  }
  __device__ __forceinline__ void lstore_one(int stage, int q, int j) {
    const uint32_t st_kr = (uint32_t)cr * 512u + ((uint32_t)(cc ^ ((cr & 3) << 2)) << 4);
    const int lr = tid >> 3;
    const uint32_t st_kc = (uint32_t)lr * 128u + ((uint32_t)((tid & 7) ^ (lr & 7) ^ ((lr >> 3) & 1)) << 4);
    char* wdst = lds + stage * kStageBytes;
    if (j < 2) {
      const int i = 2 * q + j;
      *reinterpret_cast<i32x4_t*>(wdst + (WKC ? st_kc : st_kr) + i * 4096) = wreg[i];
    } else {
      const int i = q * XQ + j - 2;
      *reinterpret_cast<i32x4_t*>(wdst + kOperandBytes + (XKC ? st_kc : st_kr) + i * 4096) = xreg[i];
    }
  }

  // The tile's part of all nk steps.
  __device__ __forceinline__ void range(const GradTile& t) {
    k0 = uniform(part_begin(nk, t.part, t.parts));
    nk = uniform(part_begin(nk, t.part + 1, t.parts)) - k0;
  }

  // rowpos (rows): the rows of the tile in the buffers, -1 for those it lacks.
  __device__ __forceinline__ void begin(const GradTile& t, const int* __restrict__ rowpos) {
    e = uniform(t.e);
    col0 = uniform(t.col0);
    if constexpr (KIND == kGradWeights) {
      row0 = uniform(t.row0);
      d = (const __bf16*)(uniform(t.second) ? p.d1 : p.d0);
      nk = weight_steps(p, offsets, e);
      range(t);
      // to the step before k0
      r = rend = sb = 0;
      for (int left = k0;;) {
        const int n = (rend - r + kBK - 1) / kBK;
        if (left <= n || sb == p.G / p.E) {
          r += (left - 1) * kBK;
          break;
        }
        left -= n;
        r = uniform(offsets[sb * p.E + e]);
        rend = uniform(offsets[sb * p.E + e + 1]);
        ++sb;
      }
      xvoff[0] = (uint32_t)cr * xpitch + (uint32_t)cc * 16u;
    } else {
      nk = (KIND == kGradRows0 ? 2 : 1) * (K / kBK);
      range(t);
      if constexpr (KIND == kKeep) {
        const uint32_t bytes = (uint32_t)min(N - col0, 128) * xpitch;
        const int64_t at = ((int64_t)e * N + col0) * K;
        rw = make_rsrc((const __bf16*)p.w0 + at, bytes);
        rw1 = make_rsrc((const __bf16*)p.w1 + at, bytes);
        rx = make_rsrc(p.x, (uint32_t)(p.R * (int64_t)xpitch));
      }
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int pos = rowpos[(tid >> 3) + 32 * i];
        // a row that the tile lacks: past the range, or (buffers over 2 GiB) another row, whose sums are not stored
        xvoff[i] = pos >= 0 ? (uint32_t)pos * xpitch + (uint32_t)(tid & 7) * 16u : 0x80000000u;
      }
    }
    if (nk > 0) {
      source(0);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < NW; ++j) gload_one(q, j);
    }
  }

  // All waves of the block call it together; every LDS use of the tile before is behind its first barrier.
  __device__ __forceinline__ void multiply() {
    // fragment addresses
    uint32_t wrd[4], xrd[4];
    {
      // lane's 16-lane group: columns 16 (g & 1), k rows 8 (g >> 1); in it, row l >> 2, 8-byte piece l & 3
      const int g = lane >> 4, l = lane & 15, lq = l >> 2;
      const uint32_t base = (uint32_t)(8 * (g >> 1) + lq) * 512u + (uint32_t)(g & 1) * 32u + (uint32_t)(l & 3) * 8u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t kc = (uint32_t)(((2 * i + lk) ^ (lrow & 7) ^ ((lrow >> 3) & 1)) << 4);  // sub-step i's chunk of a row
        wrd[i] = WKC ? (uint32_t)(wn * 64 + lrow) * 128u + kc : base + (uint32_t)(wn * 8 + ((i ^ lq) << 1)) * 32u;
        if constexpr (XKC)
          xrd[i] = (uint32_t)(kOperandBytes + (wm * (TM / 2) + lrow) * 128) + kc;
        else
          xrd[i] = (uint32_t)kOperandBytes + base + (uint32_t)(wm * 8 + ((i ^ lq) << 1)) * 32u;
      }
    }
    lds_byte* l3 = (lds_byte*)lds;
    bf16x4_t fa[2][WKC ? 1 : 4][2];
    bf16x8_t fa8[2][WKC ? 4 : 1];
    bf16x4_t fx4[2][XKC ? 1 : NJ][2];
    bf16x8_t fx8[2][XKC ? NJ : 1];
    auto read_tr = [&](uint32_t at, int stage, int ks, int h) {
      return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (lds_bf16x4*)(l3 + stage * kStageBytes + at + (uint32_t)(ks * 16 + 4 * h) * 512u));
    };
    // read j of sub-step ks, in the order the matrix instructions use them: column fragment 0, the row fragments,
    // columns 1..3
    auto read_one = [&](int set, int stage, int ks, int j) {
      if (j >= WH && j < WH + NRX) {
        const int i = j - WH;
        if constexpr (XKC)
          fx8[set][i] = *reinterpret_cast<const bf16x8_t*>(lds + stage * kStageBytes + xrd[ks] + i * 4096);
        else
          fx4[set][i / 2][i & 1] = read_tr(xrd[i / 2], stage, ks, i & 1);
      } else {
        const int i = j < WH ? j : j - NRX;
        if constexpr (WKC)  // gate rows 64 wn + 32 i (i < 2), up rows 128 + 64 wn + 32 (i - 2)
          fa8[set][i] = *reinterpret_cast<const bf16x8_t*>(lds + stage * kStageBytes + wrd[ks] + (i & 1) * 4096 + (i >> 1) * 16384);
        else
          fa[set][i / 2][i & 1] = read_tr(wrd[i / 2], stage, ks, i & 1);
      }
    };
    auto mfma_rows = [&](int set, int mi0, int mi1) {
#pragma unroll
      for (int mi = mi0; mi < mi1; ++mi)
#pragma unroll
        for (int nj = 0; nj < NJ; ++nj) {
          bf16x8_t a, b;
          if constexpr (WKC)
            a = fa8[set][mi];
          else
            a = __builtin_shufflevector(fa[set][mi][0], fa[set][mi][1], 0, 1, 2, 3, 4, 5, 6, 7);
          if constexpr (XKC)
            b = fx8[set][nj];
          else
            b = __builtin_shufflevector(fx4[set][nj][0], fx4[set][nj][1], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[mi][nj], 0, 0, 0);
        }
    };

#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
      for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[mi][nj][v] = 0.0f;
    __syncthreads();
    if (nk == 0) return;
    // prologue: step 0 into LDS, step 1 into registers, fragments of (0, 0)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NW; ++j) lstore_one(0, q, j);
    source(1);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        gload_one(q, j);
        __builtin_amdgcn_sched_barrier(0);  // in the loop body's order (see bf16_gemm_tile)
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j) read_one(0, 0, 0, j);

    for (int kt = 0; kt < nk; ++kt) {
      const int cur = kt & 1, nxt = cur ^ 1;
      source(kt + 2);
#pragma unroll
      for (int ks = 0; ks < 3; ++ks) {
        // source order = issue order; slot s of the NM matrix instructions is followed by its share of the NR reads,
        // and in some by a store of step kt + 1 or, 2 slots behind it, the load of step kt + 2 into its register
#pragma unroll
        for (int s = 0; s < NM; ++s) {
#pragma unroll
          for (int j = s * NR / NM; j < (s + 1) * NR / NM; ++j) read_one((ks + 1) & 1, cur, ks + 1, j);
#pragma unroll
          for (int j = (s + 2) * NW / NM; j < (s + 3) * NW / NM; ++j) lstore_one(nxt, ks, j);
#pragma unroll
          for (int j = s * NW / NM; j < (s + 1) * NW / NM; ++j) gload_one(ks, j);
        }
        mfma_rows(ks & 1, 0, 4);
        [&]<int... s>(std::integer_sequence<int, s...>) {
          (
              [&] {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
                if constexpr ((s + 1) * NR / NM > s * NR / NM)
                  __builtin_amdgcn_sched_group_barrier(0x100, (s + 1) * NR / NM - s * NR / NM, 0);  // DS read
                if constexpr ((s + 3) * NW / NM > (s + 2) * NW / NM)
                  __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // DS write
                if constexpr ((s + 1) * NW / NM > s * NW / NM) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
              }(),
              ...);
        }(std::make_integer_sequence<int, NM>{});
        __builtin_amdgcn_sched_barrier(0);
      }
      // sub-step 3: the last stores and loads with the first half of the matrix instructions
#pragma unroll
      for (int j = 0; j < NW; ++j) lstore_one(nxt, 3, j);
#pragma unroll
      for (int j = 0; j < NW; ++j) gload_one(3, j);
      mfma_rows(1, 0, 2);
#pragma unroll
      for (int i = 0; i < NM / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    // MFMA
        __builtin_amdgcn_sched_group_barrier(0x220, 1, 0);  // DS write, then VMEM read
      }
      if constexpr (2 * NW > NM / 2) __builtin_amdgcn_sched_group_barrier(0x220, 2 * NW - NM / 2, 0);
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NR; ++j) read_one(0, nxt, 0, j);
      mfma_rows(1, 2, 4);
      constexpr int RP = (NR + NM / 2 - 1) / (NM / 2);  // reads per matrix instruction
#pragma unroll
      for (int i = 0; i < NM / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, RP, 0);  // DS read
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Lane (lrow, lk) holds, per row fragment nj and column fragment mi, the
  // 4-column groups 8 q + 4 lk of row wm TM/2 + 32 nj + lrow.  A wave turns one
  // row fragment at a time (32 rows x 128 columns) in 32 KiB of LDS of its own,
  // in two halves by turns, so that it stores whole row segments (256 or 512 B)
  // and waits for no other wave.  After the loop's last barrier no wave uses a
  // value of the stages again.  The loads and stores are buffer ones: what lies
  // outside the tile's rows or columns has an offset past the range, so there is
  // no branch, and a fragment's accesses are in flight together.
  __device__ __forceinline__ void epilogue(const GradTile& t, const int* __restrict__ rowpos) {
    // The lane's number hidden from the optimiser: the swizzled addresses below would otherwise be computed once before
    // the tiles, some fifty registers kept (spilled) through the K loop for one instruction each.
    int lane = this->lane;
    asm volatile("" : "+v"(lane));
    const int lrow = lane & 31, lk = lane >> 5;
    char* const mine = lds + (tid >> 6) * 32768;
    const int tcol = uniform(t.col0) + wn * (KIND == kKeep ? 64 : 128);  // the wave's first column
    if constexpr (KIND == kKeep) {
      // Hact (as the forward epilogue forms it, from the f32 products), gate and up, 64 columns each: 128 B a staged row;
      // 8-byte unit u of row i at u ^ (i / 2), so that 32 rows write one unit, and 8 lanes a row read 16-byte chunks,
      // without a conflict
      const uint32_t bytes = (uint32_t)(p.R * N * 2);
      const __amdgpu_buffer_rsrc_t ro[3] = {make_rsrc(p.o2, bytes), make_rsrc(p.o0, bytes), make_rsrc(p.o1, bytes)};
      const int c = lane & 7;
#pragma unroll
      for (int nj = 0; nj < NJ; ++nj) {
        char* const stg = mine + (nj & 1) * 16384;
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            bf16x4_t o[3];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float g = acc[mi][nj][4 * q + v], u = acc[mi + 2][nj][4 * q + v];
              o[0][v] = (__bf16)silu_mul_fast(g, u);
              o[1][v] = (__bf16)g;
              o[2][v] = (__bf16)u;
            }
            const int u = mi * 8 + 2 * q + lk;
#pragma unroll
            for (int m = 0; m < 3; ++m)
              *reinterpret_cast<bf16x4_t*>(stg + m * 4096 + lrow * 128 + ((u ^ (lrow >> 1)) << 3)) = o[m];
          }
        i32x4_t v[4][3];
        uint32_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 8 * i + (lane >> 3);
          at[i] = grad_offset(rowpos[wm * (TM / 2) + nj * 32 + row], tcol + 8 * c, N);
#pragma unroll
          for (int m = 0; m < 3; ++m)
            v[i][m] = *reinterpret_cast<const i32x4_t*>(stg + m * 4096 + row * 128 + ((c ^ (row >> 2)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int m = 0; m < 3; ++m)
            buf_store16(ro[m], at[i], (lane >> 4) & 1 ? i32x4_t{v[i][m][2], v[i][m][3], v[i][m][0], v[i][m][1]} : v[i][m]);
      }
    } else if constexpr (KIND == kGradRows0) {
      // 256 B a staged row; 8-byte unit u of row i at u ^ i; read as 16-byte chunks: c ^ (i >> 1), halves swapped for
      // an odd row.  16 lanes a row, 8 columns each.
      const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.o0, (uint32_t)(p.R * N * 2));
      const int c = lane & 15;
#pragma unroll
      for (int nj = 0; nj < NJ; ++nj) {
        char* const stg = mine + (nj & 1) * 8192;
#pragma unroll
        for (int mi = 0; mi < 4; ++mi)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            bf16x4_t h;
#pragma unroll
            for (int v = 0; v < 4; ++v) h[v] = (__bf16)acc[mi][nj][4 * q + v];
            *reinterpret_cast<bf16x4_t*>(stg + lrow * 256 + (((mi * 8 + 2 * q + lk) ^ lrow) << 3)) = h;
          }
        i32x4_t v[8];
        uint32_t at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 4);
          at[i] = grad_offset(rowpos[wm * (TM / 2) + nj * 32 + row], tcol + 8 * c, N);
          v[i] = *reinterpret_cast<const i32x4_t*>(stg + row * 256 + ((c ^ (row >> 1)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          buf_store16(ro, at[i], (lane >> 4) & 1 ? i32x4_t{v[i][2], v[i][3], v[i][0], v[i][1]} : v[i]);
      }
    } else {
      // 512 B a staged row (f32): 16-byte unit u of row i at (u / 2 + 16 (u % 2)) ^ (i & 15), so that both the lanes
      // that read every unit and those that read every other one (8 columns each) read 256 bytes in a row
      auto stage = [&](int nj) {
        char* const stg = mine + (nj & 1) * 16384;
#pragma unroll
        for (int mi = 0; mi < 4; ++mi)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4_t o;
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = acc[mi][nj][4 * q + v];
            *reinterpret_cast<f32x4_t*>(stg + lrow * 512 + (((mi * 4 + q + 16 * lk) ^ (lrow & 15)) << 4)) = o;
          }
      };
      if constexpr (KIND == kGradRows1) {
        // 16 lanes a row, 8 columns each: batches of 4 x 4 rows, 2 a fragment; gate and up are loaded two batches ahead
        const uint32_t bytes = (uint32_t)(p.R * N * 2);
        const __amdgpu_buffer_rsrc_t rg = make_rsrc(p.gate, bytes), ru = make_rsrc(p.up, bytes);
        const __amdgpu_buffer_rsrc_t r0 = make_rsrc(p.o0, bytes), r1 = make_rsrc(p.o1, bytes);
        const int c = lane & 15;
        i32x4_t g[3][4], u[3][4];
        uint32_t at[3][4];
        auto load = [&](int b) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = wm * (TM / 2) + b * 16 + 4 * i + (lane >> 4);
            at[b % 3][i] = grad_offset(rowpos[row], tcol + 8 * c, N);
            g[b % 3][i] = buf_load16_once(rg, at[b % 3][i]);
            u[b % 3][i] = buf_load16_once(ru, at[b % 3][i]);
          }
        };
        load(0);
        load(1);
#pragma unroll
        for (int b = 0; b < 2 * NJ; ++b) {
          if (b % 2 == 0) stage(b / 2);
          if (b + 2 < 2 * NJ) load(b + 2);
          const char* const stg = mine + (b / 2 & 1) * 16384;
          f32x4_t dh[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = (b & 1) * 16 + 4 * i + (lane >> 4);
              dh[i][h] = *reinterpret_cast<const f32x4_t*>(stg + row * 512 + (((c + 16 * h) ^ (row & 15)) << 4));
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bf16x8_t gv = __builtin_bit_cast(bf16x8_t, g[b % 3][i]), uv = __builtin_bit_cast(bf16x8_t, u[b % 3][i]);
            bf16x8_t og, ou;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const SwigluGrad s = swiglu_grad_fast(dh[i][v / 4][v % 4], (float)gv[v], (float)uv[v]);
              og[v] = (__bf16)s.dg;
              ou[v] = (__bf16)s.du;
            }
            buf_store16(r0, at[b % 3][i], __builtin_bit_cast(i32x4_t, og));
            buf_store16(r1, at[b % 3][i], __builtin_bit_cast(i32x4_t, ou));
          }
        }
      } else {
        // 32 lanes a row, 4 columns each
        const int trow = uniform(t.row0), rows = min(DN - trow, TM), te = uniform(t.e);
        const int es = p.out_bf16 ? 2 : 4;
        const char* const out = (const char*)(uniform(t.second) ? p.o1 : p.o0) + (((int64_t)te * DN + trow) * N) * es;
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(out, (uint32_t)rows * (uint32_t)(N * es));
        const int n = tcol + 4 * (lane & 31);
        const uint32_t pitch = (uint32_t)(N * es);
        const uint32_t at0 = n < N ? (uint32_t)(wm * (TM / 2) + lk) * pitch + (uint32_t)(n * es) : 0x80000000u;
        auto each = [&](auto&& store) {
#pragma unroll
          for (int nj = 0; nj < NJ; ++nj) {
            stage(nj);
            const char* const stg = mine + (nj & 1) * 16384;
            f32x4_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = 2 * i + lk, u = lane & 31;
              v[i] = *reinterpret_cast<const f32x4_t*>(stg + row * 512 + (((u / 2 + 16 * (u % 2)) ^ (row & 15)) << 4));
            }
            store(v, at0 + (uint32_t)(nj * 32) * pitch);
          }
        };
        if (p.out_bf16) {
          each([&](f32x4_t (&v)[16], uint32_t at) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              bf16x4_t b;
#pragma unroll
              for (int j = 0; j < 4; ++j) b[j] = (__bf16)v[i][j];
              __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2_t, b), ro, (int)(at + 2u * i * pitch), 0, kOnce);
            }
          });
        } else if (p.accumulate) {
          each([&](f32x4_t (&v)[16], uint32_t at) {
            f32x4_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __builtin_bit_cast(f32x4_t, buf_load16_once(ro, at + 2u * i * pitch));
#pragma unroll
            for (int i = 0; i < 16; ++i) buf_store16(ro, at + 2u * i * pitch, __builtin_bit_cast(i32x4_t, w[i] + v[i]));
          });
        } else {
          each([&](f32x4_t (&v)[16], uint32_t at) {
#pragma unroll
            for (int i = 0; i < 16; ++i) buf_store16(ro, at + 2u * i * pitch, __builtin_bit_cast(i32x4_t, v[i]));
          });
        }
      }
    }
  }

  // The accumulators as they lie: 16 bytes a lane, fragment by fragment (mi NJ + nj) of each wave.
  __device__ __forceinline__ void store_part(int u) {
    f32x4_t* dst = reinterpret_cast<f32x4_t*>(p.split.part) + ((int64_t)u * 4 + (tid >> 6)) * 16 * 4 * 64 + lane;
#pragma unroll
    for (int mi = 0; mi < 4; ++mi)
#pragma unroll
      for (int nj = 0; nj < NJ; ++nj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t o;
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = acc[mi][nj][4 * q + v];
          dst[((mi * NJ + nj) * 4 + q) * 64] = o;
        }
  }
};

}  // namespace moe
