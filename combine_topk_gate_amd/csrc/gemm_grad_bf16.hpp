// bf16 MFMA tiles of the grouped GEMM's gradients (gfx950).
//
// The forward tile (gemm_bf16.hpp) has both operands contiguous along the
// reduction.  Here that holds for the token rows of a rows' gradient alone:
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

enum GradKind { kGradRows0, kGradRows1, kGradWeights };

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

struct GradTile {
  int e;        // weight slot
  int row0;     // weights: first row of dW (column of D)
  int col0;     // first column
  int second;   // weights: the second pair of matrices (d1, o1)
};

template <GradKind KIND, int TM>
__device__ __forceinline__ void grad_tile(const GradGemmArgs& p, const GradTile& t, char* __restrict__ lds,
                                          const int* __restrict__ rowpos) {
  constexpr bool XKC = KIND != kGradWeights;  // x operand contiguous along k
  static_assert(TM == 256 || (TM == 128 && XKC), "tile height");
  constexpr int NJ = TM / 64;                  // row fragments per wave
  constexpr int XI = XKC ? TM / 32 : 8;        // x loads per thread per K step
  constexpr int XQ = XI / 4;                   // ... per sub-step
  constexpr int NRX = XKC ? NJ : 2 * NJ;       // LDS reads of x per sub-step
  constexpr int NR = 8 + NRX;                  // LDS reads per sub-step
  constexpr int NW = 2 + XQ;                   // LDS stores (and loads) per sub-step
  constexpr int NM = 4 * NJ;                   // matrix instructions per sub-step
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wm = wave >> 1;
  const int e = uniform(t.e), col0 = uniform(t.col0), row0 = uniform(t.row0);
  // reduction length of one product and columns of the output
  const int K = KIND == kGradRows0 ? p.F : p.H;
  const int layer_cols = KIND == kGradRows0 ? p.H : p.F;
  // weights: dW is [F, H] in layer 0, [H, F] in layer 1
  const bool l0 = KIND == kGradWeights && p.layer == 0;
  const int N = KIND == kGradWeights ? (l0 ? p.H : p.F) : layer_cols;   // columns
  const int DN = KIND == kGradWeights ? (l0 ? p.F : p.H) : K;           // columns of D
  const uint32_t wpitch = (uint32_t)N * 2u, xpitch = (uint32_t)DN * 2u;

  // ---- sources of the K steps
  // current step to load: buffers, and (rows) the byte offset along k
  __amdgpu_buffer_rsrc_t rw, rx;
  uint32_t xs = 0;
  const __bf16* d = (const __bf16*)(KIND == kGradWeights && t.second ? p.d1 : p.d0);
  int nk;
  // weights: the segment's next row and end, the next source block
  int r = 0, rend = 0, sb = 0;
  const int S = p.G / p.E;
  if constexpr (KIND == kGradWeights) {
    nk = 0;
    for (int s = 0; s < S; ++s) nk += (p.offsets[s * p.E + e + 1] - p.offsets[s * p.E + e] + kBK - 1) / kBK;
    nk = uniform(nk);
  } else {
    nk = (KIND == kGradRows0 ? 2 : 1) * (K / kBK);
  }
  const int per = K / kBK;
  // steps are asked for in order, once each; past the last one it stays
  auto source = [&](int kt) {
    if constexpr (KIND == kGradWeights) {
      if (kt < nk) {
        r += kBK;
        while (r >= rend) {
          r = uniform(p.offsets[sb * p.E + e]);
          rend = uniform(p.offsets[sb * p.E + e + 1]);
          ++sb;
        }
        const uint32_t n = (uint32_t)min(rend - r, kBK);
        rw = make_rsrc((const __bf16*)p.x + (int64_t)r * N + col0, n * wpitch - (uint32_t)col0 * 2u);
        rx = make_rsrc(d + (int64_t)r * DN + row0, n * xpitch - (uint32_t)row0 * 2u);
      }
    } else {
      kt = min(kt, nk - 1);
      const bool second = KIND == kGradRows0 && kt >= per;
      const int kk = second ? kt - per : kt;
      const __bf16* w = (const __bf16*)(second ? p.w1 : p.w0) + (int64_t)e * K * N;
      rw = make_rsrc(w + (int64_t)kk * kBK * N + col0, (uint32_t)kBK * wpitch - (uint32_t)col0 * 2u);
      rx = make_rsrc(second ? p.d1 : p.d0, (uint32_t)(p.R * (int64_t)xpitch));
      xs = (uint32_t)kk * (kBK * 2);
    }
  };

  // ---- global -> register loads.  [k][columns]: thread owns 16-byte chunk
  // tid & 31 of k rows (tid >> 5) + 8 i; [rows][k]: chunk tid & 7 of rows
  // (tid >> 3) + 32 i
  const int cr = tid >> 5, cc = tid & 31;
  const uint32_t wvoff = (uint32_t)cr * wpitch + (uint32_t)cc * 16u, wstep = 8u * wpitch;
  uint32_t xvoff[XKC ? XI : 1], xstep = 8u * xpitch;
  if constexpr (XKC) {
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int pos = rowpos[(tid >> 3) + 32 * i];
      // a row that the tile lacks: past the range, or (buffers over 2 GiB) another row, whose sums are not stored
      xvoff[i] = pos >= 0 ? (uint32_t)pos * xpitch + (uint32_t)(tid & 7) * 16u : 0x80000000u;
    }
  } else {
    xvoff[0] = (uint32_t)cr * xpitch + (uint32_t)cc * 16u;
  }
  const uint32_t st_kr = (uint32_t)cr * 512u + ((uint32_t)(cc ^ ((cr & 3) << 2)) << 4);
  const int lr = tid >> 3;
  const uint32_t st_kc = (uint32_t)lr * 128u + ((uint32_t)((tid & 7) ^ (lr & 7) ^ ((lr >> 3) & 1)) << 4);

  i32x4_t wreg[8], xreg[XI];
  auto gload_one = [&](int q, int j) {
    if (j < 2) {
      const int i = 2 * q + j;
      wreg[i] = buf_load16(rw, wvoff + (uint32_t)i * wstep, 0);
    } else {
      const int i = q * XQ + j - 2;
      if constexpr (XKC)
        xreg[i] = buf_load16(rx, xvoff[i], xs);
      else
        xreg[i] = buf_load16(rx, xvoff[0] + (uint32_t)i * xstep, 0);
    }
  };
  auto lstore_one = [&](int stage, int q, int j) {
    char* wdst = lds + stage * kStageBytes;
    if (j < 2) {
      const int i = 2 * q + j;
      *reinterpret_cast<i32x4_t*>(wdst + st_kr + i * 4096) = wreg[i];
    } else {
      const int i = q * XQ + j - 2;
      *reinterpret_cast<i32x4_t*>(wdst + kOperandBytes + (XKC ? st_kc : st_kr) + i * 4096) = xreg[i];
    }
  };

  // ---- fragment addressing
  const int lrow = lane & 31, lk = lane >> 5;
  uint32_t wrd[4], xrd[4];
  {
    // lane's 16-lane group: columns 16 (g & 1), k rows 8 (g >> 1); in it, row l >> 2, 8-byte piece l & 3
    const int g = lane >> 4, l = lane & 15, lq = l >> 2;
    const uint32_t base = (uint32_t)(8 * (g >> 1) + lq) * 512u + (uint32_t)(g & 1) * 32u + (uint32_t)(l & 3) * 8u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wrd[i] = base + (uint32_t)(wn * 8 + ((i ^ lq) << 1)) * 32u;
      if constexpr (XKC)  // sub-step i of the wave's rows
        xrd[i] = (uint32_t)(kOperandBytes + (wm * (TM / 2) + lrow) * 128) +
                 (uint32_t)(((2 * i + lk) ^ (lrow & 7) ^ ((lrow >> 3) & 1)) << 4);
      else
        xrd[i] = (uint32_t)kOperandBytes + base + (uint32_t)(wm * 8 + ((i ^ lq) << 1)) * 32u;
    }
  }
  lds_byte* l3 = (lds_byte*)lds;
  bf16x4_t fa[2][4][2];
  bf16x4_t fx4[2][XKC ? 1 : NJ][2];
  bf16x8_t fx8[2][XKC ? NJ : 1];
  auto read_tr = [&](uint32_t at, int stage, int ks, int h) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (lds_bf16x4*)(l3 + stage * kStageBytes + at + (uint32_t)(ks * 16 + 4 * h) * 512u));
  };
  // read j of sub-step ks, in the order the matrix instructions use them: column fragment 0, the row fragments, columns 1..3
  auto read_one = [&](int set, int stage, int ks, int j) {
    if (j < 2) {
      fa[set][0][j] = read_tr(wrd[0], stage, ks, j);
    } else if (j < 2 + NRX) {
      if constexpr (XKC)
        fx8[set][j - 2] = *reinterpret_cast<const bf16x8_t*>(lds + stage * kStageBytes + xrd[ks] + (j - 2) * 4096);
      else
        fx4[set][(j - 2) / 2][j & 1] = read_tr(xrd[(j - 2) / 2], stage, ks, j & 1);
    } else {
      const int i = j - NRX;
      fa[set][i / 2][i & 1] = read_tr(wrd[i / 2], stage, ks, i & 1);
    }
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
      for (int nj = 0; nj < NJ; ++nj) {
        const bf16x8_t a = __builtin_shufflevector(fa[set][mi][0], fa[set][mi][1], 0, 1, 2, 3, 4, 5, 6, 7);
        bf16x8_t b;
        if constexpr (XKC)
          b = fx8[set][nj];
        else
          b = __builtin_shufflevector(fx4[set][nj][0], fx4[set][nj][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[mi][nj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[mi][nj], 0, 0, 0);
      }
  };

  if (nk > 0) {
    // prologue: step 0 into LDS, step 1 into registers, fragments of (0, 0)
    if constexpr (KIND == kGradWeights) r = -kBK;
    source(0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < NW; ++j) gload_one(q, j);
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

  // ---- epilogue, staged through LDS (free after the loop's last barrier, as
  // in bf16_gemm_tile) so that each wave stores whole row segments.  Lane
  // (lrow, lk) holds, per row fragment nj and column fragment mi, the 4-column
  // groups 8 q + 4 lk of row wm TM/2 + 32 nj + lrow.
  char* stg = lds;
  if constexpr (KIND == kGradRows0) {
    // 512 B per staged row (256 bf16); 8-byte unit u of row t at u ^ (t & 31)
#pragma unroll
    for (int nj = 0; nj < NJ; ++nj) {
      const int tr = wm * (TM / 2) + nj * 32 + lrow;
#pragma unroll
      for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bf16x4_t h;
#pragma unroll
          for (int v = 0; v < 4; ++v) h[v] = (__bf16)acc[mi][nj][4 * q + v];
          const int u = wn * 32 + mi * 8 + 2 * q + lk;
          *reinterpret_cast<bf16x4_t*>(stg + tr * 512 + ((u ^ (tr & 31)) << 3)) = h;
        }
    }
    __syncthreads();
    const int c = tid & 31, n = col0 + 8 * c;
#pragma unroll 4
    for (int tr = tid >> 5; tr < TM; tr += kGemmThreads / 32) {
      i32x4_t v = *reinterpret_cast<const i32x4_t*>(stg + tr * 512 + ((c ^ ((tr & 31) >> 1)) << 4));
      if (tr & 1) v = i32x4_t{v[2], v[3], v[0], v[1]};
      const int pos = rowpos[tr];
      if (pos >= 0 && n < N) *reinterpret_cast<i32x4_t*>((__bf16*)p.o0 + (int64_t)pos * N + n) = v;
    }
    __syncthreads();
  } else {
    // passes of 128 rows, 1 KiB per staged row (256 f32); 16-byte unit u of staged row t' at u ^ (t' & 15)
    constexpr int passes = NJ / 2;
#pragma unroll
    for (int P = 0; P < passes; ++P) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ts = wm * 64 + j * 32 + lrow;
#pragma unroll
        for (int mi = 0; mi < 4; ++mi)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4_t o;
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = acc[mi][2 * P + j][4 * q + v];
            const int u = wn * 32 + mi * 8 + 2 * q + lk;
            *reinterpret_cast<f32x4_t*>(stg + ts * 1024 + ((u ^ (ts & 15)) << 4)) = o;
          }
      }
      __syncthreads();
      if constexpr (KIND == kGradRows1) {
        // 32 threads per row, 8 columns each
        const int c = tid & 31, n = col0 + 8 * c;
#pragma unroll 4
        for (int ts = tid >> 5; ts < 128; ts += kGemmThreads / 32) {
          const int pos = rowpos[(ts >> 6) * (TM / 2) + 64 * P + (ts & 63)];
          if (pos < 0 || n >= N) continue;
          const int64_t at = (int64_t)pos * N + n;
          const bf16x8_t g = *reinterpret_cast<const bf16x8_t*>((const __bf16*)p.gate + at);
          const bf16x8_t u = *reinterpret_cast<const bf16x8_t*>((const __bf16*)p.up + at);
          bf16x8_t og, ou;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4_t dh = *reinterpret_cast<const f32x4_t*>(stg + ts * 1024 + (((2 * c + h) ^ (ts & 15)) << 4));
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const SwigluGrad s = swiglu_grad_fast(dh[v], (float)g[4 * h + v], (float)u[4 * h + v]);
              og[4 * h + v] = (__bf16)s.dg;
              ou[4 * h + v] = (__bf16)s.du;
            }
          }
          *reinterpret_cast<bf16x8_t*>((__bf16*)p.o0 + at) = og;
          *reinterpret_cast<bf16x8_t*>((__bf16*)p.o1 + at) = ou;
        }
      } else {
        void* out = t.second ? p.o1 : p.o0;
        const int c = tid & 63, n = col0 + 4 * c;
#pragma unroll 4
        for (int ts = tid >> 6; ts < 128; ts += kGemmThreads / 64) {
          const f32x4_t v = *reinterpret_cast<const f32x4_t*>(stg + ts * 1024 + ((c ^ (ts & 15)) << 4));
          const int row = row0 + (ts >> 6) * (TM / 2) + 64 * P + (ts & 63);
          if (row >= DN || n >= N) continue;
          const int64_t at = ((int64_t)e * DN + row) * N + n;
          if (p.out_bf16) {
            bf16x4_t b;
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = (__bf16)v[i];
            *reinterpret_cast<bf16x4_t*>((__bf16*)out + at) = b;
          } else {
            f32x4_t* dst = reinterpret_cast<f32x4_t*>((float*)out + at);
            *dst = p.accumulate ? *dst + v : v;
          }
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace moe
