// Gradients of the experts' products (grouped GEMM), rows and weights.
//
// "Grouped GEMM 为什么适合 MoE" (C_i = A_i B_i per expert) transposed: with the
// forward g = X Wg^T, u = X Wu^T, h = silu(g) u, Y = h Wd^T per expert,
//   rows, layer 1     dh = dY Wd;  s = 1 / (1 + e^-g);
//                     dg = dh u s (1 + g (1 - s)),  du = dh g s
//   rows, layer 0     dX = dg Wg + du Wu
//   weights, layer 1  dWd = dY^T h
//   weights, layer 0  dWg = dg^T X,  dWu = du^T X   (the sums run over rows)
// A static tile queue as in the forward grouped GEMM; each output element's sum is
// formed in a fixed order, so nothing depends on scheduling.  Three sets of tiles,
// by size: 256 x 256 (bf16), 64 or 128 square through common LDS buffers (f32), and
// 32 x 32 with the waves sharing the reduction (small problems).
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

// ------------------------------------------------------------------- split ---
// The grid's last round (or only one) of r tiles is cut along K into s units
// each, at most one a workgroup, where that is shorter: in microseconds, a K
// step (bf16 64, f32 128 terms) takes `step` with few workgroups at work and
// step + more with all, storing a unit's sums and reading them once more `store`
// of the whole card's bandwidth, the second kernel 6.  Measured (whole, split):
// layer 0's rows, 60 of 448 x 8576, one expert, 2 tiles of 268 steps: 178, 36 us.
// A weights' step, both operands read turned and none shared by many workgroups,
// takes longer: 8 experts 256 x 512, 32768 rows: 121, 57 (with the rows' cost 65);
// layer 1 of one 576 x 4224, 3311 rows, 51 tiles of 52 steps: 77, 48 (62).
struct SplitCost {
  float step, more, store;
};
constexpr SplitCost kSplitBf16{0.65f, 0.75f, 0.1f};
constexpr SplitCost kSplitWeights{1.5f, 0.4f, 0.06f};
constexpr SplitCost kSplitF32{2.0f, 0.0f, 0.01f};
__host__ __device__ inline int split_parts(const SplitCost& c, int r, int nk, int grid) {
  if (r <= 0) return 1;
  int best = 1;
  float least = 0.f;
  const int most = nk / 2 < grid / r ? nk / 2 : grid / r;
  for (int s = 1; s <= most; s += 1 + s / 8) {  // 1 .. 8, 10, 12, ...
    const float units = (float)(r * s);
    const float t = (float)((nk + s - 1) / s) * (c.step + c.more * units / (float)grid) + (s > 1 ? c.store * units + 6.0f : 0.0f);
    if (s == 1 || t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}
// ... as far as the workspace's units reach (they do for the rows that the offsets of this problem can have).
__device__ __forceinline__ int split_within(const GradGemmArgs& a, int s, int r) { return r * s <= a.split.units ? s : 1; }

// Whether an f32 product takes tiles of 128 x 128 (tiles: how many there are)
// with two groups of waves: from eight rounds of the CUs on, where their padding
// and the last round's idle CUs weigh little; below, tiles of 64 x 64.  Measured
// (128; 64, one group): layer 0's weights of 4 experts 2048 x 4096, 2048 rows each:
// 2.49, 2.57 ms; rows of layer 1, 8 of 2048 x 8192, 1024 each: 2.93, 3.01, 8 of 512
// x 2048, 4096 each: 0.97, 0.93; 64 with four groups, rows of 8 experts 2048 x 4096,
// 256 each, one round of 128: 1.24, 0.80.
static bool wide_f32(int64_t tiles, int cus) { return tiles >= 8 * cus; }

// A split tile's description for the second kernel.
struct GradDesc {
  int e, row0, col0, second, tm, rows, steps;
};
__device__ __forceinline__ void put_desc(const GradGemmArgs& a, int j, const GradDesc& d) {
  int32_t* o = a.split.desc + (int64_t)j * kGradDescInts;
  o[0] = d.e;
  o[1] = d.row0;
  o[2] = d.col0;
  o[3] = d.second;
  o[4] = d.tm;
  o[5] = d.rows;
  o[6] = d.steps;
}

// ------------------------------------------------------------------- bf16 ---
// Rows, and the forward products that are kept: the experts' rows (over all
// source blocks) in tiles of 256, or of 128 where an expert has no more and in a
// last round that would leave half the workgroups idle, in the forward queue's
// order.
template <GradKind KIND>
__global__ __launch_bounds__(kGemmThreads) void grad_rows_bf16_kernel(GradGemmArgs a, int xcd_slots) {
  __shared__ __attribute__((aligned(16))) char lds[kGemmLdsBytes];
  __shared__ TileLds tl;
  __shared__ int rowpos[2][kTileRows];  // of this tile and of the next
  constexpr int TC = KIND == kKeep ? 128 : 256;  // columns of a tile
  const int K = KIND == kGradRows0 ? a.F : a.H, N = KIND == kGradRows0 ? a.H : a.F, S = a.G / a.E;
  const int NT = (N + TC - 1) / TC;
  const int T = build_expert_tile_table(a.offsets, a.G, a.E, kTileRows, tl, (int)a.R) * NT;
  const int64_t panel = (int64_t)kTileRows * K * (KIND == kGradRows0 ? 4 : 2);
  const int grid = gridDim.x;
  // the last round's r tiles: split along K, or cut into two halves of 128 rows, or neither
  const int r = T % grid, steps = (KIND == kGradRows0 ? 2 : 1) * (K / kBK);
  const int s = a.split.hdr ? split_within(a, split_parts(kSplitBf16, r, steps, grid), r) : 1;
  const int cut = s > 1 ? s : (r > 0 && 2 * r <= grid && T > grid) ? 2 : 1;
  const int whole = cut > 1 ? T - r : T, entries = whole + (cut > 1 && s == 1 ? 2 * r : 0);
  const Shuffle sm = make_shuffle(a.shuffle, whole), sh = make_shuffle(a.shuffle, T - whole);
  if (a.split.hdr && blockIdx.x == 0 && threadIdx.x == 0) {
    a.split.hdr[0] = s > 1 ? r : 0;
    a.split.hdr[1] = s;
  }
  GradTile t{};
  bool low = false;  // 128 rows
  // Entry v or the next one of this workgroup that has rows; its rows' positions into rowpos[b].
  auto find = [&](int v, int b) {
    for (; v < entries; v += grid) {
      const int u = v - whole;  // from 0 on: halves
      const TileCoord c = tile_coord(u >= 0 ? whole + shuffled(sh, u / 2) : shuffled(sm, v), a.E, NT, kTileRows, xcd_slots,
                                     panel, tl);
      const int m0 = u >= 0 ? c.m0 + (u & 1) * (kTileRows / 2) : c.m0;
      const int n = tl.expert_rows[c.g];
      if (m0 >= n) continue;
      rowpos[b][threadIdx.x] = expert_row(tl, c.g, a.E, S, m0, threadIdx.x);
      t = {uniform(c.g), 0, uniform(c.nt) * TC, 0, 0, 1};
      low = uniform(u >= 0 || n <= kTileRows / 2);
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
  if constexpr (KIND == kKeep) return;  // (no workspace)
  // a unit of a split tile (a copy of the K loop of its own: with store_part beside the epilogue in one, the compiler
  // spills up to 130 registers a tile)
  const int slot = xcd_slot(blockIdx.x, grid), mine = slot - whole % grid + (slot < whole % grid ? grid : 0);
  if (s == 1 || mine >= r * s) return;
  const int j = mine / s, part = mine - j * s;
  const TileCoord c = tile_coord(whole + shuffled(sh, j), a.E, NT, kTileRows, xcd_slots, panel, tl);
  const int n = tl.expert_rows[c.g], pos = expert_row(tl, c.g, a.E, S, c.m0, threadIdx.x);
  low = uniform(n <= kTileRows / 2);
  t = {uniform(c.g), 0, uniform(c.nt) * 256, 0, part, s};
  __syncthreads();
  rowpos[0][threadIdx.x] = pos;
  if (part == 0) {
    if (threadIdx.x == 0) put_desc(a, j, {t.e, 0, t.col0, 0, low ? 128 : 256, min(n - c.m0, kTileRows), steps});
    a.split.desc[(int64_t)j * kGradDescInts + 8 + threadIdx.x] = pos;
  }
  __syncthreads();
  auto unit = [&]<int TM>() {
    GradWave<KIND, TM> wave(a, lds, nullptr);
    wave.begin(t, rowpos[0]);
    wave.multiply();
    wave.store_part(mine);
  };
  if (low)
    unit.template operator()<kTileRows / 2>();
  else
    unit.template operator()<kTileRows>();
}

// Weights: 256 x 256 tiles of dW, expert by expert; the row tiles (layer 0:
// of both matrices, which share x's panels) in blocks of 8, so that the 32
// tiles an XCD runs at once share 8 + 4 panels in its L2.
__global__ __launch_bounds__(kGemmThreads) void grad_weights_bf16_kernel(GradGemmArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[kGemmLdsBytes];
  __shared__ int offsets[kMaxTileSegs + 1];
  // (kept inside the rows, so that even bad ones read nothing else)
  for (int i = threadIdx.x; i <= a.G; i += kGemmThreads) offsets[i] = min(max(a.offsets[i], 0), (int)a.R);
  const bool l0 = a.layer == 0;
  const int N = l0 ? a.F : a.H, C = l0 ? a.H : a.F;
  const int NR = (N + 255) / 256, NC = (C + 255) / 256, rows = (l0 ? 2 : 1) * NR;
  const int T = a.E * rows * NC, grid = gridDim.x;
  const int r = T % grid;
  int s = 1;
  __syncthreads();
  if (a.split.hdr) {
    // steps: the experts' mean
    s = split_within(a, split_parts(kSplitWeights, r, (offsets[a.G] + a.fill + a.E * kBK - 1) / (a.E * kBK), grid), r);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.split.hdr[0] = s > 1 ? r : 0;
      a.split.hdr[1] = s;
    }
  }
  const int whole = s > 1 ? T - r : T;
  const Shuffle sm = make_shuffle(a.shuffle, whole), sh = make_shuffle(a.shuffle, T - whole);
  // tile n of the order
  auto tile = [&](int n) {
    const int e = n / (rows * NC), l = n - e * rows * NC;
    const int nb = (rows + 7) / 8, b = min((int)((int64_t)(l / NC) * nb / rows), nb - 1);
    auto first = [&](int i) { return (int)((int64_t)i * rows / nb); };
    const int bb = first(b + 1) <= l / NC ? b + 1 : b;
    const int r0 = first(bb), rb = first(bb + 1) - r0, lb = l - r0 * NC;
    const int row = r0 + lb % rb, second = row >= NR;
    return GradTile{e, (row - second * NR) * 256, lb / rb * 256, second, 0, 1};
  };
  const int slot = xcd_slot(blockIdx.x, grid);
  int v = slot;
  if (v < whole) {
    GradWave<kGradWeights, kTileRows> wave(a, lds, offsets);
    GradTile t = tile(shuffled(sm, v));
    wave.begin(t, nullptr);
    while (true) {
      wave.multiply();
      v += grid;
      const GradTile now = t;
      if (v < whole) {
        t = tile(shuffled(sm, v));
        wave.begin(t, nullptr);
      }
      wave.epilogue(now, nullptr);
      if (v >= whole) break;
    }
  }
  // a unit of a split tile
  const int mine = slot - whole % grid + (slot < whole % grid ? grid : 0);
  if (s == 1 || mine >= r * s) return;
  const int j = mine / s;
  GradTile t = tile(whole + shuffled(sh, j));
  t.part = mine - j * s;
  t.parts = s;
  if (t.part == 0 && threadIdx.x == 0)
    put_desc(a, j, {t.e, t.row0, t.col0, t.second, 256, min(N - t.row0, 256), weight_steps(a, offsets, t.e)});
  GradWave<kGradWeights, kTileRows> wave(a, lds, offsets);
  wave.begin(t, nullptr);
  wave.multiply();
  wave.store_part(mine);
}

// Second kernel of a split: a wave per fragment of 32 x 32 outputs adds the
// parts' sums (in order, from the first) and stores what the tile's epilogue
// would.  The lanes hold what they held in the tile: row lane % 32, columns 8 q
// + 4 (lane / 32).  T is the products' type: it fixes the tiles' width (256, 64)
// and the fragments of a wave (16 places in bf16, 1).
template <GradKind KIND, typename T>
__global__ __launch_bounds__(256) void grad_reduce_kernel(GradGemmArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int TC = F32 ? 64 : 256, FW = F32 ? 1 : 16, MI = TC / 64;
  const int tiles = a.split.hdr[0], parts = a.split.hdr[1];
  const int lane = threadIdx.x & 63, lrow = lane & 31, lk = lane >> 5;
  const bool l0 = KIND == kGradRows0 || (KIND == kGradWeights && a.layer == 0);
  const int N = KIND == kGradRows1 ? a.F : KIND == kGradRows0 ? a.H : (l0 ? a.H : a.F);
  const int DN = l0 ? a.F : a.H;
  for (int item = blockIdx.x * 4 + (threadIdx.x >> 6); item < tiles * 4 * FW; item += gridDim.x * 4) {
    const int j = item / (4 * FW), wave = item / FW % 4, f = item % FW;
    const int32_t* desc = a.split.desc + (int64_t)j * kGradDescInts;
    const int e = desc[0], row0 = desc[1], col0 = desc[2], second = desc[3], tm = desc[4], rows = desc[5], nk = desc[6];
    const int NJ = tm / 64, mi = f / NJ, nj = f - mi * NJ;
    if (mi >= MI) continue;
    const int row = (wave >> 1) * (tm / 2) + nj * 32, n0 = col0 + (wave & 1) * (TC / 2) + mi * 32 + 4 * lk;
    if (row >= rows || n0 - 4 * lk >= N) continue;
    const f32x4_t* src = reinterpret_cast<const f32x4_t*>(a.split.part) + (((int64_t)j * parts * 4 + wave) * FW + f) * 4 * 64 + lane;
    constexpr int64_t kUnit = 4 * FW * 4 * 64;
    f32x4_t sum[4] = {};
    for (int i = 0; i < parts; i += 4) {
      f32x4_t v[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool has = i + u < parts && part_begin(nk, i + u + 1, parts) > part_begin(nk, i + u, parts);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[u][q] = has ? src[(i + u) * kUnit + q * 64] : f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] += v[u][q];
    }
    if constexpr (KIND == kGradWeights) {
      if (row + lrow >= rows) continue;
      void* const out = second ? a.o1 : a.o0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 8 * q;
        if (n >= N) continue;
        const int64_t at = ((int64_t)e * DN + row0 + row + lrow) * N + n;
        if (a.out_bf16) {
          gf_store4((__bf16*)out + at, sum[q]);
        } else {
          float* p = (float*)out + at;
          gf_store4(p, a.accumulate ? *(const f32x4_t*)p + sum[q] : sum[q]);
        }
      }
    } else {
      const int pos = desc[8 + row + lrow];
      if (pos < 0) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 8 * q;
        if (n >= N) continue;
        const int64_t at = (int64_t)pos * N + n;
        if constexpr (KIND == kGradRows0) {
          gf_store4((T*)a.o0 + at, sum[q]);
        } else {
          typedef T T4 __attribute__((ext_vector_type(4)));
          const T4 g = *(const T4*)((const T*)a.gate + at), u = *(const T4*)((const T*)a.up + at);
          f32x4_t og, ou;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const SwigluGrad d = F32 ? swiglu_grad(sum[q][v], (float)g[v], (float)u[v])
                                     : swiglu_grad_fast(sum[q][v], (float)g[v], (float)u[v]);
            og[v] = d.dg;
            ou[v] = d.du;
          }
          gf_store4((T*)a.o0 + at, og);
          gf_store4((T*)a.o1 + at, ou);
        }
      }
    }
  }
}

template <GradKind KIND, typename T>
hipError_t grad_reduce_launch(const GradGemmArgs& a, hipStream_t s) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.split.hdr) return e;
  grad_reduce_kernel<KIND, T><<<4 * device_cu_count(), 256, 0, s>>>(a);
  return hipGetLastError();
}

// -------------------------------------------------------------------- f32 ---
// Rows (KIND) as the bf16 kernel above, tiles of TX x TX.
template <GradKind KIND, int TX, int KG>
__global__ __launch_bounds__(256 * KG) void grad_rows_f32_kernel(GradGemmArgs a) {
  typedef GfTile<TX, TX, KG> Tile;
  __shared__ __attribute__((aligned(16))) float lds[Tile::kLds];
  __shared__ TileLds tl;
  __shared__ int rowpos[TX];
  const int K = KIND == kGradRows0 ? a.F : a.H, N = KIND == kGradRows0 ? a.H : a.F;  // reduction and columns of a product
  const int NT = (N + TX - 1) / TX, S = a.G / a.E, grid = gridDim.x;
  const int T = build_expert_tile_table(a.offsets, a.G, a.E, TX, tl, (int)a.R) * NT;
  const int per = K / kGfK, steps = KIND == kGradRows0 ? 2 * per : per;
  const int r = T % grid, s = a.split.hdr ? split_within(a, split_parts(kSplitF32, r, steps / KG, grid), r) : 1;
  const int whole = s > 1 ? T - r : T, entries = whole + (s > 1 ? r * s : 0);
  const Shuffle sm = make_shuffle(a.shuffle, whole), sh = make_shuffle(a.shuffle, T - whole);
  if (a.split.hdr && blockIdx.x == 0 && threadIdx.x == 0) {
    a.split.hdr[0] = s > 1 ? r : 0;
    a.split.hdr[1] = s;
  }
  const int i = threadIdx.x & 255, g = threadIdx.x >> 8;
  for (int v = blockIdx.x; v < entries; v += grid) {
    const int u = v - whole, j = u / s, part = u >= 0 ? u - j * s : 0, parts = u >= 0 ? s : 1;
    const TileCoord c = tile_coord(u >= 0 ? whole + shuffled(sh, j) : shuffled(sm, v), a.E, NT, TX, 1, 0, tl);
    const int e = c.g, col0 = c.nt * TX;
    if (threadIdx.x < TX) {
      const int pos = expert_row(tl, e, a.E, S, c.m0, threadIdx.x);
      rowpos[threadIdx.x] = pos;
      if (u >= 0 && part == 0) a.split.desc[(int64_t)j * kGradDescInts + 8 + threadIdx.x] = pos;
    }
    if (u >= 0 && part == 0 && threadIdx.x == 0)
      put_desc(a, j, {e, 0, col0, 0, TX, min(tl.expert_rows[e] - c.m0, TX), steps});
    __syncthreads();
    const float* rows0[TX / 32];
    const float* rows1[TX / 32];
#pragma unroll
    for (int h = 0; h < TX / 32; ++h) {
      const int pos = rowpos[(i >> 3) + 32 * h];
      rows0[h] = pos >= 0 ? (const float*)a.d0 + (int64_t)pos * K : nullptr;
      rows1[h] = KIND == kGradRows0 && pos >= 0 ? (const float*)a.d1 + (int64_t)pos * K : nullptr;
    }
    const float* w0 = (const float*)a.w0 + (int64_t)e * K * N;
    const float* w1 = KIND == kGradRows0 ? (const float*)a.w1 + (int64_t)e * K * N : nullptr;
    // the unit's steps, and of them this group's
    const int k0 = part_begin(steps, part, parts), n = part_begin(steps, part + 1, parts) - k0;
    const int b = k0 + part_begin(n, g, KG), end = k0 + part_begin(n, g + 1, KG);
    GfPart<TX> pw, px;
    auto load = [&](int at) {
      const int st = b + at;
      const bool second = KIND == kGradRows0 && st >= per;
      const int k = (second ? st - per : st) * kGfK;
      px.load_k(second ? rows1 : rows0, k, i);
      pw.load_c((second ? w1 : w0) + (int64_t)k * N, N, kGfK, col0, N, i);
    };
    Tile tile;
    tile.run(lds, end - b, (n + KG - 1) / KG, load, [&](float* l) { px.store_k(l, i); }, [&](float* l) { pw.store_c(l, i); });
    tile.each(lds, [&](int fj, int q, f32x4_t (&o)[Tile::MI]) {
      if (u >= 0) {
        if constexpr (Tile::MI == 1)
          reinterpret_cast<f32x4_t*>(a.split.part)[(((int64_t)u * 4 + (i >> 6)) * 4 + q) * 64 + (i & 63)] = o[0];
        return;
      }
      const int pos = rowpos[Tile::row(fj)];
      if (pos < 0) return;
#pragma unroll
      for (int m = 0; m < Tile::MI; ++m) {
        const int col = col0 + Tile::col(m, q);
        if (col >= N) continue;
        const int64_t at = (int64_t)pos * N + col;
        if constexpr (KIND == kGradRows0) {
          gf_store4((float*)a.o0 + at, o[m]);
        } else {
          const f32x4_t gv = *(const f32x4_t*)((const float*)a.gate + at), uv = *(const f32x4_t*)((const float*)a.up + at);
          f32x4_t dg, du;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const SwigluGrad d = swiglu_grad(o[m][h], gv[h], uv[h]);
            dg[h] = d.dg;
            du[h] = d.du;
          }
          gf_store4((float*)a.o0 + at, dg);
          gf_store4((float*)a.o1 + at, du);
        }
      }
    });
    __syncthreads();  // rowpos and the buffers are free for the next tile
  }
}

// Weights: tiles of dW[e], TX of the first operand's columns (its rows) x TX of
// x's.  The K steps run over the expert's segments one after the other, the
// last step of each filled up with zero rows.
template <int TX, int KG>
__global__ __launch_bounds__(256 * KG) void grad_weights_f32_kernel(GradGemmArgs a) {
  typedef GfTile<TX, TX, KG> Tile;
  __shared__ __attribute__((aligned(16))) float lds[Tile::kLds];
  __shared__ int offsets[kMaxTileSegs + 1];
  for (int h = threadIdx.x; h <= a.G; h += 256 * KG) offsets[h] = min(max(a.offsets[h], 0), (int)a.R);
  __syncthreads();
  const bool l0 = a.layer == 0;
  const int N = l0 ? a.F : a.H, C = l0 ? a.H : a.F;  // rows and columns of dW
  const int NR = (N + TX - 1) / TX, NC = (C + TX - 1) / TX, S = a.G / a.E, mats = l0 ? 2 : 1, grid = gridDim.x;
  const int T = a.E * mats * NR * NC;
  const int r = T % grid, mean = (offsets[a.G] + a.fill + a.E * kGfK - 1) / (a.E * kGfK);
  const int s = a.split.hdr ? split_within(a, split_parts(kSplitF32, r, mean / KG, grid), r) : 1;
  const int whole = s > 1 ? T - r : T, entries = whole + (s > 1 ? r * s : 0);
  const Shuffle sm = make_shuffle(a.shuffle, whole), sh = make_shuffle(a.shuffle, T - whole);
  if (a.split.hdr && blockIdx.x == 0 && threadIdx.x == 0) {
    a.split.hdr[0] = s > 1 ? r : 0;
    a.split.hdr[1] = s;
  }
  const int i = threadIdx.x & 255, g = threadIdx.x >> 8;
  for (int v = blockIdx.x; v < entries; v += grid) {
    const int u = v - whole, j = u / s, part = u >= 0 ? u - j * s : 0, parts = u >= 0 ? s : 1;
    int l = u >= 0 ? whole + shuffled(sh, j) : shuffled(sm, v);
    const int e = l / (mats * NR * NC);
    l -= e * mats * NR * NC;
    const int m = l / (NR * NC);
    l -= m * NR * NC;
    const int row0 = l % NR * TX, col0 = l / NR * TX;
    int steps = 0;
    for (int h = 0; h < S; ++h) steps += (offsets[h * a.E + e + 1] - offsets[h * a.E + e] + kGfK - 1) / kGfK;
    if (u >= 0 && part == 0 && threadIdx.x == 0) put_desc(a, j, {e, row0, col0, m, TX, min(N - row0, TX), steps});
    const int k0 = part_begin(steps, part, parts), n = part_begin(steps, part + 1, parts) - k0;
    const int b = k0 + part_begin(n, g, KG), end = k0 + part_begin(n, g + 1, KG);
    const float* d = (const float*)(m ? a.d1 : a.d0);
    int row = 0, rend = 0, sb = 0;  // the step before b: its row, the segment's end, the next source block
    for (int left = b;;) {
      const int have = (rend - row + kGfK - 1) / kGfK;
      if (left <= have || sb == S) {
        row += (left - 1) * kGfK;
        break;
      }
      left -= have;
      row = offsets[sb * a.E + e];
      rend = offsets[sb * a.E + e + 1];
      ++sb;
    }
    GfPart<TX> pw, px;
    auto load = [&](int) {
      row += kGfK;
      while (row >= rend && sb < S) {
        row = offsets[sb * a.E + e];
        rend = offsets[sb * a.E + e + 1];
        ++sb;
      }
      pw.load_c((const float*)a.x + (int64_t)row * C, C, rend - row, col0, C, i);
      px.load_c(d + (int64_t)row * N, N, rend - row, row0, N, i);
    };
    Tile tile;
    tile.run(lds, end - b, (n + KG - 1) / KG, load, [&](float* q) { px.store_c(q, i); }, [&](float* q) { pw.store_c(q, i); });
    void* const out = m ? a.o1 : a.o0;
    tile.each(lds, [&](int fj, int q, f32x4_t (&o)[Tile::MI]) {
      if (u >= 0) {
        if constexpr (Tile::MI == 1)
          reinterpret_cast<f32x4_t*>(a.split.part)[(((int64_t)u * 4 + (i >> 6)) * 4 + q) * 64 + (i & 63)] = o[0];
        return;
      }
      const int dr = row0 + Tile::row(fj);
      if (dr >= N) return;
#pragma unroll
      for (int h = 0; h < Tile::MI; ++h) {
        const int col = col0 + Tile::col(h, q);
        if (col >= C) continue;
        const int64_t at = ((int64_t)e * N + dr) * C + col;
        if (a.out_bf16) {
          gf_store4((__bf16*)out + at, o[h]);
        } else {
          float* p = (float*)out + at;
          gf_store4(p, a.accumulate ? *(const f32x4_t*)p + o[h] : o[h]);
        }
      }
    });
    __syncthreads();
  }
}

// ------------------------------------------------------------ small tiles ---
// bf16, [64 k][32 columns] through a wave's 4 KiB of LDS: rows of 64 bytes as loaded (16-byte chunk lane % 4 of rows
// lane / 4 + 16 i); a group of 16 lanes reads 4 k x 16 columns, each lane ends with a column's 4 k.
__device__ __forceinline__ void turn_k(f32x4_t* mine, const f32x4_t (&v)[4], f32x4_t (&o)[4]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i * 64 + lane] = v[i];
  lds_byte* const at = (lds_byte*)mine + (8 * (g >> 1) + (l >> 2)) * 64 + (g & 1) * 32 + (l & 3) * 8;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(at + u * 1024));
    const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(at + u * 1024 + 256));
    o[u] = __builtin_bit_cast(f32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// The f32 kept products, and kept products and rows' gradients of small problems:
// tiles of 32 rows x 32 columns (keep: of both products), each wave a part of the
// K steps (128 bytes of a row), loaded one ahead, so that there is no barrier
// before the waves' sums are added (in order) in LDS, and the waves of several
// blocks a CU hide each other's latency.  What lies along k (x, and keep's weights)
// is loaded as whole lines (8 lanes a row) and turned by the wave in LDS of its own;
// loaded as the matrix instruction takes it, neighbouring lanes different rows, it
// comes at a third of the rate (f32 keep, 250 tokens, 8 experts 2048 x 640, top 2:
// 53 us, loaded so 74).  The weights of a rows' gradient, [k][columns], lie as the
// f32 instruction takes them; in bf16 they pass through LDS too and are read turned
// (ds_read_b64_tr_b16, as in the large tiles).
template <GradKind KIND, typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void wave_kernel(GradGemmArgs a) {
  constexpr bool KEEP = KIND == kKeep, F32 = sizeof(T) == 4;
  constexpr int NP = KEEP ? 2 : 1;      // products
  constexpr int V = 16 / sizeof(T);     // values of 16 bytes
  constexpr int KS = 8 * V;             // of a K step
  constexpr int kRegion = NP * 256;     // a wave's: 4 KiB for the operands in turn, then NP x 4 KiB of sums
  __shared__ __attribute__((aligned(16))) f32x4_t lds[WAVES][kRegion];
  __shared__ TileLds tl;
  const int K = KIND == kGradRows0 ? a.F : a.H, N = KIND == kGradRows0 ? a.H : a.F, NT = N / 32, S = a.G / a.E;
  const int tiles = build_expert_tile_table(a.offsets, a.G, a.E, 32, tl, (int)a.R) * NT;
  const Shuffle sm = make_shuffle(a.shuffle, tiles);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), lrow = lane & 31, lk = lane >> 5;
  const int lr = lane >> 3, lc = lane & 7;  // of the line loads: rows lr + 8 i, 16-byte chunk lc
  const int per = K / KS, steps = KIND == kGradRows0 ? 2 * per : per;
  const int b = part_begin(steps, wave, WAVES), end = part_begin(steps, wave + 1, WAVES);
  f32x4_t* const mine = lds[wave];
  // 32 rows x 128 bytes: chunk c of row r at c ^ (r % 8).  (A wave's LDS accesses are done in order, and the compiler
  // keeps it, as it cannot tell a lane's places of one from those of the other.)
  auto turn = [&](const f32x4_t (&v)[4], f32x4_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(lr + 8 * i) * 8 + (lc ^ lr)] = v[i];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = mine[lrow * 8 + ((2 * u + lk) ^ (lrow & 7))];
  };
  for (int v = blockIdx.x; v < tiles; v += gridDim.x) {
    const TileCoord c = tile_coord(shuffled(sm, v), a.E, NT, 32, 1, 0, tl);
    const int e = uniform(c.g), n0 = uniform(c.nt) * 32, pos = expert_row(tl, e, a.E, S, c.m0, lrow);
    // lanes' places in the operands (R times a row is below 2^31); a row that the tile lacks: the first one, not stored
    int xat[4], wat[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xat[i] = max(__shfl(pos, lr + 8 * i), 0) * K + V * lc;
      wat[i] = KEEP ? (lr + 8 * i) * K + V * lc : F32 ? 8 * i * N : 16 * i * N;
    }
    const int64_t wbase = KEEP ? ((int64_t)e * N + n0) * K
                               : ((int64_t)e * K + (F32 ? 4 * lk : lane >> 2)) * N + n0 + (F32 ? lrow : 8 * (lane & 3));
    const T* const w0 = (const T*)a.w0 + wbase;
    const T* const w1 = KIND == kGradRows1 ? nullptr : (const T*)a.w1 + wbase;
    f32x4_t xv[4], wv[NP][4], nextx[4], nextw[NP][4];
    auto load = [&](f32x4_t (&ox)[4], f32x4_t (&ow)[NP][4], int s) {
      const bool second = KIND == kGradRows0 && s >= per;
      const int k = (second ? s - per : s) * KS;
      const T* const x = (const T*)(KEEP ? a.x : second ? a.d1 : a.d0) + k;
      const T* const w = (second ? w1 : w0) + (KEEP ? k : (int64_t)k * N);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ox[i] = *reinterpret_cast<const f32x4_t*>(x + xat[i]);
        if constexpr (KEEP || !F32) {
          ow[0][i] = *reinterpret_cast<const f32x4_t*>(w + wat[i]);
          if constexpr (KEEP) ow[1][i] = *reinterpret_cast<const f32x4_t*>(w1 + k + wat[i]);
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) ow[0][i][h] = (w + wat[i])[(int64_t)h * N];
        }
      }
    };
    f32x16_t acc[NP], sum[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m)
#pragma unroll
      for (int h = 0; h < 16; ++h) acc[m][h] = sum[m][h] = 0.f;
    if (b < end) load(xv, wv, b);
    for (int s = b; s < end; ++s) {
      load(nextx, nextw, min(s + 1, end - 1));  // (with a branch here the loads are waited for at once)
      f32x4_t fx[4], fw[NP][4];
      turn(xv, fx);
#pragma unroll
      for (int m = 0; m < NP; ++m) {
        if constexpr (KEEP) {
          turn(wv[m], fw[m]);
        } else if constexpr (!F32) {
          turn_k(mine, wv[m], fw[m]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) fw[m][u] = wv[m][u];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (F32) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int m = 0; m < NP; ++m) acc[m] = __builtin_amdgcn_mfma_f32_32x32x2f32(fw[m][u][h], fx[u][h], acc[m], 0, 0, 0);
        } else {
#pragma unroll
          for (int m = 0; m < NP; ++m)
            acc[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fw[m][u]),
                                                             __builtin_bit_cast(bf16x8_t, fx[u]), acc[m], 0, 0, 0);
        }
      }
      if (F32 ? (s - b) % kGfFlush == kGfFlush - 1 || s + 1 == end : s + 1 == end) {
#pragma unroll
        for (int m = 0; m < NP; ++m) {
          sum[m] += acc[m];
#pragma unroll
          for (int h = 0; h < 16; ++h) acc[m][h] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        xv[u] = nextx[u];
#pragma unroll
        for (int m = 0; m < NP; ++m) wv[m][u] = nextw[m][u];
      }
    }
    const int q = wave, n = n0 + 8 * q + 4 * lk;
    const bool stores = q < 4 && pos >= 0;
    const int64_t at = (int64_t)pos * N + n;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 gv{}, uv{};
    if (KIND == kGradRows1 && stores) {
      gv = *(const T4*)((const T*)a.gate + at);
      uv = *(const T4*)((const T*)a.up + at);
    }
#pragma unroll
    for (int m = 0; m < NP; ++m)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        mine[(m * 4 + h) * 64 + lane] = f32x4_t{sum[m][4 * h], sum[m][4 * h + 1], sum[m][4 * h + 2], sum[m][4 * h + 3]};
    __syncthreads();
    if (stores) {
      f32x4_t o[NP] = {};
#pragma unroll
      for (int m = 0; m < NP; ++m)
#pragma unroll
        for (int w = 0; w < WAVES; ++w) o[m] += lds[w][(m * 4 + q) * 64 + lane];
      if constexpr (KIND == kGradRows0) {
        gf_store4((T*)a.o0 + at, o[0]);
      } else if constexpr (KIND == kGradRows1) {
        f32x4_t dg, du;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const SwigluGrad d = F32 ? swiglu_grad(o[0][u], (float)gv[u], (float)uv[u])
                                   : swiglu_grad_fast(o[0][u], (float)gv[u], (float)uv[u]);
          dg[u] = d.dg;
          du[u] = d.du;
        }
        gf_store4((T*)a.o0 + at, dg);
        gf_store4((T*)a.o1 + at, du);
      } else {
        f32x4_t h;
#pragma unroll
        for (int u = 0; u < 4; ++u) h[u] = F32 ? silu_f32(o[0][u]) * o[NP - 1][u] : silu_mul_fast(o[0][u], o[NP - 1][u]);
        gf_store4((T*)a.o0 + at, o[0]);
        gf_store4((T*)a.o1 + at, o[NP - 1]);
        gf_store4((T*)a.o2 + at, h);
      }
    }
    __syncthreads();  // the sums are read before the next tile's lines
  }
}

// bf16 weights' gradients of small problems: as above, tiles of 32 x 32 of dW, both
// operands [rows][columns].  A K step is 64 rows of a segment of the expert, rows
// past its end zeros.  (In f32 the tiles of 64 are as fast: 256 tokens, 8 experts 256
// x 512: 9.7 us, these 16.)
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void wave_weights_kernel(GradGemmArgs a) {
  constexpr int KS = 64;
  __shared__ __attribute__((aligned(16))) f32x4_t lds[WAVES][256];
  __shared__ int offsets[kMaxTileSegs + 1];
  for (int i = threadIdx.x; i <= a.G; i += 64 * WAVES) offsets[i] = min(max(a.offsets[i], 0), (int)a.R);
  __syncthreads();
  const bool l0 = a.layer == 0;
  const int N = l0 ? a.F : a.H, C = l0 ? a.H : a.F, NR = N / 32, NC = C / 32;  // rows and columns of dW
  const int S = a.G / a.E, mats = l0 ? 2 : 1, tiles = a.E * mats * NR * NC;
  const Shuffle sm = make_shuffle(a.shuffle, tiles);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), lrow = lane & 31, lk = lane >> 5;
  f32x4_t* const mine = lds[wave];
  for (int v = blockIdx.x; v < tiles; v += gridDim.x) {
    int l = shuffled(sm, v);
    const int e = l / (mats * NR * NC);
    l -= e * mats * NR * NC;
    const int m = l / (NR * NC);
    l -= m * NR * NC;
    const int row0 = l % NR * 32, col0 = l / NR * 32;
    int steps = 0;
    for (int h = 0; h < S; ++h) steps += (offsets[h * a.E + e + 1] - offsets[h * a.E + e] + KS - 1) / KS;
    const int b = uniform(part_begin(steps, wave, WAVES)), end = uniform(part_begin(steps, wave + 1, WAVES));
    // the step before b: its row, the segment's end, the next source block
    int row = 0, rend = 0, sb = 0;
    for (int left = b;;) {
      const int have = (rend - row + KS - 1) / KS;
      if (left <= have || sb == S) {
        row += (left - 1) * KS;
        break;
      }
      left -= have;
      row = uniform(offsets[sb * a.E + e]);
      rend = uniform(offsets[sb * a.E + e + 1]);
      ++sb;
    }
    const __bf16* const d = (const __bf16*)(m ? a.d1 : a.d0) + row0;
    const __bf16* const x = (const __bf16*)a.x + col0;
    auto advance = [&] {
      row += KS;
      while (row >= rend && sb < S) {
        row = uniform(offsets[sb * a.E + e]);
        rend = uniform(offsets[sb * a.E + e + 1]);
        ++sb;
      }
    };
    // the step's rows at `row`; those that the segment lacks are its last one, and become zeros
    auto load = [&](f32x4_t (&od)[4], f32x4_t (&ox)[4]) {
      const int64_t r0 = min(row, (int)a.R - 1);
      const int n = max(rend - row, 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = (lane >> 2) + 16 * i, r = min(k, n - 1), c = 8 * (lane & 3);
        const f32x4_t dv = *reinterpret_cast<const f32x4_t*>(d + (r0 + r) * N + c);
        const f32x4_t xv = *reinterpret_cast<const f32x4_t*>(x + (r0 + r) * C + c);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          od[i][h] = k < n ? dv[h] : 0.f;
          ox[i][h] = k < n ? xv[h] : 0.f;
        }
      }
    };
    f32x4_t dv[4], xv[4], nextd[4], nextx[4];
    f32x16_t acc;
#pragma unroll
    for (int h = 0; h < 16; ++h) acc[h] = 0.f;
    if (b < end) {
      advance();
      load(dv, xv);
    }
    for (int s = b; s < end; ++s) {
      if (s + 1 < end) advance();
      load(nextd, nextx);
      f32x4_t fd[4], fx[4];
      turn_k(mine, dv, fd);
      turn_k(mine, xv, fx);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fx[u]),
                                                      __builtin_bit_cast(bf16x8_t, fd[u]), acc, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        dv[u] = nextd[u];
        xv[u] = nextx[u];
      }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) mine[h * 64 + lane] = f32x4_t{acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]};
    __syncthreads();
    if (wave < 4) {
      f32x4_t o{};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) o += lds[w][wave * 64 + lane];
      void* const out = m ? a.o1 : a.o0;
      const int64_t at = ((int64_t)e * N + row0 + lrow) * C + col0 + 8 * wave + 4 * lk;
      if (a.out_bf16) {
        gf_store4((__bf16*)out + at, o);
      } else {
        float* p = (float*)out + at;
        gf_store4(p, a.accumulate ? *(const f32x4_t*)p + o : o);
      }
    }
    __syncthreads();  // the sums are read before the next tile's lines
  }
}

// ------------------------------------------------------------------ launch ---
// How a call splits: the units that its workspace holds (0: no tile is split),
// by sizes that the host knows.  Which tiles a call takes goes by the rows that
// an even routing keeps (a.rows: of a share of the experts its part of all R).
// The number of row tiles of a rows' gradient depends on the routing, between
// `lo` and `hi`; the workspace holds what any routing can need.
struct GradPlan {
  int units = 0;
  bool wide = false;  // f32: tiles of 128
  bool wave = false;  // tiles of 32
  bool many = false;  // f32: tiles of 64, a group of waves each
  size_t unit_bytes = 0;
  size_t bytes() const { return units ? 256 + (size_t)units * (unit_bytes + kGradDescInts * 4) : 0; }
};

// Tiles of 32 x 32 that an even routing gives, N columns wide.
// (A share of the experts taken for half of all pairs, as if it were large, and so:
// kept, 512 tokens, 2 of 8 of 2048 x 1408, top 2: 39.6, 18.4 us; rows of layer 1, 4096, 8
// of 128 of 256 x 512, top 8: 23.7, 12.3; f32, 512, 8 of 64 of 2048 x 1408: 97, 65.)
static int64_t wave_tiles(const GradGemmArgs& a, int N) {
  return (a.rows / 32 + (a.rows < a.E ? a.rows : a.E)) * (N / 32);
}
// f32: the kept products take them always (tiles of 64 x 64 of both products through
// common LDS buffers, these: 256 tokens, 8 experts 256 x 512, top 2: 18.8, 11.9
// us; 1024, 4 of 2048 x 2048, top 1: 293, 204; 4096 tokens there: 874, 714), rows'
// gradients for eight rounds of the CUs and sums of 2048 terms; longer ones are cut
// into parts in the tiles of 64, which also read less.  Measured (tiles of 64,
// these), layer 0: 256 tokens, 8 of 256 x 512, top 2 (192 tiles): 19.8, 11.8; 2000, 8
// of 512 x 512 (2128): 69, 67; 4096, 8 of 2048 x 1024 (16896): 770, 938; 64, 2 of
// 1024 x 4096, top 1 (8192 terms): 37, 57; layer 1: 512, 8 of 256 x 512, top 2 (640):
// 14.4, 12.3; 100, 4 of 4096 x 576, top 1 (4096 terms): 32.9, 31.9.
// bf16: a K step of 64 costs these about 0.2 us a CU (several waves at once) and a
// wave alone 0.9, a tile four steps' time beside; the large tiles cost 15 us and
// more but a fifth a step, and rows' gradients cut the few of them that a small
// problem has into parts.  Measured (large tiles, these) at t tiles a CU and s steps.
// Rows, 8 experts of 512 columns, layer 1: t 1, s 8: 18, 8; 64: 29, 23; 128: 34, 40; t 2.5,
// 16: 34, 19; 32: 31, 30; 64: 38, 53; t 6.5, 8: 29, 18; 32: 59, 45; t 12.5, 8: 30, 28; 16: 39,
// 43; t 16.5, 4: 28, 28; 8: 32, 37; layer 0: t 2.5, 32: 30, 28; 64: 36, 52; t 8.5, 8: 20, 19; 16:
// 28, 28; t 12.5, 8: 20, 23; 128 columns (of fewer than 256 a large tile is partly empty),
// layer 1: t 1, 64: 36, 26; 128: 44, 47; t 4, 32: 54, 31; 64: 56, 55; t 8, 16: 38, 32; 32: 56, 53; t
// 12, 8: 31, 31; 64 experts of 16 rows, layer 0: t 6, 8: 16, 18; t 12, 8: 19, 32; 58 of 6 rows, t
// 9, 4: 22, 17.  So the limits are those of middling problems, and off by up to 40% at
// t 2 to 3 with 64 steps and at t 12 with many experts.
// Kept (no parts, so the large tiles are slow where they are few): 2 experts of 256
// columns, 1024 rows, t 1: s 16: 29, 11; 128: 138, 45; 8 of 512 columns: t 1.5, 64: 65, 37;
// t 2.5, 16: 30, 20; 128: 154, 117; t 4.5, 8: 22, 19; 32: 48, 47; 64: 82, 89; t 6.5, 4: 18, 17; 8: 23,
// 23; 16: 31, 35; t 8.5, 1: 14.9, 14.9; 4: 18, 20; 17 of 3328 columns, 9 rows each, t 8.5, 3: 23, 16; 89 of
// 576, 23 each, t 10.8, 1: 18.5, 15.4; of 128 columns: t 4, 128: 169, 126; t 6, 32: 49, 46; t 8, 16: 32, 36.
static bool wave_rows(const GradGemmArgs& a, bool bf16, int N, int K, int cus) {
  const int64_t tiles = wave_tiles(a, N), steps = K / kBK;
  if (!bf16) return tiles <= 8 * cus && K <= 2048;
  return tiles * (steps + 4) <= (N < 256 ? 256 : 170) * cus && steps <= 192;
}
static bool wave_keep(const GradGemmArgs& a, bool bf16, int cus) {
  const int64_t tiles = wave_tiles(a, a.F), steps = a.H / kBK;
  // up to 4 1/4 tiles a CU whatever the steps, 6 1/4 for few of them or narrow products; more for the fewest
  return !bf16 || 4 * tiles <= (steps <= 8 || a.F < 256 ? 25 : 17) * cus || tiles * (steps + 4) <= 64 * cus;
}
// Up to a tile a CU 8 waves share one, above 4 (8, 4): layer 0's rows above 11.8,
// 13.1 us; 512 tokens there (320 tiles): 20.5, 18.8; kept, 21 rows, one of 2112 x 448:
// 28, 30; 500, 8 of 1024 x 1024: 73, 61.
template <GradKind KIND, typename T>
static hipError_t launch_wave(const GradGemmArgs& g, int N, hipStream_t s) {
  const int cus = device_cu_count();
  if (wave_tiles(g, N) <= cus)
    wave_kernel<KIND, T, 8><<<cus, 512, 0, s>>>(g);
  else  // blocks a CU as registers hold (rows of 2048 tokens above 17 us, with a fourth that waits 19)
    wave_kernel<KIND, T, 4><<<(KIND == kKeep ? 2 : 3) * cus, 256, 0, s>>>(g);
  return hipGetLastError();
}

// f32 tiles of 64 that are many for the CUs are not cut, and one group of waves
// takes a tile, several workgroups a CU.  Measured (four groups, one): weights of 6
// experts 1216 x 4224, about 300 rows each (7524 tiles): 287, 206 us; 4 of 2048 x 1024,
// 1024 rows (2048): 190, 164; 4 of 1024 x 512 (512): 54, 56; rows of layer 1, 82 experts
// 192 x 12288, 25 rows each: 572, 374; 4 of 2048 x 2048, 256 each (2.3 a CU): 123, 132;
// of layer 0, 8 of 2048 x 1024, 1024 each (17 a CU): 772, 715.
// Rows of reductions up to 1024 terms so from more than two a CU on, a third round of
// four groups being nearly empty: layer 1, 8 of 512 x K, 2.2 and 2.6 a CU, K = 256: 37,
// 28 and 36, 28; 512: 52, 41 and 52, 42; 1024: 75, 71 and 83, 72; 2048: 124, 133 and
// 151, 136; 4096: 216, 254 and 277, 257.
static bool many_rows(int64_t tiles, int K, int cus) { return K <= 1024 ? tiles > 2 * cus : tiles >= 3 * cus; }
constexpr int kManyWeights = 4;  // tiles a CU

static GradPlan plan_rows(const GradGemmArgs& a, bool bf16) {
  GradPlan p;
  const int cus = device_cu_count(), rows = bf16 ? kTileRows : 64, cols = bf16 ? 256 : 64;
  const int N = a.layer == 0 ? a.H : a.F, K = a.layer == 0 ? 2 * a.F : a.H, NT = (N + cols - 1) / cols;
  p.wide = !bf16 && wide_f32(a.rows / 128 * ((N + 127) / 128), cus);
  p.wave = !p.wide && wave_rows(a, bf16, N, K, cus);
  if (p.wide || p.wave) return p;
  // (half the experts end in a tile of their own more than their rows fill)
  p.many = !bf16 && many_rows((a.rows / 64 + (a.rows < a.E ? a.rows : a.E) / 2) * NT, K, cus);
  if (p.many) return p;
  const SplitCost& c = bf16 ? kSplitBf16 : kSplitF32;
  const int steps = bf16 ? K / kBK : K / kGfK / 4;
  const int64_t hi = a.R / rows + (a.R < a.E ? a.R : a.E), lo = a.rows == a.R ? (a.R + rows - 1) / rows : 0;
  bool split = false;
  if (hi - lo > 16)
    split = split_parts(c, 1, steps, cus) > 1;
  else
    for (int64_t mt = lo; mt <= hi && !split; ++mt) split = split_parts(c, (int)(mt * NT % cus), steps, cus) > 1;
  const int64_t most = hi * NT * (steps / 2);
  p.units = !split ? 0 : most < cus ? (int)most : cus;
  p.unit_bytes = bf16 ? 4 * 16 * 4 * 64 * 16 : 4 * 4 * 64 * 16;
  return p;
}

// Zero rows that the K steps of the weights' gradients run over beside `rows` evenly
// routed ones: they fill up every segment's last step (of `step` rows).  Of one source
// block not counted; of several half a step for each further segment, and a step for
// each at least, as far as there are rows (16 experts, 32 blocks, 8 rows a segment: 32
// steps of 64 an expert, the rows alone 4).  Measured (rows alone, so; layer 1, bf16):
// 16 experts 512 x 512, 8 blocks, 4 rows a segment: 28.6, 22.0 us; 256 x 512, 32 blocks,
// 4 rows: 41.3, 37.1; 12800 rows in 8 blocks: 33.0, 31.5; 8 experts 256 x 512, 32768 rows
// in 8: 42.6, 44.9.  (Counted from the offsets on the device, 1.2 us a call more.)
static int fill_rows(const GradGemmArgs& a, int64_t rows, int step) {
  if (a.G == a.E) return 0;
  const int64_t even = (int64_t)(a.G - a.E) * step / 2, least = (a.G < rows ? a.G : rows) * step - rows;
  return (int)(rows < a.G || least > even ? least : even);
}

// bf16 weights' gradients; steps: an expert's mean.  Measured (large tiles, these):
// layer 0, 256 tokens, 8 of 256 x 512, top 2 (2048, 1): 13.7, 9.6; 2048 there (8 steps):
// 24.2, 20.4; 4096, 2 of 16 of 1024 x 512 held, top 2 (2048, 8): 26.3, 21.4;
// 1000, 8 of 512 x 512 (4096, 3): 18.9, 25.8; layer 1 of it (2048, 3): 17.3, 14.9;
// of 8 experts 256 x C, T tiles a CU, at s steps: T 2, s 40: 30, 26; 64: 33, 38; T 4, 16:
// 27, 23; 24: 30, 31; T 6, 16: 30, 28; 24: 32, 38; T 8, 8: 25, 24; 12: 30, 30; 16: 31,
// 37; T 10, 2: 15.8, 14.9; 4: 18.7, 19.8; T 12, 1: 14.2, 14.1; 2: 15.9, 17.3; T 16, 1: 14.8, 17.3.
static bool wave_weights(const GradGemmArgs& a, int64_t tiles, int cus) {
  const int64_t steps = (a.rows + fill_rows(a, a.rows, kBK)) / (a.E * kBK);
  return tiles * (steps + 4) <= (tiles <= 4 * cus ? 104 : tiles <= 8 * cus ? 128 : 64) * cus;
}

static GradPlan plan_weights(const GradGemmArgs& a, bool bf16) {
  GradPlan p;
  const int cus = device_cu_count(), T = bf16 ? 256 : 64;
  const int64_t N = a.layer == 0 ? a.F : a.H, C = a.layer == 0 ? a.H : a.F, mats = a.layer == 0 ? 2 : 1;
  const auto tiles = [&](int t) { return a.E * mats * ((N + t - 1) / t) * ((C + t - 1) / t); };
  p.wide = !bf16 && wide_f32(tiles(128), cus);
  p.wave = bf16 && wave_weights(a, tiles(32), cus);
  p.many = !bf16 && tiles(64) >= kManyWeights * cus;
  if (p.wide || p.wave || p.many) return p;
  // f32, no split and few steps for the groups to share: one group too, below 160 rows an expert where a round holds all
  // tiles and 512 where not.  Measured (four groups, one), weights of layer 1, 8 experts 256 x 512 (a round): 64 rows
  // each 9.5, 8.6 us; 128: 12.1, 12.4; 192: 15.0, 15.9; 256: 17.4, 19.4; 384: 21.3, 25.2; 3 of 2048 x 512 (1.5): 64:
  // 18.8, 11.9; 256: 29.9, 23.3; 384: 36.8, 30.2; 512: 44.2, 37.8; 5 of 576 x 704 (2.1): 384: 30.5, 27.4.
  const bool few = !bf16 && a.rows < a.E * (tiles(64) <= cus ? 160ll : 512ll);
  // the experts' mean of steps: of an even routing, for whether a split pays, and the most (all rows kept), for its units
  const auto steps = [&](int64_t rows) {
    const int64_t step = a.E * (bf16 ? kBK : 4 * kGfK);
    return (rows + fill_rows(a, rows, bf16 ? kBK : kGfK) + step - 1) / step;
  };
  const int64_t mean = steps(a.rows), most = steps(a.R);
  const int64_t r = tiles(T) % cus;
  const bool split = split_parts(bf16 ? kSplitWeights : kSplitF32, (int)r, (int)mean, cus) > 1;
  p.units = !split ? 0 : r * (most / 2) < cus ? (int)(r * (most / 2)) : cus;
  p.many = few && !split;
  p.unit_bytes = bf16 ? 4 * 16 * 4 * 64 * 16 : 4 * 4 * 64 * 16;
  return p;
}

size_t grad_ws_bytes(const GradGemmArgs& a, bool bf16) {
  size_t most = 0;
  GradGemmArgs b = a;
  for (b.layer = 0; b.layer < 2; ++b.layer) {
    const size_t rows = plan_rows(b, bf16).bytes(), weights = plan_weights(b, bf16).bytes();
    most = rows > most ? rows : most;
    most = weights > most ? weights : most;
  }
  return most;
}

// The arguments with the workspace's parts, or without.
static GradGemmArgs with_split(const GradGemmArgs& a, const GradPlan& p, void* ws) {
  GradGemmArgs g = a;
  g.split = {nullptr, nullptr, nullptr, 0};
  if (ws && p.units) {
    g.split.part = (float*)ws;
    g.split.desc = (int32_t*)((char*)ws + p.units * p.unit_bytes);
    g.split.hdr = g.split.desc + (size_t)p.units * kGradDescInts;
    g.split.units = p.units;
  }
  return g;
}

hipError_t launch_grad_rows(const GradGemmArgs& a, bool bf16, void* ws, hipStream_t s) {
  if (a.R == 0) return hipSuccess;
  const int cus = device_cu_count(), xcd_slots = cus / kXcds > 0 ? cus / kXcds : 1;
  const GradPlan p = plan_rows(a, bf16);
  const GradGemmArgs g = with_split(a, p, ws);
  if (p.wave) {
    if (bf16) return a.layer == 0 ? launch_wave<kGradRows0, __bf16>(g, a.H, s) : launch_wave<kGradRows1, __bf16>(g, a.F, s);
    return a.layer == 0 ? launch_wave<kGradRows0, float>(g, a.H, s) : launch_wave<kGradRows1, float>(g, a.F, s);
  }
  if (bf16) {
    if (a.layer == 0) {
      grad_rows_bf16_kernel<kGradRows0><<<cus, kGemmThreads, 0, s>>>(g, xcd_slots);
      return grad_reduce_launch<kGradRows0, __bf16>(g, s);
    }
    grad_rows_bf16_kernel<kGradRows1><<<cus, kGemmThreads, 0, s>>>(g, xcd_slots);
    return grad_reduce_launch<kGradRows1, __bf16>(g, s);
  }
  if (p.wide) {
    if (a.layer == 0)
      grad_rows_f32_kernel<kGradRows0, 128, 2><<<cus, 512, 0, s>>>(g);
    else
      grad_rows_f32_kernel<kGradRows1, 128, 2><<<cus, 512, 0, s>>>(g);
    return hipGetLastError();
  }
  if (p.many) {
    if (a.layer == 0)
      grad_rows_f32_kernel<kGradRows0, 64, 1><<<3 * cus, 256, 0, s>>>(g);
    else
      grad_rows_f32_kernel<kGradRows1, 64, 1><<<3 * cus, 256, 0, s>>>(g);
    return hipGetLastError();
  }
  if (a.layer == 0) {
    grad_rows_f32_kernel<kGradRows0, 64, 4><<<cus, 1024, 0, s>>>(g);
    return grad_reduce_launch<kGradRows0, float>(g, s);
  }
  grad_rows_f32_kernel<kGradRows1, 64, 4><<<cus, 1024, 0, s>>>(g);
  return grad_reduce_launch<kGradRows1, float>(g, s);
}

static hipError_t launch_wave_weights(const GradGemmArgs& g, hipStream_t s) {
  const int cus = device_cu_count();
  const int64_t tiles = (int64_t)g.E * (g.layer == 0 ? 2 : 1) * (g.F / 32) * (g.H / 32);
  if (tiles <= cus)
    wave_weights_kernel<8><<<cus, 512, 0, s>>>(g);
  else
    wave_weights_kernel<4><<<3 * cus, 256, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_grad_weights(const GradGemmArgs& a, bool bf16, void* ws, hipStream_t s) {
  const int cus = device_cu_count();
  const GradPlan p = plan_weights(a, bf16);
  GradGemmArgs g = with_split(a, p, ws);
  g.fill = fill_rows(a, a.rows, bf16 ? kBK : kGfK);
  if (p.wave) return launch_wave_weights(g, s);
  if (bf16) {
    grad_weights_bf16_kernel<<<cus, kGemmThreads, 0, s>>>(g);
    return grad_reduce_launch<kGradWeights, __bf16>(g, s);
  }
  if (p.wide) {
    grad_weights_f32_kernel<128, 2><<<cus, 512, 0, s>>>(g);
    return hipGetLastError();
  }
  if (p.many) {  // one group a tile, four workgroups a CU
    grad_weights_f32_kernel<64, 1><<<4 * cus, 256, 0, s>>>(g);
    return hipGetLastError();
  }
  grad_weights_f32_kernel<64, 4><<<cus, 1024, 0, s>>>(g);
  return grad_reduce_launch<kGradWeights, float>(g, s);
}

hipError_t launch_keep(const GradGemmArgs& a, bool bf16, hipStream_t s) {
  if (a.R == 0) return hipSuccess;
  const int cus = device_cu_count();
  const GradGemmArgs g = with_split(a, GradPlan{}, nullptr);
  if (wave_keep(a, bf16, cus)) return bf16 ? launch_wave<kKeep, __bf16>(g, a.F, s) : launch_wave<kKeep, float>(g, a.F, s);
  grad_rows_bf16_kernel<kKeep><<<cus, kGemmThreads, 0, s>>>(g, cus / kXcds > 0 ? cus / kXcds : 1);
  return hipGetLastError();
}

}  // namespace moe
