// The shared projection with the low-rank adapters of many requests:
// moe_adapter_linear.
//
//   t[m]     = scale[a] * (x[m] . A[a])               a = adapter of row m; r values, f32
//   out[m,n] = cast(x[m] . W[n] + t[m] . B[a,n] + residual[m,n])
//
// ("Grouped GEMM 为什么适合 MoE": many small products of different row
// counts beside one large product; the row groups here are the requests of
// one adapter.)  At most 8 rows of one adapter are one launch.  Otherwise a
// first kernel computes t for every row, a second one the projection, with the
// adapters' part (t . B) added on the matrix cores or in the epilogue, the
// residual and the cast, so out is written once and nothing of the size of out
// is read back.  What bounds them: latency for a few rows, the L2 and the LDS for
// hundreds, the matrix cores beyond (adapter_gemm.hpp).
#include <math.h>

#include "adapter_gemm.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "stream.hpp"

namespace moe {

// -------------------------------------------------------------- t = x A^T ---
// Block (b, s, z): of the distinct adapters among the 16 NT rows of block b,
// those number s, s + gridDim.y, ... (none: it exits), rank rows 16 NW z .. +
// 16 NW - 1.  The waves split the reduction.  Bound by latency for short
// batches, by reading x for long ones (launch_shrink).
template <class Op, int WAVES, int NW, int NT>
__global__ __launch_bounds__(64 * WAVES) void adapter_shrink_kernel(AdapterArgs a) {
  constexpr int kLds = WAVES * imax(stream_line_bytes<Op, NW, NT>(), NW * NT * 1024);
  __shared__ __attribute__((aligned(16))) char lds[kLds];
  const int64_t m0 = (int64_t)blockIdx.x * 16 * NT;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int rows = (int)min((int64_t)16 * NT, a.M - m0);
  int id = -1;  // lane's row: m0 + lane
  if (lane < rows) {
    id = a.idx[m0 + lane];
    if ((uint32_t)id >= (uint32_t)a.P) id = -1;
  }
  const int j0 = blockIdx.z * 16 * NW;
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w_rows = min(16 * NW, a.r - j0);
  s.x = reinterpret_cast<const char*>(a.x) + m0 * a.row_bytes;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.lines = a.H / Op::kLine;
  uint64_t left = __ballot(id >= 0);
  for (int n = 0; left; ++n) {
    const int mine = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(id == mine);
    if (n % (int)gridDim.y != (int)blockIdx.y) continue;
    // (of the rows of other adapters nothing is read, computed or stored)
    s.w0 = reinterpret_cast<const char*>(a.a) + ((int64_t)mine * a.r + j0) * a.row_bytes;
    f32x4_t acc[NW][NT];
    stream_tile<Op, WAVES, NW, kOne, NT, 2, false>(s, [&](int m) { return __shfl(id, m) == mine ? (uint32_t)m * a.row_bytes : kNoRow; },
                                          lds + wave * stream_line_bytes<Op, NW, NT>(), acc);
    const float sc = a.scale[mine];
    stream_reduce<WAVES, NW, NT, NW, 1>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int g, int jt, const f32x4_t (&t)[1]) {
      f32x4_t v = t[0];
      const int i = 16 * jt + (lane & 15), j = j0 + 16 * g + 4 * (lane >> 4);
      if (__shfl(id, i) != mine || j >= a.r) return;  // r is a multiple of 8
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] *= sc;
      if (a.planes == 1) {  // f32
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.t) + (m0 + i) * a.r + j) = v;
        return;
      }
      __bf16 pl[4][3];
#pragma unroll
      for (int c = 0; c < 4; ++c) split_bf16<3>(v[c], pl[c]);
      __bf16* t16 = reinterpret_cast<__bf16*>(a.t) + (m0 + i) * a.planes * a.r + j;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        if (p >= a.planes) break;
        const bf16x4_t o = {pl[0][p], pl[1][p], pl[2][p], pl[3][p]};
        *reinterpret_cast<bf16x4_t*>(t16 + p * a.r) = o;
      }
    });
    __syncthreads();  // the sums are read before the next adapter's lines come
  }
}

// ------------------------------------------------------------- projection ---
// The adapters' part of a stream tile's outputs, in one of two ways.  Up to
// kDirectRank ranks each thread adds those of its own outputs in the epilogue
// (48 rows of 48 adapters of rank 16, 4096 x 4096: 12 us instead of 14); beyond,
// they go through the matrix cores (333 x 2048 x 1408, rank 32: 11.6 us instead
// of 13.5; 1000 x 4096 x 2048, rank 128: 41 instead of 78).
constexpr int kDirectRank = 16;

// acc[c] += t . B[id, n + c] for the columns that exist, in increasing rank (t
// in f32; the loads of 16 ranks are under way together).
template <class T>
__device__ __forceinline__ void add_adapter(const AdapterArgs& a, const float* t, int id, int n, f32x4_t& acc) {
  constexpr int V = 16 / sizeof(T), U = kDirectRank / V;  // elements per vector (r is a multiple of 8); vectors
  typedef T vec_t __attribute__((ext_vector_type(V)));
  typedef float tvec_t __attribute__((ext_vector_type(V)));
  const T* b = reinterpret_cast<const T*>(a.b) + ((int64_t)id * a.N + n) * a.r;
  for (int j0 = 0; j0 < a.r; j0 += kDirectRank) {
    tvec_t tv[U];
    vec_t bv[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * V, a.r - V);
      tv[u] = *reinterpret_cast<const tvec_t*>(t + j);
#pragma unroll
      for (int c = 0; c < 4; ++c)  // (past the last column it is read again, not used)
        bv[u][c] = *reinterpret_cast<const vec_t*>(b + (int64_t)min(c, a.N - n - 1) * a.r + j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u * V >= a.r) break;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[c] = fmaf(tv[u][v], (float)bv[u][c][v], acc[c]);
    }
  }
}

// acc += t . B for the adapters among the tile's rows, on the matrix cores: a
// unit is 16 bytes of a lane's B row (32 ranks, f32: 16) of one adapter; unit
// i of adapter a is share a + i's, whatever else the tile holds, so a row's sum
// does not depend on the other rows (SHARES > 1: the waves that split the
// reduction, whose accumulators are added later).
// A row of another adapter holds zeros, which only cancel finite values: a
// non-finite element of B is left out, and the result says so (mend_sum).
// row_id: adapter of row m0 + lane.
template <class Op, class T, int SHARES, int NW, int NT>
__device__ __forceinline__ bool add_adapters(const AdapterArgs& a, int64_t m0, int rows, int n0, int row_id, int share,
                                             f32x4_t (&acc)[NW][NT]) {
  constexpr int V = 16 / sizeof(T), K = 4 * V;  // elements of a lane, of a unit
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int cols = min(16 * NW, a.N - n0), planes = a.planes, pitch = planes * a.r;
  const __amdgpu_buffer_rsrc_t rt = make_rsrc(reinterpret_cast<const T*>(a.t) + m0 * pitch, (uint32_t)(rows * pitch) * sizeof(T));
  bool left_out = false;
  uint64_t left = __ballot(lane < rows && (uint32_t)row_id < (uint32_t)a.P &&
                           ((share - row_id) & (SHARES - 1)) * K < a.r);  // rows of adapters with a unit of this share
  int id = 0, k0 = a.r;
  auto next = [&]() {  // the share's next unit: adapter id, ranks k0 ..
    k0 += SHARES * K;
    while (k0 >= a.r) {
      if (!left) return false;
      id = __builtin_amdgcn_readlane(row_id, __ffsll((unsigned long long)left) - 1);
      left &= ~__ballot(row_id == id);
      k0 = ((share - id) & (SHARES - 1)) * K;
    }
    return true;
  };
  struct Unit {
    i32x4_t w[NW], x[NT][3];
  };
  auto load = [&](Unit& u) {
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(reinterpret_cast<const T*>(a.b) + ((int64_t)id * a.N + n0) * a.r,
                                                (uint32_t)(cols * a.r) * sizeof(T));
    const int k = k0 + V * (lane >> 4);
#pragma unroll
    for (int g = 0; g < NW; ++g)
      u.w[g] = buf_load16(rb, k < a.r ? (uint32_t)((16 * g + r) * a.r + k) * sizeof(T) : kNoRow, 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const bool mine = __shfl(row_id, 16 * j + r) == id && k < a.r;
#pragma unroll
      for (int p = 0; p < 3; ++p)
        u.x[j][p] = buf_load16(rt, mine && p < planes ? (uint32_t)((16 * j + r) * pitch + p * a.r + k) * sizeof(T) : kNoRow, 0);
    }
  };
  auto multiply = [&](Unit& u) {
#pragma unroll
    for (int g = 0; g < NW; ++g) left_out |= drop_nonfinite<T>(u.w[g]);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      if (p >= planes) break;
      i32x4_t x[NT][1];
#pragma unroll
      for (int j = 0; j < NT; ++j) x[j][0] = u.x[j][p];
#pragma unroll
      for (int g = 0; g < NW; ++g) Op::template mma<NT>(acc[g], u.w[g], 0.0f, x);
    }
  };
  Unit u0, u1;  // the next unit's loads are under way during a unit's products
  bool more = next();
  if (more) load(u0);
  while (more) {
    more = next();
    if (more) load(u1);
    multiply(u0);
    if (!more) break;
    more = next();
    if (more) load(u0);
    multiply(u1);
  }
  return __any(left_out);
}

// 16 NW columns of 16 NT rows: the weight rows stream past the token rows
// (stream.hpp).  T: the type of x, W, A and B.
template <class Op, class T, int WAVES, int NW, int NT>
__global__ __launch_bounds__(64 * WAVES) void adapter_stream_kernel(AdapterArgs a, int mb, int nb) {
  constexpr int G = NW * NT * WAVES <= 64 ? NW : NW * NT * WAVES <= 128 && NW % 2 == 0 ? NW / 2 : 1;
  constexpr int kLds = WAVES * imax(stream_line_bytes<Op, NW, NT>(), G * NT * 1024);
  __shared__ __attribute__((aligned(16))) char lds[kLds];
  __shared__ int left_out[WAVES];
  // the row blocks of one weight block run next to each other on one XCD (whose
  // workgroups come 8 apart), so its L2 reads the weights once
  const int64_t v0 = xcd_tile((int64_t)mb * nb);
  if (v0 < 0) return;
  const int64_t m0 = v0 % mb * 16 * NT;
  const int n0 = (int)(v0 / mb) * 16 * NW;
  const int lane = threadIdx.x & 63;
  const int rows = (int)min((int64_t)16 * NT, a.M - m0);
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w0 = reinterpret_cast<const char*>(a.w) + (int64_t)n0 * a.row_bytes;
  s.w_rows = min(16 * NW, a.N - n0);
  s.x = reinterpret_cast<const char*>(a.x) + m0 * a.row_bytes;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.lines = a.H / Op::kLine;
  // lane's row: m0 + lane (loaded early: t and B wait for it)
  const int row_id = a.P > 0 ? a.idx[m0 + min(lane, rows - 1)] : -1;
  f32x4_t acc[NW][NT];
  stream_tile<Op, WAVES, NW, kOne, NT, 2, false>(s, [&](int m) { return (uint32_t)min(m, rows - 1) * a.row_bytes; },
                                        lds + uniform(threadIdx.x >> 6) * stream_line_bytes<Op, NW, NT>(), acc);
  const bool direct = a.r <= kDirectRank;
  if (a.P > 0 && !direct) {
    const bool bad = add_adapters<Op, T, WAVES, NW, NT>(a, m0, rows, n0, row_id, uniform(threadIdx.x >> 6), acc);
    if (lane == 0) left_out[threadIdx.x >> 6] = bad;
  }
  stream_reduce<WAVES, NW, NT, G, 1>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int g, int j, const f32x4_t (&sum)[1]) {
    f32x4_t v = sum[0];
    const int i = 16 * j + (lane & 15);
    const int n = n0 + 16 * g + 4 * (lane >> 4);
    const int id = __shfl(row_id, i);
    if (i >= rows || n >= a.N) return;
    if (direct) {
      if ((uint32_t)id < (uint32_t)a.P) add_adapter<T>(a, reinterpret_cast<const float*>(a.t) + (m0 + i) * a.r, id, n, v);
    } else {
      bool bad = false;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) bad |= left_out[w] != 0;
      mend_sums<T>(a, m0 + i, id, n, bad, v);
    }
    adapter_store(a, m0 + i, n, v);
  });
}

// 16 NW WAVES columns of 64 rows: the waves split the columns and share the
// token rows' lines, which halves what a 64 x 64 tile reads of them for an output
// (1102 x 768 x 3020, rank 64: 25 us, 37 by the matrix-core tile; 3588 x 1216 x
// 728, rank 16: 20 us, 32 by 64 x 64 tiles).  Bound by the L2 and the LDS.
template <class Op, class T, int WAVES, int NW>
__global__ __launch_bounds__(64 * WAVES) void adapter_wide_kernel(AdapterArgs a, int mb, int nb) {
  constexpr int NT = 4;
  __shared__ __attribute__((aligned(16))) char lds[stream_wide_bytes<Op, WAVES, NW, NT>()];
  const int64_t v0 = xcd_tile((int64_t)mb * nb);
  if (v0 < 0) return;
  const int64_t m0 = v0 % mb * 16 * NT;
  const int n0 = (int)(v0 / mb) * 16 * NW * WAVES;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int rows = (int)min((int64_t)16 * NT, a.M - m0);
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w0 = reinterpret_cast<const char*>(a.w) + (int64_t)n0 * a.row_bytes;
  s.w_rows = min(16 * NW * WAVES, a.N - n0);
  s.x = reinterpret_cast<const char*>(a.x) + m0 * a.row_bytes;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.lines = a.H / Op::kLine;
  const int row_id = a.P > 0 ? a.idx[m0 + min(lane, rows - 1)] : -1;  // of row m0 + lane
  f32x4_t acc[NW][NT];
  stream_wide<Op, WAVES, NW, kOne, NT, 2, false>(
      s, [&](int m) { return (uint32_t)min(m, rows - 1) * a.row_bytes; }, lds, acc);
  const int nw = n0 + 16 * NW * wave;
  if (nw >= a.N) return;
  const bool bad = a.P > 0 && add_adapters<Op, T, 1, NW, NT>(a, m0, rows, nw, row_id, 0, acc);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 16 * j + (lane & 15), id = __shfl(row_id, i);
#pragma unroll
    for (int g = 0; g < NW; ++g) {
      const int n = nw + 16 * g + 4 * (lane >> 4);
      if (i >= rows || n >= a.N) continue;
      f32x4_t v = acc[g][j];
      mend_sums<T>(a, m0 + i, id, n, bad, v);
      adapter_store(a, m0 + i, n, v);
    }
  }
}

// At most 8 rows that use one adapter between them (one row, or one adapter),
// 16 columns a block: the adapter's A streams past the rows as NA further
// groups of 16 weight rows, so every block has t for itself and there is one
// launch (one row, 2048 x 64, rank 8: 4.3 us instead of 3.8 + 4.0 in two; 4096 x
// 4096, rank 16: 9.6 instead of 5.1 + 8.7, rank 64: 15 instead of 6.8 + 8.4).
constexpr int kOneRows = 8;

template <class Op, class T, int NA>
__global__ __launch_bounds__(512) void adapter_one_kernel(AdapterArgs a) {
  constexpr int WAVES = 8, NW = 1 + NA, kLine = stream_line_bytes<Op, NW, 1, kOneRows>();
  __shared__ __attribute__((aligned(16))) char lds[WAVES * imax(kLine, NW * 1024)];
  __shared__ __attribute__((aligned(32))) float t[kOneRows][16 * NA];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), rows = (int)a.M;
  const int n0 = blockIdx.x * 16;
  int row_id = lane < rows ? a.idx[lane] : -1;
  if ((uint32_t)row_id >= (uint32_t)a.P) row_id = -1;
  const uint64_t used = __ballot(row_id >= 0);
  const int id = used ? __builtin_amdgcn_readlane(row_id, __ffsll((unsigned long long)used) - 1) : 0;
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w0 = reinterpret_cast<const char*>(a.w) + (int64_t)n0 * a.row_bytes;
  s.w_rows = min(16, a.N - n0);
  s.w1 = reinterpret_cast<const char*>(a.a) + (int64_t)id * a.r * a.row_bytes;
  s.w1_rows = a.r;
  s.x = a.x;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.lines = a.H / Op::kLine;
  f32x4_t acc[NW][1], out = {0.f, 0.f, 0.f, 0.f};
  stream_share<Op, NW, kFirst, 1, 2, kOneRows, false>(
      s, wave, WAVES, [&](int m) { return m < rows ? (uint32_t)m * a.row_bytes : kNoRow; }, lds + wave * kLine, acc);
  const float sc = a.scale[id];
  // wave 0 gets the projection's sums, the next ones t's
  stream_reduce<WAVES, NW, 1, NW, 1>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int g, int, const f32x4_t (&sum)[1]) {
    if (g == 0) {
      out = sum[0];
    } else if ((lane & 15) < kOneRows) {
      f32x4_t v = sum[0];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] *= sc;
      *reinterpret_cast<f32x4_t*>(&t[lane & 15][16 * (g - 1) + 4 * (lane >> 4)]) = v;
    }
  });
  __syncthreads();
  const int i = lane & 15, n = n0 + 4 * (lane >> 4);
  const int mine = __shfl(row_id, i);
  if (wave > 0 || i >= rows || n >= a.N) return;
  if (mine >= 0) add_adapter<T>(a, t[i], id, n, out);
  adapter_store(a, i, n, out);
}

// ----------------------------------------------------------------- launch ---
template <class Op, int WAVES, int NW, int NT>
static void launch_shrink_as(const AdapterArgs& a, unsigned slots, hipStream_t s) {
  const dim3 grid((unsigned)((a.M + 16 * NT - 1) / (16 * NT)), slots, (unsigned)((a.r + 16 * NW - 1) / (16 * NW)));
  adapter_shrink_kernel<Op, WAVES, NW, NT><<<grid, 64 * WAVES, 0, s>>>(a);
}

// Short batches: a block of 8 waves for every adapter that 16 rows can have, or
// 8 of them beyond 64 rows, where most would find none (with 4: 200 mixed rows
// of 8 adapters 8.9 us instead of 5.5, 500 rows in runs, rank 64, 7.4 instead of
// 11), and for every 16 ranks, or 32 beyond 64 rows (16 rows, H = 6528, rank
// 32, f32: 13.5 us instead of 19; 500 rows: 13.5 instead of 10).  (16 waves a
// block: 7.5 instead of 6.3 us at 48 rows, H = 4096, rank 16.)
// Long ones: the largest tile that still gives a block for every CU (x is read
// once per 16 NW of the rank, A once per 16 NT rows), whose adapters 4 blocks
// share (1000 rows of 20 adapters, H = 4096, rank 16: 5.7 us instead of 8.7 by
// one).
struct ShrinkTile {
  int rows, ranks;
};
static ShrinkTile shrink_tile(const AdapterArgs& a) {
  const int64_t cus = device_cu_count();
  auto blocks = [&](int ranks, int rows) { return ((a.M + rows - 1) / rows) * ((a.r + ranks - 1) / ranks); };
  if (a.M <= 64) return {16, 16};
  if (a.M <= 512) return {16, a.r <= 16 ? 16 : 32};
  if (a.r > 32 && blocks(64, 32) >= cus) return {32, 64};
  if (a.r > 16 && blocks(32, 32) >= cus) return {32, 32};
  return {blocks(16, 32) >= cus ? 32 : 16, 16};
}

template <class Op>
static void launch_shrink(const AdapterArgs& a, hipStream_t s) {
  const ShrinkTile t = shrink_tile(a);
  const int most = a.M <= 64 ? 16 : 8;
  const unsigned slots = a.M > 512 ? 4 : a.P < most ? a.P : most;
  if (t.rows == 32 && t.ranks == 64)
    launch_shrink_as<Op, 8, 4, 2>(a, slots, s);
  else if (t.rows == 32 && t.ranks == 32)
    launch_shrink_as<Op, 8, 2, 2>(a, slots, s);
  else if (t.rows == 32)
    launch_shrink_as<Op, 8, 1, 2>(a, slots, s);
  else if (t.ranks == 32)
    launch_shrink_as<Op, 8, 2, 1>(a, slots, s);
  else
    launch_shrink_as<Op, 8, 1, 1>(a, slots, s);
}

template <class Op, class T, int WAVES, int NW, int NT>
static void launch_stream_as(const AdapterArgs& a, hipStream_t s) {
  const int mb = (int)((a.M + 16 * NT - 1) / (16 * NT)), nb = (a.N + 16 * NW - 1) / (16 * NW);
  adapter_stream_kernel<Op, T, WAVES, NW, NT><<<tile_grid((int64_t)mb * nb), 64 * WAVES, 0, s>>>(a, mb, nb);
}

// Which kernel: each takes about start + rounds x (round + step H / 1024) us, a
// round being one tile per CU; the rule takes the least.  Fitted to 256 tiles
// at H = 256, 1024 and 4096 (two and four rounds at 1024 for the small ones),
// in us: bf16 stream tiles of 64 x 64, 32 x 32, 16 x 16 outputs 6.6 9.4 19,
// 4.8 5.7 10, 3.7 4.0 6.5, column-splitting ones of 64 x 256 9 17 47;
// matrix-core tiles of 128 x 256 and 256 x 256 (they
// keep more of the operands in LDS, but one of them alone on a CU waits longer
// for its loads) 16 28 73, 28 46 123; f32 10 24 80, 6.4 9.8 23, 4.2 5.6 10.
// With adapters: the stream tiles' reduction is longer by the planes (one
// adapter a tile is assumed), the matrix-core tiles' by those of two adapters in
// steps of 64, and a round takes `adapters` us and `part` us for 32 ranks of a
// plane more; rows that are not whole 8-byte units take `odd` us more.
struct TileKind {
  int rows, cols;
  float start, round, step;
  float adapters = 0.0f, part = 0.0f, odd = 0.0f;
  int assumed = 1, unit = 1;  // adapters; ranks that they take a multiple of
};
constexpr TileKind kWide{64, 256, 4.3f, 2.1f, 10.1f, 2.0f, 1.0f, 1.0f};
constexpr TileKind kStream64{64, 64, 1.3f, 4.8f, 3.25f}, kStream32{32, 32, 3.2f, 1.1f, 1.4f},
    kStream16{16, 16, 3.0f, 0.25f, 0.8f}, kGemm128{128, 256, 1.5f, 10.5f, 15.3f, 3.0f, 0.0f, 2.0f, 2, kBK},
    kGemm256{256, 256, 1.5f, 20.0f, 25.2f, 3.0f, 0.0f, 8.0f, 2, kBK};
constexpr TileKind kStreamF64{64, 64, 1.3f, 3.9f, 18.5f}, kStreamF32{32, 32, 3.2f, 2.1f, 4.45f},
    kStreamF16{16, 16, 3.0f, 0.75f, 1.6f};

static float tile_cost(const AdapterArgs& a, const TileKind& t, int planes) {
  const float tiles = (float)((a.M + t.rows - 1) / t.rows) * (float)((a.N + t.cols - 1) / t.cols);
  const int ranks = planes * a.r;  // (none without adapters)
  const float more = (a.P > 0 ? t.adapters + t.part * (float)ranks / 32.0f : 0.0f) + (a.N & 3 ? t.odd : 0.0f);
  const int k = a.H + t.assumed * ((ranks + t.unit - 1) / t.unit * t.unit);
  return t.start + ceilf(tiles / (float)device_cu_count()) * (t.round + more + t.step * (float)k / 1024.0f);
}

template <class Op, class T>
static void launch_one(const AdapterArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)((a.N + 15) / 16);
  if (a.r <= 16)
    adapter_one_kernel<Op, T, 1><<<blocks, 512, 0, s>>>(a);
  else if (a.r <= 32)
    adapter_one_kernel<Op, T, 2><<<blocks, 512, 0, s>>>(a);
  else
    adapter_one_kernel<Op, T, 4><<<blocks, 512, 0, s>>>(a);
}

// One launch (adapter_one_kernel) where the blocks' reading A from the L2, at
// about 124 bytes a ns and CU, takes less than the other launch.
static bool one_launch(const AdapterArgs& a) {
  if (a.P == 0 || a.M > kOneRows || (a.M > 1 && a.P > 1) || a.r > 64) return false;
  const int64_t rounds = (a.N + 16 * device_cu_count() - 1) / (16 * device_cu_count());
  return rounds * a.r * a.row_bytes <= 768 << 10;
}

static int planes_of(const AdapterArgs& a, bool f32) { return f32 ? 1 : a.out.out_bf16 ? 2 : 3; }

AdapterTiles adapter_tiles(const AdapterArgs& a, bool f32) {
  if (one_launch(a)) return {kOneRows, 16, 0, 0};
  const int planes = planes_of(a, f32);
  const TileKind* best = f32 ? &kStreamF64 : &kStream64;
  float least = tile_cost(a, *best, planes);
  auto consider = [&](const TileKind& t) {
    const float c = tile_cost(a, t, planes);
    if (c >= least) return;
    least = c;
    best = &t;
  };
  consider(f32 ? kStreamF32 : kStream32);
  consider(f32 ? kStreamF16 : kStream16);
  if (!f32) {
    consider(kWide);
    consider(kGemm128);
    consider(kGemm256);
    if (a.H < 128 && best->cols == 256) best = &kWide;  // the matrix-core tiles take two steps of 64 at least
  }
  const ShrinkTile t = a.P > 0 ? shrink_tile(a) : ShrinkTile{0, 0};
  return {best->rows, best->cols, t.rows, t.ranks};
}

template <class Op, class T>
static void launch_tiles(const AdapterArgs& a, const AdapterTiles& t, hipStream_t s) {
  if (t.rows == kStream64.rows)
    launch_stream_as<Op, T, 8, 4, 4>(a, s);
  else if (t.rows == kStream32.rows)
    launch_stream_as<Op, T, 8, 2, 2>(a, s);
  else
    launch_stream_as<Op, T, 8, 1, 1>(a, s);
}

hipError_t launch_adapter_linear(AdapterArgs a, bool f32, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  const AdapterTiles t = adapter_tiles(a, f32);
  if (t.rows == kOneRows) {
    if (f32)
      launch_one<StreamF32, float>(a, s);
    else
      launch_one<StreamBf16<1>, __bf16>(a, s);
    return hipGetLastError();
  }
  const bool by_stream = t.cols <= kStream64.cols;
  a.planes = by_stream && a.r <= kDirectRank ? 1 : planes_of(a, f32);
  if (a.P > 0) {
    if (f32)
      launch_shrink<StreamF32>(a, s);
    else
      launch_shrink<StreamBf16<1>>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (f32) {
    launch_tiles<StreamF32, float>(a, t, s);
  } else if (by_stream) {
    launch_tiles<StreamBf16<1>, __bf16>(a, t, s);
  } else if (t.rows == kWide.rows) {
    const int mb = (int)((a.M + 63) / 64), nb = (a.N + 255) / 256;
    adapter_wide_kernel<StreamBf16<1>, __bf16, 8, 2><<<tile_grid((int64_t)mb * nb), 512, 0, s>>>(a, mb, nb);
  } else {
    const int64_t mt = (a.M + t.rows - 1) / t.rows, nt = (a.N + 255) / 256;
    const dim3 grid = tile_grid(mt * nt);
    if (t.rows == kGemm256.rows)
      adapter_gemm_kernel<256><<<grid, kGemmThreads, 0, s>>>(a, (int)mt, (int)nt);
    else
      adapter_gemm_kernel<128><<<grid, kGemmThreads, 0, s>>>(a, (int)mt, (int)nt);
  }
  return hipGetLastError();
}

}  // namespace moe
