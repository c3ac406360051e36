// The shared projection with the low-rank adapters of many requests:
// moe_adapter_linear.
//
//   t[m]     = scale[a] * (x[m] . A[a])               a = adapter of row m; r values, f32
//   out[m,n] = cast(x[m] . W[n] + t[m] . B[a,n] + residual[m,n])
//
// ("Grouped GEMM 为什么适合 MoE": many small products of different row
// counts beside one large product; the row groups here are the requests of
// one adapter.)  A first kernel computes t for every row, a second one the
// projection with the adapters' part, the residual and the cast in its
// epilogue, so out is written once and nothing of the size of out is read
// back.
#include "common.hpp"
#include "launch.hpp"
#include "stream.hpp"

namespace moe {

// -------------------------------------------------------------- t = x A^T ---
// Workgroup (b, s, z): the s-th distinct adapter among the 16 rows of block b
// (none: it exits), its rank rows 16 NW z .. + 16 NW - 1.  Rows of other
// adapters read zeros and store nothing.
template <class Op, int NW>
__global__ __launch_bounds__(kStreamThreads) void adapter_shrink_kernel(AdapterArgs a) {
  __shared__ f32x4_t lds[kStreamWaves * NW * 64];
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15;
  const int rows = (int)min((int64_t)16, a.M - m0);
  int id = -1;
  if (i < rows) {
    id = a.idx[m0 + i];
    if ((uint32_t)id >= (uint32_t)a.P) id = -1;
  }
  bool first = id >= 0;
  for (int j = 0; j < 15; ++j) {
    const int other = __shfl(id, j);  // by every lane, those that do not use it too
    if (j < i && other == id) first = false;
  }
  uint64_t firsts = __ballot(first) & 0xFFFFull;
  for (unsigned s = 0; s < blockIdx.y && firsts; ++s) firsts &= firsts - 1;
  if (!firsts) return;
  const int mine = uniform(__shfl(id, __ffsll((unsigned long long)firsts) - 1));
  const int j0 = blockIdx.z * 16 * NW;
  uint32_t xoff[1] = {id == mine ? (uint32_t)i * a.row_bytes : kNoRow};
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w0 = s.w1 = reinterpret_cast<const char*>(a.a) + ((int64_t)mine * a.r + j0) * a.row_bytes;
  s.w_bytes = (uint32_t)min(16 * NW, a.r - j0) * a.row_bytes;
  s.x = reinterpret_cast<const char*>(a.x) + m0 * a.row_bytes;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.steps = a.H / Op::kStep;
  f32x4_t acc[NW][1];
  stream_tile<Op, NW, NW, 1, 4>(s, xoff, acc);
  stream_put<NW, 1>(acc, lds);
  const float sc = a.scale[mine];
  for (int t = wave; t < NW; t += kStreamWaves) {
    f32x4_t v = stream_sum(lds, t);
    const int j = j0 + 16 * t + 4 * (lane >> 4);
    if (id != mine || j >= a.r) continue;  // r is a multiple of 8
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] *= sc;
    *reinterpret_cast<f32x4_t*>(a.t + (m0 + i) * a.r + j) = v;
  }
}

// ------------------------------------------------------------- projection ---
template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}

// acc[c] += t . B[id, n + c] for the columns that exist, in increasing rank.
template <class T>
__device__ __forceinline__ void add_adapter(const AdapterArgs& a, int64_t m, int id, int n, f32x4_t& acc) {
  const float* t = a.t + m * a.r;
  const T* b = reinterpret_cast<const T*>(a.b) + ((int64_t)id * a.N + n) * a.r;
  constexpr int V = 16 / sizeof(T);  // elements per vector; r is a multiple of 8
  typedef T vec_t __attribute__((ext_vector_type(V)));
  const int cols = min(4, a.N - n);
  for (int j = 0; j < a.r; j += V) {
    float tv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) tv[v] = t[j + v];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c >= cols) break;
      const vec_t bv = *reinterpret_cast<const vec_t*>(b + (int64_t)c * a.r + j);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[c] = fmaf(tv[v], to_f32(bv[v]), acc[c]);
    }
  }
}

// Stores 4 columns (those below N) of row m: residual, cast.
__device__ __forceinline__ void adapter_store(const AdapterArgs& a, int64_t m, int n, f32x4_t acc) {
  const int64_t i = m * a.N + n;
  if ((a.N & 3) == 0) {
    store_out(a.out, i, make_float4(acc[0], acc[1], acc[2], acc[3]));
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (n + c >= a.N) break;
    float v = acc[c];
    if (a.out.residual)
      v += a.out.res_bf16 ? (float)reinterpret_cast<const __bf16*>(a.out.residual)[i + c]
                          : reinterpret_cast<const float*>(a.out.residual)[i + c];
    if (a.out.out_bf16)
      reinterpret_cast<__bf16*>(a.out.out)[i + c] = (__bf16)v;
    else
      reinterpret_cast<float*>(a.out.out)[i + c] = v;
  }
}

// 16 NW columns of 16 NT rows: the weight rows stream past the token rows
// (stream.hpp).  T: the type of x, W, A and B.
template <class Op, class T, int NW, int NT, int U>
__global__ __launch_bounds__(kStreamThreads) void adapter_stream_kernel(AdapterArgs a) {
  __shared__ f32x4_t lds[kStreamWaves * NW * NT * 64];
  const int64_t m0 = (int64_t)blockIdx.x * 16 * NT;
  const int n0 = blockIdx.y * 16 * NW;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rows = (int)min((int64_t)16 * NT, a.M - m0);
  uint32_t xoff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 16 * j + (lane & 15);
    xoff[j] = i < rows ? (uint32_t)i * a.row_bytes : kNoRow;
  }
  StreamArgs s{};
  s.row_bytes = a.row_bytes;
  s.w0 = s.w1 = reinterpret_cast<const char*>(a.w) + (int64_t)n0 * a.row_bytes;
  s.w_bytes = (uint32_t)min(16 * NW, a.N - n0) * a.row_bytes;
  s.x = reinterpret_cast<const char*>(a.x) + m0 * a.row_bytes;
  s.x_bytes = (uint32_t)rows * a.row_bytes;
  s.steps = a.H / Op::kStep;
  f32x4_t acc[NW][NT];
  stream_tile<Op, NW, NW, NT, U>(s, xoff, acc);
  stream_put<NW, NT>(acc, lds);
  for (int t = wave; t < NW * NT; t += kStreamWaves) {
    f32x4_t v = stream_sum(lds, t);
    const int i = 16 * (t % NT) + (lane & 15);
    const int n = n0 + 16 * (t / NT) + 4 * (lane >> 4);
    if (i >= rows || n >= a.N) continue;
    const int id = a.P > 0 ? a.idx[m0 + i] : -1;
    if ((uint32_t)id < (uint32_t)a.P) add_adapter<T>(a, m0 + i, id, n, v);
    adapter_store(a, m0 + i, n, v);
  }
}

// ----------------------------------------------------------------- launch ---
template <class Op>
static void launch_shrink(const AdapterArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)((a.M + 15) / 16);
  if (a.r <= 16)
    adapter_shrink_kernel<Op, 1><<<dim3(blocks, 16, 1), kStreamThreads, 0, s>>>(a);
  else
    adapter_shrink_kernel<Op, 2><<<dim3(blocks, 16, (unsigned)((a.r + 31) / 32)), kStreamThreads, 0, s>>>(a);
}

template <class Op, class T>
static void launch_stream(const AdapterArgs& a, hipStream_t s) {
  auto grid = [&](int nt, int nw) {
    return dim3((unsigned)((a.M + 16 * nt - 1) / (16 * nt)), (unsigned)((a.N + 16 * nw - 1) / (16 * nw)));
  };
  if (a.M <= 16)
    adapter_stream_kernel<Op, T, 1, 1, 4><<<grid(1, 1), kStreamThreads, 0, s>>>(a);
  else
    adapter_stream_kernel<Op, T, 4, 4, 2><<<grid(4, 4), kStreamThreads, 0, s>>>(a);
}

hipError_t launch_adapter_linear(const AdapterArgs& a, bool f32, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  if (a.P > 0) {
    if (f32)
      launch_shrink<StreamF32>(a, s);
    else
      launch_shrink<StreamBf16<1>>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (f32)
    launch_stream<StreamF32, float>(a, s);
  else
    launch_stream<StreamBf16<1>, __bf16>(a, s);
  return hipGetLastError();
}

}  // namespace moe
