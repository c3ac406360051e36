// The MoE layer for a few tokens (a decode step): moe_layer_decode.
//
// The same layer as the kernel chain (COMET paper review §3.2: Layer0 = gate
// and up products with SwiGLU, Layer1 = down product; §4.1.1: the Top-K
// reduction), for at most MOE_DECODE_MAX_TOKENS tokens:
//   h[t,j,f] = silu(x[t].Wg[e,f]) * (x[t].Wu[e,f])         e = expert j of token t
//   out[t,n] = cast(sum_j w[t,j] (h[t,j].Wd[e,n]) + residual[t,n])
// What bounds it is reading the chosen experts' weights once from HBM (3 H F
// elements an expert; with r rows an expert there are r multiply-adds per
// weight, and the matrix cores only catch up with HBM at about 150 rows).
// So nothing is dispatched: a plan kernel routes and lists each held
// expert's pairs, and the two product kernels stream weight rows past the
// listed token rows (stream.hpp), reading x through the list.
//
// h is not rounded to the layer's type between the products as in the chain
// (there it halves the traffic of R x F values; here R is small): it is kept
// in f32, for bf16 weights as bf16 planes whose sum is the f32 value (three,
// exact, for an f32 output; two, 2^-16 of the value, for a bf16 output, whose
// own rounding is 2^-8).
// A weight that is infinite, and a product past the range, act as in f32
// (stream_resum).
#include "common.hpp"
#include "launch.hpp"
#include "stream.hpp"
#include "topk.hpp"

namespace moe {

constexpr int kStreamWaves = 4;
constexpr int kStreamThreads = 64 * kStreamWaves;
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxPairs = 256 * 16;
constexpr int kPlanMaxExperts = 512;

// ------------------------------------------------------------------ plan ---
// A token's experts and weights by its 16 lanes: softmax over the chosen
// logits, shifted by the largest, summed in slot order; a place left over
// (fewer than k logits above -inf) has weight 0 and belongs to no expert.
// Returns the held expert of slot q (-1: none).
template <int KMAX>
__device__ __forceinline__ int route_token(const float* __restrict__ logits, const DecodePlan& p, int t, int q,
                                           bool valid, bool store) {
  float vals[KMAX];
  int ids[KMAX];
  topk_row<KMAX>(logits + (int64_t)(valid ? t : 0) * p.E, p.E, q, valid, vals, ids);
  int e = -1;
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j == q && ids[j] < p.E) e = ids[j] - p.base;
  if (e >= p.EL || q >= p.k || !valid) e = -1;
  if (store && valid) {
    const float l0 = vals[0];
    float denom = 0.0f, mine = 0.0f;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (j >= p.k || ids[j] >= p.E) continue;
      const float v = expf(vals[j] - l0);
      denom += v;
      if (j == q) mine = v;
    }
    if (q < p.k) {
      const int f = t * p.k + q;
      p.w[f] = mine > 0.0f ? mine / denom : 0.0f;
      p.f2s[f] = e >= 0 ? f : -1;
    }
  }
  return e;
}

// 16 tokens a block: their weights and (in list) their pairs' experts.
template <int KMAX>
__global__ __launch_bounds__(256) void decode_route_kernel(const float* __restrict__ logits, DecodePlan p) {
  const int q = threadIdx.x % kLanesPerToken, t = blockIdx.x * 16 + threadIdx.x / kLanesPerToken;
  const int e = route_token<KMAX>(logits, p, t, q, t < p.M, true);
  if (t < p.M && q < p.k) p.list[t * p.k + q] = e;
}

// One workgroup: per held expert the list of its pairs f = t k + j, cut into
// entries of at most `rows` rows; entries past the last have none.  (Which place of an expert's list a pair
// gets is decided by an LDS atomic; a row's result does not depend on its
// place.)  KMAX 0: the route kernel has left the pairs' experts in list;
// otherwise the tokens are routed here.
template <int KMAX>
__global__ __launch_bounds__(kPlanThreads) void decode_plan_kernel(const float* __restrict__ logits, DecodePlan p) {
  __shared__ int cnt[kPlanMaxExperts], scan[kPlanMaxExperts], cur[kPlanMaxExperts];
  __shared__ short slot[kPlanMaxPairs];
  const int tid = threadIdx.x;
  for (int e = tid; e < p.EL; e += kPlanThreads) cnt[e] = 0;
  __syncthreads();
  if constexpr (KMAX == 0) {
    for (int f = tid; f < p.M * p.k; f += kPlanThreads) {
      const int e = p.list[f];
      slot[f] = (short)e;
      if (e >= 0) atomicAdd(&cnt[e], 1);
    }
  } else {
    const int q = tid % kLanesPerToken;
    for (int t0 = 0; t0 < p.M; t0 += kPlanThreads / kLanesPerToken) {
      const int t = t0 + tid / kLanesPerToken;
      const int e = route_token<KMAX>(logits, p, t, q, t < p.M, true);
      if (t < p.M && q < p.k) slot[t * p.k + q] = (short)e;
      if (e >= 0) atomicAdd(&cnt[e], 1);
    }
  }
  __syncthreads();
  // exclusive prefix over the experts of (pairs, entries), 16 bits each
  const int rows = p.rows;
  int c = 0, mine = 0;
  if (tid < p.EL) {
    c = cnt[tid];
    mine = c | (((c + rows - 1) / rows) << 16);
    scan[tid] = mine;
  }
  __syncthreads();
  for (int off = 1; off < p.EL; off <<= 1) {
    const int v = tid >= off && tid < p.EL ? scan[tid - off] : 0;
    __syncthreads();
    if (tid < p.EL) scan[tid] += v;
    __syncthreads();
  }
  if (tid < p.EL) {
    const int ex = scan[tid] - mine;
    const int start = ex & 0xFFFF, entry = ex >> 16;
    cur[tid] = start;
    for (int b = 0; b * rows < c; ++b) {
      int4 v;
      v.x = tid;
      v.y = start + b * rows;
      v.z = min(rows, c - b * rows);
      v.w = 0;
      p.entries[entry + b] = v;
    }
  }
  for (int i = (scan[p.EL - 1] >> 16) + tid; i < p.max_entries; i += kPlanThreads) p.entries[i] = int4{0, 0, 0, 0};
  __syncthreads();
  for (int f = tid; f < p.M * p.k; f += kPlanThreads)
    if (slot[f] >= 0) p.list[atomicAdd(&cur[slot[f]], 1)] = f;
}

// --------------------------------------------------------------- products ---
// Byte offset of the entry's token row i: pair list[i], at (pair / div) *
// pitch.  Past its end nothing is read.
__device__ __forceinline__ uint32_t decode_row(const DecodePlan& p, int4 ent, int i, int div, uint32_t pitch) {
  return i < ent.z ? (uint32_t)(p.list[ent.y + i] / div) * pitch : kNoRow;
}

// LDS of a product kernel: the waves' lines, then the sums of G groups.
template <class Op, int NW, int NT, int G>
constexpr int product_lds() {
  return kStreamWaves * imax(stream_line_bytes<Op, NW, NT>(), G * NT * 1024);
}

// h of one pair's 4 columns to its planes.
template <int NP>
__device__ __forceinline__ void store_h(const DecodeArgs& a, int64_t pair, int col, const f32x4_t& g, const f32x4_t& u) {
  f32x4_t h;
#pragma unroll
  for (int v = 0; v < 4; ++v) h[v] = silu_f32(g[v]) * u[v];
  if constexpr (NP == 0) {
    *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.hact) + pair * a.F + col) = h;
  } else {
    __bf16 pl[4][NP];
#pragma unroll
    for (int v = 0; v < 4; ++v) split_bf16<NP>(h[v], pl[v]);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const bf16x4_t o = {pl[0][p], pl[1][p], pl[2][p], pl[3][p]};
      *reinterpret_cast<bf16x4_t*>(reinterpret_cast<__bf16*>(a.hact) + (pair * NP + p) * a.F + col) = o;
    }
  }
}

// Layer0 of one entry: 16 columns of h for its rows.  NP: bf16 planes of h
// (0: f32).
template <class Op, int NT, int NP>
__device__ __forceinline__ void decode_l0_tile(const DecodeArgs& a, int4 ent, char* lds) {
  const int f0 = blockIdx.x * 16;
  StreamArgs s{};
  s.row_bytes = a.x_pitch;  // a gate or up row is as long as a row of x, in the same type
  const int64_t at = ((int64_t)ent.x * a.F + f0) * (int64_t)s.row_bytes;
  s.w0 = reinterpret_cast<const char*>(a.w_gate) + at;
  s.w1 = reinterpret_cast<const char*>(a.w_up) + at;
  s.w_rows = 16;
  s.x = a.x;
  s.x_bytes = (uint32_t)a.plan.M * a.x_pitch;
  s.lines = a.H / Op::kLine;
  f32x4_t acc[2][NT];
  const int wave = uniform(threadIdx.x >> 6);
  stream_tile<Op, kStreamWaves, 2, kPaired, NT, 4, true>(
      s, [&](int i) { return decode_row(a.plan, ent, i, a.plan.k, a.x_pitch); },
      lds + wave * stream_line_bytes<Op, 2, NT>(), acc);
  const int lane = threadIdx.x & 63;
  stream_reduce<kStreamWaves, 2, NT, 2, 2>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int, int j, const f32x4_t (&gu)[2]) {
    const int i = 16 * j + (lane & 15);
    if (i >= ent.z) return;
    store_h<NP>(a, a.plan.list[ent.y + i], f0 + 4 * (lane >> 4), gu[0], gu[1]);
  });
}

template <class Op, int MAXNT, int NP>
__global__ __launch_bounds__(kStreamThreads) void decode_l0_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[product_lds<Op, 2, MAXNT, 2>()];
  const int4 ent = a.plan.entries[blockIdx.y];
  if (ent.z == 0) return;
  if (MAXNT == 1 || ent.z <= 16)
    decode_l0_tile<Op, 1, NP>(a, ent, lds);
  else
    decode_l0_tile<Op, MAXNT, NP>(a, ent, lds);
}

// Layer0 where experts get many rows (entries of 64 or 128): the waves split
// the columns and share the token rows.
constexpr int kWideL0 = 4;  // waves; 16 columns each

template <class Op, int NT, int NP>
__device__ __forceinline__ void decode_l0_wide_tile(const DecodeArgs& a, int4 ent, char* lds) {
  const int f0 = blockIdx.x * 16 * kWideL0;
  StreamArgs s{};
  s.row_bytes = a.x_pitch;
  const int64_t at = ((int64_t)ent.x * a.F + f0) * (int64_t)s.row_bytes;
  s.w0 = reinterpret_cast<const char*>(a.w_gate) + at;
  s.w1 = reinterpret_cast<const char*>(a.w_up) + at;
  s.w_rows = 16 * kWideL0;
  s.x = a.x;
  s.x_bytes = (uint32_t)a.plan.M * a.x_pitch;
  s.lines = a.H / Op::kLine;
  f32x4_t acc[2][NT];
  stream_wide<Op, kWideL0, 2, kPaired, NT, 4, true>(
      s, [&](int i) { return decode_row(a.plan, ent, i, a.plan.k, a.x_pitch); }, lds, acc);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 16 * j + (lane & 15);
    if (i < ent.z) store_h<NP>(a, a.plan.list[ent.y + i], f0 + 16 * wave + 4 * (lane >> 4), acc[0][j], acc[1][j]);
  }
}

template <class Op, int MAXNT, int NP>
__global__ __launch_bounds__(64 * kWideL0) void decode_l0_wide_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[stream_wide_bytes<Op, kWideL0, 2, MAXNT>()];
  const int4 ent = a.plan.entries[blockIdx.y];
  if (ent.z == 0) return;
  if (ent.z <= 8 * MAXNT)
    decode_l0_wide_tile<Op, MAXNT / 2, NP>(a, ent, lds);
  else
    decode_l0_wide_tile<Op, MAXNT, NP>(a, ent, lds);
}

// Layer1 of one entry: 16 NW WAVES columns of y for its rows (f32, at the
// pair's own row).  Waves split the columns: h is wider than a weight row (two
// or three planes), so its lines are shared.  Block z of gridDim.z takes its
// share of the lines and has a y of its own, which the combine adds: so that
// there is a block for every CU where the tiles are large.
template <class Op, int WAVES, int NW, int NT, bool MX>
__device__ __forceinline__ void decode_l1_tile(const DecodeArgs& a, int4 ent, char* lds) {
  const int n0 = blockIdx.x * 16 * NW * WAVES;
  StreamArgs s{};
  const int64_t row0 = (int64_t)ent.x * a.H + n0;
  s.row_bytes = a.wd_pitch;
  s.w0 = reinterpret_cast<const char*>(a.w_down) + row0 * s.row_bytes;
  s.w_rows = min(16 * NW * WAVES, a.H - n0);
  s.x = a.hact;
  s.x_bytes = (uint32_t)(a.plan.M * a.plan.k) * a.h_pitch;
  s.plane = 2u * a.F;
  const int lines = a.F / Op::kLine, parts = gridDim.z;
  s.line0 = (int)blockIdx.z * lines / parts;
  s.lines = (int)(blockIdx.z + 1) * lines / parts - s.line0;
  if constexpr (MX) {
    s.scale = a.wd_scale + (row0 >> 5) * (int64_t)a.F;
    s.scale_row = (int)(row0 & 31);
    s.scale_pitch = a.F;
  }
  f32x4_t acc[NW][NT];
  constexpr int kDepth = Op::kXH * NT * Op::kP > 12 ? 2 : NW > 1 ? 3 : 4;
  float* y = a.y + (int64_t)blockIdx.z * a.plan.M * a.plan.k * a.H;
  stream_wide<Op, WAVES, NW, kOne, NT, kDepth, true>(
      s, [&](int i) { return decode_row(a.plan, ent, i, 1, a.h_pitch); }, lds, acc);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  bool nan = false;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int i = 16 * j + (lane & 15);
    if (i >= ent.z) continue;
    const int64_t pair = a.plan.list[ent.y + i];
#pragma unroll
    for (int g = 0; g < NW; ++g) {
      const int n = n0 + 16 * (wave * NW + g) + 4 * (lane >> 4);
      if (n < a.H) *reinterpret_cast<f32x4_t*>(y + pair * a.H + n) = acc[g][j];
#pragma unroll
      for (int c = 0; c < 4; ++c) nan |= n < a.H && __builtin_isnan(acc[g][j][c]);
    }
  }
  if constexpr (Op::kP > 1) {
    if (__any(nan)) {  // (after the stores, so that the usual path keeps its registers)
#pragma unroll 1
      for (int j = 0; j < NT * NW; ++j) {
        const int i = 16 * (j / NW) + (lane & 15), row = 16 * (wave * NW + j % NW) + 4 * (lane >> 4);
        const bool live = i < ent.z && n0 + row < a.H;
        const int64_t pair = live ? a.plan.list[ent.y + i] : 0;
        f32x4_t* at = reinterpret_cast<f32x4_t*>(y + pair * a.H + n0 + row);
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        if (live) v = *at;
        stream_resum<Op>(s, row, (uint32_t)pair * a.h_pitch, live, v);
        if (live) *at = v;
      }
    }
  }
}

template <class Op, int WAVES, int NW, int MAXNT, bool MX>
__global__ __launch_bounds__(64 * WAVES) void decode_l1_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[stream_wide_bytes<Op, WAVES, NW, MAXNT>()];
  const int4 ent = a.plan.entries[blockIdx.y];
  if (ent.z == 0) return;
  if (MAXNT > 1 && ent.z <= 8 * MAXNT)
    decode_l1_tile<Op, WAVES, NW, (MAXNT > 1 ? MAXNT / 2 : 1), MX>(a, ent, lds);
  else if (MAXNT == 8 && ent.z <= 96)
    decode_l1_tile<Op, WAVES, NW, (MAXNT == 8 ? 6 : MAXNT), MX>(a, ent, lds);
  else
    decode_l1_tile<Op, WAVES, NW, MAXNT, MX>(a, ent, lds);
}

// out[t, n .. n + 3] a thread: the pairs in slot order, each the sum of its
// PARTS parts in order; the loads of up to 16 of them are under way together.
template <int PARTS>
__global__ __launch_bounds__(256) void decode_combine_kernel(DecodeArgs a, OutEpilogue ep) {
  constexpr int U = PARTS > 4 ? 16 / PARTS : 4;
  const DecodePlan& p = a.plan;
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= (int64_t)p.M * a.H) return;
  const int t = (int)(i / a.H), n = (int)(i - (int64_t)t * a.H);
  const int64_t part = (int64_t)p.M * p.k * a.H;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int f0 = t * p.k; f0 < (t + 1) * p.k; f0 += U) {
    f32x4_t y[U][PARTS];
    float w[U];
    bool has[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int f = min(f0 + u, (t + 1) * p.k - 1);
      has[u] = f0 + u < (t + 1) * p.k && p.f2s[f] >= 0;
      w[u] = p.w[f];
      const float* at = a.y + (int64_t)f * a.H + n;
      if (!has[u]) continue;
#pragma unroll
      for (int s = 0; s < PARTS; ++s) y[u][s] = *reinterpret_cast<const f32x4_t*>(at + s * part);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!has[u]) continue;
#pragma unroll
      for (int s = 1; s < PARTS; ++s) y[u][0] += y[u][s];
      o.x = fmaf(w[u], y[u][0][0], o.x);
      o.y = fmaf(w[u], y[u][0][1], o.y);
      o.z = fmaf(w[u], y[u][0][2], o.z);
      o.w = fmaf(w[u], y[u][0][3], o.w);
    }
  }
  store_out(ep, i, o);
}

// ------------------------------------------------------------ few tokens ---
// At most 8 tokens and 64 pairs: two kernels.  Every Layer0 block routes the
// tokens itself (a few us that the other blocks' loads hide; a plan kernel in
// front takes 4 to 6 us alone) and its first blocks leave what Layer1 needs.
// Of the Layer1 blocks of 16 columns the one that is done last combines them
// (no block waits for another; the pairs are added in slot order whichever it
// is).  Layer1 blocks of 16 waves that own 16 columns of every pair need no
// such hand-over, but then each expert's stream starts when the one before
// has ended: 73 us at 8 tokens, 64 experts of 2048 x 1408, instead of 43.
// (Not kept: 8 waves a block, 15.2 + 11.2 us instead of 14.3 + 9.6 at one token
// and 4 such experts; every wave routing for itself without the exchange
// through LDS, 88 us instead of 78 for Layer0 of 2 experts 4096 x 14336.)
constexpr int kFewTokens = 8;
constexpr int kFewPairs = 64;
constexpr int kFewRows = 8;  // rows of one expert: one a token

// An expert and its pairs, past its rows the last one again; rows 0: none.
struct FewEntry {
  int expert, rows;
  int pair[kFewRows];
};

// The n-th distinct expert among the pairs' (lane f: pair f's, -1 none), in
// order of the first pair; rows 0: there are fewer.
__device__ __forceinline__ FewEntry few_entry(int slot, int n) {
  FewEntry e;
  uint64_t left = __ballot(slot >= 0), m = 0;
  e.expert = 0;
  for (int i = 0; i <= n; ++i) {
    if (left) e.expert = __builtin_amdgcn_readlane(slot, __ffsll((unsigned long long)left) - 1);
    m = left & __ballot(slot == e.expert);
    left &= ~m;
  }
  e.rows = __popcll(m);
  int last = 0;
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    if (m) last = __ffsll((unsigned long long)m) - 1;
    e.pair[i] = last;
    m &= m - 1;
  }
  return e;
}

template <class Op, int KMAX, int NP>
__global__ __launch_bounds__(kStreamThreads) void decode_few_l0_kernel(const float* __restrict__ logits, DecodeArgs a) {
  constexpr int kLine = stream_line_bytes<Op, 2, 1, kFewRows>();
  __shared__ __attribute__((aligned(16))) char lds[kStreamWaves * imax(kLine, 2048)];
  __shared__ int slots[kFewPairs];
  __shared__ FewEntry ent;
  const DecodePlan& p = a.plan;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int t = tid / kLanesPerToken, q = tid % kLanesPerToken;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < a.H / 16; i += kStreamThreads) a.arrived[i] = 0;
  if (wave * 64 < p.M * kLanesPerToken) {
    const int e = route_token<KMAX>(logits, p, t, q, t < p.M, blockIdx.x == 0 && blockIdx.y == 0);
    if (t < p.M && q < p.k) slots[t * p.k + q] = e;
  }
  __syncthreads();
  if (wave == 0) {
    FewEntry e;
    if (p.M == 1) {  // one token's experts are distinct
      e.expert = slots[blockIdx.y];
      e.rows = e.expert >= 0 ? 1 : 0;
#pragma unroll
      for (int i = 0; i < kFewRows; ++i) e.pair[i] = blockIdx.y;
    } else {
      e = few_entry(lane < p.M * p.k ? slots[lane] : -1, blockIdx.y);
    }
    if (lane == 0) {
      ent = e;
      if (blockIdx.x == 0) reinterpret_cast<FewEntry*>(p.entries)[blockIdx.y] = e;
    }
  }
  __syncthreads();
  const int rows = uniform(ent.rows);
  if (rows == 0) return;
  for (int f0 = blockIdx.x * 16; f0 < a.F; f0 += gridDim.x * 16) {
    StreamArgs s{};
    s.row_bytes = a.x_pitch;
    const int64_t at = ((int64_t)uniform(ent.expert) * a.F + f0) * (int64_t)s.row_bytes;
    s.w0 = reinterpret_cast<const char*>(a.w_gate) + at;
    s.w1 = reinterpret_cast<const char*>(a.w_up) + at;
    s.w_rows = 16;
    s.x = a.x;
    s.x_bytes = (uint32_t)p.M * a.x_pitch;
    s.lines = a.H / Op::kLine;
    f32x4_t acc[2][1];
    stream_share<Op, 2, kPaired, 1, 4, kFewRows, true>(
        s, wave, kStreamWaves, [&](int i) { return i < rows ? (uint32_t)(ent.pair[i] / p.k) * a.x_pitch : kNoRow; }, lds + wave * kLine, acc);
    stream_reduce<kStreamWaves, 2, 1, 2, 2>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int, int, const f32x4_t (&gu)[2]) {
      const int i = lane & 15;
      if (i < rows) store_h<NP>(a, ent.pair[i], f0 + 4 * (lane >> 4), gu[0], gu[1]);
    });
    __syncthreads();  // the sums are read before the next columns' lines come
  }
}

// 16 bytes of y between blocks: stored past the XCD's L2 and loaded past it
// (agent-scope accesses).  Ordering them with the count by waiting for the
// stores, instead of an agent-scope release, keeps the L2 from being written
// back by every block: 44 us instead of 352 for Layer1 at 8 tokens, 64
// experts of 2048 x 1408.
__device__ __forceinline__ void put_y(float* p, f32x4_t v) {
  typedef uint64_t u64x2_t __attribute__((ext_vector_type(2)));
  const u64x2_t u = __builtin_bit_cast(u64x2_t, v);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + 1, u[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t get_y(const float* p) {
  typedef uint64_t u64x2_t __attribute__((ext_vector_type(2)));
  u64x2_t u;
  u[0] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  u[1] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f32x4_t, u);
}

// Columns 16 x .. 16 x + 15 of entry y's pairs; the last block of the columns
// combines.
template <class Op, bool MX>
__global__ __launch_bounds__(kStreamThreads) void decode_few_l1_kernel(DecodeArgs a, OutEpilogue ep) {
  constexpr int kLine = stream_line_bytes<Op, 1, 1, kFewRows>();
  __shared__ __attribute__((aligned(16))) char lds[kStreamWaves * imax(kLine, 1024)];
  __shared__ int last;
  const DecodePlan& p = a.plan;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int n0 = blockIdx.x * 16;
  const FewEntry* __restrict__ ent = reinterpret_cast<const FewEntry*>(p.entries) + blockIdx.y;
  const int rows = uniform(ent->rows), expert = uniform(ent->expert);
  const int row_pair = ent->pair[lane >> 3], out_pair = ent->pair[lane & 7];  // (loaded together)
  if (rows > 0) {
    StreamArgs s{};
    const int64_t row0 = (int64_t)expert * a.H + n0;
    s.row_bytes = a.wd_pitch;
    s.w0 = reinterpret_cast<const char*>(a.w_down) + row0 * s.row_bytes;
    s.w_rows = 16;
    s.x = a.hact;
    s.x_bytes = (uint32_t)(p.M * p.k) * a.h_pitch;
    s.plane = 2u * a.F;
    s.lines = a.F / Op::kLine;
    if constexpr (MX) {
      s.scale = a.wd_scale + (row0 >> 5) * (int64_t)a.F;
      s.scale_row = (int)(row0 & 31);
      s.scale_pitch = a.F;
    }
    f32x4_t acc[1][1];
    stream_share<Op, 1, kOne, 1, 4, kFewRows, true>(
        s, wave, kStreamWaves, [&](int i) { return i < rows ? (uint32_t)(i == lane >> 3 ? row_pair : ent->pair[i]) * a.h_pitch : kNoRow; },
        lds + wave * kLine, acc);
    stream_reduce<kStreamWaves, 1, 1, 1, 1>(acc, reinterpret_cast<f32x4_t*>(lds), [&](int, int, const f32x4_t (&y)[1]) {
      f32x4_t v = y[0];
      const bool live = (lane & 15) < rows;
      stream_resum<Op>(s, 4 * (lane >> 4), (uint32_t)out_pair * a.h_pitch, live, v);
      if (live) put_y(a.y + (int64_t)out_pair * a.H + n0 + 4 * (lane >> 4), v);
    });
  }
  // wave 0 has stored the block's rows: it waits until they are at the point
  // that every XCD sees, then counts the block
  if (wave == 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (lane == 0)
      last = __hip_atomic_fetch_add(a.arrived + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             (int)gridDim.y - 1;
  }
  __syncthreads();
  if (!last) return;
  if (tid < p.M * 4) {
    const int t = tid >> 2, n = n0 + 4 * (tid & 3);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // 4 slots' loads in flight: each comes from beyond the L2
    for (int f0 = t * p.k; f0 < (t + 1) * p.k; f0 += 4) {
      f32x4_t y[4];
      float w[4];
      bool has[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int f = min(f0 + u, (t + 1) * p.k - 1);
        y[u] = get_y(a.y + (int64_t)f * a.H + n);  // (of a pair of no held expert: not used)
        w[u] = p.w[f];
        has[u] = f0 + u < (t + 1) * p.k && p.f2s[f] >= 0;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!has[u]) continue;
        o.x = fmaf(w[u], y[u][0], o.x);
        o.y = fmaf(w[u], y[u][1], o.y);
        o.z = fmaf(w[u], y[u][2], o.z);
        o.w = fmaf(w[u], y[u][3], o.w);
      }
    }
    store_out(ep, (int64_t)t * a.H + n, o);
  }
}

// ---------------------------------------------------------------- launch ---
template <class Op0, class Op1, int NP, bool MX>
static void launch_few(const DecodeArgs& a, const float* logits, const OutEpilogue& ep, hipStream_t s) {
  const DecodePlan& p = a.plan;
  const int pairs = p.M * p.k;
  // one token's entries are its slots, held or not
  const int entries = p.M == 1 ? p.k : p.EL < pairs ? p.EL : pairs;
  // Layer0 of short rows: as many blocks as are resident at once (7 on a CU),
  // each taking the same number of column groups; more of them would only route
  // again (8 tokens, k = 8, 64 experts of 2048 x 1408: 84 us instead of 109; 22
  // experts of 448 x 4992: 51 instead of 73).  Rows of more than 4 KiB hide the
  // routing (8 tokens, 8 experts of 4096 x 14336: 276 us in turn, 263 not).
  const int groups = a.F / 16, at_once = 7 * device_cu_count();
  const int turns = a.x_pitch > 4096 ? 1 : (groups * entries + at_once - 1) / at_once;
  const dim3 grid((unsigned)((groups + turns - 1) / turns), (unsigned)entries);
  if (p.k <= 2)
    decode_few_l0_kernel<Op0, 2, NP><<<grid, kStreamThreads, 0, s>>>(logits, a);
  else if (p.k <= 4)
    decode_few_l0_kernel<Op0, 4, NP><<<grid, kStreamThreads, 0, s>>>(logits, a);
  else if (p.k <= 8)
    decode_few_l0_kernel<Op0, 8, NP><<<grid, kStreamThreads, 0, s>>>(logits, a);
  else
    decode_few_l0_kernel<Op0, 16, NP><<<grid, kStreamThreads, 0, s>>>(logits, a);
  decode_few_l1_kernel<Op1, MX><<<dim3((unsigned)(a.H / 16), grid.y), kStreamThreads, 0, s>>>(a, ep);
}

// Rows an entry may hold, in 16s.  An expert gets at most one row of every
// token: 16 tokens need no more than 16.  Beyond, entries of 32 rows stream
// the weights by reduction-splitting waves, entries of 64 and 128 by
// column-splitting ones that share the rows; the latter where experts get more
// than 24 (40) rows on average, so that few experts' weights are read twice.
// (Layer0 of 8 experts 4096 x 14336: 25 rows each 305 us with 32-row entries,
// 345 with 64; 50 rows each, where every expert takes two entries of 32, 540
// and 345.)
// MXFP8's token lines are twice as long: 128 rows do not fit the LDS.
// Where the wide Layer0 would leave most CUs idle (f32, which the matrix cores
// bound: some), its entries stay at 32 rows (73 tokens, 4 experts of 2368 x
// 448, f32: 20 us instead of 91; 144 tokens, 6 experts of 1856 x 640: 25
// instead of 29; but 60 tokens, 6 experts of 512 x 2432: 20 instead of 11).
// Layer1's reduction is cut into parts until every CU has a block (29 tokens, 4
// experts of 960 x 10368, f32: 32 us instead of 217; 51 tokens, 3 experts of
// that size, bf16: 16 instead of 67; until it has four: 200 tokens, 8 experts
// of 4096 x 14336, 229 instead of 200).
DecodeSplit decode_split(int M, int k, int E, int EL, int H, int F, int dtype) {
  const bool mx = dtype == MOE_DTYPE_BF16_MXFP8, f32 = dtype == MOE_DTYPE_F32;
  const int R = M * k, cus = device_cu_count();
  const int64_t held = ((int64_t)R * EL + E - 1) / E;  // of the pairs, about
  const int experts = held < 1 ? 1 : (int)(held < EL ? held : EL);
  DecodeSplit d;
  d.nt = M <= 16 ? 1 : M <= 32 || R <= 24 * E ? 2 : mx || M <= 64 || R <= 40 * E ? 4 : 8;
  if (d.nt > 2 && F / 64 * experts < (f32 ? cus : cus / 4)) d.nt = 2;
  const int64_t rows = (held + experts - 1) / experts;
  const int64_t entries = experts * ((rows + 16 * d.nt - 1) / (16 * d.nt));
  const int64_t blocks = (H + 127) / 128 * entries / (d.nt > 2 && !mx ? 2 : 1);
  const int lines = F / (mx ? 128 : f32 ? 32 : 64);
  d.parts = d.nt > 2 ? 2 : 1;
  while (d.parts < 8 && blocks * d.parts < cus && lines >= 8 * d.parts) d.parts *= 2;
  return d;
}

int decode_max_entries(int M, int k, int EL, int nt) {
  const int R = M * k;
  return (EL < R ? EL : R) + R / (16 * nt);
}

size_t decode_entry_bytes(int max_entries) {
  const size_t many = sizeof(int4) * (size_t)max_entries, few = sizeof(FewEntry) * kFewPairs;
  return many > few ? many : few;
}

template <class Op0, class Op1, int NP, bool MX>
static void launch_products(const DecodeArgs& a, hipStream_t s) {
  const int entries = a.plan.max_entries;
  auto grid = [&](int n, int cols, int parts = 1) {
    return dim3((unsigned)((n + cols - 1) / cols), (unsigned)entries, (unsigned)parts);
  };
  const int parts = a.split.parts;
  constexpr int NW1 = MX ? 1 : 2;  // (MXFP8's lines take the registers of the second group)
  switch (a.split.nt) {
    case 1:
      decode_l0_kernel<Op0, 1, NP><<<grid(a.F, 16), kStreamThreads, 0, s>>>(a);
      decode_l1_kernel<Op1, 4, 2, 1, MX><<<grid(a.H, 128, parts), 256, 0, s>>>(a);
      break;
    case 2:
      decode_l0_kernel<Op0, 2, NP><<<grid(a.F, 16), kStreamThreads, 0, s>>>(a);
      decode_l1_kernel<Op1, 4, 2, 2, MX><<<grid(a.H, 128, parts), 256, 0, s>>>(a);
      break;
    case 4:
      decode_l0_wide_kernel<Op0, 4, NP><<<grid(a.F, 16 * kWideL0), 64 * kWideL0, 0, s>>>(a);
      decode_l1_kernel<Op1, 8, NW1, 4, MX><<<grid(a.H, 128 * NW1, parts), 512, 0, s>>>(a);
      break;
    default:
      if constexpr (!MX) {
        decode_l0_wide_kernel<Op0, 8, NP><<<grid(a.F, 16 * kWideL0), 64 * kWideL0, 0, s>>>(a);
        decode_l1_kernel<Op1, 8, NW1, 8, MX><<<grid(a.H, 128 * NW1, parts), 512, 0, s>>>(a);
      }
  }
}

template <int KMAX>
static void launch_plan(const float* logits, const DecodePlan& p, hipStream_t s) {
  // routed by the plan's one workgroup (64 tokens at a time) where that takes
  // less than a launch: 4.5 us at 17 tokens, k = 2; at 64 tokens, k = 8, 15 us
  // against 4 + 4
  if constexpr (KMAX <= 4) {
    if ((p.M + 63) / 64 * KMAX <= 4) {
      decode_plan_kernel<KMAX><<<1, kPlanThreads, 0, s>>>(logits, p);
      return;
    }
  }
  decode_route_kernel<KMAX><<<(p.M + 15) / 16, 256, 0, s>>>(logits, p);
  decode_plan_kernel<0><<<1, kPlanThreads, 0, s>>>(nullptr, p);
}

hipError_t launch_decode(const DecodeArgs& a, const float* logits, int dtype, int planes, const OutEpilogue& ep,
                         hipStream_t s) {
  const DecodePlan& p = a.plan;
  if (p.M <= kFewTokens && p.M * p.k <= kFewPairs) {
    if (dtype == MOE_DTYPE_F32)
      launch_few<StreamF32, StreamF32, 0, false>(a, logits, ep, s);
    else if (dtype == MOE_DTYPE_BF16 && planes == 3)
      launch_few<StreamBf16<1>, StreamBf16<3>, 3, false>(a, logits, ep, s);
    else if (dtype == MOE_DTYPE_BF16)
      launch_few<StreamBf16<1>, StreamBf16<2>, 2, false>(a, logits, ep, s);
    else if (planes == 3)
      launch_few<StreamBf16<1>, StreamMx<3>, 3, true>(a, logits, ep, s);
    else
      launch_few<StreamBf16<1>, StreamMx<2>, 2, true>(a, logits, ep, s);
    return hipGetLastError();
  }
  if (p.k <= 2)
    launch_plan<2>(logits, p, s);
  else if (p.k <= 4)
    launch_plan<4>(logits, p, s);
  else if (p.k <= 8)
    launch_plan<8>(logits, p, s);
  else
    launch_plan<16>(logits, p, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (dtype == MOE_DTYPE_F32)
    launch_products<StreamF32, StreamF32, 0, false>(a, s);
  else if (dtype == MOE_DTYPE_BF16 && planes == 3)
    launch_products<StreamBf16<1>, StreamBf16<3>, 3, false>(a, s);
  else if (dtype == MOE_DTYPE_BF16)
    launch_products<StreamBf16<1>, StreamBf16<2>, 2, false>(a, s);
  else if (planes == 3)
    launch_products<StreamBf16<1>, StreamMx<3>, 3, true>(a, s);
  else
    launch_products<StreamBf16<1>, StreamMx<2>, 2, true>(a, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned blocks = (unsigned)(((int64_t)p.M * a.H / 4 + 255) / 256);
  switch (a.split.parts) {
    case 1: decode_combine_kernel<1><<<blocks, 256, 0, s>>>(a, ep); break;
    case 2: decode_combine_kernel<2><<<blocks, 256, 0, s>>>(a, ep); break;
    case 4: decode_combine_kernel<4><<<blocks, 256, 0, s>>>(a, ep); break;
    default: decode_combine_kernel<8><<<blocks, 256, 0, s>>>(a, ep);
  }
  return hipGetLastError();
}

}  // namespace moe
