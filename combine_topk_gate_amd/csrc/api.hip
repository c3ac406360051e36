// C ABI of the library: host-side argument checks, workspace carving and
// kernel launches.  Every entry point only enqueues work on the caller's
// stream; none synchronises (except moe_debug_device_status, a test hook).
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <exception>
#include <vector>

#include "common.hpp"
#include "launch.hpp"
#include "layer.hpp"

namespace {

using namespace moe;

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// bytes per element of x and X_perm (and of Hact unless it is MXFP8)
size_t elem_bytes(const moe_problem_t* p) { return p->dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool is_mx(const moe_problem_t* p) { return p->dtype == MOE_DTYPE_BF16_MXFP8; }
// bytes of the Hact buffer: R x F elements, or an MXFP8 buffer (codes + scales)
size_t hact_bytes(const moe_problem_t* p, int64_t R) {
  return is_mx(p) ? (size_t)R * p->ffn + (size_t)mx_scale_bytes(R, p->ffn) : (size_t)R * p->ffn * elem_bytes(p);
}

// Whether the bf16 grouped GEMM combines each expert's segments of all the
// source blocks into one: with source blocks whose (block, expert)
// segments hold fewer rows than a tile on average (R EL / E kept pairs over
// S EL segments, i.e. R / (E S) < 256), such as the expert-parallel share
// that holds a few of many experts.
bool combine_blocks(const moe_problem_t* p) {
  return p->dtype == MOE_DTYPE_BF16 && p->num_src_blocks > 1 &&
         p->num_tokens * p->topk < 256ll * p->num_experts * p->num_src_blocks;
}

// Experts held by the call (weights it is given): EL, or all E.
int held(const moe_problem_t* p) { return p->local_experts > 0 ? p->local_experts : p->num_experts; }
int held_base(const moe_problem_t* p) { return p->local_experts > 0 ? p->expert_base : 0; }
// Segments: S * EL.
int segments(const moe_problem_t* p) { return p->num_src_blocks * held(p); }

moe_status_t check_problem(const moe_problem_t* p) {
  if (!p) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t M = p->num_tokens;
  if (M < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->hidden < 64 || p->hidden > 65536 || p->hidden % 64) return MOE_ERR_INVALID_ARGUMENT;
  if (p->ffn < 64 || p->ffn > 65536 || p->ffn % 64) return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_experts < 1 || p->num_experts > 512) return MOE_ERR_INVALID_ARGUMENT;
  if (p->topk < 1 || p->topk > 16 || p->topk > p->num_experts) return MOE_ERR_INVALID_ARGUMENT;
  if (p->local_experts < 0 || p->expert_base < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->local_experts == 0 && p->expert_base != 0) return MOE_ERR_INVALID_ARGUMENT;
  if ((int64_t)p->expert_base + p->local_experts > p->num_experts) return MOE_ERR_INVALID_ARGUMENT;
  // dropped pairs take one more segment in the bookkeeping
  const int64_t ranked = (int64_t)p->num_src_blocks * held(p) + (held(p) < p->num_experts ? 1 : 0);
  if (p->num_src_blocks < 1 || ranked > 1024) return MOE_ERR_INVALID_ARGUMENT;
  if (p->dtype != MOE_DTYPE_F32 && p->dtype != MOE_DTYPE_BF16 && p->dtype != MOE_DTYPE_BF16_MXFP8)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->dtype == MOE_DTYPE_BF16_MXFP8 && p->ffn % 128) return MOE_ERR_UNSUPPORTED;
  if (M >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;  // bounded before M * topk is formed
  const int64_t R = M * p->topk;
  if (R >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  const int64_t wide = p->hidden > p->ffn ? p->hidden : p->ffn;
  if (R * wide >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  // weights are addressed per expert with 64-bit offsets; the MXFP8 weight
  // scales are one buffer range of EL*H*F/32 bytes, below 2^32
  if ((int64_t)held(p) * p->hidden * p->ffn >= (1ll << 37)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

PermutePlan plan_of(const moe_problem_t* p) {
  return permute_plan(p->num_tokens, p->topk, p->num_src_blocks, p->num_experts, held_base(p), p->local_experts);
}

// Epilogue of the combine from the caller's description (null: plain f32).
moe_status_t epilogue_of(const moe_problem_t* p, const moe_epilogue_t* epi, void* out, OutEpilogue* ep) {
  ep->out = out;
  ep->residual = nullptr;
  ep->res_bf16 = p->dtype != MOE_DTYPE_F32;  // the dtype of x: bf16 for the bf16 and MXFP8 layers
  ep->out_bf16 = 0;
  if (epi) {
    if (epi->out_dtype != MOE_DTYPE_F32 && epi->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
    ep->out_bf16 = epi->out_dtype == MOE_DTYPE_BF16;
    ep->residual = epi->residual;
    if (epi->residual && ((uintptr_t)epi->residual % 16)) return MOE_ERR_INVALID_ARGUMENT;
  }
  if ((uintptr_t)out % 16) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status_t hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// ------------------------------------------------------ debug validation --
// MOE_DEBUG_VALIDATE=1 in the environment: before launching anything, each
// entry point copies the device-resident inputs it trusts to the host
// (synchronising the stream) and checks them: logits finite, topk_idx in
// [0, E), src_block in [0, S), offsets starting at 0, non-decreasing and
// ending at most at R, flat_to_sorted in [-1, R).  A failed check returns
// MOE_ERR_INVALID_ARGUMENT and launches nothing.  Host memory only; for
// debugging, not for timed runs.
bool debug_validate() {
  const char* v = getenv("MOE_DEBUG_VALIDATE");
  return v && v[0] == '1' && v[1] == 0;
}

// MOE_DEBUG_SHUFFLE=<n>: the seed of the reordering check (0 or unset: the
// usual order; anything but a decimal number below 2^32 counts as unset).
uint32_t debug_shuffle() {
  const char* v = getenv("MOE_DEBUG_SHUFFLE");
  if (!v || !*v) return 0;
  uint64_t n = 0;
  for (const char* c = v; *c; ++c) {
    if (*c < '0' || *c > '9') return 0;
    n = n * 10 + (uint64_t)(*c - '0');
    if (n > 0xffffffffull) return 0;
  }
  return (uint32_t)n;
}

template <typename T>
bool fetch(std::vector<T>& h, const T* d, int64_t n, hipStream_t s) {
  try {
    h.resize(n > 0 ? (size_t)n : 0);
  } catch (const std::exception&) {  // no host memory for the copy: no exception leaves the C ABI
    return false;
  }
  if (n <= 0) return true;
  if (hipMemcpyAsync(h.data(), d, (size_t)n * sizeof(T), hipMemcpyDeviceToHost, s) != hipSuccess) return false;
  return hipStreamSynchronize(s) == hipSuccess;
}

moe_status_t check_range(const int32_t* d, int64_t n, int32_t lo, int32_t hi, hipStream_t s) {
  std::vector<int32_t> h;
  if (!fetch(h, d, n, s)) return MOE_ERR_HIP;
  for (int32_t v : h)
    if (v < lo || v >= hi) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status_t validate_logits(const moe_problem_t* p, const float* logits, hipStream_t s) {
  std::vector<float> h;
  if (!fetch(h, logits, p->num_tokens * (int64_t)p->num_experts, s)) return MOE_ERR_HIP;
  for (float v : h)
    if (!isfinite(v)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status_t validate_routing(const moe_problem_t* p, const int32_t* topk_idx, const int32_t* src_block,
                              hipStream_t s) {
  moe_status_t st = check_range(topk_idx, p->num_tokens * (int64_t)p->topk, 0, p->num_experts, s);
  if (st == MOE_OK && p->num_src_blocks > 1) st = check_range(src_block, p->num_tokens, 0, p->num_src_blocks, s);
  return st;
}

moe_status_t validate_offsets(const moe_problem_t* p, const int32_t* offsets, hipStream_t s) {
  std::vector<int32_t> h;
  const int G = segments(p);
  if (!fetch(h, offsets, G + 1, s)) return MOE_ERR_HIP;
  if (h[0] != 0) return MOE_ERR_INVALID_ARGUMENT;
  for (int g = 0; g < G; ++g)
    if (h[g + 1] < h[g]) return MOE_ERR_INVALID_ARGUMENT;
  if ((int64_t)h[G] > p->num_tokens * p->topk) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// ------------------------------------------------------------ dispatch ---
// Argument checks of moe_dispatch and its allocation-free variant.
moe_status_t check_dispatch(const moe_problem_t* p, const void* x, const int32_t* topk_idx,
                            const int32_t* src_block, const int32_t* counts, const int32_t* offsets,
                            const int32_t* sorted_to_flat, const int32_t* flat_to_sorted, const void* x_perm) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!counts || !offsets) return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_src_blocks > 1 && !src_block && p->num_tokens > 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_tokens > 0) {
    if (!x || !topk_idx || !sorted_to_flat || !flat_to_sorted || !x_perm) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(x_perm, 16)) return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

// Bookkeeping and copy of the dispatch with the scratch `ws` (already sized).
moe_status_t dispatch_launch(const moe_problem_t* p, const void* x, const int32_t* topk_idx,
                             const int32_t* src_block, int32_t* counts, int32_t* offsets, int32_t* sorted_to_flat,
                             int32_t* flat_to_sorted, void* x_perm, void* ws, hipStream_t s) {
  if (debug_validate() && p->num_tokens > 0) {
    const moe_status_t st = validate_routing(p, topk_idx, src_block, s);
    if (st != MOE_OK) return st;
  }
  return hip_status(launch_dispatch(plan_of(p), topk_idx, p->num_src_blocks > 1 ? src_block : nullptr, counts,
                                    offsets, sorted_to_flat, flat_to_sorted, x, (int64_t)p->hidden * elem_bytes(p),
                                    x_perm, (int32_t*)ws, s));
}

// Workspace of the whole layer, carved in this order (each region 256-B aligned).
struct LayerWs {
  size_t status, topk_idx, topk_w, counts, offsets, s2f, f2s, perm, x_perm, hact, y, fused, gemm, total;
};

LayerWs layer_ws(const moe_problem_t* p) {
  const int64_t M = p->num_tokens, R = M * p->topk;
  const int G = segments(p);
  const size_t eb = elem_bytes(p);
  const PermutePlan pl = plan_of(p);
  LayerWs w;
  size_t o = 0;
  w.status = o; o += align_up(kAlign);
  w.topk_idx = o; o += align_up((size_t)R * 4);
  w.topk_w = o; o += align_up((size_t)R * 4);
  w.counts = o; o += align_up((size_t)G * 4);
  w.offsets = o; o += align_up((size_t)(G + 1) * 4);
  w.s2f = o; o += align_up((size_t)R * 4);
  w.f2s = o; o += align_up((size_t)R * 4);
  w.perm = o; o += align_up(permute_ws_bytes(pl));
  w.x_perm = o; o += align_up((size_t)R * p->hidden * eb);
  w.hact = o; o += align_up(hact_bytes(p, R));
  w.y = o; o += align_up((size_t)R * p->hidden * 4);
  w.fused = o; o += align_up(fused_ws_bytes(p->num_tokens, p->hidden, p->ffn, held(p), p->topk,
                                             p->num_src_blocks));
  w.gemm = o; o += align_up(p->dtype == MOE_DTYPE_BF16 ? gemm_split_ws_bytes() : 0);  // MXFP8 does not split
  w.total = o;
  return w;
}

// ------------------------------------------------------- decode layer ----
// bf16 planes of h (0: f32): three hold the f32 value exactly, two hold it
// to 2^-16, for a bf16 output.
int decode_planes(const moe_problem_t* p, const OutEpilogue& ep) {
  return p->dtype == MOE_DTYPE_F32 ? 0 : ep.out_bf16 ? 2 : 3;
}

struct DecodeWs {
  size_t entries, list, f2s, w, arrived, hact, y, total;
};

DecodeSplit split_of(const moe_problem_t* p) {
  return decode_split((int)p->num_tokens, p->topk, p->num_experts, held(p), p->hidden, p->ffn, p->dtype);
}

// The workspace does not depend on the output's type (three planes).
DecodeWs decode_ws(const moe_problem_t* p, const DecodeSplit& split) {
  const int M = (int)p->num_tokens, R = M * p->topk;
  DecodeWs w;
  size_t o = 0;
  w.entries = o; o += align_up(decode_entry_bytes(decode_max_entries(M, p->topk, held(p), split.nt)));
  w.list = o; o += align_up((size_t)R * 4);
  w.f2s = o; o += align_up((size_t)R * 4);
  w.w = o; o += align_up((size_t)R * 4);
  w.arrived = o; o += align_up((size_t)p->hidden / 16 * 4);
  w.hact = o; o += align_up((size_t)R * p->ffn * (p->dtype == MOE_DTYPE_F32 ? 4 : 6));
  w.y = o; o += align_up((size_t)R * p->hidden * 4 * split.parts);
  w.total = o;
  return w;
}

moe_status_t check_decode(const moe_problem_t* p) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  return p->num_tokens > MOE_DECODE_MAX_TOKENS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}

// out may be the residual itself (same place, same type: every element is
// read by the thread that writes it); any other overlap is an error.
bool residual_clash(const OutEpilogue& ep, int64_t n) {
  if (!ep.residual) return false;
  const size_t nr = (size_t)n * (ep.res_bf16 ? 2 : 4), no = (size_t)n * (ep.out_bf16 ? 2 : 4);
  if (ep.residual == ep.out && nr == no) return false;
  return overlap(ep.residual, nr, ep.out, no);
}

// ------------------------------------------------- adapter projection ----
moe_status_t check_adapter(const moe_adapter_problem_t* q) {
  if (!q) return MOE_ERR_INVALID_ARGUMENT;
  if (q->num_tokens < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (q->in_features < 64 || q->in_features > 65536 || q->in_features % 64) return MOE_ERR_INVALID_ARGUMENT;
  if (q->out_features < 1 || q->out_features > 65536) return MOE_ERR_INVALID_ARGUMENT;
  if (q->num_adapters < 0 || q->num_adapters > 65536) return MOE_ERR_INVALID_ARGUMENT;
  if (q->num_adapters > 0 && (q->rank < 8 || q->rank > 256 || q->rank % 8)) return MOE_ERR_INVALID_ARGUMENT;
  if (q->dtype != MOE_DTYPE_F32 && q->dtype != MOE_DTYPE_BF16)
    return q->dtype == MOE_DTYPE_BF16_MXFP8 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARGUMENT;
  // grids: 512 work items per 16 rows, below 2^32; a block per 16 x 16 outputs
  if (q->num_tokens >= (1ll << 27) || q->num_tokens * q->out_features >= (1ll << 40)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t adapter_ws(const moe_adapter_problem_t* q) {
  return q->num_adapters > 0 ? align_up((size_t)q->num_tokens * q->rank * 6) : 0;  // f32, or three bf16 planes
}

// Sizes and types of a valid problem; the pointers are left to the call.
AdapterArgs adapter_args(const moe_adapter_problem_t* q, int32_t out_dtype) {
  const bool f32 = q->dtype == MOE_DTYPE_F32;
  AdapterArgs g{};
  g.M = q->num_tokens;
  g.H = q->in_features;
  g.N = q->out_features;
  g.P = q->num_adapters;
  g.r = g.P > 0 ? q->rank : 0;
  g.out.res_bf16 = !f32;
  g.out.out_bf16 = out_dtype == MOE_DTYPE_BF16;
  g.planes = 1;  // set by the launcher
  g.row_bytes = (uint32_t)(g.H * (f32 ? 4 : 2));
  return g;
}

// ------------------------------------------------------------- training ---
// Pairs that an even routing keeps.
int64_t kept_rows(const moe_problem_t* p) { return p->num_tokens * p->topk * held(p) / p->num_experts; }

// A buffer of a call, for the checks: bytes, and whether the call writes it.
struct Span {
  const void* p;
  size_t n;
  bool out;
};

// Every tensor given and 16-byte aligned, and no output overlaps another span.
moe_status_t check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (!s[i].p && s[i].n) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(s[i].p, 16)) return MOE_ERR_INVALID_ARGUMENT;
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((s[i].out || s[j].out) && overlap(s[i].p, s[i].n, s[j].p, s[j].n)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// An index or per-pair array: given and 4-byte aligned, and apart from the outputs.
moe_status_t check_words(const void* p, size_t n, const Span* s, int ns) {
  if ((!p && n) || !aligned(p, 4)) return MOE_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < ns; ++i)
    if (s[i].out && overlap(p, n, s[i].p, s[i].n)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// The kernels' dropout from the caller's description (null: none, rng null).
moe_status_t dropout_of(const moe_dropout_t* drop, Dropout* d) {
  d->rng = nullptr;
  d->threshold = 0;
  d->scale = 1.0f;
  if (!drop) return MOE_OK;
  if (!(drop->p >= 0.0 && drop->p < 1.0)) return MOE_ERR_INVALID_ARGUMENT;  // NaN too
  if (!drop->rng || !aligned(drop->rng, 8)) return MOE_ERR_INVALID_ARGUMENT;
  d->rng = drop->rng;
  d->threshold = (uint32_t)(drop->p * 4294967296.0);
  d->scale = (float)(1.0 / (1.0 - drop->p));
  return MOE_OK;
}

// Problem and layer of a gradient of the grouped GEMM.
moe_status_t check_grad_gemm(const moe_problem_t* p, int32_t layer) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (layer != 0 && layer != 1) return MOE_ERR_INVALID_ARGUMENT;
  return is_mx(p) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The workspace of a gradient of the grouped GEMM, and that it overlaps nothing.
moe_status_t check_grad_ws(const moe_problem_t* p, const void* ws, size_t ws_bytes, const Span* s, int n,
                           const int32_t* offsets) {
  const size_t need = moe_workspace_bytes(p, MOE_OP_GROUPED_GEMM_BACKWARD);
  if (need == 0) return MOE_OK;
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, kAlign) || overlap(ws, need, offsets, (size_t)(segments(p) + 1) * 4)) return MOE_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < n; ++i)
    if (overlap(ws, need, s[i].p, s[i].n)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

GradGemmArgs grad_args(const moe_problem_t* p, int layer, const int32_t* offsets) {
  GradGemmArgs g{};
  g.layer = layer;
  g.offsets = offsets;
  g.R = p->num_tokens * p->topk;
  g.rows = kept_rows(p);
  g.H = p->hidden;
  g.F = p->ffn;
  g.E = held(p);
  g.G = segments(p);
  g.shuffle = debug_shuffle();
  return g;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(ws) + off);
}

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return (2 << 16) | 3; }

const char* moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARGUMENT: return "MOE_ERR_INVALID_ARGUMENT";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_WORKSPACE_TOO_SMALL: return "MOE_ERR_WORKSPACE_TOO_SMALL";
    case MOE_ERR_HIP: return "MOE_ERR_HIP";
    case MOE_ERR_DEVICE_TIMEOUT: return "MOE_ERR_DEVICE_TIMEOUT";
  }
  return "MOE_ERR_UNKNOWN";
}

size_t moe_workspace_bytes(const moe_problem_t* p, int32_t op) {
  if (check_problem(p) != MOE_OK) return 0;
  switch (op) {
    case MOE_OP_DISPATCH: return permute_ws_bytes(plan_of(p));
    case MOE_OP_GROUPED_GEMM: return p->dtype == MOE_DTYPE_BF16 ? gemm_split_ws_bytes() : 0;
    case MOE_OP_LAYER: return layer_ws(p).total;
    case MOE_OP_GROUPED_GEMM_BACKWARD:
      return is_mx(p) ? 0 : align_up(grad_ws_bytes(grad_args(p, 0, nullptr), p->dtype == MOE_DTYPE_BF16));
    case MOE_OP_LAYER_DECODE: return check_decode(p) == MOE_OK ? decode_ws(p, split_of(p)).total : 0;
  }
  return 0;
}

moe_status_t moe_route(const moe_problem_t* p, const float* logits, int32_t* topk_idx, float* topk_w, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (debug_validate()) {
    st = validate_logits(p, logits, (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  return hip_status(launch_route(logits, p->num_tokens, p->num_experts, p->topk, topk_idx, topk_w,
                                 (hipStream_t)stream));
}

moe_status_t moe_dispatch(const moe_problem_t* p, const void* x, const int32_t* topk_idx, const int32_t* src_block,
                          int32_t* counts, int32_t* offsets, int32_t* sorted_to_flat, int32_t* flat_to_sorted,
                          void* x_perm, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = check_dispatch(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm);
  if (st != MOE_OK) return st;
  if (ws_bytes < permute_ws_bytes(plan_of(p)) || !ws) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return dispatch_launch(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm, ws,
                         (hipStream_t)stream);
}

moe_status_t moe_dispatch_noalloc(const moe_problem_t* p, const void* x, const int32_t* topk_idx,
                                  const int32_t* src_block, int32_t* counts, int32_t* offsets,
                                  int32_t* sorted_to_flat, int32_t* flat_to_sorted, void* x_perm, void* stream) {
  moe_status_t st = check_dispatch(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm);
  if (st != MOE_OK) return st;
  if (permute_ws_bytes(plan_of(p)) > MOE_NOALLOC_SCRATCH_BYTES) return MOE_ERR_UNSUPPORTED;
  void* scratch_addr = nullptr;
  if (static_scratch(&scratch_addr) != hipSuccess) return MOE_ERR_HIP;
  return dispatch_launch(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm,
                         scratch_addr, (hipStream_t)stream);
}

moe_status_t moe_grouped_gemm(const moe_problem_t* p, int32_t layer, const void* a, const void* w0, const void* w1,
                              const int32_t* offsets, void* c, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (layer != 0 && layer != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!offsets || !w0 || (layer == 0 && !w1)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t R = p->num_tokens * p->topk;
  if (R > 0 && (!a || !c)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(a, 16) || !aligned(c, 16) || !aligned(w0, 16) || (layer == 0 && !aligned(w1, 16)))
    return MOE_ERR_INVALID_ARGUMENT;
  GemmProblem gp;
  gp.layer = layer;
  gp.a = a;
  gp.w0 = w0;
  gp.w1 = layer == 0 ? w1 : nullptr;
  gp.offsets = offsets;
  gp.c = c;
  gp.R = R;
  gp.K = layer == 0 ? p->hidden : p->ffn;
  gp.N = layer == 0 ? p->ffn : p->hidden;
  gp.E = held(p);
  gp.G = segments(p);
  // a workspace smaller than moe_workspace_bytes(p, MOE_OP_GROUPED_GEMM)
  // (or none) only disables the split of the last round
  if (ws && !aligned(ws, 16)) return MOE_ERR_INVALID_ARGUMENT;
  gp.ws = ws;
  gp.ws_bytes = ws ? ws_bytes : 0;
  gp.rowmap = combine_blocks(p);
  gp.shuffle = debug_shuffle();
  hipStream_t s = (hipStream_t)stream;
  if (debug_validate()) {
    st = validate_offsets(p, offsets, s);
    if (st != MOE_OK) return st;
  }
  if (is_mx(p)) return hip_status(launch_grouped_gemm_mx(gp, s));
  return hip_status(p->dtype == MOE_DTYPE_BF16 ? launch_grouped_gemm_bf16(gp, s) : launch_grouped_gemm_f32(gp, s));
}

moe_status_t moe_combine_ex(const moe_problem_t* p, const float* y, const float* topk_w,
                            const int32_t* flat_to_sorted, const moe_epilogue_t* epi, void* out, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  if (!y || !topk_w || !flat_to_sorted || !out) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(y, 16) || !aligned(topk_w, 4)) return MOE_ERR_INVALID_ARGUMENT;
  OutEpilogue ep;
  st = epilogue_of(p, epi, out, &ep);
  if (st != MOE_OK) return st;
  if (debug_validate()) {
    st = check_range(flat_to_sorted, p->num_tokens * (int64_t)p->topk, -1, (int32_t)(p->num_tokens * p->topk),
                     (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  return hip_status(launch_combine(y, topk_w, flat_to_sorted, p->num_tokens, p->hidden, p->topk, ep,
                                   (hipStream_t)stream));
}

moe_status_t moe_combine(const moe_problem_t* p, const float* y, const float* topk_w, const int32_t* flat_to_sorted,
                         float* out, void* stream) {
  return moe_combine_ex(p, y, topk_w, flat_to_sorted, nullptr, out, stream);
}

int32_t moe_layer_default_movers(const moe_problem_t* p) {
  if (check_problem(p) != MOE_OK || p->dtype != MOE_DTYPE_BF16) return -1;
  return fused_default_movers(p->num_tokens, p->hidden, p->ffn, p->num_experts, p->topk, p->num_src_blocks,
                              held(p), p->dtype, device_cu_count());
}

moe_status_t moe_layer_ex(const moe_problem_t* p, const void* x, const float* logits, const int32_t* src_block,
                          const void* w_gate, const void* w_up, const void* w_down, const moe_epilogue_t* epi,
                          void* out, const moe_layer_aux_t* aux, const moe_layer_opts_t* opts, void* ws,
                          size_t ws_bytes, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  const int64_t M = p->num_tokens;
  if (!w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARGUMENT;
  if (M > 0 && (!x || !logits || !out)) return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_src_blocks > 1 && !src_block && M > 0) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  OutEpilogue ep;
  st = epilogue_of(p, epi, out, &ep);
  if (st != MOE_OK) return st;
  const LayerWs L = layer_ws(p);
  if (!ws || ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, kAlign)) return MOE_ERR_INVALID_ARGUMENT;
  moe_layer_aux_t a;
  memset(&a, 0, sizeof a);
  if (aux) a = *aux;
  if (a.x_perm && !aligned(a.x_perm, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (a.hact && !aligned(a.hact, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (a.y && !aligned(a.y, 16)) return MOE_ERR_INVALID_ARGUMENT;
  const int G = segments(p);
  int32_t* idx = a.topk_idx ? a.topk_idx : at<int32_t>(ws, L.topk_idx);
  float* w = a.topk_w ? a.topk_w : at<float>(ws, L.topk_w);
  int32_t* counts = a.counts ? a.counts : at<int32_t>(ws, L.counts);
  int32_t* offsets = a.offsets ? a.offsets : at<int32_t>(ws, L.offsets);
  int32_t* s2f = a.sorted_to_flat ? a.sorted_to_flat : at<int32_t>(ws, L.s2f);
  int32_t* f2s = a.flat_to_sorted ? a.flat_to_sorted : at<int32_t>(ws, L.f2s);
  void* xp = a.x_perm ? a.x_perm : at<void>(ws, L.x_perm);
  void* hact = a.hact ? a.hact : at<void>(ws, L.hact);
  float* y = a.y ? a.y : at<float>(ws, L.y);
  int32_t* status = at<int32_t>(ws, L.status);
  const int32_t* src = p->num_src_blocks > 1 ? src_block : nullptr;
  hipStream_t s = (hipStream_t)stream;

  moe_layer_opts_t o;
  o.n_mover = -1;
  o.grid = 0;
  o.fused = 1;
  o.spin_limit = 0;
  o.gather = -1;
  if (opts) o = *opts;

  const int cus = device_cu_count();
  // n_mover < 0 asks the profiled table, which may pick the kernel chain
  const int movers = o.n_mover >= 0 ? o.n_mover
                                    : fused_default_movers(M, p->hidden, p->ffn, p->num_experts, p->topk,
                                                           p->num_src_blocks, held(p), p->dtype, cus);
  if (movers == kTableUnusable) return MOE_ERR_INVALID_ARGUMENT;
  if (debug_validate() && M > 0) {
    st = validate_logits(p, (const float*)logits, s);
    if (st == MOE_OK && p->num_src_blocks > 1) st = check_range(src_block, M, 0, p->num_src_blocks, s);
    if (st != MOE_OK) return st;
  }
  // zeroed by kernels rather than memset nodes, so that the call can be
  // captured into a HIP graph
  hipError_t e;
  if (M == 0) {
    // nothing routed: counts and offsets are all zero
    e = launch_fill_i32(status, 1, 0, s);
    if (e == hipSuccess) e = launch_fill_i32(counts, G, 0, s);
    if (e == hipSuccess) e = launch_fill_i32(offsets, G + 1, 0, s);
    return hip_status(e);
  }
  const bool fused = o.fused != 0 && p->dtype == MOE_DTYPE_BF16 && movers >= 0;
  // Layer0 of the fused kernel gathers its token rows from x unless the
  // caller asks for the X_perm copy (o.gather == 0)
  const bool gather = o.gather != 0;
  FusedArgs fa;
  if (fused) {
    fa.M = M;
    fa.H = p->hidden;
    fa.F = p->ffn;
    fa.E = held(p);
    fa.k = p->topk;
    fa.G = G;
    fa.x = x;
    fa.x_perm = gather ? nullptr : xp;
    fa.w_gate = w_gate;
    fa.w_up = w_up;
    fa.w_down = w_down;
    fa.topk_w = w;
    fa.offsets = offsets;
    fa.s2f = s2f;
    fa.f2s = f2s;
    fa.hact = hact;
    fa.y = y;
    fa.out = ep;
    fa.status = status;
    fa.flags = at<int32_t>(ws, L.fused);
    fa.mt_max = fused_mt_max(M, p->hidden, p->topk, G);
    fa.grid = o.grid > 0 ? o.grid : cus;
    fa.n_mover = movers;
    fa.spin_limit = o.spin_limit;
    fa.shuffle = debug_shuffle();
    // checked before anything is launched
    const moe_status_t fs = fused_check(fa, cus);
    if (fs != MOE_OK) return fs;
  }
  // the route kernel also clears the status word and (fused) the ready counters
  e = launch_route(logits, M, p->num_experts, p->topk, idx, w, s, status, 1, fused ? fa.flags : nullptr,
                   fused ? fused_flag_words(M, p->hidden, p->topk, G) : 0);
  if (e != hipSuccess) return MOE_ERR_HIP;
  if (fused) {
    // gathering, the kernel reads token rows straight from x and X_perm is
    // produced only when the caller asks for it
    e = launch_dispatch(plan_of(p), idx, src, counts, offsets, s2f, f2s, x, (int64_t)p->hidden * elem_bytes(p),
                        (!gather || a.x_perm) ? xp : nullptr, at<int32_t>(ws, L.perm), s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    return hip_status(launch_fused_layer(fa, s));
  }
  e = launch_dispatch(plan_of(p), idx, src, counts, offsets, s2f, f2s, x, (int64_t)p->hidden * elem_bytes(p), xp,
                      at<int32_t>(ws, L.perm), s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  GemmProblem gp;
  gp.R = M * p->topk;
  gp.E = held(p);
  gp.G = G;
  gp.offsets = offsets;
  gp.layer = 0;
  gp.a = xp;
  gp.w0 = w_gate;
  gp.w1 = w_up;
  gp.c = hact;
  gp.K = p->hidden;
  gp.N = p->ffn;
  gp.ws = at<void>(ws, L.gemm);
  gp.ws_bytes = L.total - L.gemm;
  gp.rowmap = combine_blocks(p);
  gp.shuffle = debug_shuffle();
  e = is_mx(p) ? launch_grouped_gemm_mx(gp, s)
              : (p->dtype == MOE_DTYPE_BF16 ? launch_grouped_gemm_bf16(gp, s) : launch_grouped_gemm_f32(gp, s));
  if (e != hipSuccess) return MOE_ERR_HIP;
  gp.layer = 1;
  gp.a = hact;
  gp.w0 = w_down;
  gp.w1 = nullptr;
  gp.c = y;
  gp.K = p->ffn;
  gp.N = p->hidden;
  e = is_mx(p) ? launch_grouped_gemm_mx(gp, s)
              : (p->dtype == MOE_DTYPE_BF16 ? launch_grouped_gemm_bf16(gp, s) : launch_grouped_gemm_f32(gp, s));
  if (e != hipSuccess) return MOE_ERR_HIP;
  return hip_status(launch_combine(y, w, f2s, M, p->hidden, p->topk, ep, s));
}

moe_status_t moe_layer(const moe_problem_t* p, const void* x, const float* logits, const int32_t* src_block,
                       const void* w_gate, const void* w_up, const void* w_down, float* out,
                       const moe_layer_aux_t* aux, const moe_layer_opts_t* opts, void* ws, size_t ws_bytes,
                       void* stream) {
  return moe_layer_ex(p, x, logits, src_block, w_gate, w_up, w_down, nullptr, out, aux, opts, ws, ws_bytes, stream);
}

moe_status_t moe_layer_decode(const moe_problem_t* p, const void* x, const float* logits, const void* w_gate,
                              const void* w_up, const void* w_down, const moe_epilogue_t* epi, void* out, void* ws,
                              size_t ws_bytes, void* stream) {
  moe_status_t st = check_decode(p);
  if (st != MOE_OK) return st;
  if (!w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16)) return MOE_ERR_INVALID_ARGUMENT;
  OutEpilogue ep;
  st = epilogue_of(p, epi, out, &ep);
  if (st != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  if (!x || !logits || !out) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(logits, 4)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t n = p->num_tokens * p->hidden;
  const DecodeSplit split = split_of(p);
  const DecodeWs L = decode_ws(p, split);
  if (!ws || ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, kAlign)) return MOE_ERR_INVALID_ARGUMENT;
  const size_t nout = (size_t)n * (ep.out_bf16 ? 2 : 4);
  if (overlap(out, nout, x, (size_t)n * elem_bytes(p)) || overlap(out, nout, ws, L.total) || residual_clash(ep, n) ||
      overlap(out, nout, logits, (size_t)p->num_tokens * p->num_experts * 4))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t nw = (size_t)held(p) * p->hidden * p->ffn;
  if (overlap(out, nout, w_gate, nw * elem_bytes(p)) || overlap(out, nout, w_up, nw * elem_bytes(p)) ||
      overlap(out, nout, w_down, is_mx(p) ? nw + nw / 32 : nw * elem_bytes(p)))
    return MOE_ERR_INVALID_ARGUMENT;
  hipStream_t s = (hipStream_t)stream;
  if (debug_validate()) {
    // -inf is an expert the token may not choose; NaN and +inf are errors
    std::vector<float> h;
    if (!fetch(h, logits, p->num_tokens * (int64_t)p->num_experts, s)) return MOE_ERR_HIP;
    for (float v : h)
      if (!(v < INFINITY)) return MOE_ERR_INVALID_ARGUMENT;
  }
  const bool mx = is_mx(p);
  const int planes = decode_planes(p, ep);
  DecodeArgs a;
  a.plan.M = (int)p->num_tokens;
  a.plan.k = p->topk;
  a.plan.E = p->num_experts;
  a.plan.EL = held(p);
  a.plan.base = held_base(p);
  a.plan.rows = 16 * split.nt;
  a.split = split;
  a.plan.max_entries = decode_max_entries(a.plan.M, a.plan.k, a.plan.EL, split.nt);
  a.plan.entries = at<int4>(ws, L.entries);
  a.plan.list = at<int32_t>(ws, L.list);
  a.plan.f2s = at<int32_t>(ws, L.f2s);
  a.plan.w = at<float>(ws, L.w);
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.wd_scale = mx ? reinterpret_cast<const uint8_t*>(w_down) + (int64_t)held(p) * p->hidden * p->ffn : nullptr;
  a.hact = at<void>(ws, L.hact);
  a.y = at<float>(ws, L.y);
  a.arrived = at<int32_t>(ws, L.arrived);
  a.H = p->hidden;
  a.F = p->ffn;
  a.x_pitch = (uint32_t)(p->hidden * elem_bytes(p));
  a.h_pitch = (uint32_t)p->ffn * (planes ? 2u * planes : 4u);
  a.wd_pitch = (uint32_t)p->ffn * (mx ? 1u : (uint32_t)elem_bytes(p));
  return hip_status(launch_decode(a, logits, p->dtype, planes, ep, s));
}

size_t moe_adapter_workspace_bytes(const moe_adapter_problem_t* q) {
  return check_adapter(q) == MOE_OK ? adapter_ws(q) : 0;
}

moe_status_t moe_adapter_tiles(const moe_adapter_problem_t* q, int32_t out_dtype, int32_t tiles[4]) {
  const moe_status_t st = check_adapter(q);
  if (st != MOE_OK) return st;
  if (!tiles || (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)) return MOE_ERR_INVALID_ARGUMENT;
  const AdapterTiles t =
      q->num_tokens > 0 ? adapter_tiles(adapter_args(q, out_dtype), q->dtype == MOE_DTYPE_F32) : AdapterTiles{};
  tiles[0] = t.rows;
  tiles[1] = t.cols;
  tiles[2] = t.t_rows;
  tiles[3] = t.t_ranks;
  return MOE_OK;
}

moe_status_t moe_adapter_linear(const moe_adapter_problem_t* q, const void* x, const void* w, const void* a,
                                const void* b, const float* scale, const int32_t* adapter_idx,
                                const moe_epilogue_t* epi, void* out, void* ws, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_adapter(q);
  if (st != MOE_OK) return st;
  const bool f32 = q->dtype == MOE_DTYPE_F32;
  const size_t eb = f32 ? 4 : 2;
  AdapterArgs g = adapter_args(q, epi ? epi->out_dtype : MOE_DTYPE_F32);
  g.out.out = out;
  g.out.residual = epi ? epi->residual : nullptr;
  if (epi && epi->out_dtype != MOE_DTYPE_F32 && epi->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (!w || (g.P > 0 && (!a || !b || !scale))) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) ||
      !aligned(g.out.residual, 16) || !aligned(scale, 4) || !aligned(adapter_idx, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  if (g.M == 0) return MOE_OK;
  if (!x || !out || (g.P > 0 && !adapter_idx)) return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = adapter_ws(q);
  if (need > 0) {
    if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, kAlign)) return MOE_ERR_INVALID_ARGUMENT;
  }
  const size_t nout = (size_t)g.M * g.N * (g.out.out_bf16 ? 2 : 4);
  if (overlap(out, nout, x, (size_t)g.M * g.H * eb) || overlap(out, nout, w, (size_t)g.N * g.H * eb) ||
      (need > 0 && overlap(out, nout, ws, need)) || residual_clash(g.out, g.M * g.N))
    return MOE_ERR_INVALID_ARGUMENT;
  if (g.P > 0 && (overlap(out, nout, a, (size_t)g.P * g.r * g.H * eb) || overlap(out, nout, b, (size_t)g.P * g.N * g.r * eb) ||
                  overlap(out, nout, scale, (size_t)g.P * 4) || overlap(out, nout, adapter_idx, (size_t)g.M * 4)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (debug_validate() && g.P > 0) {
    const moe_status_t sv = check_range(adapter_idx, g.M, -1, g.P, (hipStream_t)stream);
    if (sv != MOE_OK) return sv;
  }
  g.x = x;
  g.w = w;
  g.a = a;
  g.b = b;
  g.scale = scale;
  g.idx = adapter_idx;
  g.t = need > 0 ? ws : nullptr;
  return hip_status(launch_adapter_linear(g, f32, (hipStream_t)stream));
}

moe_status_t moe_combine_dropout(const moe_problem_t* p, const float* y, const float* topk_w,
                                 const int32_t* flat_to_sorted, const moe_epilogue_t* epi, const moe_dropout_t* drop,
                                 void* out, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  Dropout d;
  OutEpilogue ep;
  if ((st = dropout_of(drop, &d)) != MOE_OK || (st = epilogue_of(p, epi, out, &ep)) != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  const int64_t R = p->num_tokens * p->topk, n = p->num_tokens * p->hidden;
  const Span s[] = {{y, (size_t)R * p->hidden * 4, false}, {out, (size_t)n * (ep.out_bf16 ? 2 : 4), true}};
  if ((st = check_spans(s, 2)) != MOE_OK || (st = check_words(topk_w, (size_t)R * 4, s, 2)) != MOE_OK ||
      (st = check_words(flat_to_sorted, (size_t)R * 4, s, 2)) != MOE_OK ||
      (st = check_words(d.rng, d.rng ? 16 : 0, s, 2)) != MOE_OK)
    return st;
  if (residual_clash(ep, n)) return MOE_ERR_INVALID_ARGUMENT;
  if (debug_validate()) {
    st = check_range(flat_to_sorted, R, -1, (int32_t)R, (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  if (!d.rng)
    return hip_status(launch_combine(y, topk_w, flat_to_sorted, p->num_tokens, p->hidden, p->topk, ep, (hipStream_t)stream));
  return hip_status(launch_combine_dropout(y, topk_w, flat_to_sorted, p->num_tokens, kept_rows(p), p->hidden, p->topk, ep,
                                           d, (hipStream_t)stream));
}

moe_status_t moe_combine_backward(const moe_problem_t* p, const void* dout, int32_t dout_dtype, const float* y,
                                  const float* topk_w, const int32_t* flat_to_sorted, const moe_dropout_t* drop,
                                  void* dy, float* dtopk_w, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  CombineBackwardArgs a;
  if ((st = dropout_of(drop, &a.drop)) != MOE_OK) return st;
  if (dout_dtype != MOE_DTYPE_F32 && dout_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_tokens == 0) return MOE_OK;
  const int64_t R = p->num_tokens * p->topk, n = p->num_tokens * p->hidden;
  // dtopk_w is an output, but as the other per-pair arrays 4-byte aligned
  const Span s[] = {{dout, (size_t)n * (dout_dtype == MOE_DTYPE_BF16 ? 2 : 4), false},
                    {y, (size_t)R * p->hidden * 4, false},
                    {dy, (size_t)R * p->hidden * elem_bytes(p), true}};
  const Span w[] = {{dtopk_w, (size_t)R * 4, true}};
  if ((st = check_spans(s, 3)) != MOE_OK || (st = check_words(dtopk_w, (size_t)R * 4, s, 3)) != MOE_OK) return st;
  for (const Span& b : s)
    if (overlap(dtopk_w, (size_t)R * 4, b.p, b.n)) return MOE_ERR_INVALID_ARGUMENT;
  const void* words[] = {topk_w, flat_to_sorted};
  for (const void* b : words)
    if ((st = check_words(b, (size_t)R * 4, s, 3)) != MOE_OK || (st = check_words(b, (size_t)R * 4, w, 1)) != MOE_OK)
      return st;
  if (a.drop.rng && ((st = check_words(a.drop.rng, 16, s, 3)) != MOE_OK || (st = check_words(a.drop.rng, 16, w, 1)) != MOE_OK))
    return st;
  if (debug_validate()) {
    st = check_range(flat_to_sorted, R, -1, (int32_t)R, (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  a.dout = dout;
  a.dout_bf16 = dout_dtype == MOE_DTYPE_BF16;
  a.y = y;
  a.topk_w = topk_w;
  a.f2s = flat_to_sorted;
  a.dy = dy;
  a.dy_bf16 = p->dtype != MOE_DTYPE_F32;
  a.dtopk_w = dtopk_w;
  a.M = p->num_tokens;
  a.rows = kept_rows(p);
  a.H = p->hidden;
  a.k = p->topk;
  return hip_status(launch_combine_backward(a, (hipStream_t)stream));
}

moe_status_t moe_dispatch_backward(const moe_problem_t* p, const void* dx_perm, const int32_t* flat_to_sorted,
                                   const moe_epilogue_t* epi, void* dx, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  OutEpilogue ep;
  if ((st = epilogue_of(p, epi, dx, &ep)) != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  const int64_t R = p->num_tokens * p->topk, n = p->num_tokens * p->hidden;
  const Span s[] = {{dx_perm, (size_t)R * p->hidden * elem_bytes(p), false},
                    {dx, (size_t)n * (ep.out_bf16 ? 2 : 4), true}};
  if ((st = check_spans(s, 2)) != MOE_OK || (st = check_words(flat_to_sorted, (size_t)R * 4, s, 2)) != MOE_OK) return st;
  if (residual_clash(ep, n)) return MOE_ERR_INVALID_ARGUMENT;
  if (debug_validate()) {
    st = check_range(flat_to_sorted, R, -1, (int32_t)R, (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  return hip_status(launch_dispatch_backward(dx_perm, p->dtype != MOE_DTYPE_F32, flat_to_sorted, p->num_tokens,
                                             kept_rows(p), p->hidden, p->topk, ep, (hipStream_t)stream));
}

moe_status_t moe_route_backward(const moe_problem_t* p, const int32_t* topk_idx, const float* topk_w,
                                const float* dtopk_w, float* dlogits, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (p->num_tokens == 0) return MOE_OK;
  const int64_t R = p->num_tokens * p->topk;
  const Span s[] = {{dlogits, (size_t)p->num_tokens * p->num_experts * 4, true}};
  if ((st = check_spans(s, 1)) != MOE_OK || (st = check_words(topk_idx, (size_t)R * 4, s, 1)) != MOE_OK ||
      (st = check_words(topk_w, (size_t)R * 4, s, 1)) != MOE_OK ||
      (st = check_words(dtopk_w, (size_t)R * 4, s, 1)) != MOE_OK)
    return st;
  if (debug_validate()) {
    st = check_range(topk_idx, R, 0, p->num_experts, (hipStream_t)stream);
    if (st != MOE_OK) return st;
  }
  return hip_status(launch_route_backward(topk_idx, topk_w, dtopk_w, p->num_tokens, p->num_experts, p->topk, dlogits,
                                          (hipStream_t)stream));
}

moe_status_t moe_grouped_gemm_aux(const moe_problem_t* p, const void* a, const void* w0, const void* w1,
                                  const int32_t* offsets, void* gate, void* up, void* c, void* stream) {
  moe_status_t st = check_grad_gemm(p, 0);
  if (st != MOE_OK) return st;
  const int64_t R = p->num_tokens * p->topk;
  const size_t nh = (size_t)R * p->hidden * elem_bytes(p), nf = (size_t)R * p->ffn * elem_bytes(p);
  const size_t nw = (size_t)held(p) * p->hidden * p->ffn * elem_bytes(p);
  const Span s[] = {{a, nh, false}, {w0, nw, false}, {w1, nw, false}, {gate, nf, true}, {up, nf, true}, {c, nf, true}};
  if ((st = check_spans(s, 6)) != MOE_OK || (st = check_words(offsets, (size_t)(segments(p) + 1) * 4, s, 6)) != MOE_OK)
    return st;
  if (R == 0) return MOE_OK;
  hipStream_t hs = (hipStream_t)stream;
  if (debug_validate()) {
    st = validate_offsets(p, offsets, hs);
    if (st != MOE_OK) return st;
  }
  GradGemmArgs g = grad_args(p, 0, offsets);
  g.x = a;
  g.w0 = w0;
  g.w1 = w1;
  g.o0 = gate;
  g.o1 = up;
  g.o2 = c;
  return hip_status(launch_keep(g, p->dtype == MOE_DTYPE_BF16, hs));
}

moe_status_t moe_grouped_gemm_backward(const moe_problem_t* p, int32_t layer, const void* d0, const void* d1,
                                       const void* w0, const void* w1, const void* gate, const void* up,
                                       const int32_t* offsets, void* o0, void* o1, void* ws, size_t ws_bytes,
                                       void* stream) {
  moe_status_t st = check_grad_gemm(p, layer);
  if (st != MOE_OK) return st;
  const int64_t R = p->num_tokens * p->topk;
  const size_t eb = elem_bytes(p), nh = (size_t)R * p->hidden * eb, nf = (size_t)R * p->ffn * eb;
  const size_t nw = (size_t)held(p) * p->hidden * p->ffn * eb;
  if (layer == 0 ? (gate || up || o1) : (d1 || w1)) return MOE_ERR_INVALID_ARGUMENT;
  const Span rows1[] = {{d0, nh, false}, {w0, nw, false}, {gate, nf, false}, {up, nf, false}, {o0, nf, true}, {o1, nf, true}};
  const Span rows0[] = {{d0, nf, false}, {d1, nf, false}, {w0, nw, false}, {w1, nw, false}, {o0, nh, true}};
  const Span* s = layer == 0 ? rows0 : rows1;
  const int n = layer == 0 ? 5 : 6;
  if ((st = check_spans(s, n)) != MOE_OK || (st = check_words(offsets, (size_t)(segments(p) + 1) * 4, s, n)) != MOE_OK)
    return st;
  if (R == 0) return MOE_OK;
  if ((st = check_grad_ws(p, ws, ws_bytes, s, n, offsets)) != MOE_OK) return st;
  hipStream_t hs = (hipStream_t)stream;
  if (debug_validate()) {
    st = validate_offsets(p, offsets, hs);
    if (st != MOE_OK) return st;
  }
  GradGemmArgs g = grad_args(p, layer, offsets);
  g.d0 = d0;
  g.d1 = d1;
  g.w0 = w0;
  g.w1 = w1;
  g.gate = gate;
  g.up = up;
  g.o0 = o0;
  g.o1 = o1;
  return hip_status(launch_grad_rows(g, p->dtype == MOE_DTYPE_BF16, ws, hs));
}

moe_status_t moe_grouped_gemm_backward_weights(const moe_problem_t* p, int32_t layer, const void* d0, const void* d1,
                                               const void* a, const int32_t* offsets, int32_t dw_dtype,
                                               int32_t accumulate, void* dw0, void* dw1, void* ws, size_t ws_bytes,
                                               void* stream) {
  moe_status_t st = check_grad_gemm(p, layer);
  if (st != MOE_OK) return st;
  if (dw_dtype != MOE_DTYPE_F32 && dw_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  if (accumulate && dw_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  const int64_t R = p->num_tokens * p->topk;
  const size_t eb = elem_bytes(p), nh = (size_t)R * p->hidden * eb, nf = (size_t)R * p->ffn * eb;
  const size_t nw = (size_t)held(p) * p->hidden * p->ffn * (dw_dtype == MOE_DTYPE_BF16 ? 2 : 4);
  if (layer == 1 && (d1 || dw1)) return MOE_ERR_INVALID_ARGUMENT;
  const Span w1[] = {{d0, nh, false}, {a, nf, false}, {dw0, nw, true}};
  const Span w0[] = {{d0, nf, false}, {d1, nf, false}, {a, nh, false}, {dw0, nw, true}, {dw1, nw, true}};
  const Span* s = layer == 0 ? w0 : w1;
  const int n = layer == 0 ? 5 : 3;
  if ((st = check_spans(s, n)) != MOE_OK || (st = check_words(offsets, (size_t)(segments(p) + 1) * 4, s, n)) != MOE_OK)
    return st;
  if ((st = check_grad_ws(p, ws, ws_bytes, s, n, offsets)) != MOE_OK) return st;
  hipStream_t hs = (hipStream_t)stream;
  if (debug_validate()) {
    st = validate_offsets(p, offsets, hs);
    if (st != MOE_OK) return st;
  }
  GradGemmArgs g = grad_args(p, layer, offsets);
  g.d0 = d0;
  g.d1 = d1;
  g.x = a;
  g.o0 = dw0;
  g.o1 = dw1;
  g.out_bf16 = dw_dtype == MOE_DTYPE_BF16;
  g.accumulate = accumulate != 0;
  return hip_status(launch_grad_weights(g, p->dtype == MOE_DTYPE_BF16, ws, hs));
}

moe_status_t moe_quantize_mxfp8(int64_t rows, int32_t cols, int32_t src_dtype, const void* src, void* dst,
                                void* stream) {
  if (rows < 0 || cols < 128 || cols % 128) return MOE_ERR_INVALID_ARGUMENT;
  if (src_dtype != MOE_DTYPE_BF16 && src_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 16) || !aligned(dst, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (rows >= (1ll << 40) / cols) return MOE_ERR_UNSUPPORTED;  // rows * cols < 2^40, checked without forming it
  return hip_status(launch_mx_quantize(src, src_dtype == MOE_DTYPE_BF16, rows, cols, dst, (hipStream_t)stream));
}

moe_status_t moe_transpose_weights(int64_t batch, int32_t rows, int32_t cols, int32_t dtype, const void* src,
                                   void* dst, void* stream) {
  if (batch < 0 || rows <= 0 || cols <= 0 || rows % 64 || cols % 64) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARGUMENT;
  if (batch == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 16) || !aligned(dst, 16)) return MOE_ERR_INVALID_ARGUMENT;
  // sizes bounded before any product that could wrap: batch * rows * cols < 2^40
  const uint64_t elems = (uint64_t)rows * (uint64_t)cols;  // < 2^62
  if (elems >= (1ull << 40) || (uint64_t)batch >= (1ull << 40) / elems) return MOE_ERR_UNSUPPORTED;
  const uint64_t bytes = (uint64_t)batch * elems * (dtype == MOE_DTYPE_BF16 ? 2u : 4u);
  const uintptr_t a = (uintptr_t)src, b = (uintptr_t)dst;
  if (a < b + bytes && b < a + bytes) return MOE_ERR_INVALID_ARGUMENT;  // overlapping buffers
  return hip_status(launch_transpose(src, dst, batch, rows, cols, dtype == MOE_DTYPE_BF16, (hipStream_t)stream));
}

moe_status_t moe_debug_device_status(const moe_problem_t* p, void* ws, size_t ws_bytes, void* stream) {
  moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  const LayerWs L = layer_ws(p);
  if (!ws || ws_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int32_t v = 0;
  hipStream_t s = (hipStream_t)stream;
  if (hipMemcpyAsync(&v, at<int32_t>(ws, L.status), sizeof v, hipMemcpyDeviceToHost, s) != hipSuccess)
    return MOE_ERR_HIP;
  if (hipStreamSynchronize(s) != hipSuccess) return MOE_ERR_HIP;
  return v == 0 ? MOE_OK : (moe_status_t)v;
}

}  // extern "C"
