"""Python binding of the MoE layer library (``lib/libmoe.so``, C ABI in
``include/moe.h``).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch device tensors (row-major, contiguous); the
binding passes their data pointers and the current HIP stream of torch (or
the stream given) straight through.  There is no fallback: if the library is
missing, loading it raises.

The entry points keep the C names: ``moe_route``, ``moe_dispatch``,
``moe_dispatch_noalloc``, ``moe_grouped_gemm``, ``moe_combine``, ``moe_combine_ex``, ``moe_layer``,
``moe_layer_ex``, ``moe_layer_decode``, ``moe_adapter_linear``, and for training
``moe_combine_dropout``, ``moe_combine_backward``, ``moe_dispatch_backward``, ``moe_route_backward``,
``moe_grouped_gemm_aux``, ``moe_grouped_gemm_backward``, ``moe_grouped_gemm_backward_weights`` (plus
``moe_workspace_bytes``, ``moe_adapter_workspace_bytes``, ``moe_adapter_tiles``, ``moe_layer_default_movers``,
``moe_debug_device_status``, ``moe_status_string``, ``moe_abi_version``).
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARGUMENT = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_HIP = 4
MOE_ERR_DEVICE_TIMEOUT = 5

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_BF16_MXFP8 = 2

MOE_OP_DISPATCH = 0
MOE_OP_GROUPED_GEMM = 1
MOE_OP_LAYER = 2
MOE_OP_LAYER_DECODE = 3
MOE_OP_GROUPED_GEMM_BACKWARD = 4

MOE_DECODE_MAX_TOKENS = 256

MOE_NOALLOC_SCRATCH_BYTES = 1 << 20

EXPORTED = ("moe_workspace_bytes", "moe_route", "moe_dispatch", "moe_dispatch_noalloc", "moe_grouped_gemm", "moe_combine", "moe_combine_ex",
            "moe_layer", "moe_layer_ex", "moe_layer_decode", "moe_adapter_linear", "moe_adapter_workspace_bytes", "moe_adapter_tiles",
            "moe_combine_dropout", "moe_combine_backward", "moe_dispatch_backward", "moe_route_backward",
            "moe_grouped_gemm_aux", "moe_grouped_gemm_backward", "moe_grouped_gemm_backward_weights",
            "moe_quantize_mxfp8", "moe_transpose_weights", "moe_layer_default_movers",
            "moe_debug_device_status",
            "moe_status_string", "moe_abi_version")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_name(status)} ({status})")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("num_src_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("expert_base", ctypes.c_int32), ("local_experts", ctypes.c_int32)]


class AdapterProblem(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("num_adapters", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("out_dtype", ctypes.c_int32)]
    tensor = None  # the residual's tensor, where epilogue() was given one


class Dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("rng", ctypes.c_void_p)]
    tensor = None  # the {seed, offset} tensor, where dropout() was given one


class LayerAux(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "counts", "offsets", "sorted_to_flat",
                                              "flat_to_sorted", "x_perm", "hact", "y")]


class LayerOpts(ctypes.Structure):
    _fields_ = [("n_mover", ctypes.c_int32), ("grid", ctypes.c_int32), ("fused", ctypes.c_int32),
                ("spin_limit", ctypes.c_int32), ("gather", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"MoE HIP library not built: {path} missing "
                           "(run python -m combine_topk_gate_amd.build)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    PP = ctypes.POINTER(Problem)
    PA = ctypes.POINTER(AdapterProblem)
    sig = {
        "moe_workspace_bytes": ([PP, I32], SZ),
        "moe_route": ([PP, P, P, P, P], I32),
        "moe_dispatch": ([PP, P, P, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_dispatch_noalloc": ([PP, P, P, P, P, P, P, P, P, P], I32),
        "moe_grouped_gemm": ([PP, I32, P, P, P, P, P, P, SZ, P], I32),
        "moe_combine": ([PP, P, P, P, P, P], I32),
        "moe_combine_ex": ([PP, P, P, P, ctypes.POINTER(Epilogue), P, P], I32),
        "moe_layer": ([PP, P, P, P, P, P, P, P, ctypes.POINTER(LayerAux), ctypes.POINTER(LayerOpts), P, SZ, P], I32),
        "moe_layer_ex": ([PP, P, P, P, P, P, P, ctypes.POINTER(Epilogue), P, ctypes.POINTER(LayerAux),
                          ctypes.POINTER(LayerOpts), P, SZ, P], I32),
        "moe_layer_decode": ([PP, P, P, P, P, P, ctypes.POINTER(Epilogue), P, P, SZ, P], I32),
        "moe_adapter_workspace_bytes": ([PA], SZ),
        "moe_adapter_tiles": ([PA, I32, ctypes.POINTER(I32)], I32),
        "moe_adapter_linear": ([PA, P, P, P, P, P, P, ctypes.POINTER(Epilogue), P, P, SZ, P], I32),
        "moe_combine_dropout": ([PP, P, P, P, ctypes.POINTER(Epilogue), ctypes.POINTER(Dropout), P, P], I32),
        "moe_combine_backward": ([PP, P, I32, P, P, P, ctypes.POINTER(Dropout), P, P, P], I32),
        "moe_dispatch_backward": ([PP, P, P, ctypes.POINTER(Epilogue), P, P], I32),
        "moe_route_backward": ([PP, P, P, P, P, P], I32),
        "moe_grouped_gemm_aux": ([PP, P, P, P, P, P, P, P, P], I32),
        "moe_grouped_gemm_backward": ([PP, I32, P, P, P, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_grouped_gemm_backward_weights": ([PP, I32, P, P, P, P, I32, I32, P, P, P, SZ, P], I32),
        "moe_quantize_mxfp8": ([ctypes.c_int64, I32, I32, P, P, P], I32),
        "moe_transpose_weights": ([ctypes.c_int64, I32, I32, I32, P, P, P], I32),
        "moe_layer_default_movers": ([PP], I32),
        "moe_debug_device_status": ([PP, P, SZ, P], I32),
        "moe_status_string": ([I32], ctypes.c_char_p),
        "moe_abi_version": ([], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def status_name(status: int) -> str:
    try:
        return load_library().moe_status_string(status).decode()
    except Exception:  # library not loadable: plain number
        return str(status)


_DTYPES = {"bf16": MOE_DTYPE_BF16, "f32": MOE_DTYPE_F32, "bf16_mxfp8": MOE_DTYPE_BF16_MXFP8,
           MOE_DTYPE_BF16: MOE_DTYPE_BF16, MOE_DTYPE_F32: MOE_DTYPE_F32, MOE_DTYPE_BF16_MXFP8: MOE_DTYPE_BF16_MXFP8}


def mx_bytes(rows: int, cols: int) -> int:
    """Bytes of an MXFP8 buffer of rows x cols (cols a multiple of 128): the
    codes, then one scale byte per 32 values with rows padded to a multiple
    of 32."""
    return rows * cols + (rows + 31) // 32 * 32 * (cols // 32)


def problem(M, H, F, E, k, S=1, dtype="bf16", expert_base=0, local_experts=0) -> Problem:
    return Problem(int(M), int(H), int(F), int(E), int(k), int(S), _DTYPES[dtype], int(expert_base),
                   int(local_experts))


def adapter_problem(M, H, N, rank, num_adapters, dtype="bf16") -> AdapterProblem:
    return AdapterProblem(int(M), int(H), int(N), int(rank), int(num_adapters), _DTYPES[dtype])


def epilogue(residual=None, out_dtype="f32") -> Epilogue:
    """The combine's output epilogue: out = cast(acc + residual).  It holds the
    residual's tensor."""
    epi = Epilogue(None if residual is None else residual.data_ptr(), _DTYPES[out_dtype])
    epi.tensor = residual
    return epi


def dropout(p, rng) -> Dropout:
    """Dropout with probability p (0 <= p < 1) whose mask comes from rng, a device
    int64 tensor {seed, offset} that the kernels read: one of its own for every
    layer, step and data-parallel rank, whose masks are else the same.  It holds
    the tensor."""
    drop = Dropout(float(p), None if rng is None else rng.data_ptr())
    drop.tensor = rng
    return drop


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


def moe_abi_version() -> int:
    return load_library().moe_abi_version()


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_workspace_bytes(p: Problem, op: int) -> int:
    return load_library().moe_workspace_bytes(ctypes.byref(p), op)


def moe_layer_default_movers(p: Problem) -> int:
    return load_library().moe_layer_default_movers(ctypes.byref(p))


def moe_route(p, logits, topk_idx, topk_w, stream=None):
    _check(load_library().moe_route(ctypes.byref(p), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_route")


def moe_dispatch(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm, ws,
                 stream=None):
    _check(load_library().moe_dispatch(ctypes.byref(p), _ptr(x), _ptr(topk_idx), _ptr(src_block), _ptr(counts),
                                       _ptr(offsets), _ptr(sorted_to_flat), _ptr(flat_to_sorted), _ptr(x_perm),
                                       _ptr(ws), _nbytes(ws), _stream(stream)), "moe_dispatch")


def moe_dispatch_noalloc(p, x, topk_idx, src_block, counts, offsets, sorted_to_flat, flat_to_sorted, x_perm,
                         stream=None):
    _check(load_library().moe_dispatch_noalloc(ctypes.byref(p), _ptr(x), _ptr(topk_idx), _ptr(src_block),
                                               _ptr(counts), _ptr(offsets), _ptr(sorted_to_flat),
                                               _ptr(flat_to_sorted), _ptr(x_perm), _stream(stream)),
           "moe_dispatch_noalloc")


def moe_grouped_gemm(p, layer, a, w0, w1, offsets, c, ws=None, stream=None):
    _check(load_library().moe_grouped_gemm(ctypes.byref(p), int(layer), _ptr(a), _ptr(w0), _ptr(w1), _ptr(offsets),
                                           _ptr(c), _ptr(ws), _nbytes(ws), _stream(stream)), "moe_grouped_gemm")


def moe_combine(p, y, topk_w, flat_to_sorted, out, stream=None):
    _check(load_library().moe_combine(ctypes.byref(p), _ptr(y), _ptr(topk_w), _ptr(flat_to_sorted), _ptr(out),
                                      _stream(stream)), "moe_combine")


def moe_combine_ex(p, y, topk_w, flat_to_sorted, epi, out, stream=None):
    _check(load_library().moe_combine_ex(ctypes.byref(p), _ptr(y), _ptr(topk_w), _ptr(flat_to_sorted),
                                         ctypes.byref(epi) if epi is not None else None, _ptr(out),
                                         _stream(stream)), "moe_combine_ex")


def moe_quantize_mxfp8(src, dst, stream=None):
    """MXFP8 quantisation of a 2-D (or stacked) bf16/f32 tensor along its last
    dimension into dst (uint8, mx_bytes(rows, cols) bytes)."""
    import torch
    cols = src.shape[-1]
    rows = src.numel() // cols
    dt = MOE_DTYPE_BF16 if src.dtype == torch.bfloat16 else MOE_DTYPE_F32
    _check(load_library().moe_quantize_mxfp8(rows, cols, dt, _ptr(src), _ptr(dst), _stream(stream)),
           "moe_quantize_mxfp8")


def moe_transpose_weights(src, dst, stream=None):
    """dst[b] = src[b].T for a [batch, rows, cols] bf16/f32 tensor src and a
    [batch, cols, rows] tensor dst of the same dtype (weights given as the
    math writes them -> the storage the layer reads)."""
    import torch
    batch, rows, cols = (1,) * (3 - src.dim()) + tuple(src.shape)
    dt = MOE_DTYPE_BF16 if src.dtype == torch.bfloat16 else MOE_DTYPE_F32
    _check(load_library().moe_transpose_weights(batch, rows, cols, dt, _ptr(src), _ptr(dst), _stream(stream)),
           "moe_transpose_weights")


def moe_layer(p, x, logits, src_block, w_gate, w_up, w_down, out, ws, aux: dict | None = None,
              n_mover: int = -1, grid: int = 0, fused: int = 1, spin_limit: int = 0,
              gather: int = -1, stream=None):
    a = None
    if aux:
        a = LayerAux(**{k: (v.data_ptr() if v is not None else None) for k, v in aux.items()})
    o = LayerOpts(int(n_mover), int(grid), int(fused), int(spin_limit), int(gather))
    _check(load_library().moe_layer(ctypes.byref(p), _ptr(x), _ptr(logits), _ptr(src_block), _ptr(w_gate),
                                    _ptr(w_up), _ptr(w_down), _ptr(out), ctypes.byref(a) if a else None,
                                    ctypes.byref(o), _ptr(ws), _nbytes(ws), _stream(stream)), "moe_layer")


def moe_layer_ex(p, x, logits, src_block, w_gate, w_up, w_down, epi, out, ws, aux: dict | None = None,
                 n_mover: int = -1, grid: int = 0, fused: int = 1, spin_limit: int = 0,
                 gather: int = -1, stream=None):
    a = None
    if aux:
        a = LayerAux(**{k: (v.data_ptr() if v is not None else None) for k, v in aux.items()})
    o = LayerOpts(int(n_mover), int(grid), int(fused), int(spin_limit), int(gather))
    _check(load_library().moe_layer_ex(ctypes.byref(p), _ptr(x), _ptr(logits), _ptr(src_block), _ptr(w_gate),
                                       _ptr(w_up), _ptr(w_down), ctypes.byref(epi) if epi is not None else None,
                                       _ptr(out), ctypes.byref(a) if a else None, ctypes.byref(o), _ptr(ws),
                                       _nbytes(ws), _stream(stream)), "moe_layer_ex")


def _refuse(what, name, t, dtype, shape):
    raise MoeError(MOE_ERR_INVALID_ARGUMENT,
                   f"{what}: {name} must be a contiguous {dtype} tensor of shape {shape} on the call's GPU; "
                   f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _gpu_of(what, name, t):
    if t is None:
        raise MoeError(MOE_ERR_INVALID_ARGUMENT, f"{what}: {name} is missing")
    return t.get_device()


def _addr(what, name, t, dtype, shape, gpu):
    """The data pointer of t (None: NULL), which must be what the call reads:
    contiguous, of this type and shape, on GPU number `gpu` (-1, no GPU, never
    is); otherwise MoeError with MOE_ERR_INVALID_ARGUMENT, before the library
    sees it."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == gpu >= 0 and t.is_contiguous():
        return t.data_ptr()
    _refuse(what, name, t, dtype, shape)


def _epilogue(what, epi, dtype, shape, gpu):
    """The epilogue for the library; its residual is checked as the other
    tensors are (one given as a bare address is the caller's word)."""
    if epi is None:
        return None
    if epi.tensor is not None and epi.residual:
        if _addr(what, "residual", epi.tensor, dtype, shape, gpu) != epi.residual:
            raise MoeError(MOE_ERR_INVALID_ARGUMENT, f"{what}: the residual has moved since its epilogue was made")
    return ctypes.byref(epi)


def _workspace(what, ws, gpu):
    """(pointer, bytes) of a workspace: any contiguous tensor on the GPU."""
    if ws is None:
        return None, 0
    if ws.get_device() != gpu or not ws.is_contiguous():
        _refuse(what, "ws", ws, "uint8", "any")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _call_on(gpu, stream, f, *args):
    """f(*args, stream) with GPU number `gpu` current, on the stream given or
    torch's current one of that GPU."""
    import torch
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(gpu)
    else:
        raw = stream if isinstance(stream, int) else stream.cuda_stream
    if torch._C._cuda_getDevice() == gpu:
        return f(*args, raw)
    with torch.cuda.device(gpu):
        return f(*args, raw)


def moe_layer_decode(p, x, logits, w_gate, w_up, w_down, epi, out, ws, stream=None):
    """The layer for at most MOE_DECODE_MAX_TOKENS tokens (a decode step): out
    [M, H] of x [M, H] and logits [M, E] (-inf: an expert the token may not
    choose; an all -inf row is idle), epi as in moe_layer_ex or None, ws
    moe_workspace_bytes(p, MOE_OP_LAYER_DECODE) bytes."""
    import torch
    what = "moe_layer_decode"
    f32 = torch.float32
    M, H, F, E, dtype = p.num_tokens, p.hidden, p.ffn, p.num_experts, p.dtype
    EL, gpu = p.local_experts or E, _gpu_of(what, "x", x)
    act = f32 if dtype == MOE_DTYPE_F32 else torch.bfloat16
    odt = torch.bfloat16 if epi is not None and epi.out_dtype == MOE_DTYPE_BF16 else f32
    if dtype == MOE_DTYPE_BF16_MXFP8:
        down = _addr(what, "w_down", w_down, torch.uint8, (mx_bytes(EL * H, F),), gpu)
    else:
        down = _addr(what, "w_down", w_down, act, (EL, H, F), gpu)
    _check(_call_on(gpu, stream, load_library().moe_layer_decode, ctypes.byref(p),
                    _addr(what, "x", x, act, (M, H), gpu), _addr(what, "logits", logits, f32, (M, E), gpu),
                    _addr(what, "w_gate", w_gate, act, (EL, F, H), gpu),
                    _addr(what, "w_up", w_up, act, (EL, F, H), gpu), down,
                    _epilogue(what, epi, act, (M, H), gpu), _addr(what, "out", out, odt, (M, H), gpu),
                    *_workspace(what, ws, gpu)), what)


def moe_adapter_workspace_bytes(q: AdapterProblem) -> int:
    return load_library().moe_adapter_workspace_bytes(ctypes.byref(q))


def moe_adapter_tiles(q: AdapterProblem, out_dtype="f32"):
    """(rows, columns) of the projection's tile and (rows, ranks) of t's that
    moe_adapter_linear takes, as one tuple (moe.h)."""
    tiles = (ctypes.c_int32 * 4)()
    _check(load_library().moe_adapter_tiles(ctypes.byref(q), _DTYPES[out_dtype], tiles), "moe_adapter_tiles")
    return tuple(tiles)


def moe_adapter_linear(q, x, w, a, b, scale, adapter_idx, epi, out, ws, stream=None):
    """out[m] = x[m] W^T + scale[a] (x[m] A[a]^T) B[a]^T (+ residual) with a =
    adapter_idx[m] (-1: none): x [M, H], w [N, H], a [P, rank, H], b [P, N,
    rank], scale [P] f32, adapter_idx [M] int32, out [M, N]; epi as in
    moe_combine_ex or None; ws moe_adapter_workspace_bytes(q) bytes.  With
    num_adapters 0: a, b, scale, adapter_idx and ws may be None."""
    import torch
    what = "moe_adapter_linear"
    f32 = torch.float32
    M, H, N, r, P = q.num_tokens, q.in_features, q.out_features, q.rank, q.num_adapters
    gpu = _gpu_of(what, "x", x)
    act = f32 if q.dtype == MOE_DTYPE_F32 else torch.bfloat16
    odt = torch.bfloat16 if epi is not None and epi.out_dtype == MOE_DTYPE_BF16 else f32
    _check(_call_on(gpu, stream, load_library().moe_adapter_linear, ctypes.byref(q),
                    _addr(what, "x", x, act, (M, H), gpu), _addr(what, "w", w, act, (N, H), gpu),
                    _addr(what, "a", a, act, (P, r, H), gpu), _addr(what, "b", b, act, (P, N, r), gpu),
                    _addr(what, "scale", scale, f32, (P,), gpu),
                    _addr(what, "adapter_idx", adapter_idx, torch.int32, (M,), gpu),
                    _epilogue(what, epi, act, (M, N), gpu), _addr(what, "out", out, odt, (M, N), gpu),
                    *_workspace(what, ws, gpu)), what)


def _dropout(what, drop, gpu):
    """The dropout for the library; its rng is checked as the other tensors are."""
    if drop is None:
        return None
    if drop.tensor is not None:
        import torch
        if _addr(what, "rng", drop.tensor, torch.int64, (2,), gpu) != drop.rng:
            raise MoeError(MOE_ERR_INVALID_ARGUMENT, f"{what}: the rng tensor has moved since its dropout was made")
    return ctypes.byref(drop)


def _dtypes(p, epi=None):
    """(dtype of the problem's activations, dtype of an output under epi)."""
    import torch
    act = torch.float32 if p.dtype == MOE_DTYPE_F32 else torch.bfloat16
    return act, torch.bfloat16 if epi is not None and epi.out_dtype == MOE_DTYPE_BF16 else torch.float32


def moe_combine_dropout(p, y, topk_w, flat_to_sorted, epi, drop, out, stream=None):
    """moe_combine_ex with a dropout (dropout(p, rng), or None) on the sum before
    the epilogue: y [R, H] f32, topk_w [M, k] f32, flat_to_sorted [R] int32, out
    [M, H] in epi's type."""
    import torch
    what = "moe_combine_dropout"
    M, H, k, gpu = p.num_tokens, p.hidden, p.topk, _gpu_of(what, "y", y)
    act, odt = _dtypes(p, epi)
    _check(_call_on(gpu, stream, load_library().moe_combine_dropout, ctypes.byref(p),
                    _addr(what, "y", y, torch.float32, (M * k, H), gpu),
                    _addr(what, "topk_w", topk_w, torch.float32, (M, k), gpu),
                    _addr(what, "flat_to_sorted", flat_to_sorted, torch.int32, (M * k,), gpu),
                    _epilogue(what, epi, act, (M, H), gpu), _dropout(what, drop, gpu),
                    _addr(what, "out", out, odt, (M, H), gpu)), what)


def moe_combine_backward(p, dout, y, topk_w, flat_to_sorted, drop, dy, dtopk_w, stream=None):
    """Gradient of the combine: dout [M, H] f32 or bf16, y [R, H] f32, topk_w [M,
    k], flat_to_sorted [R], drop as in the forward call (or None) -> dy [R, H] in
    the problem's dtype, dtopk_w [M, k] f32."""
    import torch
    what = "moe_combine_backward"
    M, H, k, gpu = p.num_tokens, p.hidden, p.topk, _gpu_of(what, "dout", dout)
    bf16 = dout.dtype is torch.bfloat16
    _check(_call_on(gpu, stream, load_library().moe_combine_backward, ctypes.byref(p),
                    _addr(what, "dout", dout, torch.bfloat16 if bf16 else torch.float32, (M, H), gpu),
                    MOE_DTYPE_BF16 if bf16 else MOE_DTYPE_F32, _addr(what, "y", y, torch.float32, (M * k, H), gpu),
                    _addr(what, "topk_w", topk_w, torch.float32, (M, k), gpu),
                    _addr(what, "flat_to_sorted", flat_to_sorted, torch.int32, (M * k,), gpu),
                    _dropout(what, drop, gpu), _addr(what, "dy", dy, _dtypes(p)[0], (M * k, H), gpu),
                    _addr(what, "dtopk_w", dtopk_w, torch.float32, (M, k), gpu)), what)


def moe_dispatch_backward(p, dx_perm, flat_to_sorted, epi, dx, stream=None):
    """Gradient of the dispatch's copy: dx_perm [R, H] in the problem's dtype,
    flat_to_sorted [R] -> dx [M, H] in epi's type (its residual added)."""
    import torch
    what = "moe_dispatch_backward"
    M, H, k, gpu = p.num_tokens, p.hidden, p.topk, _gpu_of(what, "dx_perm", dx_perm)
    act, odt = _dtypes(p, epi)
    _check(_call_on(gpu, stream, load_library().moe_dispatch_backward, ctypes.byref(p),
                    _addr(what, "dx_perm", dx_perm, act, (M * k, H), gpu),
                    _addr(what, "flat_to_sorted", flat_to_sorted, torch.int32, (M * k,), gpu),
                    _epilogue(what, epi, act, (M, H), gpu), _addr(what, "dx", dx, odt, (M, H), gpu)), what)


def moe_route_backward(p, topk_idx, topk_w, dtopk_w, dlogits, stream=None):
    """Gradient of the router: topk_idx [M, k] int32, topk_w and dtopk_w [M, k] f32
    -> dlogits [M, E] f32."""
    import torch
    what = "moe_route_backward"
    M, E, k, gpu = p.num_tokens, p.num_experts, p.topk, _gpu_of(what, "topk_idx", topk_idx)
    f32 = torch.float32
    _check(_call_on(gpu, stream, load_library().moe_route_backward, ctypes.byref(p),
                    _addr(what, "topk_idx", topk_idx, torch.int32, (M, k), gpu),
                    _addr(what, "topk_w", topk_w, f32, (M, k), gpu), _addr(what, "dtopk_w", dtopk_w, f32, (M, k), gpu),
                    _addr(what, "dlogits", dlogits, f32, (M, E), gpu)), what)


def _segments(p):
    return p.num_src_blocks * (p.local_experts or p.num_experts)


def moe_grouped_gemm_aux(p, a, w0, w1, offsets, gate, up, c, stream=None):
    """Layer 0 of the grouped GEMM that keeps its products for the gradient: a
    [R, H], w0, w1 [EL, F, H], offsets [G + 1] -> gate, up, c (Hact) [R, F]."""
    import torch
    what = "moe_grouped_gemm_aux"
    R, H, F, gpu = p.num_tokens * p.topk, p.hidden, p.ffn, _gpu_of(what, "a", a)
    EL, act = p.local_experts or p.num_experts, _dtypes(p)[0]
    _check(_call_on(gpu, stream, load_library().moe_grouped_gemm_aux, ctypes.byref(p),
                    _addr(what, "a", a, act, (R, H), gpu), _addr(what, "w0", w0, act, (EL, F, H), gpu),
                    _addr(what, "w1", w1, act, (EL, F, H), gpu),
                    _addr(what, "offsets", offsets, torch.int32, (_segments(p) + 1,), gpu),
                    _addr(what, "gate", gate, act, (R, F), gpu), _addr(what, "up", up, act, (R, F), gpu),
                    _addr(what, "c", c, act, (R, F), gpu)), what)


def moe_grouped_gemm_backward(p, layer, d0, d1, w0, w1, gate, up, offsets, o0, o1, ws=None, stream=None):
    """Gradient of the grouped GEMM for its rows.  Layer 1: d0 = dY [R, H], w0 =
    W_down, gate, up [R, F] -> o0 = dgate, o1 = dup [R, F] (d1, w1 None).  Layer 0:
    d0 = dgate, d1 = dup, w0 = W_gate, w1 = W_up -> o0 = dX_perm [R, H] (gate, up,
    o1 None).  ws moe_workspace_bytes(p, MOE_OP_GROUPED_GEMM_BACKWARD) bytes."""
    import torch
    what = "moe_grouped_gemm_backward"
    R, H, F, gpu = p.num_tokens * p.topk, p.hidden, p.ffn, _gpu_of(what, "d0", d0)
    EL, act = p.local_experts or p.num_experts, _dtypes(p)[0]
    din, dout = (F, H) if layer == 0 else (H, F)
    wshape = (EL, F, H) if layer == 0 else (EL, H, F)
    _check(_call_on(gpu, stream, load_library().moe_grouped_gemm_backward, ctypes.byref(p), int(layer),
                    _addr(what, "d0", d0, act, (R, din), gpu), _addr(what, "d1", d1, act, (R, din), gpu),
                    _addr(what, "w0", w0, act, wshape, gpu), _addr(what, "w1", w1, act, wshape, gpu),
                    _addr(what, "gate", gate, act, (R, F), gpu), _addr(what, "up", up, act, (R, F), gpu),
                    _addr(what, "offsets", offsets, torch.int32, (_segments(p) + 1,), gpu),
                    _addr(what, "o0", o0, act, (R, dout), gpu), _addr(what, "o1", o1, act, (R, dout), gpu),
                    *_workspace(what, ws, gpu)), what)


def moe_grouped_gemm_backward_weights(p, layer, d0, d1, a, offsets, dw0, dw1, accumulate=False, ws=None, stream=None):
    """Gradient of the grouped GEMM for its weights.  Layer 1: d0 = dY [R, H], a =
    Hact [R, F] -> dw0 = dW_down [EL, H, F] (d1, dw1 None).  Layer 0: d0 = dgate, d1
    = dup [R, F], a = X_perm [R, H] -> dw0 = dW_gate, dw1 = dW_up [EL, F, H].  dw0
    and dw1 f32 or bf16; accumulate (f32): added to what they hold."""
    import torch
    what = "moe_grouped_gemm_backward_weights"
    R, H, F, gpu = p.num_tokens * p.topk, p.hidden, p.ffn, _gpu_of(what, "a", a)
    EL, act = p.local_experts or p.num_experts, _dtypes(p)[0]
    n, m = (F, H) if layer == 0 else (H, F)
    bf16 = dw0 is not None and dw0.dtype is torch.bfloat16
    odt = torch.bfloat16 if bf16 else torch.float32
    _check(_call_on(gpu, stream, load_library().moe_grouped_gemm_backward_weights, ctypes.byref(p), int(layer),
                    _addr(what, "d0", d0, act, (R, n), gpu), _addr(what, "d1", d1, act, (R, n), gpu),
                    _addr(what, "a", a, act, (R, m), gpu),
                    _addr(what, "offsets", offsets, torch.int32, (_segments(p) + 1,), gpu),
                    MOE_DTYPE_BF16 if bf16 else MOE_DTYPE_F32, int(bool(accumulate)),
                    _addr(what, "dw0", dw0, odt, (EL, n, m), gpu), _addr(what, "dw1", dw1, odt, (EL, n, m), gpu),
                    *_workspace(what, ws, gpu)), what)


def moe_debug_device_status(p, ws, stream=None) -> int:
    return load_library().moe_debug_device_status(ctypes.byref(p), _ptr(ws), _nbytes(ws), _stream(stream))
