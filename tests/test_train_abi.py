"""The training operators' host checks: every refusal before anything is
launched (CPU only: no call here reaches a kernel)."""
import ctypes
import os

import pytest
import torch

import combine_topk_gate_amd as moe
from test_serving_abi import INV, UNS, OnGpu, P, at, on_gpu

B = ctypes.byref
OK = moe.MOE_OK
M, H, F, E, k = 4, 64, 128, 8, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from combine_topk_gate_amd import build
        build.build()
    return moe.load_library()


def drop(p=0.5, rng=None):
    return moe.Dropout(p, at(20).value if rng is None else rng)


# name -> (arguments in order; "problem", "epi", "drop" and numbers by name too)
CALLS = {
    "combine_dropout": ("problem", "y", "topk_w", "f2s", "epi", "drop", "out"),
    "combine_backward": ("problem", "dout", "dout_dtype", "y", "topk_w", "f2s", "drop", "dy", "dtopk_w"),
    "dispatch_backward": ("problem", "dx_perm", "f2s", "epi", "dx"),
    "route_backward": ("problem", "topk_idx", "topk_w", "dtopk_w", "dlogits"),
    "grouped_gemm_aux": ("problem", "a", "w0", "w1", "offsets", "gate", "up", "c"),
    "rows1": ("problem", "layer", "d0", "d1", "w0", "w1", "gate", "up", "offsets", "o0", "o1", "ws", "ws_bytes"),
    "rows0": ("problem", "layer", "d0", "d1", "w0", "w1", "gate", "up", "offsets", "o0", "o1", "ws", "ws_bytes"),
    "weights1": ("problem", "layer", "d0", "d1", "a", "offsets", "dw_dtype", "accumulate", "dw0", "dw1", "ws", "ws_bytes"),
    "weights0": ("problem", "layer", "d0", "d1", "a", "offsets", "dw_dtype", "accumulate", "dw0", "dw1", "ws", "ws_bytes"),
}
NUMBERS = {"rows1": dict(layer=1), "rows0": dict(layer=0), "weights1": dict(layer=1, dw_dtype=0, accumulate=0),
           "weights0": dict(layer=0, dw_dtype=0, accumulate=0), "combine_backward": dict(dout_dtype=0)}
ABSENT = {"rows1": ("d1", "w1"), "rows0": ("gate", "up", "o1"), "weights1": ("d1", "dw1"), "weights0": ()}
WORDS = ("topk_w", "f2s", "dtopk_w", "topk_idx", "offsets")
OUTPUTS = {"combine_dropout": ("out",), "combine_backward": ("dy", "dtopk_w"), "dispatch_backward": ("dx",),
           "route_backward": ("dlogits",), "grouped_gemm_aux": ("gate", "up", "c"), "rows1": ("o0", "o1"), "rows0": ("o0",),
           "weights1": ("dw0",), "weights0": ("dw0", "dw1")}


def tensors(name):
    skip = ("problem", "epi", "drop", "ws", "ws_bytes", *NUMBERS.get(name, {}), *ABSENT.get(name, ()))
    return [a for a in CALLS[name] if a not in skip]


def call(lib, name, **kw):
    problem = kw.pop("problem", moe.problem(M, H, F, E, k, dtype="f32"))
    v = {a: at(i) for i, a in enumerate(CALLS[name])}
    v.update(NUMBERS.get(name, {}), epi=None, ws=at(15), ws_bytes=1 << 28)
    v.update({a: None for a in ABSENT.get(name, ())})
    v["drop"] = drop()
    v.update(kw)
    v["problem"] = B(problem) if problem is not None else None
    for n in ("epi", "drop"):
        v[n] = B(v[n]) if v[n] is not None else None
    fn = {"rows1": "grouped_gemm_backward", "rows0": "grouped_gemm_backward", "weights1": "grouped_gemm_backward_weights",
          "weights0": "grouped_gemm_backward_weights"}.get(name, name)
    return getattr(lib, "moe_" + fn)(*[v[a] for a in CALLS[name]], None)


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_problems(lib, name):
    assert call(lib, name, problem=None) == INV
    for kw in (dict(M=-1), dict(H=100), dict(F=32), dict(E=0), dict(E=513), dict(k=0), dict(k=9), dict(S=0),
               dict(expert_base=3), dict(expert_base=6, local_experts=3)):
        assert call(lib, name, problem=moe.problem(**dict(dict(M=M, H=H, F=F, E=E, k=k), **kw))) == INV, kw
    assert call(lib, name, problem=moe.problem(1 << 26, 64, 64, 8, 2)) == UNS
    if name not in ("combine_dropout", "combine_backward", "dispatch_backward", "route_backward"):
        assert call(lib, name, problem=moe.problem(M, H, F, E, k, dtype="bf16_mxfp8")) == UNS


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_pointers(lib, name):
    for a in tensors(name):
        assert call(lib, name, **{a: None}) == INV, a
        assert call(lib, name, **{a: P((1 << 50) + (2 if a in WORDS else 8))}) == INV, a


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_overlap_nothing(lib, name):
    v = {a: at(i) for i, a in enumerate(CALLS[name])}
    for o in OUTPUTS[name]:
        for a in tensors(name):
            if a != o:
                assert call(lib, name, **{o: v[a]}) == INV, (o, a)
                if a not in WORDS and o not in WORDS:
                    assert call(lib, name, **{o: P(v[a].value + 16)}) == INV, (o, a)


@pytest.mark.parametrize("name", ["rows1", "rows0", "weights1", "weights0"])
def test_layers_and_their_operands(lib, name):
    for layer in (-1, 2):
        assert call(lib, name, layer=layer) == INV
    for a in ABSENT[name]:  # an operand of the other layer is a mistake, not something to ignore
        assert call(lib, name, **{a: at(17)}) == INV, a


@pytest.mark.parametrize("name", ["rows1", "rows0", "weights1", "weights0"])
def test_workspaces(lib, name):
    op = moe.MOE_OP_GROUPED_GEMM_BACKWARD
    for dtype in ("f32", "bf16"):
        p = moe.problem(60, 448, 8576, 2, 1, dtype=dtype)  # few tiles with long reductions
        need = moe.moe_workspace_bytes(p, op)
        assert need > 0
        assert call(lib, name, problem=p, ws=None) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
        assert call(lib, name, problem=p, ws_bytes=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
        assert call(lib, name, problem=p, ws=P(at(15).value + 128)) == INV
        for a in tensors(name):  # no buffer of the call lies in it
            assert call(lib, name, problem=p, ws=at(CALLS[name].index(a))) == INV, a
    assert moe.moe_workspace_bytes(moe.problem(0, H, F, E, k), op) == 0
    # no tile would be split: none is needed, and one that is given is not looked at
    assert moe.moe_workspace_bytes(moe.problem(M, H, F, E, k), op) == 0
    assert moe.moe_workspace_bytes(moe.problem(M, H, F, E, k, dtype="bf16_mxfp8"), op) == 0


def test_weights_types(lib):
    for name in ("weights1", "weights0"):
        for bad in (-1, 2, 7):
            assert call(lib, name, dw_dtype=bad) == INV
        assert call(lib, name, dw_dtype=moe.MOE_DTYPE_BF16, accumulate=1) == UNS
    for bad in (-1, 2, 7):
        assert call(lib, "combine_backward", dout_dtype=bad) == INV


@pytest.mark.parametrize("name", ["combine_dropout", "combine_backward"])
def test_dropouts(lib, name):
    for bad in (drop(-0.1), drop(1.0), drop(2.0), drop(float("nan")), drop(float("inf")), drop(rng=0),
                drop(rng=(1 << 50) + 4), drop(rng=at(len(CALLS[name]) - 1).value)):  # the last one: in the output
        assert call(lib, name, drop=bad) == INV, (bad.p, bad.rng)


@pytest.mark.parametrize("name,out", [("combine_dropout", "out"), ("dispatch_backward", "dx")])
def test_epilogues(lib, name, out):
    v = {a: at(i) for i, a in enumerate(CALLS[name])}
    for bad in (moe.Epilogue(None, 7), moe.Epilogue((1 << 50) + 8, moe.MOE_DTYPE_F32),
                moe.Epilogue(v[out].value + 128, moe.MOE_DTYPE_F32), moe.Epilogue(v[out].value, moe.MOE_DTYPE_BF16)):
        assert call(lib, name, epi=bad) == INV


def test_no_tokens_launch_nothing(lib):
    p = moe.problem(0, H, F, E, k, dtype="f32")
    none = lambda *names: dict.fromkeys(names)
    assert call(lib, "combine_dropout", problem=p, **none("y", "topk_w", "f2s", "out")) == OK
    assert call(lib, "combine_backward", problem=p, **none("dout", "y", "topk_w", "f2s", "dy", "dtopk_w")) == OK
    assert call(lib, "dispatch_backward", problem=p, **none("dx_perm", "f2s", "dx")) == OK
    assert call(lib, "route_backward", problem=p, **none("topk_idx", "topk_w", "dtopk_w", "dlogits")) == OK
    assert call(lib, "grouped_gemm_aux", problem=p, **none("a", "gate", "up", "c")) == OK
    assert call(lib, "rows1", problem=p, **none("d0", "gate", "up", "o0", "o1")) == OK
    assert call(lib, "rows0", problem=p, **none("d0", "d1", "o0")) == OK
    assert call(lib, "combine_dropout", problem=p, drop=drop(1.5)) == INV


# ----------------------------------------------------------------- binding ---


def binding_calls():
    f32, i32 = torch.float32, torch.int32
    p = moe.problem(M, H, F, E, k)
    R, t = M * k, on_gpu
    w = dict(topk_w=t(M, k, dtype=f32), f2s=t(R, dtype=i32))
    rng = t(2, dtype=torch.int64)

    def combine(y, topk_w, f2s, residual, rng, out):
        moe.moe_combine_dropout(p, y, topk_w, f2s, moe.epilogue(residual, "bf16"), moe.dropout(0.5, rng), out, stream=0)

    def combine_backward(dout, y, topk_w, f2s, rng, dy, dtopk_w):
        moe.moe_combine_backward(p, dout, y, topk_w, f2s, moe.dropout(0.5, rng), dy, dtopk_w, stream=0)

    def dispatch_backward(dx_perm, f2s, residual, dx):
        moe.moe_dispatch_backward(p, dx_perm, f2s, moe.epilogue(residual, "bf16"), dx, stream=0)

    def route_backward(topk_idx, topk_w, dtopk_w, dlogits):
        moe.moe_route_backward(p, topk_idx, topk_w, dtopk_w, dlogits, stream=0)

    def aux(a, w0, w1, offsets, gate, up, c):
        moe.moe_grouped_gemm_aux(p, a, w0, w1, offsets, gate, up, c, stream=0)

    def rows1(d0, w0, gate, up, offsets, o0, o1, ws):
        moe.moe_grouped_gemm_backward(p, 1, d0, None, w0, None, gate, up, offsets, o0, o1, ws, stream=0)

    def rows0(d0, d1, w0, w1, offsets, o0, ws):
        moe.moe_grouped_gemm_backward(p, 0, d0, d1, w0, w1, None, None, offsets, o0, None, ws, stream=0)

    def weights1(d0, a, offsets, dw0, ws):
        moe.moe_grouped_gemm_backward_weights(p, 1, d0, None, a, offsets, dw0, None, False, ws, stream=0)

    def weights0(d0, d1, a, offsets, dw0, dw1, ws):
        moe.moe_grouped_gemm_backward_weights(p, 0, d0, d1, a, offsets, dw0, dw1, False, ws, stream=0)

    rows = lambda n: t(R, n)
    off = t(E + 1, dtype=i32)
    ws = t(1 << 20, dtype=torch.uint8)
    return {
        "combine": (combine, dict(y=t(R, H, dtype=f32), residual=t(M, H), rng=rng, out=t(M, H), **w)),
        "combine_backward": (combine_backward, dict(dout=t(M, H), y=t(R, H, dtype=f32), rng=rng, dy=rows(H),
                                                    dtopk_w=t(M, k, dtype=f32), **w)),
        "dispatch_backward": (dispatch_backward, dict(dx_perm=rows(H), f2s=w["f2s"], residual=t(M, H), dx=t(M, H))),
        "route_backward": (route_backward, dict(topk_idx=t(M, k, dtype=i32), topk_w=t(M, k, dtype=f32),
                                                dtopk_w=t(M, k, dtype=f32), dlogits=t(M, E, dtype=f32))),
        "aux": (aux, dict(a=rows(H), w0=t(E, F, H), w1=t(E, F, H), offsets=off, gate=rows(F), up=rows(F), c=rows(F))),
        "rows1": (rows1, dict(d0=rows(H), w0=t(E, H, F), gate=rows(F), up=rows(F), offsets=off, o0=rows(F), o1=rows(F), ws=ws)),
        "rows0": (rows0, dict(d0=rows(F), d1=rows(F), w0=t(E, F, H), w1=t(E, F, H), offsets=off, o0=rows(H), ws=ws)),
        "weights1": (weights1, dict(d0=rows(H), a=rows(F), offsets=off, dw0=t(E, H, F, dtype=f32), ws=ws)),
        "weights0": (weights0, dict(d0=rows(F), d1=rows(F), a=rows(H), offsets=off, dw0=t(E, F, H, dtype=f32),
                                    dw1=t(E, F, H, dtype=f32), ws=ws)),
    }


class Elsewhere(OnGpu):
    def get_device(self):
        return 1


@pytest.mark.parametrize("name", list(binding_calls()))
def test_binding_refuses_tensors_it_would_misread(lib, name, monkeypatch):
    reached = []
    monkeypatch.setattr(moe, "_call_on", lambda gpu, stream, f, *args: reached.append(gpu) or OK)
    call, ok = binding_calls()[name]
    call(**ok)
    assert reached == [0]
    for n, t in ok.items():
        other = torch.float64
        bad = [t.as_subclass(Elsewhere), t.as_subclass(torch.Tensor)]  # on another GPU, on the host
        if n != "ws":
            bad += [t.to(other).as_subclass(OnGpu), torch.zeros((*t.shape, 1), dtype=t.dtype).as_subclass(OnGpu)]
        if t.dim() > 1:
            bad.append(torch.zeros((*t.shape[:-2], t.shape[-1], t.shape[-2]), dtype=t.dtype).transpose(-1, -2).as_subclass(OnGpu))
        for b in bad:
            del reached[:]
            with pytest.raises(moe.MoeError) as ex:
                call(**dict(ok, **{n: b}))
            assert ex.value.status == INV, (name, n)
            assert not reached, (name, n)


def test_a_dropout_holds_its_tensor_and_notices_when_it_moved(lib):
    rng = on_gpu(2, dtype=torch.int64)
    d = moe.dropout(0.25, rng)
    assert d.tensor is rng and d.rng == rng.data_ptr()
    d.tensor = on_gpu(2, dtype=torch.int64)
    with pytest.raises(moe.MoeError):
        moe._dropout("x", d, 0)
