"""The serving operators' host checks (moe_layer_decode, moe_adapter_linear):
every refusal before anything is launched (CPU only: no call here reaches a
kernel)."""
import ctypes
import os

import pytest
import torch

import combine_topk_gate_amd as moe
import serving_ref as ref

INV, UNS, SMALL = moe.MOE_ERR_INVALID_ARGUMENT, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE_TOO_SMALL
B = ctypes.byref
P = ctypes.c_void_p
MiB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from combine_topk_gate_amd import build
        build.build()
    return moe.load_library()


def at(i):
    """A fake device address, far from the others (never dereferenced)."""
    return P((1 << 32) + i * (1 << 32))


def decode(lib, p, epi=None, ws_bytes=None, **ptr):
    a = dict(x=at(0), logits=at(1), w_gate=at(2), w_up=at(3), w_down=at(4), out=at(5), ws=at(6))
    a.update(ptr)
    n = moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE) if ws_bytes is None else ws_bytes
    return lib.moe_layer_decode(B(p), a["x"], a["logits"], a["w_gate"], a["w_up"], a["w_down"],
                                B(epi) if epi else None, a["out"], a["ws"], n, None)


def adapter(lib, q, epi=None, ws_bytes=None, **ptr):
    a = dict(x=at(0), w=at(1), a=at(2), b=at(3), scale=at(4), idx=at(5), out=at(6), ws=at(7))
    a.update(ptr)
    n = moe.moe_adapter_workspace_bytes(q) if ws_bytes is None else ws_bytes
    return lib.moe_adapter_linear(B(q), a["x"], a["w"], a["a"], a["b"], a["scale"], a["idx"],
                                  B(epi) if epi else None, a["out"], a["ws"], n, None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(H=100), dict(F=32), dict(E=0), dict(E=513), dict(k=0), dict(k=9),
                                dict(S=0), dict(expert_base=3), dict(expert_base=6, local_experts=3)])
def test_decode_refuses_bad_problems(lib, kw):
    p = moe.problem(**dict(dict(M=4, H=64, F=64, E=8, k=2), **kw))
    assert moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE) == 0
    assert decode(lib, p, ws_bytes=1 << 30) == INV
    assert lib.moe_layer_decode(None, *[None] * 8, 0, None) == INV


def test_decode_token_limit(lib):
    assert moe.MOE_DECODE_MAX_TOKENS == 256
    ok, over = moe.problem(256, 64, 64, 8, 2), moe.problem(257, 64, 64, 8, 2)
    assert moe.moe_workspace_bytes(ok, moe.MOE_OP_LAYER_DECODE) > 0
    assert moe.moe_workspace_bytes(over, moe.MOE_OP_LAYER_DECODE) == 0
    assert decode(lib, over, ws_bytes=1 << 30) == UNS
    # MXFP8 needs whole 128-column quads
    assert decode(lib, moe.problem(4, 64, 192, 8, 2, dtype="bf16_mxfp8"), ws_bytes=1 << 30) == UNS


def test_decode_refuses_bad_pointers(lib):
    p = moe.problem(4, 64, 64, 8, 2)
    for name in ("x", "logits", "w_gate", "w_up", "w_down", "out"):
        assert decode(lib, p, **{name: None}) == INV, name
    for name in ("x", "w_gate", "w_up", "w_down", "out"):
        assert decode(lib, p, **{name: P((1 << 40) + 8)}) == INV, name
    assert decode(lib, p, logits=P((1 << 40) + 2)) == INV
    assert decode(lib, p, ws=None) == SMALL
    assert decode(lib, p, ws_bytes=moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE) - 1) == SMALL
    assert decode(lib, p, ws=P((1 << 40) + 128)) == INV
    for bad in (moe.Epilogue(None, 7), moe.Epilogue((1 << 40) + 8, moe.MOE_DTYPE_BF16)):
        assert decode(lib, p, epi=bad) == INV


def test_decode_refuses_overlaps(lib):
    p = moe.problem(4, 64, 64, 8, 2)
    assert decode(lib, p, out=at(0)) == INV  # x
    assert decode(lib, p, out=P(at(1).value + 64)) == INV  # logits
    assert decode(lib, p, out=P(at(6).value + 256)) == INV  # ws
    for i in (2, 3, 4):  # the last bytes of the weights
        assert decode(lib, p, out=P(at(i).value + 8 * 64 * 64 * 2 - 16)) == INV
    # the residual one row further, or in place with another type
    assert decode(lib, p, epi=moe.Epilogue(at(5).value + 128, moe.MOE_DTYPE_BF16)) == INV
    assert decode(lib, p, epi=moe.Epilogue(at(5).value, moe.MOE_DTYPE_F32)) == INV


def test_decode_without_tokens_launches_nothing(lib):
    p = moe.problem(0, 64, 64, 8, 2)
    assert decode(lib, p, x=None, logits=None, out=None, ws=None, ws_bytes=0) == moe.MOE_OK


def test_workspace_sizes_without_tokens(lib):
    for dtype in ("bf16", "f32", "bf16_mxfp8"):
        for E, k, held in ((1, 1, 0), (512, 16, 3)):
            p = moe.problem(0, 64, 128, E, k, dtype=dtype, local_experts=held)
            assert 0 <= moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE) < 1 << 16


def test_decode_workspace_covers_the_intermediates(lib):
    for M, H, F, E, k in ((1, 64, 64, 1, 1), (200, 4096, 14336, 8, 2), (256, 64, 64, 512, 16)):
        p = moe.problem(M, H, F, E, k)
        assert moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE) >= M * k * (6 * F + 4 * H + 12)


@pytest.mark.parametrize("kw,err", [(dict(M=-1), INV), (dict(H=32), INV), (dict(H=100), INV), (dict(H=1 << 17), INV),
                                    (dict(N=0), INV), (dict(N=65537), INV), (dict(rank=0), INV), (dict(rank=12), INV),
                                    (dict(rank=264), INV), (dict(num_adapters=-1), INV),
                                    (dict(num_adapters=65537), INV), (dict(M=1 << 27), UNS),
                                    (dict(M=1 << 62), UNS), (dict(M=1 << 25, N=1 << 15), UNS),
                                    (dict(dtype="bf16_mxfp8"), UNS)])
def test_adapter_refuses_bad_problems(lib, kw, err):
    q = moe.adapter_problem(**dict(dict(M=4, H=64, N=8, rank=8, num_adapters=2), **kw))
    assert moe.moe_adapter_workspace_bytes(q) == 0
    assert adapter(lib, q, ws_bytes=1 << 30) == err
    assert lib.moe_adapter_linear(None, *[None] * 9, 0, None) == INV


def test_adapter_refuses_bad_types(lib):
    q = moe.AdapterProblem(4, 64, 8, 8, 2, 9)
    assert adapter(lib, q, ws_bytes=1 << 30) == INV


def test_adapter_refuses_bad_pointers(lib):
    q = moe.adapter_problem(4, 64, 8, 8, 2)
    for name in ("x", "w", "a", "b", "scale", "idx", "out"):
        assert adapter(lib, q, **{name: None}) == INV, name
    for name in ("x", "w", "a", "b", "out"):
        assert adapter(lib, q, **{name: P((1 << 40) + 8)}) == INV, name
    for name in ("scale", "idx"):
        assert adapter(lib, q, **{name: P((1 << 40) + 2)}) == INV, name
    assert adapter(lib, q, ws=None) == SMALL
    assert adapter(lib, q, ws_bytes=moe.moe_adapter_workspace_bytes(q) - 1) == SMALL
    assert adapter(lib, q, ws=P((1 << 40) + 64)) == INV
    for bad in (moe.Epilogue(None, 7), moe.Epilogue((1 << 40) + 8, moe.MOE_DTYPE_BF16)):
        assert adapter(lib, q, epi=bad) == INV


def test_adapter_refuses_overlaps(lib):
    q = moe.adapter_problem(64, 64, 64, 8, 2)
    assert adapter(lib, q, out=P(at(0).value + 64)) == INV  # x
    assert adapter(lib, q, out=at(1)) == INV  # w
    assert adapter(lib, q, out=P(at(2).value + 2 * 8 * 64 * 2 - 16)) == INV  # a
    assert adapter(lib, q, out=P(at(3).value + 2 * 64 * 8 * 2 - 16)) == INV  # b
    assert adapter(lib, q, out=at(4)) == INV  # scale
    assert adapter(lib, q, out=P(at(5).value + 240)) == INV  # adapter_idx
    assert adapter(lib, q, out=at(7)) == INV  # ws
    assert adapter(lib, q, epi=moe.Epilogue(at(6).value + 128, moe.MOE_DTYPE_BF16)) == INV
    assert adapter(lib, q, epi=moe.Epilogue(at(6).value, moe.MOE_DTYPE_F32)) == INV


def test_adapter_without_rows_or_adapters(lib):
    q = moe.adapter_problem(0, 64, 8, 8, 2)
    assert adapter(lib, q, x=None, idx=None, out=None, ws=None, ws_bytes=0) == moe.MOE_OK
    # no adapters: no workspace, any rank, and none of their pointers
    q = moe.adapter_problem(0, 64, 8, 0, 0)
    assert moe.moe_adapter_workspace_bytes(moe.adapter_problem(100, 64, 8, 0, 0)) == 0
    assert adapter(lib, q, a=None, b=None, scale=None, idx=None, ws=None, ws_bytes=0) == moe.MOE_OK


def test_binding_refuses_tensors_it_would_misread(lib):
    """Host tensors, other shapes, types and strides end in MoeError before the
    library sees a pointer."""
    def t(*shape, dtype=torch.bfloat16, device="meta"):
        return torch.empty(shape, dtype=dtype, device=device)

    p = moe.problem(4, 64, 128, 8, 2)
    w = (t(8, 128, 64), t(8, 128, 64), t(8, 64, 128))
    for x in (t(4, 64), torch.zeros(4, 64).bfloat16()):
        with pytest.raises(moe.MoeError) as ex:
            moe.moe_layer_decode(p, x, t(4, 8, dtype=torch.float32), *w, None, t(4, 64, dtype=torch.float32), None)
        assert ex.value.status == INV
    q = moe.adapter_problem(4, 64, 8, 8, 2)
    with pytest.raises(moe.MoeError) as ex:
        moe.moe_adapter_linear(q, t(4, 64, device="cpu"), t(8, 64, device="cpu"), None, None, None, None, None,
                               t(4, 8, device="cpu"), None)
    assert ex.value.status == INV


def test_reference_quantiser_matches_its_values():
    """The reference's MXFP8 buffer and the values it returns are the same
    tensor, and a value is off by at most half an e4m3 step."""
    g = torch.Generator()
    g.manual_seed(3)
    w = torch.randn((64, 256), generator=g) * 0.05
    buf, v = ref.quantize_mxfp8(w)
    assert buf.numel() == moe.mx_bytes(64, 256)
    codes = buf[:64 * 256].view(torch.float8_e4m3fn).double().view(64, 8, 32)
    for r in (0, 31, 32, 63):
        for b in range(8):
            s = int(buf[64 * 256 + (r // 32) * 256 + (b // 4) * 128 + (r % 32) * 4 + b % 4])
            assert torch.equal(codes[r, b] * 2.0 ** (s - 127), v[r, 32 * b:32 * b + 32])
    # With the block's scale S = 2^X, amax / S lies in [256, 512).  A value of
    # magnitude in [2^e, 2^(e+1)) S is rounded to steps of 2^(e-3) S: off by at
    # most 2^(e-4) S <= 2^-4 of it; below 2^-6 S the steps are 2^-9 S, half of
    # one 2^-10 S; above 448 S (e4m3's largest) it becomes 448 S.
    a = w.double().view(64, 8, 32).abs()
    S = torch.exp2(torch.floor(torch.log2(a.amax(-1, keepdim=True))) - 8)
    err = (v.view(64, 8, 32) - w.double().view(64, 8, 32)).abs()
    bound = torch.maximum(torch.maximum(2.0 ** -4 * a, 2.0 ** -10 * S), a - 448 * S)
    assert bool((err <= bound).all())


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0: what the binding looks at."""

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def binding_calls():
    """name -> (call, its tensors by name): calls that the binding passes on."""
    f32 = torch.float32
    p = moe.problem(4, 64, 128, 8, 2)
    q = moe.adapter_problem(4, 64, 16, 8, 3)

    def decode(x, logits, w_gate, w_up, w_down, residual, out, ws):
        moe.moe_layer_decode(p, x, logits, w_gate, w_up, w_down, moe.epilogue(residual, "bf16"), out, ws, stream=0)

    def linear(x, w, a, b, scale, adapter_idx, residual, out, ws):
        moe.moe_adapter_linear(q, x, w, a, b, scale, adapter_idx, moe.epilogue(residual, "bf16"), out, ws, stream=0)

    return {
        "decode": (decode, dict(x=on_gpu(4, 64), logits=on_gpu(4, 8, dtype=f32), w_gate=on_gpu(8, 128, 64),
                                w_up=on_gpu(8, 128, 64), w_down=on_gpu(8, 64, 128), residual=on_gpu(4, 64),
                                out=on_gpu(4, 64), ws=on_gpu(1 << 20, dtype=torch.uint8))),
        "linear": (linear, dict(x=on_gpu(4, 64), w=on_gpu(16, 64), a=on_gpu(3, 8, 64), b=on_gpu(3, 16, 8),
                                scale=on_gpu(3, dtype=f32), adapter_idx=on_gpu(4, dtype=torch.int32),
                                residual=on_gpu(4, 16), out=on_gpu(4, 16), ws=on_gpu(1 << 20, dtype=torch.uint8))),
    }


BINDING_TENSORS = [("decode", n) for n in ("x", "logits", "w_gate", "w_up", "w_down", "residual", "out", "ws")] + \
                  [("linear", n) for n in ("x", "w", "a", "b", "scale", "adapter_idx", "residual", "out", "ws")]


@pytest.fixture
def passed_on(lib, monkeypatch):
    """The calls that the binding has passed on to the library (which is not called)."""
    calls = []
    monkeypatch.setattr(moe, "_call_on", lambda gpu, stream, f, *args: calls.append(args) or moe.MOE_OK)
    return calls


@pytest.mark.parametrize("which,name", BINDING_TENSORS)
def test_binding_checks_each_tensor(which, name, passed_on):
    """Right but for one tensor's type, shape, strides or device."""
    call, t = binding_calls()[which]
    call(**t)
    assert len(passed_on) == 1
    good = t[name]
    wide = torch.zeros(good.shape[:-1] + (2 * good.shape[-1],), dtype=good.dtype).as_subclass(OnGpu)
    bad = {"strides": wide[..., ::2], "device": good.as_subclass(torch.Tensor)}
    if name != "ws":
        bad["type"] = good.to(torch.float16)
        bad["shape"] = torch.cat([good, good]).as_subclass(OnGpu)
        if good.dim() > 1:
            bad["transposed"] = good.transpose(0, 1)
    assert bad["strides"].shape == good.shape and bad["device"].get_device() == -1
    for what, b in bad.items():
        with pytest.raises(moe.MoeError) as ex:
            call(**dict(t, **{name: b}))
        assert ex.value.status == INV, what
    assert len(passed_on) == 1


def test_epilogue_keeps_its_residual():
    r = torch.zeros(4, 64)
    at = r.data_ptr()
    epi = moe.epilogue(r)
    del r
    assert epi.tensor.data_ptr() == at == epi.residual
    assert moe.epilogue().tensor is None and moe.epilogue().residual is None


def test_a_residual_that_moved_is_refused(passed_on):
    call, t = binding_calls()["decode"]
    p = moe.problem(4, 64, 128, 8, 2)
    epi = moe.epilogue(t["residual"], "bf16")
    args = [t[n] for n in ("x", "logits", "w_gate", "w_up", "w_down")]
    moe.moe_layer_decode(p, *args, epi, t["out"], t["ws"], stream=0)
    epi.tensor.set_(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(moe.MoeError):
        moe.moe_layer_decode(p, *args, epi, t["out"], t["ws"], stream=0)
    # an address without a tensor is passed on as it is
    moe.moe_layer_decode(p, *args, moe.Epilogue(1 << 40, moe.MOE_DTYPE_BF16), t["out"], t["ws"], stream=0)
    assert len(passed_on) == 2


def test_binding_refuses_calls_without_x(passed_on):
    for which in ("decode", "linear"):
        call, t = binding_calls()[which]
        with pytest.raises(moe.MoeError) as ex:
            call(**dict(t, x=None))
        assert ex.value.status == INV
    assert not passed_on


def tiles_of(shape, out="f32"):
    s = dict(dict(r=0, dtype="bf16"), **shape)
    return moe.moe_adapter_tiles(moe.adapter_problem(s["M"], s["H"], s["N"], s["r"], s["P"], s["dtype"]), out)


@pytest.mark.parametrize("shape,tiles", ref.TILES)
def test_adapter_tiles(lib, shape, tiles):
    """The rule on sizes: the shapes that the GPU tests run take the kernels
    that they are there for."""
    assert tiles_of(shape) == tiles


def test_adapter_tiles_covers_every_kernel(lib):
    bf16 = [t for s, t in ref.TILES if s.get("dtype") != "f32"]
    f32 = [t for s, t in ref.TILES if s.get("dtype") == "f32"]
    streamed = {(16, 16), (32, 32), (64, 64)}
    assert {t[:2] for t in bf16} == streamed | {(8, 16), (64, 256), (128, 256), (256, 256)}
    assert {t[:2] for t in f32} == streamed
    t_tiles = {(16, 16), (16, 32), (32, 16), (32, 32), (32, 64)}
    assert {t[2:] for t in bf16} == {t[2:] for t in f32} | {(0, 0)} == t_tiles | {(0, 0)}


def test_adapter_tiles_refuses_bad_arguments(lib):
    q = moe.adapter_problem(4, 64, 8, 8, 2)
    tiles = (ctypes.c_int32 * 4)()
    assert lib.moe_adapter_tiles(None, moe.MOE_DTYPE_F32, tiles) == INV
    assert lib.moe_adapter_tiles(B(q), moe.MOE_DTYPE_BF16_MXFP8, tiles) == INV
    assert lib.moe_adapter_tiles(B(q), moe.MOE_DTYPE_F32, None) == INV
    assert lib.moe_adapter_tiles(B(moe.adapter_problem(4, 64, 8, 12, 2)), moe.MOE_DTYPE_F32, tiles) == INV
    assert lib.moe_adapter_tiles(B(moe.adapter_problem(4, 64, 8, 8, 2, "bf16_mxfp8")), moe.MOE_DTYPE_F32, tiles) == UNS
    assert tiles_of(dict(M=0, H=64, N=8, r=8, P=2)) == (0, 0, 0, 0)
