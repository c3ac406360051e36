"""moe_layer_decode against a plain 64-bit layer: types, head counts of the
routing, held experts, odd batches, masked logits, idle rows, blocks of rows
of one expert, epilogues, graph replays and concurrent calls."""
import pytest
import torch

import combine_topk_gate_amd as moe
import serving_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(M, H, F, E, k, held=0, base=0, dtype="bf16", out="f32", residual=False, logits="random", seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 + seed)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    EL = held or E

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(act)

    d = dict(x=normal(M, H), w_gate=normal(EL, F, H, std=0.05), w_up=normal(EL, F, H, std=0.05),
             w_down=normal(EL, H, F, std=0.05), residual=normal(M, H) if residual else None)
    lg = torch.randn((M, E), generator=g, device=DEV)
    if logits == "ties":
        lg = torch.round(lg)  # many equal logits, zeros of both signs
    elif logits == "equal":
        lg = torch.zeros_like(lg)
    elif logits == "masked":  # a third of the experts closed to each token
        lg[torch.rand(lg.shape, generator=g, device=DEV) < 0.33] = float("-inf")
    elif logits == "idle":  # whole rows without a token
        lg[::3] = float("-inf")
    elif logits == "empty":
        lg[:] = float("-inf")
    elif logits == "few":  # fewer open experts than k
        lg[:, 1:] = float("-inf")
    elif logits == "one":  # every token to the same experts
        lg += 50.0 * torch.arange(E, device=DEV)
    elif logits == "lowest":  # the type's lowest value is a value, not a mask
        lg[:, ::2] = torch.finfo(torch.float32).min
    elif logits == "elsewhere":  # only experts that are not held
        lg[:, base:base + EL] = float("-inf")
    d["logits"] = lg
    d["values_down"] = d["w_down"]
    if dtype == "bf16_mxfp8":
        d["w_down"], v = ref.quantize_mxfp8(d["w_down"].view(EL * H, F))
        d["values_down"] = v.view(EL, H, F)
    p = moe.problem(M, H, F, E, k, 1, dtype, base, held)
    odt = torch.bfloat16 if out == "bf16" else torch.float32
    # the output between guard rows, the workspace full of NaN bits
    guard = torch.full((M + 2, H), 7.0, dtype=odt, device=DEV)
    ws = torch.full((moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE),), 0xFF, dtype=torch.uint8, device=DEV)
    out_t = guard[1:M + 1]
    out_t.fill_(float("nan"))
    return p, d, moe.epilogue(d["residual"], out), out_t, ws, guard


def call(p, d, epi, out, ws, stream=None):
    moe.moe_layer_decode(p, d["x"], d["logits"], d["w_gate"], d["w_up"], d["w_down"], epi, out, ws, stream=stream)


def want(p, d, dtype, out):
    return ref.layer(d["x"], d["logits"], d["w_gate"], d["w_up"], d["values_down"], p.topk, p.expert_base,
                     d["residual"], dtype == "f32", out == "bf16")


def run_and_check(**kw):
    print(f"[decode] {kw}", flush=True)
    p, d, epi, out, ws, guard = make(**kw)
    dtype, odt = kw.get("dtype", "bf16"), kw.get("out", "f32")
    y, bound = want(p, d, dtype, odt)
    call(p, d, epi, out, ws)
    torch.cuda.synchronize()
    ref.check(out, y, bound, kw)
    ref.check_norm(out, y, p.hidden + 3 * p.ffn, odt == "bf16", kw)
    assert bool((guard[0] == 7.0).all()) and bool((guard[-1] == 7.0).all())
    return p, d, epi, out, ws


SHAPES = [
    # one token; more tokens than one 16-row group; the 32- and 64-row variants; the limit
    dict(M=1, H=64, F=64, E=1, k=1),
    dict(M=1, H=256, F=192, E=8, k=2),
    dict(M=1, H=2048, F=1408, E=64, k=4),
    dict(M=3, H=320, F=448, E=8, k=8),
    dict(M=16, H=128, F=320, E=5, k=3),
    dict(M=17, H=128, F=320, E=5, k=3),
    dict(M=32, H=192, F=128, E=4, k=2),
    dict(M=33, H=192, F=128, E=4, k=2),
    dict(M=100, H=448, F=576, E=60, k=6),
    dict(M=255, H=128, F=192, E=3, k=2),
    dict(M=256, H=256, F=256, E=16, k=16),
    dict(M=64, H=128, F=128, E=512, k=10),
]


# entries of 64 and 128 rows (Layer0 wide enough for every CU), with 1 to 128
# rows in them; Layer1's reduction in 4 and 8 parts; Layer0 blocks of few
# tokens that take several column groups
SPLITS = [
    dict(M=60, H=192, F=1408, E=3, k=2),
    dict(M=100, H=128, F=1408, E=3, k=2),
    dict(M=255, H=64, F=1408, E=3, k=2),
    dict(M=256, H=320, F=1024, E=4, k=4),
    dict(M=97, H=64, F=4096, E=1, k=1),
    dict(M=20, H=64, F=8192, E=2, k=2),
    dict(M=9, H=192, F=2560, E=8, k=1),
    dict(M=8, H=64, F=8576, E=22, k=5),
]


@pytest.mark.parametrize("out,residual", [("f32", False), ("bf16", True)])
@pytest.mark.parametrize("shape", SHAPES + SPLITS)
def test_shapes_bf16(shape, out, residual):
    run_and_check(**shape, out=out, residual=residual)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SPLITS)
def test_splits_mxfp8(shape, out):
    run_and_check(**shape, dtype="bf16_mxfp8", out=out, seed=5)


@pytest.mark.parametrize("shape", [dict(M=60, H=64, F=5504, E=3, k=2), dict(M=120, H=64, F=5504, E=3, k=2),
                                   dict(M=255, H=64, F=5504, E=3, k=2), dict(M=73, H=192, F=448, E=4, k=2),
                                   dict(M=29, H=64, F=4096, E=4, k=4), dict(M=8, H=64, F=8576, E=22, k=5)])
def test_splits_f32(shape):
    run_and_check(**shape, dtype="f32", residual=True, seed=6)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s["E"] <= 64])
def test_shapes_f32(shape):
    run_and_check(**shape, dtype="f32", residual=True, seed=1)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [dict(M=1, H=64, F=128, E=4, k=2), dict(M=16, H=192, F=384, E=6, k=2),
                                   dict(M=24, H=192, F=640, E=6, k=3), dict(M=130, H=128, F=256, E=3, k=2)])
def test_shapes_mxfp8(shape, out):
    run_and_check(**shape, dtype="bf16_mxfp8", out=out, seed=2)


def test_bf16_output_of_the_f32_layer():
    run_and_check(M=9, H=128, F=192, E=4, k=2, dtype="f32", out="bf16", residual=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "bf16_mxfp8"])
@pytest.mark.parametrize("M", [1, 12, 70])
@pytest.mark.parametrize("logits", ["ties", "equal", "masked", "idle", "empty", "few", "one", "lowest"])
def test_logits(logits, M, dtype):
    p, d, epi, out, ws = run_and_check(M=M, H=128, F=256, E=9, k=3, dtype=dtype, residual=M == 12, logits=logits, seed=3)
    if logits == "empty":
        want = d["residual"].float() if d["residual"] is not None else torch.zeros_like(out)
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [4, 40, 200])
def test_every_token_to_one_expert(M):
    # blocks of rows of one expert, the last one ragged
    run_and_check(M=M, H=192, F=320, E=4, k=1, logits="one", seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "bf16_mxfp8"])
@pytest.mark.parametrize("M,held,base,logits", [(1, 2, 3, "random"), (20, 4, 0, "random"), (50, 3, 13, "masked"),
                                                (50, 16, 0, "random"), (7, 5, 6, "elsewhere"), (1, 5, 6, "elsewhere")])
def test_held_experts(M, held, base, logits, dtype):
    run_and_check(M=M, H=128, F=128, E=16, k=4, held=held, base=base, dtype=dtype, logits=logits, residual=M == 20, seed=5)


def test_the_shares_of_two_holders_add_up_to_the_layer():
    kw = dict(M=21, H=128, F=192, E=8, k=3, seed=6)
    p, d, epi, out, ws, _ = make(**kw)
    call(p, d, epi, out, ws)
    parts = []
    for base, held in ((0, 3), (3, 5)):
        q = moe.problem(21, 128, 192, 8, 3, 1, "bf16", base, held)
        w = {k: d[k][base:base + held].contiguous() for k in ("w_gate", "w_up", "w_down")}
        o = torch.empty_like(out)
        call(q, dict(d, **w), None, o, torch.empty(moe.moe_workspace_bytes(q, moe.MOE_OP_LAYER_DECODE),
                                                    dtype=torch.uint8, device=DEV))
        parts.append(o.double())
    y, bound = want(p, d, "bf16", "f32")
    ref.check(parts[0] + parts[1], y, bound, "sum of shares")


def test_agrees_with_the_layer_call():
    # the layer call rounds Hact to bf16: 2^-8 of each |h| at most
    M, H, F, E, k = 48, 256, 384, 8, 2
    p, d, epi, out, ws, _ = make(M, H, F, E, k, seed=7)
    call(p, d, epi, out, ws)
    big = torch.empty((M, H), device=DEV)
    lws = torch.empty(moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER), dtype=torch.uint8, device=DEV)
    moe.moe_layer(p, d["x"], d["logits"], None, d["w_gate"], d["w_up"], d["w_down"], big, lws)
    rel = float((big.double() - out.double()).norm() / out.double().norm())
    assert rel <= ref.BF16, rel


def test_source_blocks_do_not_matter():
    p, d, epi, out, ws, _ = make(M=10, H=128, F=128, E=4, k=2, seed=8)
    call(p, d, epi, out, ws)
    first = out.clone()
    q = moe.problem(10, 128, 128, 4, 2, 3)
    out.fill_(float("nan"))
    call(q, d, epi, out, torch.empty(moe.moe_workspace_bytes(q, moe.MOE_OP_LAYER_DECODE), dtype=torch.uint8, device=DEV))
    assert torch.equal(out, first)


def test_output_in_place_of_the_residual():
    p, d, epi, out, ws, _ = make(M=13, H=192, F=128, E=4, k=2, out="bf16", residual=True, seed=9)
    call(p, d, epi, out, ws)
    first = out.clone()
    r = d["residual"]
    call(p, d, moe.epilogue(r, "bf16"), r, ws)
    assert torch.equal(r, first)


@pytest.mark.parametrize("what", ["x", "weights"])
def test_infinities_and_nan_stay_in_their_rows(what):
    # a row of x, or an expert that only some tokens choose, is not finite: the others are as without it
    M, H, F, E, k = 20, 128, 192, 6, 1
    p, d, epi, out, ws, _ = make(M, H, F, E, k, seed=10)
    call(p, d, epi, out, ws)
    clean = out.clone()
    chosen = d["logits"].argmax(1)
    if what == "x":
        d["x"][5] = float("nan")
        d["x"][6, 3] = float("inf")
        touched = torch.zeros(M, dtype=torch.bool, device=DEV)
        touched[5:7] = True
    else:
        e = int(chosen[0])
        d["w_gate"][e, 7] = float("nan")
        d["w_down"][e, 9] = float("inf")
        touched = chosen == e
    out.fill_(0.0)
    call(p, d, epi, out, ws)
    assert torch.equal(out[~touched], clean[~touched])
    assert not bool(torch.isfinite(out[touched]).all())


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 12, 60])
def test_an_activation_past_the_range_is_infinite(M, out):
    # h = silu(1e25) * 1e25 overflows f32; 3.4e38 does not, and rounds past bf16's largest value
    H, F = 64, 64
    p, d, epi, o, ws, _ = make(M, H, F, 1, 1, out=out, seed=14)
    for k in ("x", "w_gate", "w_up", "w_down"):
        d[k].zero_()
    d["x"][:, 0] = 1.0
    d["w_gate"][0, 0, 0] = d["w_up"][0, 0, 0] = 1e25
    d["w_down"][0, 3, 0] = 1.0
    call(p, d, epi, o, ws)
    assert bool((o[:, 3] == float("inf")).all())
    # (in a call of its own: every other column is 0 times that infinity)
    a, b = 127 / 64 * 2.0 ** 63, 129 / 128 * 2.0 ** 64  # both bf16 values
    assert torch.finfo(torch.bfloat16).max * (1 + 2.0 ** -9) < a * b < torch.finfo(torch.float32).max
    d["w_gate"][0, 0, 0], d["w_up"][0, 0, 0] = a, b
    d["w_down"][0, 3, 0] = 2.0 ** -100
    call(p, d, epi, o, ws)
    err = (o[:, 3].double() / (a * b * 2.0 ** -100) - 1).abs().max()
    # f32 roundings; with a bf16 output two planes, the first cut off (2^-7) instead of rounded, and the cast
    assert float(err) <= 8 * ref.U + (2.0 ** -7 * ref.BF16 + ref.BF16 if out == "bf16" else 0), float(err)


@pytest.mark.parametrize("M", [1, 6, 40])
def test_same_bits_on_every_call(M):
    p, d, epi, out, ws, _ = make(M=M, H=512, F=704, E=16, k=4, out="bf16", residual=True, seed=11)
    call(p, d, epi, out, ws)
    first = out.clone()
    for _ in range(5):
        out.zero_()
        call(p, d, epi, out, ws)
        assert torch.equal(out, first)


@pytest.mark.parametrize("M,dtype", [(1, "bf16"), (5, "f32"), (40, "bf16"), (40, "bf16_mxfp8")])
def test_graph_replays_equal_eager(M, dtype):
    p, d, epi, out, ws, _ = make(M=M, H=256, F=384, E=8, k=2, dtype=dtype, seed=12)
    eager, ws2 = torch.empty_like(out), torch.empty_like(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(p, d, epi, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, d, epi, out, ws)
    x0, l0 = d["x"].clone(), d["logits"].clone()
    idle = l0.clone()
    idle[::2] = float("-inf")
    for x, lg in ((x0, l0), (-0.5 * x0, l0.flip(1)), (x0, idle), (x0, l0)):
        d["x"].copy_(x)
        d["logits"].copy_(lg)
        call(p, d, epi, eager, ws2)
        torch.cuda.synchronize()
        float((eager * 2.0).sum())  # unrelated eager work between the replays
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_calls_on_two_streams():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    cases = [make(M=M, H=512, F=1408, E=16, k=4, seed=13 + i) for i, M in enumerate((4, 50))]
    serial = []
    for p, d, epi, out, ws, _ in cases:
        call(p, d, epi, out, ws)
        serial.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (p, d, epi, out, ws, _) in zip(sides, cases):
            call(p, d, epi, out, ws, stream=s)
    torch.cuda.synchronize()
    for (p, d, epi, out, ws, _), first in zip(cases, serial):
        assert torch.equal(out, first)


def test_no_tokens():
    p, d, epi, out, ws, guard = make(M=0, H=128, F=128, E=4, k=2)
    call(p, d, epi, out, ws)
    torch.cuda.synchronize()
    assert bool((guard == 7.0).all())


def test_weights_past_32_bit_offsets():
    # 40 experts of 8192 x 8192: the last one starts past 2^31 elements and 2^32 bytes
    M, H, F, E = 3, 8192, 8192, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    w = [torch.empty((E, F, H), dtype=torch.bfloat16, device=DEV).normal_(0, 0.02, generator=g) for _ in range(3)]
    x = torch.randn((M, H), generator=g, device=DEV).bfloat16()
    lg = torch.full((M, E), float("-inf"), device=DEV)
    lg[:, 39], lg[1:, 35] = 1.0, 2.0
    p = moe.problem(M, H, F, E, 2)
    out = torch.empty((M, H), device=DEV)
    ws = torch.empty(moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE), dtype=torch.uint8, device=DEV)
    moe.moe_layer_decode(p, x, lg, *w, None, out, ws)
    y, bound = ref.layer(x, lg, w[0], w[1], w[2], 2, 0, None, False, False)
    ref.check(out, y, bound, "large weights")


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("bf16_mxfp8", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("shape", [dict(M=100, H=128, F=1408, E=3, k=2), dict(M=255, H=64, F=1408, E=3, k=2),
                                   dict(M=256, H=320, F=1024, E=4, k=4), dict(M=200, H=1024, F=2048, E=8, k=2)])
def test_same_bits_whichever_place_a_row_gets(shape, dtype, out):
    # entries of 64 and 128 rows, whose places, and an expert's two entries, are dealt by atomics
    p, d, epi, o, ws, _ = make(**shape, dtype=dtype, out=out, residual=True, seed=15)
    call(p, d, epi, o, ws)
    first = o.clone()
    for _ in range(12):
        o.zero_()
        call(p, d, epi, o, ws)
        assert torch.equal(o, first)


# both few-token kernels, entries of 16 to 128 rows, the reduction in parts
NONFINITE = [dict(M=1, H=128, F=192, E=4, k=2), dict(M=6, H=128, F=192, E=6, k=2), dict(M=12, H=128, F=2560, E=4, k=2),
             dict(M=30, H=192, F=320, E=5, k=3), dict(M=60, H=192, F=1408, E=3, k=2), dict(M=100, H=128, F=1408, E=3, k=2),
             dict(M=255, H=64, F=1408, E=3, k=2)]


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape", NONFINITE)
def test_infinite_down_weights(shape, dtype, out):
    # an infinity of W_down makes its column infinite, with the sign of the activation; the rest keeps its bits
    p, d, epi, o, ws, _ = make(**shape, dtype=dtype, out=out, residual=True, seed=15)
    call(p, d, epi, o, ws)
    clean = o.clone()
    e = int(d["logits"][0].argmax())
    d["w_down"][e, 9, 5] = float("inf")
    d["w_down"][e, 40, p.ffn - 1] = float("-inf")
    y, _ = want(p, d, dtype, out)
    y = y.float()
    assert not bool(torch.isnan(y).any()) and bool(torch.isinf(y[0, [9, 40]]).all())
    o.fill_(0.0)
    call(p, d, epi, o, ws)
    there = torch.isinf(y)
    assert torch.equal(o.float()[there], y[there])
    assert torch.equal(o[~there], clean[~there])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 12, 60])
def test_an_infinite_weight_and_short_activations(M, dtype):
    # h = silu(64) * 2 = 128, one plane; 0 * inf is NaN, an infinity of each sign too
    p, d, epi, o, ws, _ = make(M, 64, 128, 1, 1, dtype=dtype, seed=16)
    for k in ("x", "w_gate", "w_up", "w_down"):
        d[k].zero_()
    d["x"][:, 0] = 1.0
    d["w_gate"][0, :2, 0], d["w_up"][0, 0, 0], d["w_up"][0, 1, 0] = 64.0, 2.0, -1.0
    d["w_down"][0, 3, 0] = d["w_down"][0, 4, 1] = d["w_down"][0, 5, 7] = float("inf")
    d["w_down"][0, 6, :2] = float("inf")
    d["w_down"][0, 7, 0], d["w_down"][0, 7, 1] = float("inf"), float("-inf")
    d["w_down"][0, 8, 2] = float("nan")
    call(p, d, epi, o, ws)
    assert bool((o[:, [3, 7]] == float("inf")).all()) and bool((o[:, 4] == float("-inf")).all())
    assert bool(torch.isnan(o[:, [5, 6, 8]]).all())
    assert not bool(o[:, :3].any()) and not bool(o[:, 9:].any())


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("bf16_mxfp8", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M", [1, 12, 60])
def test_a_product_past_the_range_is_infinite(M, dtype, out):
    # h = 16383 2^27 takes two planes of opposite sign (2^41, -2^27); times 2^110 each is past the range
    H, F = 64, 128
    p, d, epi, o, ws, _ = make(M, H, F, 1, 1, dtype=dtype, out=out, seed=17)
    for k in ("x", "w_gate", "w_up"):
        d[k].zero_()
    d["x"][:, 0] = 1.0
    d["w_gate"][0, 0, 0], d["w_up"][0, 0, 0] = 127 / 64 * 2.0 ** 20, 129 / 128 * 2.0 ** 20
    w = torch.zeros((H, F), device=DEV)
    w[3, 0], w[4, 0], w[5, 0] = 2.0 ** 110, -2.0 ** 110, 2.0 ** 80
    if dtype == "bf16_mxfp8":
        d["w_down"], _ = ref.quantize_mxfp8(w)
    else:
        d["w_down"][0] = w.to(d["w_down"].dtype)
    call(p, d, epi, o, ws)
    assert bool((o[:, 3] == float("inf")).all()) and bool((o[:, 4] == float("-inf")).all())
    h = 127 / 64 * 129 / 128 * 2.0 ** 40
    err = (o[:, 5].double() / (h * 2.0 ** 80) - 1).abs().max()
    assert float(err) <= 8 * ref.U + (ref.BF16 * ref.BF16 + ref.BF16 if out == "bf16" else 0), float(err)


# few tokens with k of 9 to 16 (up to 64 pairs: two kernels; 72: the plan)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "bf16_mxfp8"])
@pytest.mark.parametrize("logits,held,base", [("random", 0, 0), ("masked", 7, 5), ("idle", 0, 0), ("few", 0, 0),
                                              ("ties", 20, 0)])
@pytest.mark.parametrize("M,k", [(1, 16), (4, 16), (7, 9), (8, 8), (8, 9)])
def test_many_experts_of_few_tokens(M, k, logits, held, base, dtype):
    run_and_check(M=M, H=128, F=256, E=24, k=k, held=held, base=base, dtype=dtype, logits=logits, residual=M == 7, seed=18)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,F", [(1, 384), (6, 1280), (12, 2560), (24, 640), (130, 1408)])
def test_mxfp8_products_past_the_range(M, F, out):
    # in any row of a group of 32, line and part of the reduction, beside ordinary weights, which keep their bits
    H, E = 192, 2
    p, d, epi, o, ws, _ = make(M, H, F, E, 1, dtype="bf16_mxfp8", out=out, seed=19)
    d["x"][:, 0] = 1.0
    at = [(0, 3), (37, F - 1), (63, F // 2 + 1), (64, 130), (191, F - 70)]
    for _, f in at:  # h = 16383 2^27, as planes 2^41 and -2^27
        for k in ("w_gate", "w_up"):
            d[k][:, f] = 0
        d["w_gate"][:, f, 0], d["w_up"][:, f, 0] = 127 / 64 * 2.0 ** 20, 129 / 128 * 2.0 ** 20
    w = d["values_down"].float().clone()
    for _, f in at:
        w[:, :, f] = 0
    buf, values = ref.quantize_mxfp8(w.view(E * H, F))
    d["w_down"], d["values_down"] = buf, values.view(E, H, F)
    call(p, d, epi, o, ws)
    clean = o.clone()
    assert bool(torch.isfinite(clean).all())
    for i, (n, f) in enumerate(at):  # (the other weights of the element's block round to zero beside it)
        w[:, n, f] = 2.0 ** 110 * (-1) ** i
    d["w_down"], v = ref.quantize_mxfp8(w.view(E * H, F))
    o.fill_(0.0)
    call(p, d, epi, o, ws)
    rows = [n for n, _ in at]
    keep = torch.ones(H, dtype=torch.bool, device=DEV)
    keep[rows] = False
    sign = torch.tensor([(-1.0) ** i for i in range(len(at))], device=DEV)
    assert torch.equal(o[:, rows].float(), (sign * float("inf")).expand(M, -1))
    assert torch.equal(o[:, keep], clean[:, keep])
