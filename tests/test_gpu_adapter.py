"""moe_adapter_linear against a plain 64-bit projection: types, odd widths and
row counts, ranks, mixes of adapters, rows without one, epilogues, offsets
past 32 bits, graph replays; and a decode step made of both serving
operators."""
import pytest
import torch

import combine_topk_gate_amd as moe
import serving_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(M, H, N, r=16, P=4, dtype="bf16", out="f32", residual=False, mix="rows", seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(2000 + seed)
    act = torch.float32 if dtype == "f32" else torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(act)

    d = dict(x=normal(M, H), w=normal(N, H, std=0.05), a=None, b=None, scale=None, idx=None,
             residual=normal(M, N) if residual else None)
    if P > 0:
        d.update(a=normal(P, r, H, std=0.1), b=normal(P, N, r, std=0.2),
                 scale=torch.rand(P, generator=g, device=DEV) * 2 - 0.5)
        idx = torch.randint(-1, P, (M,), generator=g, device=DEV, dtype=torch.int32)
        if mix == "none":
            idx[:] = -1
        elif mix == "one":
            idx[:] = P - 1
        elif mix == "runs":
            idx = torch.sort(idx).values.contiguous()
        elif mix == "outside":  # not an adapter: as -1
            idx[::2] = P
            idx[1::4] = -(2 ** 31)
            idx[3::4] = 2 ** 31 - 1
        elif mix == "distinct":
            idx = (torch.arange(M, device=DEV) % P).to(torch.int32)
        d["idx"] = idx
    q = moe.adapter_problem(M, H, N, r if P else 0, P, dtype)
    odt = torch.bfloat16 if out == "bf16" else torch.float32
    guard = torch.full((M * N + 16,), 7.0, dtype=odt, device=DEV)
    o = guard[8:8 + M * N].view(M, N)
    o.fill_(float("nan"))
    ws = torch.full((moe.moe_adapter_workspace_bytes(q),), 0xFF, dtype=torch.uint8, device=DEV)
    return q, d, moe.epilogue(d["residual"], out), o, ws, guard


def call(q, d, epi, out, ws, stream=None):
    moe.moe_adapter_linear(q, d["x"], d["w"], d["a"], d["b"], d["scale"], d["idx"], epi, out, ws, stream=stream)


def want(d, dtype, out):
    return ref.linear(d["x"], d["w"], d["a"], d["b"], d["scale"], d["idx"], d["residual"], dtype == "f32", out == "bf16")


def run_and_check(**kw):
    print(f"[adapter] {kw}", flush=True)
    q, d, epi, out, ws, guard = make(**kw)
    dtype, odt = kw.get("dtype", "bf16"), kw.get("out", "f32")
    y, bound = want(d, dtype, odt)
    call(q, d, epi, out, ws)
    torch.cuda.synchronize()
    ref.check(out, y, bound, kw)
    ref.check_norm(out, y, 2 * q.in_features + 3 * q.rank, odt == "bf16", kw)
    assert bool((guard[:8] == 7.0).all()) and bool((guard[-8:] == 7.0).all())
    return q, d, epi, out, ws


SHAPES = [
    dict(M=1, H=64, N=1, r=8, P=1),
    dict(M=1, H=2048, N=64, r=8, P=4),
    dict(M=2, H=192, N=60, r=24, P=3),
    dict(M=16, H=128, N=100, r=16, P=5),
    dict(M=17, H=320, N=257, r=40, P=9),
    dict(M=48, H=512, N=640, r=16, P=64),
    dict(M=65, H=128, N=31, r=256, P=3),
    dict(M=130, H=256, N=516, r=64, P=7),
    dict(M=300, H=192, N=130, r=8, P=20),
    dict(M=515, H=448, N=1030, r=32, P=6),
]


@pytest.mark.parametrize("out,residual", [("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes_bf16(shape, out, residual):
    run_and_check(**shape, out=out, residual=residual)


@pytest.mark.parametrize("shape", SHAPES)
def test_shapes_f32(shape):
    run_and_check(**shape, dtype="f32", out="bf16" if shape["M"] == 48 else "f32", residual=shape["M"] % 2 == 0, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 24, 200, 700])
@pytest.mark.parametrize("mix", ["none", "one", "runs", "outside", "distinct"])
def test_mixes(mix, M, dtype):
    run_and_check(M=M, H=256, N=272, r=16, P=40, mix=mix, dtype=dtype, seed=2)


@pytest.mark.parametrize("M", [1, 30, 260])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_adapters_is_the_projection(M, dtype):
    q, d, epi, out, ws, _ = make(M=M, H=192, N=100, P=0, dtype=dtype, seed=3)
    assert ws.numel() == 0
    moe.moe_adapter_linear(q, d["x"], d["w"], None, None, None, None, None, out, None)
    y, bound = want(d, dtype, "f32")
    ref.check(out, y, bound, (M, dtype))


@pytest.mark.parametrize("M,r", [(16, 16), (16, 48), (100, 40)])
def test_rows_do_not_depend_on_the_other_rows(M, r):
    # a row's bits are the same whatever the other rows and their adapters are
    q, d, epi, out, ws, _ = make(M=M, H=512, N=256, r=r, P=8, seed=4)
    call(q, d, epi, out, ws)
    first = out.clone()
    for m in (0, 7, M - 1):
        other = dict(d, x=-2 * d["x"], idx=d["idx"].flip(0).contiguous())
        other["x"][m], other["idx"][m] = d["x"][m], d["idx"][m]
        call(q, other, epi, out, ws)
        assert torch.equal(out[m], first[m])


# at most 8 rows and one adapter between them: one launch, up to rank 64
@pytest.mark.parametrize("dtype,out,residual", [("bf16", "f32", False), ("bf16", "bf16", True), ("f32", "f32", True)])
@pytest.mark.parametrize("shape", [dict(M=1, H=64, N=1, r=8, P=3), dict(M=1, H=320, N=1001, r=24, P=3),
                                   dict(M=1, H=4096, N=257, r=64, P=9), dict(M=1, H=192, N=40, r=72, P=2),
                                   dict(M=8, H=256, N=60, r=40, P=1), dict(M=5, H=1024, N=130, r=16, P=1),
                                   dict(M=9, H=256, N=60, r=16, P=1), dict(M=2, H=256, N=60, r=16, P=2)])
def test_few_rows_of_one_adapter(shape, dtype, out, residual):
    for mix in ("one", "none", "rows", "outside"):
        run_and_check(**shape, dtype=dtype, out=out, residual=residual, mix=mix, seed=14)


# the column-splitting and the matrix-core tiles, with rows at any address,
# residuals, many adapters a tile
@pytest.mark.parametrize("out,residual", [("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("shape", [dict(M=700, H=256, N=3020, r=40, P=5, mix="runs"),
                                   dict(M=900, H=64, N=3333, r=16, P=30, mix="rows"),
                                   dict(M=641, H=192, N=4099, r=8, P=2, mix="distinct"),
                                   dict(M=3000, H=320, N=2049, r=72, P=7, mix="runs"),
                                   dict(M=3001, H=320, N=2052, r=16, P=40, mix="rows"),
                                   dict(M=5004, H=192, N=1753, r=16, P=5, mix="runs"),
                                   dict(M=4100, H=128, N=1999, r=8, P=3, mix="one")])
def test_long_batches(shape, out, residual):
    run_and_check(**shape, out=out, residual=residual, seed=13)


def test_output_in_place_of_the_residual():
    q, d, epi, out, ws, _ = make(M=37, H=192, N=136, out="bf16", residual=True, seed=5)
    call(q, d, epi, out, ws)
    first, r = out.clone(), d["residual"]
    call(q, d, moe.epilogue(r, "bf16"), r, ws)
    assert torch.equal(r, first)


@pytest.mark.parametrize("M,N,r,dtype", [(20, 72, 16, "bf16"), (300, 72, 16, "bf16"), (20, 72, 40, "bf16"),
                                         (300, 72, 40, "bf16"), (20, 72, 40, "f32"), (300, 72, 72, "f32"),
                                         (700, 3001, 40, "bf16"), (900, 3020, 16, "bf16"),
                                         (3000, 2052, 40, "bf16"), (4000, 2049, 24, "bf16")])
def test_nan_in_an_unused_adapter_and_in_a_row_stays_there(M, N, r, dtype):
    q, d, epi, out, ws, _ = make(M=M, H=128, N=N, r=r, P=6, mix="rows", dtype=dtype, seed=6)
    d["idx"][d["idx"] == 2] = 1
    d["a"][2], d["b"][2], d["scale"][2] = float("nan"), float("inf"), float("nan")
    y, bound = want(d, dtype, "f32")
    call(q, d, epi, out, ws)
    ref.check(out, y, bound, "unused adapter")
    clean = out.clone()
    d["x"][3] = float("nan")
    d["b"][4, 5] = float("inf")
    d["b"][4, N - 1, r - 1] = float("-inf")
    call(q, d, epi, out, ws)
    same = torch.ones((M, N), dtype=torch.bool, device=DEV)
    same[3] = False
    rows = d["idx"] == 4
    same[rows, 5] = same[rows, N - 1] = False
    assert torch.equal(out[same], clean[same])
    assert bool(torch.isnan(out[3]).all())
    # one infinite element, the others finite: t's sign decides
    rows[3] = False
    assert bool(torch.isinf(out[rows, N - 1]).all()) and not bool(torch.isfinite(out[rows, 5]).any())


def test_same_bits_on_every_call():
    for M in (3, 70, 600):
        q, d, epi, out, ws, _ = make(M=M, H=512, N=384, r=32, P=9, out="bf16", residual=True, seed=7)
        call(q, d, epi, out, ws)
        first = out.clone()
        for _ in range(4):
            out.zero_()
            call(q, d, epi, out, ws)
            assert torch.equal(out, first), M


@pytest.mark.parametrize("M", [1, 40, 500])
def test_graph_replays_equal_eager(M):
    q, d, epi, out, ws, _ = make(M=M, H=256, N=320, r=16, P=6, out="bf16", residual=True, seed=8)
    eager, ws2 = torch.empty_like(out), torch.empty_like(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(q, d, epi, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, d, epi, out, ws)
    x0, i0 = d["x"].clone(), d["idx"].clone()
    for x, idx in ((x0, i0), (-x0, i0.flip(0)), (x0, torch.full_like(i0, -1)), (x0, i0)):
        d["x"].copy_(x)
        d["idx"].copy_(idx)
        call(q, d, epi, eager, ws2)
        torch.cuda.synchronize()
        float((eager * 2.0).sum())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_calls_on_two_streams():
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    cases = [make(M=M, H=1024, N=768, r=16, P=12, seed=9 + i) for i, M in enumerate((9, 333))]
    serial = []
    for q, d, epi, out, ws, _ in cases:
        call(q, d, epi, out, ws)
        serial.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (q, d, epi, out, ws, _) in zip(sides, cases):
            call(q, d, epi, out, ws, stream=s)
    torch.cuda.synchronize()
    for (q, d, epi, out, ws, _), first in zip(cases, serial):
        assert torch.equal(out, first)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_output_past_32_bit_offsets(out):
    # 2^31 output elements are passed inside the last rows
    M, H, N, P = 33000, 64, 65536, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    x = torch.randn((M, H), generator=g, device=DEV).bfloat16()
    w = torch.randn((N, H), generator=g, device=DEV).bfloat16()
    a = torch.randn((P, 8, H), generator=g, device=DEV).bfloat16()
    b = torch.randn((P, N, 8), generator=g, device=DEV).bfloat16()
    scale = torch.ones(P, device=DEV)
    idx = (torch.arange(M, device=DEV) >= M - 100).to(torch.int32)
    q = moe.adapter_problem(M, H, N, 8, P)
    o = torch.empty((M, N), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=DEV)
    ws = torch.empty(moe.moe_adapter_workspace_bytes(q), dtype=torch.uint8, device=DEV)
    moe.moe_adapter_linear(q, x, w, a, b, scale, idx, moe.epilogue(None, out), o, ws)
    for rows in (slice(0, 64), slice(M - 120, M)):
        y, bound = ref.linear(x[rows], w, a, b, scale, idx[rows], None, False, out == "bf16")
        ref.check(o[rows], y, bound, rows)


def test_adapters_past_32_bit_offsets():
    # the last of 1030 adapters: B past 2^32 elements
    M, H, N, r, P = 5, 128, 65536, 64, 1030
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    x = torch.randn((M, H), generator=g, device=DEV).bfloat16()
    w = torch.randn((N, H), generator=g, device=DEV).bfloat16()
    a = torch.randn((P, r, H), generator=g, device=DEV).bfloat16()
    b = torch.empty((P, N, r), dtype=torch.bfloat16, device=DEV)
    for i in (0, P - 1):
        b[i] = torch.randn((N, r), generator=g, device=DEV).bfloat16()
    idx = torch.tensor([P - 1, 0, -1, P - 1, P - 1], dtype=torch.int32, device=DEV)
    scale = torch.full((P,), 0.5, device=DEV)
    q = moe.adapter_problem(M, H, N, r, P)
    o = torch.empty((M, N), device=DEV)
    ws = torch.empty(moe.moe_adapter_workspace_bytes(q), dtype=torch.uint8, device=DEV)
    moe.moe_adapter_linear(q, x, w, a, b, scale, idx, None, o, ws)
    y, bound = ref.linear(x, w, a, b, scale, idx, None, False, False)
    ref.check(o, y, bound, "last adapter")


def test_no_rows():
    q, d, epi, out, ws, guard = make(M=0, H=128, N=64)
    call(q, d, epi, out, ws)
    torch.cuda.synchronize()
    assert bool((guard == 7.0).all())


@pytest.mark.parametrize("M", [1, 7, 64])
def test_a_decode_step_of_both_operators(M):
    """Gate logits with the requests' adapters, the layer on them with the
    residual, and an output projection: the logits the layer routes by are
    the operator's own, so its routing is compared on those."""
    H, F, E, k, P, N = 256, 384, 8, 2, 5, 200
    qr, dr, er, logits, wsr, _ = make(M=M, H=H, N=E, r=8, P=P, seed=20)
    call(qr, dr, er, logits, wsr)
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    w_gate, w_up, w_down = ((torch.randn(s, generator=g, device=DEV) * 0.05).bfloat16()
                            for s in ((E, F, H), (E, F, H), (E, H, F)))
    p = moe.problem(M, H, F, E, k)
    y = torch.empty((M, H), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE), dtype=torch.uint8, device=DEV)
    moe.moe_layer_decode(p, dr["x"], logits, w_gate, w_up, w_down, moe.epilogue(dr["x"], "bf16"), y, ws)
    qo, do, eo, out, wso, _ = make(M=M, H=H, N=N, r=16, P=P, seed=22)
    do["x"], do["idx"] = y, dr["idx"]
    call(qo, do, eo, out, wso)
    torch.cuda.synchronize()
    l64, bl = want(dr, "bf16", "f32")
    ref.check(logits, l64, bl, "logits")
    y64, by = ref.layer(dr["x"], logits, w_gate, w_up, w_down, k, 0, dr["x"], False, True)
    ref.check(y, y64, by, "layer")
    o64, bo = want(do, "bf16", "f32")
    ref.check(out, o64, bo, "projection")


# the tiles of 16, 32 and 64 rows, the column-splitting one, both matrix-core ones
OVER = [(20, 128, 72, 24, "bf16"), (20, 128, 72, 40, "f32"), (333, 2048, 1408, 32, "bf16"), (1000, 128, 516, 40, "f32"),
        (2048, 64, 516, 64, "bf16"), (700, 128, 3001, 40, "bf16"), (2100, 320, 2049, 72, "bf16"),
        (8191, 1024, 2048, 24, "bf16")]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,H,N,r,dtype", OVER)
def test_values_past_the_range_of_a_row_and_its_adapter(M, H, N, r, dtype, out):
    # one value of t is infinite (1e30 * 1e30) in two rows; B has infinities of both signs in its column, and
    # products past the range without any; the rows beside them keep their bits
    q, d, epi, o, ws, _ = make(M=M, H=H, N=N, r=r, P=3, mix="rows", dtype=dtype, out=out, residual=True, seed=15)
    rows = torch.tensor([3, M - 2], device=DEV)
    d["idx"][rows] = 1
    d["w"][:, 7] = 0
    d["a"][:, :, 7] = 0
    d["a"][1, 4, 7] = 1e30
    d["x"][:, 7] = 0
    d["scale"][1] = 1.0
    d["b"][1, :, 4] = d["b"][1, :, 4].abs() + 0.5
    call(q, d, epi, o, ws)
    clean = o.clone()
    d["x"][rows, 7] = 1e30
    d["b"][1, 5, 4], d["b"][1, N - 1, 4], d["b"][1, 6, 4] = float("inf"), float("-inf"), -1.0
    d["b"][1, 8, 4], d["b"][1, 8, 0] = float("inf"), float("nan")
    call(q, d, epi, o, ws)
    got = o[rows].float()
    sign = torch.ones(N, device=DEV)
    sign[6] = sign[N - 1] = -1
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[8] = False
    assert torch.equal(got[:, keep], (sign * float("inf"))[keep].expand(2, -1)), got
    assert bool(torch.isnan(got[:, 8]).all())
    same = torch.ones((M, N), dtype=torch.bool, device=DEV)
    same[rows] = False
    one = d["idx"] == 1
    one[rows] = False
    for n in (5, 6, 8, N - 1):
        same[one, n] = False
    assert torch.equal(o[same], clean[same])
    # the other rows of that adapter: t is finite there
    t4 = d["x"].double()[one] @ d["a"][1, 4].double()
    assert torch.equal(o[one, 5].float(), (torch.sign(t4) * float("inf")).float())
    assert torch.equal(o[one, N - 1].float(), (torch.sign(t4) * float("-inf")).float())
    # t = 16383 2^27, in planes 2^41 and -2^27: each times 2^110 is past the range
    d["x"][rows, 7], d["a"][1, 4, 7] = 127 / 64 * 2.0 ** 20, 129 / 128 * 2.0 ** 20
    d["b"][1, 5, 4], d["b"][1, N - 1, 4] = 2.0 ** 110, -2.0 ** 110
    call(q, d, epi, o, ws)
    got = o[rows].float()
    assert bool((got[:, 5] == float("inf")).all()) and bool((got[:, N - 1] == float("-inf")).all()), got[:, [5, N - 1]]
    assert bool(torch.isfinite(got[:, :5]).all())


def on_tiles(shape, tiles, out="f32"):
    s = dict(dict(r=0, dtype="bf16"), **shape)
    got = moe.moe_adapter_tiles(moe.adapter_problem(s["M"], s["H"], s["N"], s["r"], s["P"], s["dtype"]), out)
    assert got == tiles, (shape, got)


@pytest.mark.parametrize("shape,tiles", ref.TILES)
def test_every_tile(shape, tiles):
    on_tiles(shape, tiles)
    run_and_check(**shape, residual=shape["N"] % 2 == 1, seed=16)


# tiles that a bf16 output and a residual in place take too
WIDE = [(dict(M=1001, H=1024, N=1022, r=40, P=5), (64, 64, 16, 16)), (dict(M=700, H=128, N=3001, r=40, P=6), (64, 256, 16, 16)),
        (dict(M=2001, H=512, N=4093, r=24, P=6), (128, 256, 16, 16)), (dict(M=2001, H=1024, N=7167, r=24, P=6), (256, 256, 16, 16)),
        (dict(M=2000, H=192, N=7168, r=24, P=5), (256, 256, 16, 16))]


@pytest.mark.parametrize("shape,tiles", WIDE)
def test_long_batches_in_place_of_the_residual(shape, tiles):
    on_tiles(shape, tiles, "bf16")
    q, d, epi, out, ws = run_and_check(**shape, out="bf16", residual=True, seed=17)
    r = d["residual"]
    call(q, d, moe.epilogue(r, "bf16"), r, ws)
    assert torch.equal(r, out)


@pytest.mark.parametrize("shape,tiles", WIDE)
def test_rows_of_long_batches_do_not_depend_on_the_others(shape, tiles):
    on_tiles(shape, tiles)
    M = shape["M"]
    q, d, epi, out, ws, _ = make(**shape, seed=18)
    call(q, d, epi, out, ws)
    first = out.clone()
    other = dict(d, x=-2 * d["x"], idx=d["idx"].flip(0).contiguous())
    rows = [0, 70, 255, 256, M // 2, M - 1]
    for m in rows:
        other["x"][m], other["idx"][m] = d["x"][m], d["idx"][m]
    call(q, other, epi, out, ws)
    assert torch.equal(out[rows], first[rows])


@pytest.mark.parametrize("M,N,r,tiles", [(2001, 7168, 24, (256, 256, 16, 16)), (700, 3001, 40, (64, 256, 16, 16)),
                                         (3000, 2052, 40, (128, 256, 32, 16))])
def test_nan_and_infinities_on_the_long_tiles(M, N, r, tiles):
    on_tiles(dict(M=M, H=128, N=N, r=r, P=6), tiles)
    test_nan_in_an_unused_adapter_and_in_a_row_stays_there(M, N, r, "bf16")


def test_same_bits_on_the_long_tiles():
    for shape, tiles in WIDE:
        on_tiles(shape, tiles, "bf16")
        q, d, epi, out, ws, _ = make(**shape, out="bf16", residual=True, seed=19)
        call(q, d, epi, out, ws)
        first = out.clone()
        for _ in range(4):
            out.zero_()
            call(q, d, epi, out, ws)
            assert torch.equal(out, first), shape
