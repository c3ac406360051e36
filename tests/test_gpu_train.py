"""The training operators against plain 64-bit references: types, ragged and
empty segments, source blocks, held experts, odd sizes, dropout masks, values
that are not finite in places that do not count, graphs, streams, reordering;
and a whole training step of them against the layer's gradient."""
import os

import pytest
import torch

import combine_topk_gate_amd as moe
import serving_ref
import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(7000 + seed)
    return g


def act_of(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def routing(M, E, k, S=1, held=0, base=0, seed=0, crowd=0.0, skip=()):
    """topk_idx, topk_w, flat_to_sorted, offsets as moe_route and moe_dispatch leave them; crowd: how much likelier
    expert 0 of those held is, skip: experts that no token chooses."""
    g = gen(seed + 100)
    logits = torch.randn(M, E, generator=g, device=DEV)
    logits[:, base] += crowd
    for e in skip:
        logits[:, e] = -1e9
    EL = held or E
    vals, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    vals, idx = vals[:, :k], idx[:, :k]
    slot = idx.reshape(-1) - (base if held else 0)
    block = (torch.arange(M, device=DEV) * 7 % S).repeat_interleave(k)  # blocks interleaved
    seg = torch.where((slot >= 0) & (slot < EL), block * EL + slot, torch.full_like(slot, S * EL))
    order = torch.sort(seg, stable=True).indices
    offsets = torch.zeros(S * EL + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(seg, minlength=S * EL + 1)[:S * EL], 0)
    f2s = torch.empty_like(order)
    f2s[order] = torch.arange(M * k, device=DEV)
    f2s[f2s >= offsets[-1]] = -1
    return (idx.to(torch.int32).contiguous(), torch.softmax(vals, 1).contiguous(), f2s.to(torch.int32), offsets)


def guarded(shape, dtype, fill=NAN):
    """A tensor between two guard zones, and a check of them."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 32,), 7.0, dtype=dtype, device=DEV)
    t = buf[16:16 + n].view(shape)
    t.fill_(fill)

    def intact():
        assert bool((buf[:16] == 7.0).all()) and bool((buf[16 + n:] == 7.0).all())

    return t, intact


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


# ------------------------------------------------------------------ router ---


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 3), (17, 64, 4), (64, 127, 8), (65, 128, 1), (200, 512, 16),
                                   (1000, 8, 2), (1001, 33, 16), (5000, 130, 6)])
def test_route_backward(M, E, k):
    idx, w, _, _ = routing(M, E, k, seed=M)
    dw = normal(gen(M), M, k)
    out, intact = guarded((M, E), torch.float32)
    moe.moe_route_backward(moe.problem(M, 64, 64, E, k), idx, w, dw, out)
    want, bound = ref.route_backward(idx, w, dw, E)
    serving_ref.check(out, want, bound, (M, E, k))
    intact()
    if k == 1:
        assert not bool(out.any())  # a single choice always has the weight 1


def test_route_backward_equal_slots_and_foreign_indices():
    # the same expert in two slots adds up; an index that is no expert writes nothing
    M, E, k = 70, 9, 4
    idx, w, _, _ = routing(M, E, k, seed=5)
    dw = normal(gen(6), M, k)
    idx[::3, 2] = idx[::3, 0]
    p = moe.problem(M, 64, 64, E, k)
    out, intact = guarded((M, E), torch.float32)
    moe.moe_route_backward(p, idx, w, dw, out)
    want, bound = ref.route_backward(idx, w, dw, E)
    serving_ref.check(out, want, bound, "equal slots")
    bad = idx.clone()
    bad[1::5, 1], bad[2::5, 3] = E, -1
    moe.moe_route_backward(p, bad, w, dw, out)
    serving_ref.check(out, *ref.route_backward(bad, w, dw, E), "foreign")
    intact()


# ----------------------------------------------------------------- combine ---

COMBINE = [dict(M=1, H=64, E=1, k=1), dict(M=1, H=4096, E=8, k=2), dict(M=7, H=128, E=6, k=3, held=2, base=1),
           dict(M=33, H=192, E=4, k=4), dict(M=50, H=512, E=16, k=8, S=3), dict(M=19, H=576, E=20, k=16, held=7, base=9),
           dict(M=129, H=1088, E=8, k=2, S=2, held=3, base=5), dict(M=300, H=2112, E=5, k=5)]
KINDS = [("f32", "f32", False, 0.0), ("bf16", "bf16", True, 0.1), ("bf16", "f32", True, 0.5), ("f32", "bf16", False, 0.9)]


def combine_inputs(M, H, E, k, dtype, S=1, held=0, base=0, seed=0):
    idx, w, f2s, offsets = routing(M, E, k, S, held, base, seed=seed + M)
    y = normal(gen(seed + 1), M * k, H)
    y[int(offsets[-1]):] = NAN  # rows that no pair has
    return moe.problem(M, H, 64, E, k, S, dtype, base if held else 0, held), w, f2s, y


@pytest.mark.parametrize("dtype,out,residual,p", KINDS)
@pytest.mark.parametrize("shape", COMBINE)
def test_combine_dropout(shape, dtype, out, residual, p):
    print(f"[combine dropout] {shape} {dtype} {out} {residual} {p}", flush=True)
    prob, w, f2s, y = combine_inputs(**shape, dtype=dtype)
    M, H = shape["M"], shape["H"]
    res = normal(gen(2), M, H, dtype=act_of(dtype)) if residual else None
    rng = rng_of(-(2 ** 61) + M, 2 ** 40 + H)
    o, intact = guarded((M, H), act_of(out))
    moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(res, out), moe.dropout(p, rng), o)
    keep = ref.mask(M, H, p, rng, DEV)
    want, bound = ref.combine(y, w, f2s, keep, p, res, out == "bf16")
    serving_ref.check(o, want, bound, (shape, dtype, out, p))
    intact()
    if res is None:
        assert not bool(o[~keep].any())
    plain, _ = guarded((M, H), act_of(out))
    moe.moe_combine_ex(prob, y, w, f2s, moe.epilogue(res, out), plain)
    none, _ = guarded((M, H), act_of(out))
    moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(res, out), None, none)
    assert torch.equal(plain, none)
    moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(res, out), moe.dropout(0.0, rng), none)
    assert torch.equal(plain, none)


def test_dropout_reads_its_generator_on_the_device_and_in_place():
    M, H = 40, 256
    prob, w, f2s, y = combine_inputs(M, H, 8, 2, "f32")
    rng = rng_of(11, 0)
    drop = moe.dropout(0.5, rng)
    seen = []
    for offset in (0, 1, 2 ** 33):
        rng[1] = offset
        x = normal(gen(3), M, H)
        out, intact = guarded((M, H), torch.float32)
        moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(x, "f32"), drop, out)
        want, bound = ref.combine(y, w, f2s, ref.mask(M, H, 0.5, rng, DEV), 0.5, x, False)
        serving_ref.check(out, want, bound, offset)
        moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(x, "f32"), drop, x)  # onto the residual
        assert torch.equal(x, out)
        seen.append(out)
        intact()
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_dropped_elements_are_zero_whatever_was_there():
    M, H = 9, 128
    prob, w, f2s, y = combine_inputs(M, H, 4, 2, "f32")
    rng = rng_of(3, 4)
    keep = ref.mask(M, H, 0.6, rng, DEV)
    f, _ = ref._rows(f2s, M, 2)
    y[f[:, 0]] = torch.where(keep, y[f[:, 0]], float("inf"))
    y[f[:, 1]] = torch.where(keep, y[f[:, 1]], NAN)
    out, _ = guarded((M, H), torch.float32)
    moe.moe_combine_dropout(prob, y, w, f2s, None, moe.dropout(0.6, rng), out)
    assert bool(torch.isfinite(out).all()) and not bool(out[~keep].any())
    dout = torch.where(keep, normal(gen(5), M, H), float("inf"))
    dy, _ = guarded((M * 2, H), torch.float32)
    dw, _ = guarded((M, 2), torch.float32)
    moe.moe_combine_backward(prob, dout, y, w, f2s, moe.dropout(0.6, rng), dy, dw)
    want = ref.combine_backward(torch.where(keep, dout, 0.0), y, w, f2s, keep, 0.6, False)
    serving_ref.check(dy, want[0], want[1], "dy")
    serving_ref.check(dw, want[2], want[3], "dw")


@pytest.mark.parametrize("dtype,out,residual,p", KINDS)
@pytest.mark.parametrize("shape", COMBINE)
def test_combine_backward(shape, dtype, out, residual, p):
    print(f"[combine backward] {shape} {dtype} {out} {p}", flush=True)
    prob, w, f2s, y = combine_inputs(**shape, dtype=dtype)
    M, H, k = shape["M"], shape["H"], shape["k"]
    dout = normal(gen(4), M, H, dtype=act_of(out))
    rng = rng_of(M, H)
    dy, i1 = guarded((M * k, H), act_of(dtype), fill=5.0)
    dw, i2 = guarded((M, k), torch.float32)
    moe.moe_combine_backward(prob, dout, y, w, f2s, moe.dropout(p, rng) if p else None, dy, dw)
    wy, by, ww, bw = ref.combine_backward(dout, y, w, f2s, ref.mask(M, H, p, rng, DEV) if p else None, p, dtype == "bf16")
    rest = torch.isnan(wy)
    assert bool((dy[rest] == 5.0).all())  # rows behind the kept pairs' are left as they were
    serving_ref.check(dy[~rest], wy[~rest], by[~rest], (shape, "dy"))
    serving_ref.check(dw, ww, bw, (shape, "dw"))
    check_norm(dw, ww, H + 3, False, (shape, "dw"))
    i1()
    i2()


# ---------------------------------------------------------------- dispatch ---


@pytest.mark.parametrize("dtype,out,residual,p", KINDS)
@pytest.mark.parametrize("shape", COMBINE)
def test_dispatch_backward(shape, dtype, out, residual, p):
    print(f"[dispatch backward] {shape} {dtype} {out} {residual}", flush=True)
    M, H, k = shape["M"], shape["H"], shape["k"]
    prob, _, f2s, y = combine_inputs(**shape, dtype=dtype)
    dxp = y.to(act_of(dtype))
    res = normal(gen(8), M, H, dtype=act_of(dtype)) if residual else None
    dx, intact = guarded((M, H), act_of(out))
    moe.moe_dispatch_backward(prob, dxp, f2s, moe.epilogue(res, out), dx)
    want, bound = ref.dispatch_backward(dxp, f2s, M, k, res, out == "bf16")
    serving_ref.check(dx, want, bound, (shape, dtype, out))
    intact()
    if res is not None and out == dtype:
        moe.moe_dispatch_backward(prob, dxp, f2s, moe.epilogue(res, out), res)
        assert torch.equal(res, dx)


# ------------------------------------------------------- experts' products ---

EXPERTS = [dict(M=1, H=64, F=64, E=1, k=1), dict(M=1, H=256, F=320, E=8, k=2), dict(M=5, H=128, F=64, E=3, k=3),
           dict(M=64, H=192, F=128, E=4, k=2, skip=(0, 3)), dict(M=200, H=320, F=448, E=3, k=1, crowd=1.5),
           dict(M=129, H=64, F=576, E=16, k=4, S=3), dict(M=300, H=448, F=192, E=12, k=3, held=3, base=4, S=2),
           dict(M=700, H=512, F=256, E=2, k=1), dict(M=520, H=256, F=704, E=4, k=2, held=2, base=1, crowd=3.0),
           dict(M=90, H=128, F=128, E=40, k=2), dict(M=257, H=576, F=320, E=1, k=1),
           # few tiles with long reductions: split along K
           dict(M=70, H=1088, F=2112, E=2, k=1), dict(M=1500, H=64, F=128, E=1, k=1),
           dict(M=1400, H=128, F=64, E=3, k=2, S=3, held=2, base=1), dict(M=300, H=1024, F=1024, E=2, k=1, skip=(1,)),
           dict(M=3000, H=320, F=64, E=2, k=1, crowd=2.5),
           # many tiles: the larger f32 ones
           dict(M=8200, H=64, F=4096, E=2, k=1), dict(M=4100, H=4160, F=64, E=3, k=2), dict(M=100, H=1088, F=1152, E=32, k=2),
           dict(M=90, H=128, F=448, E=40, k=2),
           # the larger bf16 tiles: ragged segments over source blocks, a share, few rows an expert, split along K
           dict(M=3000, H=832, F=1088, E=5, k=2, S=3, skip=(1,), crowd=1.0),
           dict(M=5000, H=704, F=960, E=12, k=3, held=3, base=4, S=2), dict(M=300, H=1024, F=1408, E=64, k=4),
           dict(M=60, H=448, F=6272, E=1, k=1), dict(M=60, H=12352, F=448, E=1, k=1),
           dict(M=90, H=320, F=6272, E=12, k=3, S=3, held=3, base=4),
           # ... of few weights over many rows
           dict(M=20000, H=256, F=320, E=4, k=2, S=3, held=2, base=1),
           # the largest number of segments, the longest rows
           dict(M=100, H=64, F=64, E=512, k=16, S=2), dict(M=3, H=65536, F=64, E=2, k=1), dict(M=3, H=64, F=65536, E=2, k=1)]


def experts(M, H, F, E, k, dtype, S=1, held=0, base=0, crowd=0.0, skip=(), seed=0):
    _, _, _, offsets = routing(M, E, k, S, held, base, seed=seed + M, crowd=crowd, skip=skip)
    EL, R, act, g = held or E, M * k, act_of(dtype), gen(seed + 20)
    end = int(offsets[-1])

    def rows(n, std=1.0):
        t = normal(g, R, n, std=std, dtype=act)
        t[end:] = NAN  # rows of no segment count for nothing
        return t

    d = dict(offsets=offsets, xp=rows(H), gate=rows(F), up=rows(F), h=rows(F), dy=rows(H), dgate=rows(F), dup=rows(F),
             wg=normal(g, EL, F, H, std=0.1, dtype=act), wu=normal(g, EL, F, H, std=0.1, dtype=act),
             wd=normal(g, EL, H, F, std=0.1, dtype=act))
    prob = moe.problem(M, H, F, E, k, S, dtype, base if held else 0, held)
    ws = torch.full((max(moe.moe_workspace_bytes(prob, moe.MOE_OP_GROUPED_GEMM_BACKWARD), 1),), 0xFF, dtype=torch.uint8, device=DEV)
    return prob, d, ws


def check_norm(got, want, n, bf16, what):
    # The norm's bounds are means over many outputs of like size.  A single sum can cancel (64 terms of mean size 0.64,
    # 40.7 in all, that add up to 0.0163: 64 roundings of 2^-24 of partial sums of a few units are 1e-7, 7e-6 of it);
    # and products of three normal factors have a fourth moment of 27 squares of the second, so the mean square of n of
    # them rests on n / 27: on two values of 64 (1.4948 and 0.8732 of dup, 0.0026 and 0.0018 from their bf16 values with
    # half steps of 0.0039 and 0.00195, are 2.7e-3 of the norm together).  From 4096 on it rests on 150 values, and the
    # rms of a rounding, at most 2^-8 / sqrt(3) where it is worst, is below 2/3 of that over values spread in size.
    if got.numel() >= 4096:
        serving_ref.check_norm(got, want, n, bf16, what)


def check_rows(got, want, bound, n, bf16, what):
    rest = torch.isnan(want)
    assert bool((got[rest] == 5.0).all()), what  # rows of no segment are left as they were
    serving_ref.check(got[~rest], want[~rest], bound[~rest], what)
    if int((~rest).sum()):
        check_norm(got[~rest], want[~rest], n, bf16, what)


def run_all(prob, d, ws, dw_dtype=torch.float32, accumulate=False, start=0.0, fill=5.0):
    """Every call of the experts' products on the inputs d; a dict of outputs and the guards' check."""
    R, H, F, EL = prob.num_tokens * prob.topk, prob.hidden, prob.ffn, prob.local_experts or prob.num_experts
    act = torch.float32 if prob.dtype == moe.MOE_DTYPE_F32 else torch.bfloat16
    o, checks = {}, []
    for name, shape, dt, f in (("gate", (R, F), act, fill), ("up", (R, F), act, fill), ("c", (R, F), act, fill),
                               ("dgate", (R, F), act, fill), ("dup", (R, F), act, fill), ("dxp", (R, H), act, fill),
                               ("dwd", (EL, H, F), dw_dtype, start), ("dwg", (EL, F, H), dw_dtype, start),
                               ("dwu", (EL, F, H), dw_dtype, start)):
        o[name], c = guarded(shape, dt, fill=f)
        checks.append(c)
    moe.moe_grouped_gemm_aux(prob, d["xp"], d["wg"], d["wu"], d["offsets"], o["gate"], o["up"], o["c"])
    moe.moe_grouped_gemm_backward(prob, 1, d["dy"], None, d["wd"], None, d["gate"], d["up"], d["offsets"], o["dgate"],
                                  o["dup"], ws)
    moe.moe_grouped_gemm_backward(prob, 0, d["dgate"], d["dup"], d["wg"], d["wu"], None, None, d["offsets"], o["dxp"], None, ws)
    moe.moe_grouped_gemm_backward_weights(prob, 1, d["dy"], None, d["h"], d["offsets"], o["dwd"], None, accumulate, ws)
    moe.moe_grouped_gemm_backward_weights(prob, 0, d["dgate"], d["dup"], d["xp"], d["offsets"], o["dwg"], o["dwu"], accumulate, ws)
    torch.cuda.synchronize()
    for c in checks:
        c()
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", EXPERTS)
def test_experts(shape, dtype):
    print(f"[experts] {shape} {dtype}", flush=True)
    prob, d, ws = experts(**shape, dtype=dtype)
    bf16, H, F, EL, R = dtype == "bf16", shape["H"], shape["F"], d["wg"].shape[0], d["xp"].shape[0]
    o = run_all(prob, d, ws, start=NAN)
    g, bg, u, bu = ref.products(d["xp"], d["wg"], d["wu"], d["offsets"], bf16)
    check_rows(o["gate"], g, bg, 2 * H, bf16, (shape, "gate"))
    check_rows(o["up"], u, bu, 2 * H, bf16, (shape, "up"))
    check_rows(o["c"], *ref.hact(d["xp"], d["wg"], d["wu"], d["offsets"], bf16), 2 * H + 8, bf16, (shape, "hact"))
    g, bg, u, bu = ref.rows1(d["dy"], d["wd"], d["gate"], d["up"], d["offsets"], bf16)
    check_rows(o["dgate"], g, bg, 2 * H + 64, bf16, (shape, "dgate"))
    check_rows(o["dup"], u, bu, 2 * H + 64, bf16, (shape, "dup"))
    check_rows(o["dxp"], *ref.rows0(d["dgate"], d["dup"], d["wg"], d["wu"], d["offsets"], bf16), 4 * F, bf16, (shape, "dxp"))
    for name, a, b in (("dwd", "dy", "h"), ("dwg", "dgate", "xp"), ("dwu", "dup", "xp")):
        want, bound = ref.weights(d[a], d[b], d["offsets"], EL, False)
        serving_ref.check(o[name], want, bound, (shape, name))
        check_norm(o[name], want, 2 * R, False, (shape, name))
    low = run_all(prob, d, ws, dw_dtype=torch.bfloat16, start=NAN)
    for name, a, b in (("dwd", "dy", "h"), ("dwg", "dgate", "xp"), ("dwu", "dup", "xp")):
        want, bound = ref.weights(d[a], d[b], d["offsets"], EL, True)
        serving_ref.check(low[name], want, bound, (shape, name, "bf16"))
    more = run_all(prob, d, ws, accumulate=True, start=3.0)
    for name, a, b in (("dwd", "dy", "h"), ("dwg", "dgate", "xp"), ("dwu", "dup", "xp")):
        want, bound = ref.weights(d[a], d[b], d["offsets"], EL, False, start=torch.full((), 3.0, device=DEV))
        serving_ref.check(more[name], want, bound, (shape, name, "accumulated"))


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("M,H", [(3333, 4160), (16500, 832), (33333, 448)])
def test_rows_larger_than_the_cache(M, H, p):
    # f32 rows of over 96 MiB take other loads
    E, k = 8, 2
    prob, w, f2s, y = combine_inputs(M, H, E, k, "bf16")
    rng = rng_of(7, 8)
    keep = ref.mask(M, H, p, rng, DEV) if p else None
    drop = moe.dropout(p, rng) if p else None
    x = normal(gen(31), M, H, dtype=torch.bfloat16)
    out, i1 = guarded((M, H), torch.bfloat16)
    moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(x, "bf16"), drop, out)
    serving_ref.check(out, *ref.combine(y, w, f2s, keep, p, x, True), "out")
    dy, i2 = guarded((M * k, H), torch.bfloat16, fill=5.0)
    dw, i3 = guarded((M, k), torch.float32)
    moe.moe_combine_backward(prob, x, y, w, f2s, drop, dy, dw)
    wy, by, ww, bw = ref.combine_backward(x, y, w, f2s, keep, p, True)
    serving_ref.check(dy, wy, by, "dy")
    serving_ref.check(dw, ww, bw, "dw")
    dx, i4 = guarded((M, H), torch.float32)
    moe.moe_dispatch_backward(moe.problem(M, H, 64, E, k, dtype="f32"), y, f2s, None, dx)
    serving_ref.check(dx, *ref.dispatch_backward(y, f2s, M, k, None, False), "dx")
    for c in (i1, i2, i3, i4):
        c()


def test_offsets_past_32_bits():
    # y of 5.2 GB, and buffers of the experts' products of 2.6 GB: the first and the last tokens and rows
    M, H, E, k = 40000, 16384, 3, 2
    idx, w, f2s, offsets = routing(M, E, k, seed=77)
    prob = moe.problem(M, H, 64, E, k)
    y = torch.empty((M * k, H), device=DEV)
    dout = normal(gen(5), M, H, dtype=torch.bfloat16)
    ends = torch.cat([torch.arange(5), torch.arange(M - 5, M)]).to(DEV)
    f = f2s.long().view(M, k)
    y.normal_()
    y[f[ends].flatten()] = normal(gen(6), 10 * k, H)
    dy = torch.zeros((M * k, H), dtype=torch.bfloat16, device=DEV)
    dw = torch.zeros((M, k), device=DEV)
    rng = rng_of(1, 2)
    moe.moe_combine_backward(prob, dout, y, w, f2s, None, dy, dw)
    for t in ends.tolist():
        r = f[t]
        small = torch.arange(k, dtype=torch.int32, device=DEV)
        wy, by, ww, bw = ref.combine_backward(dout[t:t + 1], y[r], w[t:t + 1], small, None, 0.0, True)
        serving_ref.check(dy[r], wy, by, ("dy", t))
        serving_ref.check(dw[t:t + 1], ww, bw, ("dw", t))
    out = torch.zeros((M, H), device=DEV)
    moe.moe_combine_dropout(prob, y, w, f2s, None, moe.dropout(0.5, rng), out)
    words = ref.philox_words(M * H, 1, 2).reshape(M, H)
    for t in ends.tolist():
        keep = torch.from_numpy(words[t:t + 1] >= 2 ** 31).to(DEV)
        small = torch.arange(k, dtype=torch.int32, device=DEV)
        serving_ref.check(out[t:t + 1], *ref.combine(y[f[t]], w[t:t + 1], small, keep, 0.5, None, False), ("out", t))
    dx = torch.zeros((M, H), device=DEV)
    moe.moe_dispatch_backward(prob, dy, f2s, None, dx)
    for t in ends.tolist():
        small = torch.arange(k, dtype=torch.int32, device=DEV)
        serving_ref.check(dx[t:t + 1], *ref.dispatch_backward(dy[f[t]], small, 1, k, None, False), ("dx", t))


def test_product_buffers_past_two_gib():
    M, H, F, E = 20011, 64, 65536, 2  # R F = 1.3e9: 2.6 GB a buffer
    _, _, _, offsets = routing(M, E, 1, seed=78)
    prob = moe.problem(M, H, F, E, 1)
    ws = torch.empty(moe.moe_workspace_bytes(prob, moe.MOE_OP_GROUPED_GEMM_BACKWARD), dtype=torch.uint8, device=DEV)
    g = gen(40)
    n = lambda *s, std=1.0: torch.empty(s, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)
    xp, dy, wg, wu, wd = n(M, H), n(M, H), n(E, F, H, std=0.1), n(E, F, H, std=0.1), n(E, H, F, std=0.1)
    gate, up, h = (torch.zeros((M, F), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    moe.moe_grouped_gemm_aux(prob, xp, wg, wu, offsets, gate, up, h)
    cut = int(offsets[1])
    rows = [0, 1, cut - 1, cut, cut + 1, M - 2, M - 1]
    part = lambda lo, hi: torch.tensor([0, 1, 1] if hi <= cut else [0, 0, 1], dtype=torch.int32)
    for r in rows:
        gw, bg, uw, bu = ref.products(xp[r:r + 1], wg, wu, part(r, r + 1), True)
        serving_ref.check(gate[r:r + 1], gw, bg, ("gate", r))
        serving_ref.check(up[r:r + 1], uw, bu, ("up", r))
    dgate, dup = torch.zeros_like(gate), torch.zeros_like(up)
    moe.moe_grouped_gemm_backward(prob, 1, dy, None, wd, None, gate, up, offsets, dgate, dup, ws)
    for r in rows:
        gw, bg, uw, bu = ref.rows1(dy[r:r + 1], wd, gate[r:r + 1], up[r:r + 1], part(r, r + 1), True)
        serving_ref.check(dgate[r:r + 1], gw, bg, ("dgate", r))
        serving_ref.check(dup[r:r + 1], uw, bu, ("dup", r))
    dxp = torch.zeros_like(xp)
    moe.moe_grouped_gemm_backward(prob, 0, dgate, dup, wg, wu, None, None, offsets, dxp, None, ws)
    for r in rows:
        serving_ref.check(dxp[r:r + 1], *ref.rows0(dgate[r:r + 1], dup[r:r + 1], wg, wu, part(r, r + 1), True), ("dxp", r))
    dwg, dwu = (torch.zeros((E, F, H), device=DEV) for _ in range(2))
    moe.moe_grouped_gemm_backward_weights(prob, 0, dgate, dup, xp, offsets, dwg, dwu, False, ws)
    cols = torch.tensor([0, 5, 255, 256, F - 2, F - 1], device=DEV)
    for d, o in ((dgate, dwg), (dup, dwu)):
        want, bound = ref.weights(d[:, cols].contiguous(), xp, offsets, E, False)
        serving_ref.check(o[:, cols], want, bound, "weights")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    # nothing to read: the weights' gradients are zero, or unchanged where they accumulate
    prob = moe.problem(0, 64, 128, 4, 2, dtype=dtype)
    act, offsets = act_of(dtype), torch.zeros(5, dtype=torch.int32, device=DEV)
    e = lambda n: torch.empty((0, n), dtype=act, device=DEV)
    for accumulate, want in ((False, 0.0), (True, 2.0)):
        dw, intact = guarded((4, 128, 64), torch.float32, fill=2.0)
        dw1, intact1 = guarded((4, 128, 64), torch.float32, fill=2.0)
        moe.moe_grouped_gemm_backward_weights(prob, 0, e(128), e(128), e(64), offsets, dw, dw1, accumulate)
        assert bool((dw == want).all()) and bool((dw1 == want).all())
        intact()
        intact1()
    w = normal(gen(1), 4, 128, 64, dtype=act)
    moe.moe_grouped_gemm_backward(prob, 0, e(128), e(128), w, w.clone(), None, None, offsets, e(64), None)
    moe.moe_grouped_gemm_aux(prob, e(64), w, w.clone(), offsets, e(128), e(128), e(128))
    f = torch.empty((0, 64), device=DEV)
    i32 = torch.empty((0,), dtype=torch.int32, device=DEV)
    moe.moe_dispatch_backward(prob, e(64), i32, None, f)
    moe.moe_combine_backward(prob, f, f, torch.empty((0, 2), device=DEV), i32, None, e(64), torch.empty((0, 2), device=DEV))
    moe.moe_combine_dropout(prob, f, torch.empty((0, 2), device=DEV), i32, None, moe.dropout(0.5, rng_of(1, 2)), f)
    moe.moe_route_backward(prob, i32.view(0, 2), torch.empty((0, 2), device=DEV), torch.empty((0, 2), device=DEV),
                           torch.empty((0, 4), device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(M=150, H=192, F=320, E=3, k=2), dict(M=3000, H=832, F=1088, E=5, k=2)])
def test_infinities_and_nan_stay_in_their_row_or_column(shape, dtype):
    # a value that is not finite reaches what the formula says and nothing else
    prob, d, ws = experts(**shape, dtype=dtype, seed=3)
    first = run_all(prob, d, ws)
    r = int(d["offsets"][1]) + 3  # a row of expert 1
    bad = {n: v.clone() for n, v in d.items()}
    bad["dgate"][r, 7], bad["dy"][r, 5], bad["up"][r + 1, 9] = NAN, float("inf"), float("inf")
    o = run_all(prob, bad, ws)
    hit = {n: torch.zeros_like(v, dtype=torch.bool) for n, v in o.items()}
    hit["dxp"][r], hit["dgate"][r], hit["dup"][r] = True, True, True
    hit["dgate"][r + 1, 9] = True
    hit["dwg"][1, 7], hit["dwd"][1, 5] = True, True
    for n, v in o.items():
        assert torch.equal(v[~hit[n]], first[n][~hit[n]]), n
        assert not bool(torch.isfinite(v[hit[n]]).any()), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [dict(M=600, H=320, F=448, E=6, k=2, S=2), dict(M=900, H=256, F=576, E=3, k=2),
                                   dict(M=70, H=2176, F=2112, E=2, k=1), dict(M=3000, H=832, F=1088, E=5, k=2, S=3),
                                   dict(M=60, H=448, F=6272, E=1, k=1),
                                   dict(M=12000, H=256, F=320, E=2, k=1, S=2)])
def test_order_does_not_change_a_bit(shape, dtype):
    prob, d, ws = experts(**shape, dtype=dtype, seed=4)
    first = run_all(prob, d, ws)
    try:
        for seed in (1, 12345):
            os.environ["MOE_DEBUG_SHUFFLE"] = str(seed)
            o = run_all(prob, d, ws)
            for n, v in o.items():
                assert torch.equal(v, first[n]), (n, seed)
    finally:
        os.environ.pop("MOE_DEBUG_SHUFFLE", None)
    again = run_all(prob, d, ws)
    assert all(torch.equal(v, first[n]) for n, v in again.items())


# ------------------------------------------------------- streams and graphs ---


class Step:
    """A training step of the layer by the operators: buffers, forward and backward."""

    def __init__(self, M, H, F, E, k, dtype, p, out="f32", S=1, held=0, base=0, seed=0):
        g, act, EL, R = gen(seed + 50), act_of(dtype), held or E, M * k
        self.out, self.p, self.dtype, self.base, self.shape = out, p, dtype, base, (M, H, F, E, k, S, EL)
        self.x, self.logits = normal(g, M, H, dtype=act), normal(g, M, E)
        self.wg, self.wu = normal(g, EL, F, H, std=0.1, dtype=act), normal(g, EL, F, H, std=0.1, dtype=act)
        self.wd = normal(g, EL, H, F, std=0.1, dtype=act)
        self.dout = normal(g, M, H, dtype=act_of(out))
        self.rng = rng_of(seed + 99, 5)
        self.src = (torch.arange(M, device=DEV) % S).to(torch.int32) if S > 1 else None
        self.prob = moe.problem(M, H, F, E, k, S, dtype, base if held else 0, held)
        e = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
        i32 = torch.int32
        self.idx, self.w = e(M, k, dt=i32), e(M, k)
        self.counts, self.offsets = e(S * EL, dt=i32), e(S * EL + 1, dt=i32)
        self.s2f, self.f2s = e(R, dt=i32), e(R, dt=i32)
        self.xp, self.gate, self.up, self.h = e(R, H, dt=act), e(R, F, dt=act), e(R, F, dt=act), e(R, F, dt=act)
        self.y, self.o = e(R, H), e(M, H, dt=act_of(out))
        self.dy, self.dw, self.dgate, self.dup = e(R, H, dt=act), e(M, k), e(R, F, dt=act), e(R, F, dt=act)
        self.dxp, self.dx, self.dl = e(R, H, dt=act), e(M, H, dt=act), e(M, E)
        self.dwg, self.dwu, self.dwd = e(EL, F, H), e(EL, F, H), e(EL, H, F)
        ws = lambda op: torch.empty(max(moe.moe_workspace_bytes(self.prob, op), 256), dtype=torch.uint8, device=DEV)
        self.ws_d, self.ws_g, self.ws_b = ws(moe.MOE_OP_DISPATCH), ws(moe.MOE_OP_GROUPED_GEMM), ws(moe.MOE_OP_GROUPED_GEMM_BACKWARD)

    def run(self, stream=None):
        p, s = self.prob, stream
        drop = moe.dropout(self.p, self.rng) if self.p else None
        moe.moe_route(p, self.logits, self.idx, self.w, stream=s)
        moe.moe_dispatch(p, self.x, self.idx, self.src, self.counts, self.offsets, self.s2f, self.f2s, self.xp, self.ws_d, stream=s)
        moe.moe_grouped_gemm_aux(p, self.xp, self.wg, self.wu, self.offsets, self.gate, self.up, self.h, stream=s)
        moe.moe_grouped_gemm(p, 1, self.h, self.wd, None, self.offsets, self.y, self.ws_g, stream=s)
        moe.moe_combine_dropout(p, self.y, self.w, self.f2s, moe.epilogue(self.x, self.out), drop, self.o, stream=s)
        moe.moe_combine_backward(p, self.dout, self.y, self.w, self.f2s, drop, self.dy, self.dw, stream=s)
        moe.moe_grouped_gemm_backward(p, 1, self.dy, None, self.wd, None, self.gate, self.up, self.offsets, self.dgate,
                                      self.dup, self.ws_b, stream=s)
        moe.moe_grouped_gemm_backward_weights(p, 1, self.dy, None, self.h, self.offsets, self.dwd, None, False, self.ws_b, stream=s)
        moe.moe_grouped_gemm_backward(p, 0, self.dgate, self.dup, self.wg, self.wu, None, None, self.offsets, self.dxp, None,
                                      self.ws_b, stream=s)
        moe.moe_grouped_gemm_backward_weights(p, 0, self.dgate, self.dup, self.xp, self.offsets, self.dwg, self.dwu, False,
                                              self.ws_b, stream=s)
        # the residual of the layer passes dout on to x
        res = self.dout if self.out == self.dtype else self.dout.to(act_of(self.dtype))
        moe.moe_dispatch_backward(p, self.dxp, self.f2s, moe.epilogue(res, self.dtype), self.dx, stream=s)
        moe.moe_route_backward(p, self.idx, self.w, self.dw, self.dl, stream=s)
        return {n: getattr(self, n) for n in ("o", "dx", "dl", "dwg", "dwu", "dwd", "dgate", "dup", "dy", "dw")}


@pytest.mark.parametrize("dtype,p,kw", [("f32", 0.0, {}), ("f32", 0.25, dict(S=2, held=4, base=2)),
                                        ("bf16", 0.25, {}), ("bf16", 0.0, dict(S=3, held=5, base=1))])
def test_a_training_step_is_the_layers_gradient(dtype, p, kw):
    M, H, F, E, k = 203, 192, 320, 8, 3
    s = Step(M, H, F, E, k, dtype, p, out=dtype, seed=8, **kw)
    got = {n: v.clone() for n, v in s.run().items()}
    torch.cuda.synchronize()
    keep = ref.mask(M, H, p, s.rng, DEV) if p else None
    leaves = {n: getattr(s, n).double().requires_grad_() for n in ("x", "logits", "wg", "wu", "wd")}
    out = ref.layer(leaves["x"], leaves["logits"], leaves["wg"], leaves["wu"], leaves["wd"], s.idx.long(), s.base, leaves["x"],
                    keep, p)
    out.backward(s.dout.double())
    # f32: chains of sums of up to 2 F terms.  bf16: eight roundings of 2^-8 / sqrt(3) rms on the way (gate, up, h, dy,
    # dgate, dup, dX_perm, the output), of which independent ones add in squares: below 4 of them in all; a softmax's
    # gradient is a difference of such sums, twice as much
    tol = 4 * (8 * F) ** 0.5 * serving_ref.U if dtype == "f32" else 4 * serving_ref.BF16 / 3 ** 0.5
    for n, want in (("o", out), ("dx", leaves["x"].grad), ("dl", leaves["logits"].grad), ("dwg", leaves["wg"].grad),
                    ("dwu", leaves["wu"].grad), ("dwd", leaves["wd"].grad)):
        rel = float((got[n].double() - want).norm() / want.norm())
        assert rel <= (2 * tol if n == "dl" else tol), (n, rel, tol)
    if dtype == "f32":
        # and against differences of the layer along a direction, in 64 bits
        for n, grad in (("x", got["dx"]), ("logits", got["dl"]), ("wg", got["dwg"]), ("wu", got["dwu"]), ("wd", got["dwd"])):
            base = {m: v.detach() for m, v in leaves.items()}
            way = grad.double() / grad.double().norm()  # along the gradient, where the difference is largest

            def loss(h):
                d = dict(base, **{n: base[n] + h * way})
                return float((ref.layer(d["x"], d["logits"], d["wg"], d["wu"], d["wd"], s.idx.long(), s.base, d["x"], keep, p)
                              * s.dout.double()).sum())

            h = 1e-4
            diff, mine = (loss(h) - loss(-h)) / (2 * h), float((grad.double() * way).sum())
            assert abs(diff - mine) <= 1e-4 * abs(mine), (n, diff, mine)


# small tiles; large ones; reductions cut into parts (rows, weights)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [(300, 256, 320, 8, 2), (2500, 832, 1088, 4, 2), (60, 448, 6272, 1, 1), (12000, 256, 320, 2, 1)])
def test_graph_replays_equal_eager(sizes, dtype):
    a = Step(*sizes, dtype, 0.25, out=dtype, seed=12)
    b = Step(*sizes, dtype, 0.25, out=dtype, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.run()
    for rep in range(4):
        for s in (a, b):
            s.x.mul_(-0.75)
            s.logits.copy_(s.logits.flip(1))
            s.rng[1] += 17  # another mask, without another capture
        want = a.run()
        torch.cuda.synchronize()
        float((want["dwg"] * 2).sum())  # eager work between replays
        for v in got.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[n]), (rep, n)


@pytest.mark.parametrize("first,second", [((800, 256, 448, 8, 2), (500, 512, 256, 16, 4)),
                                          ((2500, 832, 1088, 4, 2), (60, 448, 6272, 1, 1))])
def test_two_steps_at_once_on_two_streams(first, second):
    steps = [Step(*first, "bf16", 0.1, seed=1), Step(*second, "bf16", 0.5, seed=2)]
    serial = []
    for s in steps:
        serial.append({n: v.clone() for n, v in s.run().items()})
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for s, st in zip(steps, streams):
            for v in (s.o, s.dx, s.dwg, s.dy):
                v.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for s, st in zip(steps, streams):
                with torch.cuda.stream(st):
                    got = s.run(stream=st)
        torch.cuda.synchronize()
        for s, want in zip(steps, serial):
            for n, v in want.items():
                assert torch.equal(getattr(s, n), v), (rep, n)


# -------------------------------------------------------------- validation ---


def test_debug_validate_refuses_bad_indices():
    M, H, F, E, k = 20, 64, 128, 4, 2
    prob, w, f2s, y = combine_inputs(M, H, E, k, "f32")
    idx, _, _, offsets = routing(M, E, k)
    prob = moe.problem(M, H, F, E, k, dtype="f32")
    dw, dl = torch.zeros(M, k, device=DEV), torch.zeros(M, E, device=DEV)
    z = lambda *s: torch.zeros(s, device=DEV)
    wt, rows, rowsf = z(E, F, H), z(M * k, H), z(M * k, F)
    ws = torch.empty(moe.moe_workspace_bytes(prob, moe.MOE_OP_GROUPED_GEMM_BACKWARD), dtype=torch.uint8, device=DEV)
    bad_f2s, bad_idx, bad_off = f2s.clone(), idx.clone(), offsets.clone()
    bad_f2s[3], bad_idx[5, 1], bad_off[2] = M * k, E, -1
    calls = [(lambda i: moe.moe_route_backward(prob, i, w, dw, dl), idx, bad_idx),
             (lambda i: moe.moe_combine_dropout(prob, y, w, i, None, None, z(M, H)), f2s, bad_f2s),
             (lambda i: moe.moe_combine_backward(prob, z(M, H), y, w, i, None, rows, dw), f2s, bad_f2s),
             (lambda i: moe.moe_dispatch_backward(prob, y, i, None, z(M, H)), f2s, bad_f2s),
             (lambda i: moe.moe_grouped_gemm_aux(prob, y, wt, wt, i, rowsf, z(M * k, F), z(M * k, F)), offsets, bad_off),
             (lambda i: moe.moe_grouped_gemm_backward(prob, 0, rowsf, rowsf, wt, wt, None, None, i, rows, None, ws), offsets, bad_off),
             (lambda i: moe.moe_grouped_gemm_backward_weights(prob, 0, rowsf, rowsf, y, i, z(E, F, H), z(E, F, H), False, ws), offsets, bad_off)]
    os.environ["MOE_DEBUG_VALIDATE"] = "1"
    try:
        for n, (call, good, bad) in enumerate(calls):
            call(good)
            with pytest.raises(moe.MoeError) as ex:
                call(bad)
            assert ex.value.status == moe.MOE_ERR_INVALID_ARGUMENT, n
    finally:
        os.environ.pop("MOE_DEBUG_VALIDATE", None)
