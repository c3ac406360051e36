"""The training operators' cases: the gradients of the MoE layer's steps (route,
dispatch, grouped GEMM, combine) and the combine with dropout.

A case is a dict of sizes; ``prepare`` makes its inputs on the GPU from a
seed, ``run`` is one call (plain torch operations where ``own`` is false, the
library where it is true), ``work`` what the call cannot do without and
``exact`` its result in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"

# ------------------------------------------------------------------ cases ---


def listed():
    return [
        # the router's gradient of a short sequence: nothing but latency
        case("route backward, 256 tokens, 8 experts", "route", M=256, E=8, k=2),
        # ... and of a long batch over many experts
        case("route backward, 65536 tokens, 128 experts", "route", M=65536, E=128, k=8),
        # the layer's output in the residual stream's type, dropout before the residual
        case("combine with dropout, 8192 tokens", "combine", M=8192, H=4096, E=8, k=2, p=0.1, out="bf16", residual=True),
        # an odd number of tokens, plain f32 output
        case("combine with dropout, 333 tokens", "combine", M=333, H=2048, E=64, k=4, p=0.5),
        # its gradient, with the same mask again
        case("combine backward, 8192 tokens, dropout", "combine_backward", M=8192, H=4096, E=8, k=2, p=0.1, out="bf16"),
        # one card's expert-parallel share: an eighth of the pairs is held here
        case("combine backward, 16 of 128 held", "combine_backward", M=4096, H=7168, E=128, k=8, held=16, S=8),
        # gradient of many small experts' rows back to the tokens, onto the residual stream's gradient
        case("dispatch backward, 4096 tokens, top 4", "dispatch_backward", M=4096, H=2048, E=64, k=4, out="bf16",
             residual=True),
        case("dispatch backward, 16384 tokens, top 2", "dispatch_backward", M=16384, H=4096, E=16, k=2),
        # forward gate/up product of many small experts that keeps gate and up for the gradient
        case("experts, gate and up kept, 64 small", "keep", M=4096, H=2048, F=1408, E=64, k=4),
        # gradient through the down product and SwiGLU of few large experts
        case("experts, rows of layer 1, 8 large", "rows1", M=8192, H=4096, F=14336, E=8, k=2),
        # gradient of the small f32 layer's token rows
        case("experts, rows of layer 0, f32", "rows0", M=256, H=256, F=512, E=8, k=2, dtype="f32"),
        # gradient of the gate and up weights, f32 as an optimizer's main gradient
        case("experts, weights of layer 0, 16 of 4096 x 6400", "weights0", M=16384, H=4096, F=6400, E=16, k=2),
    ]


def case(name=None, op="route", *, M, H=64, F=64, E, k, held=0, S=1, dtype="bf16", out="f32", residual=False, p=0.0):
    """`op` for M tokens (H hidden, F expert width) that choose k of E experts, of which `held` (0: all) are here, from
    the middle on; the tokens come in S equal source blocks; p: dropout; out: the type of the output (of the incoming
    gradient in combine_backward, of the weights' gradient in weights0 and weights1)."""
    c = dict(op=op, M=M, H=H, F=F, E=E, k=k, held=held, S=S, dtype=dtype, out=out, residual=residual, p=p)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["route", "combine", "combine", "combine_backward", "combine_backward", "dispatch_backward",
                         "dispatch_backward", "keep", "rows1", "rows0", "weights1", "weights0"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        M, E = _log_int(rng, 1, 16384), _log_int(rng, 1, 128)
        k = min(E, _log_int(rng, 1, 8))
        held = 0 if rng.random() < 0.7 else max(1, E // rng.choice([2, 4, 8]))
        S = 1 if rng.random() < 0.7 else rng.choice([2, 3, 8])
        out = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
        c = case(op=op, M=M, H=64 * _log_int(rng, 1, 112), F=64 * _log_int(rng, 1, 224), E=E, k=k,
                 held=0 if held == E else held, S=S, dtype=dtype, out=out,
                 residual=op in ("combine", "dispatch_backward") and rng.random() < 0.5,
                 p=0.0 if "combine" not in op or rng.random() < 0.3 else rng.choice([0.1, 0.25, 0.5]))
        if op == "combine" and not c["p"]:
            c["p"] = 0.1
        if op == "route":
            c.update(M=_log_int(rng, 1, 65536), H=64, F=64, held=0, S=1, dtype="bf16", out="f32")
        if op not in ("keep", "rows1", "rows0", "weights1", "weights0"):
            c["F"] = 64
        w = work(c)
        rows = c["M"] * c["k"]
        f32 = c["dtype"] == "f32"
        if (w["bytes"] <= 3.5e9 and w["flops"] <= (1e11 if f32 else 1.5e12) and rows * max(c["H"], c["F"]) <= 4e8
                and _held(c) * c["H"] * c["F"] <= 6e8):
            return c


# ----------------------------------------------------------------- inputs ---


def _size(dtype):
    return 4 if dtype == "f32" else 2


def _held(c):
    return c["held"] or c["E"]


def _base(c):
    return (c["E"] - _held(c)) // 2


def work(case):
    c = case
    M, H, F, E, k, EL = c["M"], c["H"], c["F"], c["E"], c["k"], _held(c)
    b, o, R = _size(c["dtype"]), _size(c["out"]), M * k
    kept = R * EL / E
    used = EL * (1.0 - (1.0 - k / E) ** M)  # experts held that some token chooses
    res = M * H * b if c["residual"] else 0
    op = c["op"]
    if op == "route":
        n, f = 12 * R + 4 * M * E, 4 * R
    elif op == "combine":
        n, f = kept * H * 4 + M * H * o + res + 8 * R, 2 * kept * H + M * H
    elif op == "combine_backward":
        n, f = M * H * o + kept * H * (4 + b) + 12 * R, 3 * kept * H
    elif op == "dispatch_backward":
        n, f = kept * H * b + M * H * o + res + 4 * R, kept * H
    elif op == "keep":
        n, f = (2 * used * H * F + kept * (H + 3 * F)) * b, 4 * kept * H * F
    elif op == "rows1":
        n, f = (used * H * F + kept * (H + 4 * F)) * b, 2 * kept * H * F
    elif op == "rows0":
        n, f = (2 * used * H * F + kept * (H + 2 * F)) * b, 4 * kept * H * F
    elif op == "weights1":
        n, f = kept * (H + F) * b + EL * H * F * o, 2 * kept * H * F
    else:
        n, f = kept * (H + 2 * F) * b + 2 * EL * H * F * o, 4 * kept * H * F
    return {"bytes": float(n), "flops": float(f)}


def _routing(c, normal):
    """What a forward pass leaves: the chosen experts, their weights, and the order of the rows sorted by segment."""
    M, E, k, S, EL = c["M"], c["E"], c["k"], c["S"], _held(c)
    R, G = M * k, S * EL
    logits = normal(M, E, dtype=torch.float32) + 0.3 * normal(E, dtype=torch.float32)  # some experts get more than others
    vals, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    vals, idx = vals[:, :k].contiguous(), idx[:, :k].contiguous()
    e = torch.exp(vals - vals[:, :1])
    slot = idx.reshape(-1) - _base(c)
    block = torch.arange(M, device=DEV) * S // M
    seg = block.repeat_interleave(k) * EL + slot
    seg = torch.where((slot >= 0) & (slot < EL), seg, torch.full_like(seg, G))
    order = torch.sort(seg, stable=True).indices
    n = torch.bincount(seg, minlength=G + 1)
    offsets = torch.zeros(G + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(n[:G], 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(R, device=DEV)
    kept = offsets[-1]
    f2s = torch.where(place < kept, place, torch.full_like(place, -1))
    return dict(topk_idx=idx.to(torch.int32), topk_w=e / e.sum(1, keepdim=True), f2s=f2s.to(torch.int32),
                offsets=offsets.to(torch.int32))


def _tensors(c, seed):
    """The inputs of a case: what both sides, and the result in 64 bits, are computed from.  Gradients are of a mean
    loss's size; rows past the kept pairs hold whatever they hold."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * (seed + 1) + 11)
    act = torch.float32 if c["dtype"] == "f32" else torch.bfloat16

    def normal(*shape, std=1.0, dtype=act):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)

    M, H, F, k, EL, R, op = c["M"], c["H"], c["F"], c["k"], _held(c), c["M"] * c["k"], c["op"]
    d = _routing(c, normal)
    grad = 1e-2
    if op == "route":
        d["dw"] = normal(M, k, std=grad, dtype=torch.float32)
    elif op == "combine":
        d["y"] = normal(R, H, dtype=torch.float32)
    elif op == "combine_backward":
        d["y"] = normal(R, H, dtype=torch.float32)
        d["dout"] = normal(M, H, std=grad, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    elif op == "dispatch_backward":
        d["dxp"] = normal(R, H, std=grad)
    if op in ("keep", "weights0"):
        d["xp"] = normal(R, H)
    if op in ("keep", "rows0"):
        d.update(w_gate=normal(EL, F, H, std=0.02), w_up=normal(EL, F, H, std=0.02))
    if op in ("rows1", "weights1"):
        d["dy"] = normal(R, H, std=grad)
    if op == "rows1":
        d.update(w_down=normal(EL, H, F, std=0.02), gate=normal(R, F), up=normal(R, F))
    if op in ("rows0", "weights0"):
        d.update(dgate=normal(R, F, std=grad), dup=normal(R, F, std=grad))
    if op == "weights1":
        d["h"] = normal(R, F)
    if c["residual"]:
        d["residual"] = normal(M, H)
    if c["p"]:
        d["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device=DEV, dtype=torch.int64)
    return d


def prepare(case, seed):
    c = dict(case)
    d = _tensors(c, seed)
    s = dict(c=c, d=d)
    if not own:
        s["cuts"] = d["offsets"].tolist()  # the segments' bounds, for the plain form's loop
        return s
    import combine_topk_gate_amd as moe
    M, H, F, EL, R, op = c["M"], c["H"], c["F"], _held(c), c["M"] * c["k"], c["op"]
    act = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    odt = torch.bfloat16 if c["out"] == "bf16" else torch.float32

    def rows(n, dtype=act):
        return torch.zeros((R, n), dtype=dtype, device=DEV)

    out = {"route": lambda: [torch.empty((M, c["E"]), device=DEV)],
           "combine": lambda: [torch.empty((M, H), dtype=odt, device=DEV)],
           "combine_backward": lambda: [rows(H), torch.empty((M, c["k"]), device=DEV)],
           "dispatch_backward": lambda: [torch.empty((M, H), dtype=odt, device=DEV)],
           "keep": lambda: [rows(F), rows(F), rows(F)],
           "rows1": lambda: [rows(F), rows(F)],
           "rows0": lambda: [rows(H)],
           "weights1": lambda: [torch.empty((EL, H, F), dtype=odt, device=DEV)],
           "weights0": lambda: [torch.empty((EL, F, H), dtype=odt, device=DEV) for _ in range(2)]}[op]()
    p = moe.problem(M, H, F, c["E"], c["k"], c["S"], c["dtype"], _base(c) if c["held"] else 0, c["held"])
    need = moe.moe_workspace_bytes(p, moe.MOE_OP_GROUPED_GEMM_BACKWARD)
    s.update(moe=moe, p=p, out=out, ws=torch.empty(max(need, 256), dtype=torch.uint8, device=DEV))
    return s


# -------------------------------------------------------------- one call ---


def run(state):
    c, d = state["c"], state["d"]
    if not own:
        return _PLAIN[c["op"]](c, d, state["cuts"])
    moe, p, out, ws, op = state["moe"], state["p"], state["out"], state["ws"], c["op"]
    drop = moe.dropout(c["p"], d["rng"]) if c["p"] else None
    if op == "route":
        moe.moe_route_backward(p, d["topk_idx"], d["topk_w"], d["dw"], out[0])
    elif op == "combine":
        moe.moe_combine_dropout(p, d["y"], d["topk_w"], d["f2s"], moe.epilogue(d.get("residual"), c["out"]), drop, out[0])
    elif op == "combine_backward":
        moe.moe_combine_backward(p, d["dout"], d["y"], d["topk_w"], d["f2s"], drop, out[0], out[1])
    elif op == "dispatch_backward":
        moe.moe_dispatch_backward(p, d["dxp"], d["f2s"], moe.epilogue(d.get("residual"), c["out"]), out[0])
    elif op == "keep":
        moe.moe_grouped_gemm_aux(p, d["xp"], d["w_gate"], d["w_up"], d["offsets"], *out)
    elif op == "rows1":
        moe.moe_grouped_gemm_backward(p, 1, d["dy"], None, d["w_down"], None, d["gate"], d["up"], d["offsets"], out[0],
                                      out[1], ws)
    elif op == "rows0":
        moe.moe_grouped_gemm_backward(p, 0, d["dgate"], d["dup"], d["w_gate"], d["w_up"], None, None, d["offsets"], out[0],
                                      None, ws)
    elif op == "weights1":
        moe.moe_grouped_gemm_backward_weights(p, 1, d["dy"], None, d["h"], d["offsets"], out[0], None, False, ws)
    else:
        moe.moe_grouped_gemm_backward_weights(p, 0, d["dgate"], d["dup"], d["xp"], d["offsets"], out[0], out[1], False, ws)
    return out


def _act(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _out(c, v):
    return v.to(torch.bfloat16) if c["out"] == "bf16" else v


LOW = 0xFFFFFFFF


def _kept(c, d):
    """Philox 4x32 in ten rounds (Salmon et al. 2011): word n % 4 of the block with counter {n / 4, offset} and key
    seed decides element n; it stays where the word is at least p 2^32.  64-bit products wrap, and their halves are
    masked out."""
    n = c["M"] * c["H"]
    i = torch.arange(n // 4, device=DEV, dtype=torch.int64)
    seed, offset = d["rng"][0], d["rng"][1]
    x = [i & LOW, (i >> 32) & LOW, (offset & LOW).expand_as(i), ((offset >> 32) & LOW).expand_as(i)]
    key = [seed & LOW, (seed >> 32) & LOW]
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [((b >> 32) & LOW) ^ x[1] ^ key[0], b & LOW, ((a >> 32) & LOW) ^ x[3] ^ key[1], a & LOW]
        key = [(key[0] + 0x9E3779B9) & LOW, (key[1] + 0xBB67AE85) & LOW]
    return (torch.stack(x, dim=1) >= int(c["p"] * 2.0 ** 32)).view(c["M"], c["H"])


def _dropped(c, d, v):
    return torch.where(_kept(c, d), v * (1.0 / (1.0 - c["p"])), torch.zeros_like(v)) if c["p"] else v


def _gathered(c, d, rows, weights=None):
    """Per token the (weighted) sum over its kept pairs of their rows."""
    f2s = d["f2s"].long().view(c["M"], c["k"])
    acc = torch.zeros((c["M"], c["H"]), device=DEV)
    for j in range(c["k"]):
        here = (f2s[:, j] >= 0)[:, None]
        v = rows[f2s[:, j].clamp(min=0)].float()
        acc += torch.where(here, v if weights is None else weights[:, j:j + 1] * v, torch.zeros_like(v))
    return acc


def _plain_route(c, d, cuts):
    w, dw = d["topk_w"], d["dw"]
    dl = w * (dw - (w * dw).sum(1, keepdim=True))
    out = torch.zeros((c["M"], c["E"]), device=DEV)
    out.scatter_(1, d["topk_idx"].long(), dl)
    return [out]


def _plain_combine(c, d, cuts):
    acc = _dropped(c, d, _gathered(c, d, d["y"], d["topk_w"]))
    return [_out(c, acc + d["residual"].float() if "residual" in d else acc)]


def _plain_combine_backward(c, d, cuts):
    M, H, k = c["M"], c["H"], c["k"]
    g = _dropped(c, d, d["dout"].float())
    f2s = d["f2s"].long().view(M, k)
    dy = torch.zeros((M * k + 1, H), dtype=_act(c), device=DEV)  # the last row takes the dropped pairs'
    dw = torch.zeros((M, k), device=DEV)
    for j in range(k):
        here = f2s[:, j] >= 0
        row = torch.where(here, f2s[:, j], torch.full_like(f2s[:, j], M * k))
        dy[row] = (d["topk_w"][:, j:j + 1] * g).to(dy.dtype)
        s = (g * d["y"][f2s[:, j].clamp(min=0)]).sum(1)
        dw[:, j] = torch.where(here, s, torch.zeros_like(s))
    return [dy[:-1], dw]


def _plain_dispatch_backward(c, d, cuts):
    acc = _gathered(c, d, d["dxp"])
    return [_out(c, acc + d["residual"].float() if "residual" in d else acc)]


def _segments(c, cuts):
    """(weight slot, first row, end) of the segments that hold rows."""
    return [(g % _held(c), lo, hi) for g, (lo, hi) in enumerate(zip(cuts, cuts[1:])) if hi > lo]


def _rows(c, n):
    return torch.zeros((c["M"] * c["k"], n), dtype=_act(c), device=DEV)


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_keep(c, d, cuts):
    gate, up, h = (_rows(c, c["F"]) for _ in range(3))
    for e, lo, hi in _segments(c, cuts):
        x = d["xp"][lo:hi].float()
        g, u = torch.matmul(x, d["w_gate"][e].float().t()), torch.matmul(x, d["w_up"][e].float().t())
        gate[lo:hi], up[lo:hi], h[lo:hi] = g, u, _silu(g) * u
    return [gate, up, h]


def _plain_rows1(c, d, cuts):
    dgate, dup = _rows(c, c["F"]), _rows(c, c["F"])
    for e, lo, hi in _segments(c, cuts):
        dh = torch.matmul(d["dy"][lo:hi].float(), d["w_down"][e].float())
        g, u = d["gate"][lo:hi].float(), d["up"][lo:hi].float()
        s = 1.0 / (1.0 + torch.exp(-g))
        dgate[lo:hi] = dh * u * (s * (1.0 + g * (1.0 - s)))
        dup[lo:hi] = dh * (g * s)
    return [dgate, dup]


def _plain_rows0(c, d, cuts):
    dxp = _rows(c, c["H"])
    for e, lo, hi in _segments(c, cuts):
        dxp[lo:hi] = (torch.matmul(d["dgate"][lo:hi].float(), d["w_gate"][e].float())
                      + torch.matmul(d["dup"][lo:hi].float(), d["w_up"][e].float()))
    return [dxp]


def _plain_weights(c, d, cuts, a, rows):
    n = _held(c), a[0].shape[1], rows.shape[1]
    out = [torch.zeros(n, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV) for _ in a]
    by_expert = {}
    for e, lo, hi in _segments(c, cuts):
        by_expert.setdefault(e, []).append((lo, hi))
    for e, parts in by_expert.items():
        x = torch.cat([rows[lo:hi] for lo, hi in parts]).float()
        for o, g in zip(out, a):
            o[e] = torch.matmul(torch.cat([g[lo:hi] for lo, hi in parts]).float().t(), x)
    return out


def _plain_weights1(c, d, cuts):
    return _plain_weights(c, d, cuts, [d["dy"]], d["h"])


def _plain_weights0(c, d, cuts):
    return _plain_weights(c, d, cuts, [d["dgate"], d["dup"]], d["xp"])


_PLAIN = {"route": _plain_route, "combine": _plain_combine, "combine_backward": _plain_combine_backward,
          "dispatch_backward": _plain_dispatch_backward, "keep": _plain_keep, "rows1": _plain_rows1, "rows0": _plain_rows0,
          "weights1": _plain_weights1, "weights0": _plain_weights0}


# ------------------------------------------------------ the exact result ---


def _exact_mask(c, d):
    """The mask with unsigned 64-bit arithmetic on the host."""
    seed, offset = (int(v) for v in d["rng"].tolist())
    u = np.uint64
    low, up = u(0xFFFFFFFF), u(32)
    n = np.arange(c["M"] * c["H"] // 4, dtype=np.uint64)
    c0, c1 = n & low, n >> up
    c2, c3 = np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (p1 >> up) ^ c1 ^ u(k0), p1 & low, (p0 >> up) ^ c3 ^ u(k1), p0 & low
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    keep = np.stack([c0, c1, c2, c3], axis=-1).reshape(c["M"], c["H"]) >= u(math.floor(c["p"] * 2 ** 32))
    return torch.from_numpy(keep).to(DEV).double() / (1.0 - c["p"])


def exact(case, seed):
    """The definition in 64 bits, over the pairs that are held."""
    c = dict(case)
    d = _tensors(c, seed)
    M, H, F, k, EL, op = c["M"], c["H"], c["F"], c["k"], _held(c), c["op"]
    R = M * k
    f64 = dict(dtype=torch.float64, device=DEV)
    if op == "route":
        w = d["topk_w"].double()
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        dl = (jac * d["dw"].double()[:, None, :]).sum(2)
        return [torch.zeros(M, c["E"], **f64).scatter_add_(1, d["topk_idx"].long(), dl)]
    flat = torch.nonzero(d["f2s"] >= 0).flatten()  # the held pairs, their rows and tokens
    row, tok = d["f2s"].long()[flat], flat // k
    mask = _exact_mask(c, d) if c["p"] else None
    if op in ("combine", "dispatch_backward"):
        out = torch.zeros(M, H, **f64)
        for lo in range(0, flat.numel(), 8192):
            s = slice(lo, lo + 8192)
            v = d["y"][row[s]].double() * d["topk_w"].double().flatten()[flat[s], None] if op == "combine" else d["dxp"][row[s]].double()
            out.index_add_(0, tok[s], v)
        out = out * mask if mask is not None else out
        return [out + d["residual"].double() if c["residual"] else out]
    if op == "combine_backward":
        g = d["dout"].double() * (mask if mask is not None else 1.0)
        dy, dw = torch.zeros(R, H, **f64), torch.zeros(R, **f64)
        for lo in range(0, flat.numel(), 8192):
            s = slice(lo, lo + 8192)
            dy[row[s]] = g[tok[s]] * d["topk_w"].double().flatten()[flat[s], None]
            dw[flat[s]] = (g[tok[s]] * d["y"][row[s]].double()).sum(1)
        return [dy, dw.view(M, k)]
    off = d["offsets"].tolist()
    bounds = [[(off[s * EL + e], off[s * EL + e + 1]) for s in range(c["S"])] for e in range(EL)]
    where = [torch.cat([torch.arange(lo, hi, device=DEV) for lo, hi in b]) for b in bounds]
    shape = {"keep": [(R, F)] * 3, "rows1": [(R, F)] * 2, "rows0": [(R, H)], "weights1": [(EL, H, F)],
             "weights0": [(EL, F, H)] * 2}[op]
    out = [torch.zeros(n, **f64) for n in shape]
    for e, r in enumerate(where):
        if op == "keep":
            g, u = d["xp"][r].double() @ d["w_gate"][e].double().T, d["xp"][r].double() @ d["w_up"][e].double().T
            out[0][r], out[1][r], out[2][r] = g, u, g * torch.sigmoid(g) * u
        elif op == "rows1":
            dh, g = d["dy"][r].double() @ d["w_down"][e].double(), d["gate"][r].double()
            s = torch.sigmoid(g)
            out[0][r] = dh * d["up"][r].double() * (s + g * s * torch.sigmoid(-g))
            out[1][r] = dh * g * s
        elif op == "rows0":
            out[0][r] = (torch.cat([d["dgate"][r], d["dup"][r]], 1).double()
                         @ torch.cat([d["w_gate"][e], d["w_up"][e]], 0).double())
        elif op == "weights1":
            out[0][e] = d["dy"][r].double().T @ d["h"][r].double()
        else:
            x = d["xp"][r].double()
            out[0][e], out[1][e] = d["dgate"][r].double().T @ x, d["dup"][r].double().T @ x
    return out
