"""The serving operators' cases: the MoE layer for a few tokens
(moe_layer_decode) and the projection with low-rank adapters of many requests
(moe_adapter_linear).

A case is a dict of sizes; ``prepare`` makes its inputs on the GPU from a
seed, ``run`` is one call (plain torch operations where ``own`` is false, the
library where it is true), ``work`` what the call cannot do without and
``exact`` its result in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"

# ------------------------------------------------------------------ cases ---


def listed():
    return [
        # one token of a model of many small experts: the smallest weights a
        # decode step reads, where the launches and the routing latency count
        layer("layer, 1 token, 64 small experts", M=1, H=2048, F=1408, E=64, k=4),
        # one token of a model of few large experts, in the residual stream's type
        layer("layer, 1 token, 8 large experts", M=1, H=4096, F=14336, E=8, k=2, out="bf16", residual=True),
        # a small decode batch of odd size: most experts get one to four rows
        layer("layer, 17 tokens, 16 experts", M=17, H=4096, F=6400, E=16, k=2, out="bf16", residual=True),
        # one card's expert-parallel share in a decode step (16 of 128 experts,
        # W_down in MXFP8) of a fixed batch of which an eighth is idle
        layer("layer, 64 tokens, 16 of 128 held, mxfp8", M=64, H=7168, F=4096, E=128, k=8, held=16, dtype="bf16_mxfp8",
              idle=8),
        # a large decode batch: about 50 rows an expert, every weight read once
        layer("layer, 200 tokens, 8 large experts", M=200, H=4096, F=14336, E=8, k=2),
        # the f32 layer at the size of the f32 workload's matrices
        layer("layer, 5 tokens, f32", M=5, H=256, F=512, E=8, k=2, dtype="f32"),
        # the router of one token: gate logits from the hidden state, with the request's adapter
        linear("linear, router of 1 token", M=1, H=2048, N=64, r=8, P=4, mix="rows"),
        # a decode batch where nearly every request has an adapter of its own
        linear("linear, 48 requests of one token", M=48, H=4096, N=4096, r=16, P=64, out="bf16", residual=True, mix="rows"),
        # ragged prompts of a few requests, an odd number of rows
        linear("linear, 333 rows of 6 prompts", M=333, H=2048, N=1408, r=32, P=8, mix="runs", requests=6),
        # prompts of a full batch: the projection's product bounds it
        linear("linear, 8192 rows of 24 prompts", M=8192, H=4096, N=4096, r=16, P=16, out="bf16", residual=True, mix="runs",
               requests=24),
        # a wide input and a larger rank
        linear("linear, 2048 rows, rank 64", M=2048, H=7168, N=4096, r=64, P=12, out="bf16", mix="runs", requests=9),
        # f32, with an output width that is no multiple of anything
        linear("linear, 100 rows, f32", M=100, H=1024, N=1001, r=8, P=5, dtype="f32", mix="runs", requests=7),
    ]


def layer(name=None, *, M, H, F, E, k, held=0, dtype="bf16", out="f32", residual=False, idle=0):
    """A call of the MoE layer: `held` of the E experts are here (0: all), from the middle on; every `idle`-th row of
    the batch holds no token (its logits are all -inf)."""
    c = dict(op="layer", M=M, H=H, F=F, E=E, k=k, held=held, dtype=dtype, out=out, residual=residual, idle=idle)
    return dict(c, name=name) if name else c


def linear(name=None, *, M, H, N, r, P, dtype="bf16", out="f32", residual=False, mix, requests=0):
    """A call of the projection: P adapters of rank r; mix "rows": each row a request of its own, "runs": the rows of
    `requests` prompts one after the other.  One request in eight or so uses no adapter."""
    c = dict(op="linear", M=M, H=H, N=N, r=r, P=P, dtype=dtype, out=out, residual=residual, mix=mix, requests=requests)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        if rng.random() < 0.5:
            dtype = rng.choice(["bf16", "bf16", "bf16", "bf16_mxfp8", "f32"])
            unit = 128 if dtype == "bf16_mxfp8" else 64
            H = 64 * _log_int(rng, 4, 112)
            F = unit * _log_int(rng, 4, 14336 // unit)
            E = _log_int(rng, 4, 128)
            held = E if rng.random() < 0.7 else max(1, E // rng.choice([2, 4, 8]))
            k = min(E, _log_int(rng, 1, 8))
            out = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
            c = layer(M=_log_int(rng, 1, 200), H=H, F=F, E=E, k=k, held=0 if held == E else held, dtype=dtype, out=out,
                      residual=rng.random() < 0.5, idle=rng.choice([0, 0, 5]))
        else:
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            M = _log_int(rng, 1, 8192 if dtype == "bf16" else 600)
            mix = "rows" if M <= 200 and rng.random() < 0.6 else "runs"
            out = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
            c = linear(M=M, H=64 * _log_int(rng, 4, 112), N=_log_int(rng, 8, 7168), r=rng.choice([8, 16, 24, 32, 64]),
                       P=_log_int(rng, 1, 64), dtype=dtype, out=out, residual=rng.random() < 0.5, mix=mix,
                       requests=0 if mix == "rows" else _log_int(rng, 1, min(M, 40)))
        w = work(c)
        if w["bytes"] <= 2.5e9 and w["flops"] <= 2.5e11 and _weight_bytes(c) <= 3e9:
            return c


# ----------------------------------------------------------------- inputs ---


def _bytes_of(dtype):
    return 4 if dtype == "f32" else 2


def _held(c):
    return c["held"] or c["E"]


def _base(c):
    return (c["E"] - _held(c)) // 2


def _down_bytes(c):
    """Bytes of one expert's W_down: MXFP8 has one byte an element and one scale byte for 32."""
    n = c["H"] * c["F"]
    return n + n // 32 if c["dtype"] == "bf16_mxfp8" else n * _bytes_of(c["dtype"])


def _weight_bytes(c):
    if c["op"] == "linear":
        return (c["N"] * c["H"] + c["P"] * c["r"] * (c["H"] + c["N"])) * _bytes_of(c["dtype"])
    return _held(c) * (2 * c["H"] * c["F"] * _bytes_of(c["dtype"]) + _down_bytes(c))


def _live(c):
    """Rows of the batch that hold a token."""
    return c["M"] - (c["M"] // c["idle"] if c["idle"] else 0)


def work(case):
    c = case
    b = _bytes_of(c["dtype"])
    ob = 2 if c["out"] == "bf16" else 4
    if c["op"] == "linear":
        M, H, N, r = c["M"], c["H"], c["N"], c["r"]
        requests = M if c["mix"] == "rows" else min(c["requests"], M)
        used = c["P"] * (1.0 - (1.0 - 0.875 / c["P"]) ** requests)  # adapters that some request uses
        nbytes = (N * H + used * r * (H + N) + M * H) * b + M * N * (ob + (b if c["residual"] else 0)) + 4 * (M + c["P"])
        return {"bytes": float(nbytes), "flops": 2.0 * M * N * H + 2.0 * 0.875 * M * r * (H + N)}
    M, H, F, E, k = c["M"], c["H"], c["F"], c["E"], c["k"]
    live = _live(c)
    used = _held(c) * (1.0 - (1.0 - k / E) ** live)  # experts held that some token chooses
    pairs = live * k * _held(c) / E
    nbytes = (used * (2 * H * F * b + _down_bytes(c)) + M * H * (b + ob + (b if c["residual"] else 0)) + 4 * M * E)
    return {"bytes": float(nbytes), "flops": 6.0 * pairs * H * F}


def _quantize(w):
    """MXFP8 of w [rows, cols] (rows a multiple of 32, cols of 128), as the layer stores it: the e4m3 codes, then one
    scale byte per 32 values, those of 32 rows and 128 columns together."""
    rows, cols = w.shape
    v = w.float().view(rows, cols // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, torch.full_like(amax, -127.0).int()).clamp(min=-127)
    codes = torch.ldexp(v, -X).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(rows * cols)
    s = (X.squeeze(-1) + 127).to(torch.uint8).view(rows // 32, 32, cols // 128, 4).permute(0, 2, 1, 3).reshape(-1)
    return codes, s


def _dequantize(buf, rows, cols, lo, hi, to):
    """Rows [lo, hi) (multiples of 32) of an MXFP8 buffer of rows x cols, as the values they stand for."""
    codes = buf[lo * cols:hi * cols].view(torch.float8_e4m3fn).to(to).view(hi - lo, cols // 32, 32)
    s = buf[rows * cols:].view(rows // 32, cols // 128, 32, 4)[lo // 32:hi // 32]
    s = s.permute(0, 2, 1, 3).reshape(hi - lo, cols // 32, 1)
    return (codes * torch.exp2(s.to(to) - 127.0)).view(hi - lo, cols)


def _tensors(c, seed):
    """The inputs of a case: what both sides, and the result in 64 bits, are computed from."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * (seed + 1) + 7)
    act = torch.float32 if c["dtype"] == "f32" else torch.bfloat16

    def normal(*shape, std=1.0, dtype=act):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)

    M, H = c["M"], c["H"]
    d = dict(x=normal(M, H))
    if c["op"] == "layer":
        F, E, EL = c["F"], c["E"], _held(c)
        logits = normal(M, E, dtype=torch.float32)
        if c["idle"]:
            logits[c["idle"] - 1::c["idle"]] = float("-inf")
        d.update(logits=logits, w_gate=normal(EL, F, H, std=0.02), w_up=normal(EL, F, H, std=0.02))
        if c["dtype"] == "bf16_mxfp8":
            codes, scales = [], []
            for _ in range(EL):
                a, s = _quantize(normal(H, F, std=0.02))
                codes.append(a)
                scales.append(s)
            d["w_down"] = torch.cat(codes + scales)
        else:
            d["w_down"] = normal(EL, H, F, std=0.02)
        if c["residual"]:
            d["residual"] = normal(M, H)
        return d
    N, r, P = c["N"], c["r"], c["P"]
    d.update(w=normal(N, H, std=0.02), a=normal(P, r, H, std=H ** -0.5), b=normal(P, N, r, std=0.02),
             scale=torch.empty(P, device=DEV).uniform_(0.5, 2.0, generator=g))
    n = M if c["mix"] == "rows" else min(c["requests"], M)
    which = torch.randint(0, P, (n,), generator=g, device=DEV, dtype=torch.int32)
    which[torch.rand(n, generator=g, device=DEV) < 0.125] = -1  # no adapter
    if c["mix"] == "rows":
        d["idx"] = which
    else:
        cuts = torch.sort(torch.randint(0, M + 1, (n - 1,), generator=g, device=DEV)).values
        d["idx"] = which[torch.searchsorted(cuts, torch.arange(M, device=DEV), right=True)].contiguous()
    if c["residual"]:
        d["residual"] = normal(M, N)
    return d


def prepare(case, seed):
    c = dict(case)
    s = dict(c=c, d=_tensors(c, seed))
    if own:
        import combine_topk_gate_amd as moe
        odt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        if c["op"] == "layer":
            p = moe.problem(c["M"], c["H"], c["F"], c["E"], c["k"], 1, c["dtype"], _base(c) if c["held"] else 0, c["held"])
            need = moe.moe_workspace_bytes(p, moe.MOE_OP_LAYER_DECODE)
            out = torch.empty((c["M"], c["H"]), dtype=odt, device=DEV)
        else:
            p = moe.adapter_problem(c["M"], c["H"], c["N"], c["r"], c["P"], c["dtype"])
            need = moe.moe_adapter_workspace_bytes(p)
            out = torch.empty((c["M"], c["N"]), dtype=odt, device=DEV)
        s.update(moe=moe, p=p, out=out, ws=torch.empty(max(need, 256), dtype=torch.uint8, device=DEV))
    return s


# -------------------------------------------------------------- one call ---


def run(state):
    c, d = state["c"], state["d"]
    if own:
        moe, p, out, ws = state["moe"], state["p"], state["out"], state["ws"]
        epi = moe.epilogue(d.get("residual"), c["out"])
        if c["op"] == "layer":
            moe.moe_layer_decode(p, d["x"], d["logits"], d["w_gate"], d["w_up"], d["w_down"], epi, out, ws)
        else:
            moe.moe_adapter_linear(p, d["x"], d["w"], d["a"], d["b"], d["scale"], d["idx"], epi, out, ws)
        return out
    y = _plain_layer(c, d) if c["op"] == "layer" else _plain_linear(c, d)
    if "residual" in d:
        y = y + d["residual"].float()
    return y.to(torch.bfloat16) if c["out"] == "bf16" else y


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_layer(c, d):
    M, H, F, k, EL, base = c["M"], c["H"], c["F"], c["k"], _held(c), _base(c)
    vals, idx = torch.sort(d["logits"], dim=1, descending=True, stable=True)  # ties: the lower expert first
    vals, idx = vals[:, :k], idx[:, :k]
    chosen = vals > float("-inf")
    top = torch.where(chosen[:, :1], vals[:, :1], torch.zeros_like(vals[:, :1]))
    e = torch.where(chosen, torch.exp(vals - top), torch.zeros_like(vals))
    w = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    slot = idx - base
    w = torch.where((slot >= 0) & (slot < EL), w, torch.zeros_like(w))
    x = d["x"].float()

    def down(e):
        if c["dtype"] == "bf16_mxfp8":
            return _dequantize(d["w_down"], EL * H, F, e * H, (e + 1) * H, torch.float32)
        return d["w_down"][e].float()

    if M == 1 and c["dtype"] != "bf16_mxfp8":
        # one token: only its own experts' matrices
        i = slot[0].clamp(0, EL - 1)
        h = _silu(torch.matmul(d["w_gate"][i].float(), x[0])) * torch.matmul(d["w_up"][i].float(), x[0])  # [k, F]
        y = torch.matmul(d["w_down"][i].float(), h[:, :, None])[:, :, 0]
        return (w[0][:, None] * y).sum(0, keepdim=True)
    out = torch.zeros((M, H), dtype=torch.float32, device=DEV)
    for e in range(EL):
        share = torch.where(slot == e, w, torch.zeros_like(w)).sum(1, keepdim=True)
        h = _silu(torch.matmul(x, d["w_gate"][e].float().t())) * torch.matmul(x, d["w_up"][e].float().t())
        out += share * torch.matmul(h, down(e).t())
    return out


def _plain_linear(c, d):
    x = d["x"].float()
    y = torch.matmul(x, d["w"].float().t())
    zero = torch.zeros((), device=DEV)
    for p in range(c["P"]):
        t = torch.matmul(x, d["a"][p].float().t()) * d["scale"][p]
        t = torch.where((d["idx"] == p)[:, None], t, zero)
        y += torch.matmul(t, d["b"][p].float().t())
    return y


# ------------------------------------------------------ the exact result ---


def exact(case, seed):
    """The definition in 64 bits, row by row of what each row needs."""
    c = dict(case)
    d = _tensors(c, seed)
    x = d["x"].double()
    if c["op"] == "linear":
        y = x @ d["w"].double().T
        for p in sorted(set(d["idx"].tolist())):
            if p >= 0:
                rows = torch.nonzero(d["idx"] == p).flatten()
                y[rows] += float(d["scale"][p]) * ((x[rows] @ d["a"][p].double().T) @ d["b"][p].double().T)
    else:
        y = torch.zeros(c["M"], c["H"], dtype=torch.float64, device=DEV)
        todo = {}  # held expert -> its (row, weight)
        for t, row in enumerate(d["logits"].double().tolist()):
            best = sorted((-v, e) for e, v in enumerate(row) if v > -math.inf)[:c["k"]]
            share = [math.exp(best[0][0] - v) for v, _ in best]
            for (_, e), s in zip(best, share):
                if 0 <= e - _base(c) < _held(c):
                    todo.setdefault(e - _base(c), []).append((t, s / math.fsum(share)))
        for e, pairs in todo.items():
            rows = torch.tensor([t for t, _ in pairs], device=DEV)
            share = torch.tensor([s for _, s in pairs], dtype=torch.float64, device=DEV)
            g, u = x[rows] @ d["w_gate"][e].double().T, x[rows] @ d["w_up"][e].double().T
            if c["dtype"] == "bf16_mxfp8":
                wd = _dequantize(d["w_down"], _held(c) * c["H"], c["F"], e * c["H"], (e + 1) * c["H"], torch.float64)
            else:
                wd = d["w_down"][e].double()
            y[rows] += share[:, None] * ((g * torch.sigmoid(g) * u) @ wd.T)
    return y + d["residual"].double() if "residual" in d else y
