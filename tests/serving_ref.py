"""Plain 64-bit references of the serving operators (moe_layer_decode,
moe_adapter_linear), with element-wise error bounds derived from the
arithmetic.  torch float64 on whatever device the inputs are; nothing here is
shared with the library.

Bounds.  u = 2^-24 is the largest relative error of one f32 rounding.  A sum
of n terms accumulated in f32 in any order is off by at most n u sum|terms|
to first order; the matrix cores may truncate where an f32 addition rounds,
so 2 n u is counted.  bf16 x bf16 products are exact in f32.  An f32 value
kept as two bf16 planes is off by at most 2^-8 2^-8 of itself (each plane
rounds what is left to 8 bits, half a step: eps / 2 = 2^-8); three planes
hold all 24 bits.  A cast to bf16 is off by at most 2^-8 of the value.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def quantize_mxfp8(w):
    """MXFP8 buffer of w [rows, cols] (rows a multiple of 32) and the values it
    stands for, in float64."""
    rows, cols = w.shape
    v = w.double().view(rows, cols // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp(min=1e-300))) - 8, torch.full_like(amax, -127.0))
    X = X.clamp(min=-127.0)
    codes = (v / torch.exp2(X)).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    values = (codes.double() * torch.exp2(X)).view(rows, cols)
    s = (X.squeeze(-1) + 127).to(torch.uint8).view(rows // 32, 32, cols // 128, 4).permute(0, 2, 1, 3).reshape(-1)
    return torch.cat([codes.view(torch.uint8).reshape(-1), s]), values


def silu(z):
    return z * torch.sigmoid(z)


def route(logits, k):
    """Per token the chosen experts (best first, ties to the lower index, -inf
    never) and their softmax weights: two lists of lists."""
    experts, weights = [], []
    for row in logits.double().cpu().tolist():
        best = sorted((e for e in range(len(row)) if row[e] > float("-inf")), key=lambda e: (-row[e], e))[:k]
        v = torch.tensor([row[e] for e in best], dtype=torch.float64)
        experts.append(best)
        weights.append(torch.softmax(v, 0).tolist() if best else [])
    return experts, weights


def layer(x, logits, w_gate, w_up, w_down, k, base, residual, f32, out_bf16):
    """(out, bound) in float64; w_* hold the experts from `base` on (values)."""
    M, H = x.shape
    EL, F = w_gate.shape[0], w_gate.shape[1]
    dev = x.device
    out = torch.zeros(M, H, dtype=torch.float64, device=dev)
    bound, mag = torch.zeros_like(out), torch.zeros_like(out)
    experts, weights = route(logits, k)
    rows_of = {}
    for t in range(M):
        for e, w in zip(experts[t], weights[t]):
            if 0 <= e - base < EL:
                rows_of.setdefault(e - base, []).append((t, w))
    x = x.double()
    for e, pairs in rows_of.items():
        rows = torch.tensor([t for t, _ in pairs], device=dev)
        w = torch.tensor([s for _, s in pairs], dtype=torch.float64, device=dev)[:, None]
        wg, wu, wd = w_gate[e].double(), w_up[e].double(), w_down[e].double()
        xr = x[rows]
        g, u = xr @ wg.T, xr @ wu.T
        n = 2 * H + (1 if f32 else 0)  # f32 products round too
        eg, eu = n * U * (xr.abs() @ wg.abs().T), n * U * (xr.abs() @ wu.abs().T)
        h = silu(g) * u
        # |silu'| <= 1.1; the exponential (its argument's rounding is in eg), the division, the product: 8 u
        eh = 1.1 * eg * (u.abs() + eu) + silu(g).abs() * eu + 8 * U * h.abs()
        if out_bf16 and not f32:
            eh = eh + BF16 * BF16 * h.abs()
        y, ay = h @ wd.T, h.abs() @ wd.abs().T
        ey = eh @ wd.abs().T + (2 * (1 if f32 else 3) * F + 1) * U * (ay + eh @ wd.abs().T)
        out[rows] += w * y
        # the weight: exponentials, their sum, a division
        bound[rows] += w * ey + (k + 8) * U * w * (y.abs() + ey)
        mag[rows] += w * y.abs()
    bound += 2 * k * U * mag
    return _finish(out, bound, residual, out_bf16)


def linear(x, w, a, b, scale, idx, residual, f32, out_bf16):
    M, H = x.shape
    x, w = x.double(), w.double()
    out = x @ w.T
    n = 2 * H + (1 if f32 else 0)
    mag = x.abs() @ w.abs().T
    bound = n * U * mag
    P = 0 if a is None else a.shape[0]
    for p in sorted(set(idx.cpu().tolist())) if P else []:
        if not 0 <= p < P:
            continue
        rows = torch.nonzero(idx == p).flatten()
        A, B, s = a[p].double(), b[p].double(), float(scale[p])
        t = s * (x[rows] @ A.T)
        et = (n + 1) * U * abs(s) * (x[rows].abs() @ A.abs().T)
        if out_bf16 and not f32:  # long batches: two planes of t
            et = et + BF16 * BF16 * t.abs()
        r = A.shape[0]
        at = t.abs() @ B.abs().T
        out[rows] += t @ B.T
        bound[rows] += et @ B.abs().T + (2 * 3 * r + 1) * U * (at + et @ B.abs().T) + (3 * r + 1) * U * mag[rows]
    bound += U * out.abs()
    return _finish(out, bound, residual, out_bf16)


def _finish(out, bound, residual, out_bf16):
    if residual is not None:
        out = out + residual.double()
        bound = bound + U * (out.abs() + bound)
    if out_bf16:
        bound = bound + BF16 * (out.abs() + bound)
    return out, bound


def check(got, want, bound, what):
    """got within bound of want, element by element, and its error's 2-norm
    within what roundings of independent signs give."""
    assert got.shape == want.shape, what
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 1e-30)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at {i}: got "
                             f"{float(got[tuple(i)])}, want {float(want[tuple(i)])}, bound {float(bound[tuple(i)])}")


def check_norm(got, want, roundings, out_bf16, what):
    """Relative 2-norm of the error: `roundings` f32 roundings of independent
    signs, each at most u of a partial sum, whose rms is at most the sum's:
    sqrt(roundings) u, times 4 for the stages; plus the cast's rms, half a
    step / sqrt(3) at most, for a bf16 output.  That is a mean over many
    elements: a single one may be off by the whole half step (0.6078 lies
    between the bf16 values 0.60547 and 0.60938, 0.0016 from the nearer: 2.6e-3
    of it, above 2^-8 / sqrt(3) = 2.3e-3 and below 2^-8 = 3.9e-3), so outputs of
    fewer than 64 elements get the half step itself."""
    ref = want.norm()
    if float(ref) == 0.0:
        assert not bool(got.double().any()), what
        return
    rel = float((got.double() - want).norm() / ref)
    bound = 4 * roundings ** 0.5 * U + ((BF16 / 3 ** 0.5 if got.numel() >= 64 else BF16) if out_bf16 else 0.0)
    assert rel <= bound, (what, rel, bound)


# Projections (bf16 unless dtype says) with the tiles that 256 CUs take for
# them, rows and columns of the projection's, rows and ranks of t's: every
# kernel, with ragged rows and columns, rows at any address, one to many
# adapters a tile, none at all.
TILES = [
    (dict(M=1, H=320, N=1001, r=24, P=3), (8, 16, 0, 0)),
    (dict(M=20, H=128, N=72, r=24, P=3), (16, 16, 16, 16)),
    (dict(M=20, H=128, N=70, r=16, P=3), (16, 16, 16, 16)),
    (dict(M=48, H=4096, N=4096, r=16, P=64), (32, 32, 16, 16)),
    (dict(M=333, H=2048, N=1408, r=32, P=6, mix="runs"), (32, 32, 16, 32)),
    (dict(M=335, H=1024, N=1021, r=8, P=9), (32, 32, 16, 16)),
    (dict(M=130, H=2048, N=1001, P=0), (32, 32, 0, 0)),
    (dict(M=1001, H=1024, N=1022, r=40, P=5, mix="runs"), (64, 64, 16, 16)),
    (dict(M=1001, H=1024, N=1021, r=8, P=5), (64, 64, 16, 16)),
    (dict(M=1000, H=1024, N=1021, P=0), (64, 64, 0, 0)),
    (dict(M=700, H=128, N=3001, r=40, P=6), (64, 256, 16, 16)),
    (dict(M=900, H=64, N=3333, r=16, P=30), (64, 256, 16, 16)),
    (dict(M=3000, H=320, N=2049, P=0), (64, 256, 0, 0)),
    (dict(M=1900, H=2048, N=4090, r=16, P=40), (128, 256, 16, 16)),
    (dict(M=2001, H=512, N=4093, r=24, P=6, mix="runs"), (128, 256, 16, 16)),
    (dict(M=3500, H=1024, N=2302, r=72, P=9, mix="runs"), (128, 256, 32, 32)),
    (dict(M=2001, H=1024, N=4093, P=0), (128, 256, 0, 0)),
    (dict(M=2000, H=192, N=7168, r=24, P=5), (256, 256, 16, 16)),
    (dict(M=2001, H=1024, N=7167, r=24, P=6, mix="runs"), (256, 256, 16, 16)),
    (dict(M=8191, H=1024, N=2045, r=16, P=33), (256, 256, 32, 16)),
    (dict(M=8191, H=1024, N=2048, r=24, P=3, mix="runs"), (256, 256, 32, 32)),
    (dict(M=8192, H=1024, N=2046, r=40, P=7), (256, 256, 32, 64)),
    (dict(M=4001, H=1024, N=4093, P=0), (256, 256, 0, 0)),
    # t's tiles for long batches beside short projections
    (dict(M=8200, H=128, N=64, r=64, P=3), (64, 64, 32, 64)),
    (dict(M=8200, H=128, N=66, r=24, P=300), (16, 16, 32, 32)),
    (dict(M=8200, H=128, N=64, r=16, P=3, mix="runs"), (16, 16, 32, 16)),
    (dict(M=20, H=128, N=72, r=40, P=3, dtype="f32"), (16, 16, 16, 16)),
    (dict(M=333, H=256, N=1001, r=40, P=5, dtype="f32"), (32, 32, 16, 32)),
    (dict(M=500, H=256, N=257, r=16, P=5, dtype="f32"), (32, 32, 16, 16)),
    (dict(M=1000, H=128, N=515, r=40, P=3, dtype="f32"), (64, 64, 16, 16)),
    (dict(M=700, H=128, N=700, r=16, P=3, dtype="f32", mix="runs"), (64, 64, 16, 16)),
    (dict(M=8200, H=64, N=40, r=64, P=3, dtype="f32"), (64, 64, 32, 64)),
    (dict(M=8200, H=64, N=40, r=24, P=30, dtype="f32"), (64, 64, 32, 32)),
    (dict(M=8200, H=64, N=39, r=8, P=3, dtype="f32", mix="runs"), (64, 64, 32, 16)),
]
