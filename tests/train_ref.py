"""Plain 64-bit references of the training operators (moe_combine_dropout,
moe_combine_backward, moe_dispatch_backward, moe_route_backward,
moe_grouped_gemm_aux, moe_grouped_gemm_backward,
moe_grouped_gemm_backward_weights), each with element-wise error bounds
derived from the arithmetic.  torch float64 on whatever device the inputs
are; nothing here is shared with the library.

Bounds.  u = 2^-24 is the largest relative error of one f32 rounding.  A sum
of n terms accumulated in f32 in any order is off by at most n u sum|terms| to
first order; products of bf16 values are exact in f32, products of f32 values
round once more, and the matrix cores may truncate where an f32 addition
rounds, so a product's sum counts (2 n + 1) u.  A cast to bf16 is off by at
most 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np
import torch

from serving_ref import BF16, U


def cast(value, bound, bf16):
    return (value, bound + BF16 * (value.abs() + bound)) if bf16 else (value, bound)


def philox_words(n, seed, offset):
    """Words of elements 0 .. n - 1 (n a multiple of 4): Philox 4x32-10, block i =
    element / 4 with key {seed low, high} and counter {i low, high, offset low,
    high}; unsigned 64-bit numpy."""
    u, low, up = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    i = np.arange(n // 4, dtype=np.uint64)
    c = [i & low, i >> up, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> up) ^ c[1] ^ u(k[0]), b & low, (a >> up) ^ c[3] ^ u(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).reshape(-1)


def mask(M, H, p, rng, device):
    """The kept elements [M, H] under dropout p with rng {seed, offset}."""
    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    keep = philox_words(M * H, seed, offset) >= np.uint64(int(p * 2.0 ** 32))
    return torch.from_numpy(keep.reshape(M, H)).to(device)


def _rows(f2s, M, k):
    f = f2s.long().view(M, k)
    return f, f >= 0


def combine(y, w, f2s, keep, p, residual, bf16):
    """(out, bound); keep: the kept elements, or None."""
    M, k = w.shape
    f, here = _rows(f2s, M, k)
    acc = torch.zeros(M, y.shape[1], dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(acc)
    for j in range(k):
        t = torch.nonzero(here[:, j]).flatten()
        v = w[t, j:j + 1].double() * y[f[t, j]].double()
        acc[t] += v
        mag[t] += v.abs()
    bound = (k + 1) * U * mag
    if keep is not None:
        s = 1.0 / (1.0 - p)
        # the scale's own rounding and the product's
        acc, bound = torch.where(keep, acc * s, 0.0), torch.where(keep, s * (bound + 2 * U * mag), 0.0)
    if residual is not None:
        acc = acc + residual.double()
        bound = bound + U * (acc.abs() + bound)
    return cast(acc, bound, bf16)


def combine_backward(dout, y, w, f2s, keep, p, bf16):
    """(dy, its bound, dw, its bound); rows of dy that no pair has are NaN."""
    M, k = w.shape
    H = y.shape[1]
    f, here = _rows(f2s, M, k)
    g = dout.double()
    if keep is not None:
        g = torch.where(keep, g / (1.0 - p), 0.0)
    dy = torch.full((M * k, H), float("nan"), dtype=torch.float64, device=y.device)
    by = torch.zeros_like(dy)
    dw, bw = torch.zeros(M, k, dtype=torch.float64, device=y.device), torch.zeros(M, k, dtype=torch.float64, device=y.device)
    for j in range(k):
        t = torch.nonzero(here[:, j]).flatten()
        dy[f[t, j]] = w[t, j:j + 1].double() * g[t]
        terms = g[t] * y[f[t, j]].double()
        if keep is not None:
            terms = torch.where(keep[t], terms, 0.0)  # what is dropped adds nothing, whatever y holds
        dw[t, j] = terms.sum(1)
        bw[t, j] = (H + 3) * U * terms.abs().sum(1)  # H terms, the scale twice, a product each
    by = 3 * U * dy.abs()
    dy, by = cast(dy, by, bf16)
    return dy, by, dw, bw


def dispatch_backward(dxp, f2s, M, k, residual, bf16):
    f, here = _rows(f2s, M, k)
    acc = torch.zeros(M, dxp.shape[1], dtype=torch.float64, device=dxp.device)
    mag = torch.zeros_like(acc)
    for j in range(k):
        t = torch.nonzero(here[:, j]).flatten()
        acc[t] += dxp[f[t, j]].double()
        mag[t] += dxp[f[t, j]].double().abs()
    bound = (k - 1) * U * mag
    if residual is not None:
        acc = acc + residual.double()
        bound = bound + U * (acc.abs() + bound)
    return cast(acc, bound, bf16)


def route_backward(idx, w, dw, E):
    M, k = idx.shape
    w, dw = w.double(), dw.double()
    mean, mag = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    v = w * (dw - mean)
    # the mean's k products and sums, the difference, the product, sums of equal slots
    b = w.abs() * ((k + 1) * U * mag + U * (dw - mean).abs()) + (k + 1) * U * v.abs()
    here = (idx >= 0) & (idx < E)  # an index that is no expert writes nothing
    at, out = torch.where(here, idx, 0).long(), torch.zeros(M, E, dtype=torch.float64, device=idx.device)
    return out.scatter_add(1, at, torch.where(here, v, 0.0)), out.scatter_add(1, at, torch.where(here, b, 0.0))


# ------------------------------------------------------- experts' products ---


def segments(offsets, EL):
    """(weight slot, first row, end) of the segments that hold rows."""
    cuts = offsets.tolist()
    return [(g % EL, lo, hi) for g, (lo, hi) in enumerate(zip(cuts, cuts[1:])) if hi > lo]


def _matmul(a, b):
    """a b and the bound of an f32 sum over its terms."""
    a, b = a.double(), b.double()
    return a @ b, (2 * a.shape[1] + 1) * U * (a.abs() @ b.abs())


def _empty(R, n, dev, count=1):
    return [torch.full((R, n), float("nan"), dtype=torch.float64, device=dev) for _ in range(2 * count)]


def products(xp, wg, wu, offsets, bf16):
    """gate, its bound, up, its bound (rows of no segment NaN)."""
    o = _empty(xp.shape[0], wg.shape[1], xp.device, 2)
    for e, lo, hi in segments(offsets, wg.shape[0]):
        for i, w in enumerate((wg, wu)):
            o[2 * i][lo:hi], o[2 * i + 1][lo:hi] = cast(*_matmul(xp[lo:hi], w[e].T), bf16)
    return o


def hact(xp, wg, wu, offsets, bf16=False):
    """silu(gate) up of the f32 products, and its bound: |silu'| <= 1.1; the exponential, the division and the products
    8 u; in bf16 |gate| u more, as the argument of the exponential is a rounded product (gate / ln 2)."""
    g, bg, u, bu = products(xp, wg, wu, offsets, False)
    silu = g * torch.sigmoid(g)
    h = silu * u
    return cast(h, 1.1 * bg * (u.abs() + bu) + silu.abs() * bu + (8 + (g.abs() if bf16 else 0)) * U * h.abs(), bf16)


def rows1(dy, wd, gate, up, offsets, bf16):
    """dgate, its bound, dup, its bound."""
    o = _empty(gate.shape[0], gate.shape[1], dy.device, 2)
    for e, lo, hi in segments(offsets, wd.shape[0]):
        dh, bh = _matmul(dy[lo:hi], wd[e])
        g, u = gate[lo:hi].double(), up[lo:hi].double()
        s, c = torch.sigmoid(g), torch.sigmoid(-g)
        dsilu, silu = s + g * s * c, g * s
        # s from an exponential whose argument rounds (|g| u), then the exponential, a sum and a division (at most
        # 4 u in all): |ds| <= s c (|g| + 4) u + u s.  In g s that is multiplied by |g|, in s (1 + g (1 - s)) by at
        # most 1 + 2 |g|, with a few roundings more: 16 u (1 + |g|)^2 covers both.
        es = 16 * U * (1 + g.abs()) ** 2
        dg, du = dh * u * dsilu, dh * silu
        bg = u.abs() * (bh * dsilu.abs() + (dh.abs() + bh) * es) + 4 * U * dg.abs()
        bu = bh * silu.abs() + (dh.abs() + bh) * es + 4 * U * du.abs()
        o[0][lo:hi], o[1][lo:hi] = cast(dg, bg, bf16)
        o[2][lo:hi], o[3][lo:hi] = cast(du, bu, bf16)
    return o


def rows0(dg, du, wg, wu, offsets, bf16):
    o = _empty(dg.shape[0], wg.shape[2], dg.device)
    for e, lo, hi in segments(offsets, wg.shape[0]):
        o[0][lo:hi], o[1][lo:hi] = cast(*_matmul(torch.cat([dg[lo:hi], du[lo:hi]], 1), torch.cat([wg[e], wu[e]], 0)), bf16)
    return o


def weights(d, a, offsets, EL, bf16, start=None):
    """dW [EL, columns of d, columns of a] and its bound; start: what it is added to."""
    out = torch.zeros(EL, d.shape[1], a.shape[1], dtype=torch.float64, device=d.device)
    bound, parts = torch.zeros_like(out), {}
    for e, lo, hi in segments(offsets, EL):
        parts.setdefault(e, []).append(torch.arange(lo, hi, device=d.device))
    for e, r in parts.items():
        r = torch.cat(r)
        out[e], bound[e] = _matmul(d[r].T, a[r])
    if start is not None:
        out = out + start.double()
        bound = bound + U * (out.abs() + bound)
    return cast(out, bound, bf16)


# ---------------------------------------------------------- the whole layer ---


def layer(x, logits, wg, wu, wd, idx, base, residual, keep, p):
    """The layer's output in float64 as a function of its inputs, for the experts
    idx [M, k] that the router chose (held: base .. base + EL): differentiable."""
    M, k = idx.shape
    EL = wg.shape[0]
    w = torch.softmax(torch.gather(logits, 1, idx.long()), 1)
    out = torch.zeros_like(x)
    for e in range(EL):
        share = torch.where(idx == e + base, w, torch.zeros_like(w)).sum(1, keepdim=True)
        g, u = x @ wg[e].T, x @ wu[e].T
        out = out + share * ((g * torch.sigmoid(g) * u) @ wd[e].T)
    if keep is not None:
        out = torch.where(keep, out / (1.0 - p), torch.zeros_like(out))
    return out if residual is None else out + residual
