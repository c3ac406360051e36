"""The 64-bit references of the training operators against differences of the
layer itself and against closed forms (CPU only)."""
import numpy as np
import pytest
import torch

import train_ref as ref


def test_philox_known_answers():
    # the published vectors of Philox 4x32-10 (counter, key -> block)
    def block(ctr, key):
        i = ctr[0] | ctr[1] << 32
        n = 4 * (i % 2 ** 12)  # the words of block i, when i is small
        assert i < 2 ** 12
        return ref.philox_words(n + 4, key[0] | key[1] << 32, ctr[2] | ctr[3] << 32)[n:].tolist()

    assert block((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_philox_is_uniform_and_depends_on_everything():
    a = ref.philox_words(1 << 16, 5, 7)
    assert abs(float(a.mean()) / 2 ** 32 - 0.5) < 4 / np.sqrt(12 * a.size)
    for bit in range(32):
        assert abs(float(((a >> np.uint64(bit)) & np.uint64(1)).mean()) - 0.5) < 4 * 0.5 / np.sqrt(a.size)
    for other in ((6, 7), (5 + 2 ** 32, 7), (5, 8), (5, 7 + 2 ** 32)):
        assert float((ref.philox_words(1 << 16, *other) == a).mean()) < 1e-3


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_the_chain_of_references_is_the_gradient(p):
    """Every reference in turn, as the operators are chained, against autograd of
    the layer and against its differences."""
    M, H, F, E, k, base, EL, S = 13, 8, 12, 6, 3, 1, 4, 2
    g = torch.Generator().manual_seed(3)
    f64 = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    ins = dict(x=f64(M, H), logits=f64(M, E), wg=f64(EL, F, H), wu=f64(EL, F, H), wd=f64(EL, H, F), residual=f64(M, H))
    dout = f64(M, H)
    idx = torch.sort(ins["logits"], dim=1, descending=True, stable=True).indices[:, :k]
    keep = torch.rand(M, H, generator=g) >= p if p else None
    loss = lambda d: (ref.layer(d["x"], d["logits"], d["wg"], d["wu"], d["wd"], idx, base, d["residual"], keep, p) * dout).sum()

    # as the framework lays it out
    seg = torch.full((M * k,), S * EL)
    for f, e in enumerate(idx.flatten().tolist()):
        if base <= e < base + EL:
            seg[f] = (f // k * S // M) * EL + e - base
    order = torch.sort(seg, stable=True).indices
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(torch.bincount(seg, minlength=S * EL + 1)[:S * EL], 0)])
    f2s = torch.empty_like(order)
    f2s[order] = torch.arange(M * k)
    f2s[f2s >= offsets[-1]] = -1
    xp = ins["x"][order // k]
    w = torch.softmax(torch.gather(ins["logits"], 1, idx), 1)
    gate, _, up, _ = ref.products(xp, ins["wg"], ins["wu"], offsets, False)
    h = gate * torch.sigmoid(gate) * up
    y = torch.zeros(M * k, H, dtype=torch.float64)
    for e, lo, hi in ref.segments(offsets, EL):
        y[lo:hi] = h[lo:hi] @ ins["wd"][e].T
    out, _ = ref.combine(y, w, f2s, keep, p, ins["residual"], False)
    assert torch.allclose((out * dout).sum(), loss(ins), rtol=1e-12)
    dy, _, dw, _ = ref.combine_backward(dout, y, w, f2s, keep, p, False)
    dgate, _, dup, _ = ref.rows1(dy, ins["wd"], gate, up, offsets, False)
    dxp, _ = ref.rows0(dgate, dup, ins["wg"], ins["wu"], offsets, False)
    mine = dict(x=ref.dispatch_backward(dxp, f2s, M, k, None, False)[0], logits=ref.route_backward(idx, w, dw, E)[0],
                wg=ref.weights(dgate, xp, offsets, EL, False)[0], wu=ref.weights(dup, xp, offsets, EL, False)[0],
                wd=ref.weights(dy, h, offsets, EL, False)[0], residual=dout)

    leaves = {n: v.clone().requires_grad_() for n, v in ins.items()}
    loss(leaves).backward()
    for n, v in leaves.items():
        assert torch.allclose(mine[n], v.grad, rtol=1e-9, atol=1e-9), n
        way = f64(*v.shape)
        step = 1e-5
        diff = (loss(dict(ins, **{n: ins[n] + step * way})) - loss(dict(ins, **{n: ins[n] - step * way}))) / (2 * step)
        # third derivatives of the softmax and the SwiGLU are of order 1 to 100 here: step^2 of them
        assert abs(float(diff) - float((mine[n] * way).sum())) < 1e-6 * (1 + abs(float(diff))), n
