"""The combine's and the dispatch's gradients in the forms that many slots take:
every group of slots (1, 2, 4, 8, 16) in the three row lengths, experts all held
and a share whose tokens hold some or none of their pairs, small and large rows
(other loads); and the kernels' mask where all words of seed and offset differ."""
import pytest
import torch

import combine_topk_gate_amd as moe
import serving_ref
import train_ref as ref
from test_gpu_train import DEV, act_of, check_norm, combine_inputs, gen, guarded, normal, rng_of

pytestmark = pytest.mark.gpu

FORMS = [dict(M=37, H=2112, E=32, k=8, held=4, base=9), dict(M=37, H=2112, E=32, k=8), dict(M=21, H=1152, E=40, k=16, held=5),
         dict(M=21, H=1152, E=40, k=16), dict(M=45, H=1600, E=24, k=11, held=6, base=3, S=2), dict(M=30, H=4096, E=16, k=3, held=2, base=14),
         dict(M=64, H=1088, E=9, k=7, S=3), dict(M=50, H=960, E=64, k=8, held=8, base=20), dict(M=50, H=1024, E=20, k=13),
         dict(M=70, H=128, E=40, k=16, held=6, base=30), dict(M=70, H=64, E=9, k=9)]
# 96 MiB of held f32 rows and more: loads of rows used once
LARGE = [dict(M=3000, H=1152, E=16, k=8), dict(M=14000, H=1152, E=32, k=8, held=8, base=11), dict(M=2100, H=832, E=32, k=16)]


@pytest.mark.parametrize("dtype,out,p", [("f32", "f32", 0.0), ("bf16", "bf16", 0.3), ("bf16", "f32", 0.0)])
@pytest.mark.parametrize("shape", FORMS + LARGE)
def test_many_slots(shape, dtype, out, p):
    print(f"[many slots] {shape} {dtype} {out} {p}", flush=True)
    prob, w, f2s, y = combine_inputs(**shape, dtype=dtype, seed=3)
    M, H, k = shape["M"], shape["H"], shape["k"]
    held = int((f2s.view(M, k) >= 0).any(1).sum())
    if shape.get("held") and M >= 37 and k <= 8:
        assert held < M  # some tokens hold no pair at all
    dout = normal(gen(4), M, H, dtype=act_of(out))
    rng = rng_of(0x299F31D0A4093822, 0x0370734413198A2E)
    keep = ref.mask(M, H, p, rng, DEV) if p else None
    drop = moe.dropout(p, rng) if p else None
    dy, i1 = guarded((M * k, H), act_of(dtype), fill=5.0)
    dw, i2 = guarded((M, k), torch.float32)
    moe.moe_combine_backward(prob, dout, y, w, f2s, drop, dy, dw)
    wy, by, ww, bw = ref.combine_backward(dout, y, w, f2s, keep, p, dtype == "bf16")
    rest = torch.isnan(wy)
    assert bool((dy[rest] == 5.0).all())
    serving_ref.check(dy[~rest], wy[~rest], by[~rest], (shape, "dy"))
    serving_ref.check(dw, ww, bw, (shape, "dw"))
    check_norm(dw, ww, H + 3, False, (shape, "dw"))
    res = normal(gen(8), M, H, dtype=act_of(dtype))
    dx, i3 = guarded((M, H), act_of(out))
    moe.moe_dispatch_backward(prob, y.to(act_of(dtype)), f2s, moe.epilogue(res, out), dx)
    serving_ref.check(dx, *ref.dispatch_backward(y.to(act_of(dtype)), f2s, M, k, res, out == "bf16"), (shape, "dx"))
    o, i4 = guarded((M, H), act_of(out))
    moe.moe_combine_dropout(prob, y, w, f2s, moe.epilogue(res, out), drop, o)
    serving_ref.check(o, *ref.combine(y, w, f2s, keep, p, res, out == "bf16"), (shape, "out"))
    for c in (i1, i2, i3, i4):
        c()
