"""Offsets that do not fit the rows: the grouped GEMM keeps every access inside
the buffers, as the header says of device-resident inputs.  An end past the last
row counts as that row, a negative start as row 0."""
import pytest
import torch

import combine_topk_gate_amd as moe
from test_gpu_train import DEV, gen, guarded, normal

pytestmark = pytest.mark.gpu

M, H, F, E, k = 300, 192, 256, 4, 2
R = M * k


def inputs(dtype, S):
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    g = gen(S)
    d = dict(x=normal(g, R, H, dtype=act), h=normal(g, R, F, dtype=act), wg=normal(g, E, F, H, std=0.1, dtype=act),
             wu=normal(g, E, F, H, std=0.1, dtype=act), wd=normal(g, E, H, F, std=0.1, dtype=act))
    if dtype == "bf16_mxfp8":
        for n, cols in (("h", F), ("wd", F)):
            q = torch.empty(moe.mx_bytes(d[n].numel() // cols, cols), dtype=torch.uint8, device=DEV)
            moe.moe_quantize_mxfp8(d[n], q)
            d[n] = q
    return moe.problem(M, H, F, E, k, S, dtype), d


def run(p, d, offsets, dtype):
    """Both layers between guard zones; (Hact, Y) as bytes."""
    offsets = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if dtype == "bf16_mxfp8":
        h, i1 = guarded((moe.mx_bytes(R, F),), torch.uint8, fill=0)
    else:
        h, i1 = guarded((R, F), d["x"].dtype, fill=0.0)
    y, i2 = guarded((R, H), torch.float32, fill=0.0)
    ws = torch.empty(max(moe.moe_workspace_bytes(p, moe.MOE_OP_GROUPED_GEMM), 256), dtype=torch.uint8, device=DEV)
    moe.moe_grouped_gemm(p, 0, d["x"], d["wg"], d["wu"], offsets, h, ws)
    moe.moe_grouped_gemm(p, 1, d["h"], d["wd"], None, offsets, y, ws)
    torch.cuda.synchronize()
    i1()
    i2()
    return h, y


@pytest.mark.parametrize("S", [1, 2])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "bf16_mxfp8"])
def test_offsets_outside_the_rows_reach_nothing_else(dtype, S):
    p, d = inputs(dtype, S)
    cuts = [i * R // (S * E) for i in range(S * E)] + [R]
    want = run(p, d, cuts, dtype)
    for first, last in ((0, R + 1), (0, R + 5000), (-1, R), (-(2 ** 31), 2 ** 31 - 1)):
        print(f"[offsets] {dtype} S {S} first {first} last {last}", flush=True)
        got = run(p, d, [first] + cuts[1:-1] + [last], dtype)
        for a, b in zip(got, want):
            assert torch.equal(a, b), (first, last)
    # decreasing, past the rows in the middle: unspecified results, inside the buffers
    for i, v in ((1, R + 77), (2, -9), (3, 0)):
        print(f"[offsets] {dtype} S {S} offsets[{i}] {v}", flush=True)
        run(p, d, cuts[:i] + [v] + cuts[i + 1:], dtype)
