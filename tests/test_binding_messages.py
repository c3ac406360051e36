"""What the binding says of a tensor that is missing: its name (CPU only)."""
import pytest
import torch

import combine_topk_gate_amd as moe
from test_serving_abi import INV, on_gpu
from test_train_abi import binding_calls

# the tensor by whose GPU each call goes
FIRST = {"combine": "y", "combine_backward": "dout", "dispatch_backward": "dx_perm", "route_backward": "topk_idx", "aux": "a",
         "rows1": "d0", "rows0": "d0", "weights1": "a", "weights0": "a"}


@pytest.mark.parametrize("name", list(FIRST))
def test_a_missing_tensor_is_named(name):
    call, ok = binding_calls()[name]
    with pytest.raises(moe.MoeError, match=rf": {FIRST[name]} is missing") as ex:
        call(**dict(ok, **{FIRST[name]: None}))
    assert ex.value.status == INV


def test_serving_calls_still_name_x():
    q = moe.adapter_problem(4, 64, 64, 8, 0)
    with pytest.raises(moe.MoeError, match="x is missing"):
        moe.moe_adapter_linear(q, None, on_gpu(64, 64), None, None, None, None, None, on_gpu(4, 64, dtype=torch.float32), None, stream=0)
    p = moe.problem(4, 64, 64, 8, 2)
    with pytest.raises(moe.MoeError, match="x is missing"):
        moe.moe_layer_decode(p, None, on_gpu(4, 8, dtype=torch.float32), None, None, None, None, on_gpu(4, 64), None, stream=0)
