"""Which tiles the experts' gradients take, as far as their workspace shows it on
the host (CPU only): 0 where no reduction is cut into parts."""
import os

import pytest

import combine_topk_gate_amd as moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from combine_topk_gate_amd import build
        build.build()
    return moe.load_library()


def need(*args, **kw):
    return moe.moe_workspace_bytes(moe.problem(*args, **kw), moe.MOE_OP_GROUPED_GEMM_BACKWARD)


# M, H, F, E, held, k
SMALL = [(512, 1024, 512, 128, 16, 8), (512, 2048, 1408, 16, 2, 2), (4096, 256, 512, 64, 8, 8), (512, 2048, 1408, 16, 1, 2)]
LONG = [(4096, 2048, 1408, 128, 16, 2), (512, 4096, 2048, 64, 8, 8), (4096, 4096, 2048, 16, 2, 2)]


@pytest.mark.parametrize("M,H,F,E,held,k", SMALL)
def test_a_small_share_takes_small_tiles(M, H, F, E, held, k):
    # the rows that an even routing keeps, of experts all held, take tiles that are not cut; so does the share
    assert need(M * k * held // E, H, F, held, 1) == 0
    assert need(M, H, F, E, k, expert_base=E // 2, local_experts=held) == 0


@pytest.mark.parametrize("M,H,F,E,held,k", LONG)
def test_a_share_of_long_f32_products_is_cut_as_its_rows_are(M, H, F, E, held, k):
    assert need(M * k * held // E, H, F, held, 1, dtype="f32") > 0
    assert need(M, H, F, E, k, dtype="f32", expert_base=E // 2, local_experts=held) > 0


@pytest.mark.parametrize("M,H,F,E,S", [(4096, 256, 512, 16, 32), (2048, 512, 512, 16, 32)])
def test_short_segments_of_many_blocks_count_a_step_each(M, H, F, E, S):
    # the rows alone are two to four steps of 64 an expert, its segments 32: a long reduction, which is cut
    assert need(M, H, F, E, 1) == 0
    assert need(M, H, F, E, 1, S) > 0
