"""GPU: the adapters' product over runs long enough and parts of columns wide enough that every stage of its rings is used
again, after results have stood in it, against float64."""
import pytest
import torch

from helpers import dev
from test_lora import case, check, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


# 16 to 20 steps of 64 columns a workgroup, rings of three or four stages; whole waves of 16 rows (N a multiple of 64:
# their stores count among what a stage is waited for) and runs that end inside one
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [8, 16, 32, 56, 64, 128])
@pytest.mark.parametrize("M,N,run", [(4096, 4096, 512), (4096, 4104, 512), (2100, 8192, 150)])
def test_lora_rings_refilled(gmi, dtype, M, N, rank, run):
    X, A, B, index, scales, base = case(M, N, 128, rank, 5, dtype, run=run)
    d = up(X, A, B, index, scales, base)
    order = gmi.group_rows(d[3], 5).order
    got = gmi.gemm_lora(*d[:4], scales=d[4], order=order, base=d[5])
    check(got, X, A, B, index, scales, base)
    gmi.gemm_lora(*d[:4], scales=d[4], order=order, base=d[5], Y=d[5])
    assert torch.equal(d[5], got), "in the place of the base"
    check(gmi.gemm_lora(*d[:4], order=order), X, A, B, index, None, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_lora_long_sums(gmi, dtype):
    # 65 steps of K a workgroup, the last one partial
    X, A, B, index, scales, base = case(4096, 136, 16424, 48, 3, dtype, run=700)
    d = up(X, A, B, index, scales, base)
    check(gmi.gemm_lora(*d[:4], scales=d[4], base=d[5]), X, A, B, index, scales, base)
