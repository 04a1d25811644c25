"""The workspace of the adapters' product: what it is asked for, and that this is what is used."""
import pytest
import torch

from helpers import dev
from test_lora import case, check, up


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    if not g.LIB_PATH.exists():
        from grouped_mixed_input_amd import build

        build.build()
    g.lib()
    return g


# runs of K whose sums a call may hold at most: of 256 k, 16 up to 511 rows and up to rank 16, else eight, and from 512
# rows on 256 over all tiles of 64 rows
@pytest.mark.parametrize("M,K,rank,runs", [(1, 8, 8, 1), (511, 8192, 128, 16), (511, 2056, 64, 8), (512, 8192, 16, 16),
                                           (512, 8192, 24, 8), (1000, 8192, 128, 8), (2048, 1 << 20, 64, 8),
                                           (8192, 8192, 128, 2), (8192, 8192, 16, 2), (1 << 20, 8192, 64, 1)])
def test_lora_workspace_holds_the_runs_that_can_be(gmi, M, K, rank, runs):
    assert gmi.lib().gmi_gemm_lora_workspace_bytes(M, 256, K, rank) == runs * M * rank * 4


@pytest.mark.gpu
@pytest.mark.parametrize("M,rank", [(512, 16), (512, 24), (1000, 64), (4096, 128), (40000, 64)])
def test_lora_sums_are_the_workspace(gmi, M, rank):
    # no byte behind the size that is asked for is touched
    X, A, B, index, scales, base = case(M, 72, 4096, rank, 4, torch.bfloat16, run=100)
    d = up(X, A, B, index, scales, base)
    need = gmi.lib().gmi_gemm_lora_workspace_bytes(M, 72, 4096, rank)
    ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device=dev())
    got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], workspace=ws[:need])
    assert (ws[need:] == 0x5a).all()
    check(got, X, A, B, index, scales, base)
