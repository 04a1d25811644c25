"""GPU: ends of the block-scaled fp8 GEMM's argument ranges."""
import pytest
import torch

from helpers import SENTINEL, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.mark.parametrize("M", [1, 40, 70, 300])
@pytest.mark.parametrize("ld", [0, -1, 1 << 40, -(1 << 62)])
def test_no_k_gives_zeros_whatever_the_unused_operands_are(gmi, M, ld):
    # with K = 0 there is nothing to read: NULL operands and any leading dimension, up to ones that as byte counts
    # would pass 2^31
    N, G = 72, 3
    off = torch.tensor([0, M // 2, M // 2, M], dtype=torch.int32, device=dev())
    work = torch.empty(gmi.lib().gmi_gemm_f8_block_grouped_workspace_bytes(G), dtype=torch.uint8, device=dev())
    for grouped in (False, True):
        Y = torch.full((M, N + 8), SENTINEL, dtype=torch.int16, device=dev())
        st = torch.cuda.current_stream().cuda_stream
        if grouped:
            got = gmi.lib().gmi_gemm_f8_block_grouped(G, off.data_ptr(), M, N, 0, None, ld, None, ld, None, ld,
                                                      abs(ld) // 16 * 16, None, ld, abs(ld), Y.data_ptr(), N + 8,
                                                      work.data_ptr(), work.numel(), st)
        else:
            got = gmi.lib().gmi_gemm_f8_block(M, N, 0, None, ld, None, ld, None, ld, None, ld, Y.data_ptr(), N + 8, None,
                                              0, st)
        torch.cuda.synchronize()
        assert got == gmi.GMI_OK
        assert (Y[:, :N] == 0).all() and (Y[:, N:] == SENTINEL).all()
