"""The norm's backward without the gradient of its weight."""
import pytest
import torch

import moe_ref as ref
from helpers import dev


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def test_a_given_dweight_is_refused(gmi):
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="weight_grad"):
        gmi.rmsnorm_bwd(x, x, w, dweight=torch.zeros(256), weight_grad=False)
    with pytest.raises(ValueError, match="device"):
        gmi.rmsnorm_bwd(x, x, w, weight_grad=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 8), (333, 2000), (2100, 2048), (9, 16384)])
def test_same_dh_and_no_workspace(gmi, dtype, rows, K):
    gen = torch.Generator().manual_seed(rows + K)
    h, dy, dres = (torch.randn(rows, K, generator=gen).to(dtype).to(dev()) for _ in range(3))
    w = (1 + 0.2 * torch.randn(K, generator=gen)).to(dtype).to(dev())
    want, _ = gmi.rmsnorm_bwd(dy, h, w, dres=dres)
    none = torch.empty(0, dtype=torch.uint8, device=dev())
    dh, dw = gmi.rmsnorm_bwd(dy, h, w, dres=dres, workspace=none, weight_grad=False)
    again, _ = gmi.rmsnorm_bwd(dy, h, w, dres=dres, weight_grad=False)
    torch.cuda.synchronize()
    assert dw is None and torch.equal(dh, want) and torch.equal(again, want)
    rdh, _, mag, _ = ref.norm_bwd(dy.cpu(), h.cpu(), w.cpu(), dres.cpu(), 1e-6)
    hs, tiny = ref.half_step(dtype), torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert ((dh.cpu().double() - rdh).abs() <= hs * rdh.abs() + 2e-5 * mag + tiny).all()


@pytest.mark.gpu
def test_no_rows(gmi):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=dev()), torch.ones(64, dtype=torch.bfloat16, device=dev())
    dh, dw = gmi.rmsnorm_bwd(x, x, w, weight_grad=False)
    assert dh.shape == (0, 64) and dw is None
