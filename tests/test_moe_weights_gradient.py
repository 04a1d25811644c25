"""GPU: the gradient of the routing weights to the last bits of fp32."""
import pytest
import torch

from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.mark.parametrize("k,cols", [(1, 8), (3, 512), (8, 1024), (16, 520)])
@pytest.mark.parametrize("dtype,ed,ey", [(torch.bfloat16, 0, 0), (torch.bfloat16, -128, 110), (torch.float16, 0, 0),
                                         (torch.float16, -14, 2)])
def test_weights_gradient_of_two_terms(gmi, dtype, ed, ey, k, cols):
    # two neighbouring columns: the first product is an fp32 number, so their sum is rounded once, however far they
    # cancel, and also where dout is subnormal
    gen = torch.Generator().manual_seed(k + cols)
    T = 500
    y, dout = torch.zeros(T, k, cols), torch.zeros(T, cols)
    for t in range(T):
        c = 2 * int(torch.randint(0, cols // 2, (1,), generator=gen))
        dout[t, c:c + 2] = torch.randn(2, generator=gen)
        y[t, :, c] = torch.randn(k, generator=gen)
        y[t, :, c + 1] = torch.randn(k, generator=gen) * 2.0 ** -12
        if t % 2:  # the terms nearly cancel
            y[t, :, c + 1] = -y[t, :, c] * dout[t, c] / dout[t, c + 1]
    dout, y = (dout.double() * 2.0 ** ed).to(dtype), (y.double().clamp(-1e4, 1e4) * 2.0 ** ey).to(dtype)
    slots = torch.arange(T * k, dtype=torch.int32).view(T, k)
    _, dw = gmi.moe_unpermute_bwd(dout.to(dev()), slots.to(dev()), rows=y.view(T * k, cols).to(dev()), row_grad=False)
    want = (dout.double()[:, None] * y.double()).sum(2)
    assert torch.equal(dw.cpu(), want.float())
