"""GPU: roundings of the fp8 mixture-of-experts calls where one step too many shows.

The norm's codes: with h = 1 everywhere, eps = 0 and power-of-two sums, v is the weight itself.  Each block's largest
value is 448 s with s a small odd multiple of a power of two, so s is exact, and the others are s times a midpoint of two
fp8 codes: v / s is that midpoint and goes to the even code.  A reciprocal's rounding on the way moves it to either side."""
import pytest
import torch

import moe_ref as ref
from helpers import dev


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.mark.gpu
def test_norm_codes_are_of_the_quotient(gmi):
    odd = range(1, 67, 2)
    w = torch.zeros(len(odd), 128)
    mids = torch.arange(17, 32, 2) / 16.0  # midpoints of neighbouring codes in [1, 2)
    for i, m in enumerate(odd):
        s = m * 2.0 ** -6
        w[i, 0] = 448.0 * s
        w[i, 1:105] = (mids[:, None] * torch.pow(2.0, torch.arange(-5.0, 8.0)[None])).reshape(-1) * s
    want = torch.tensor([m * 2.0 ** -6 for m in odd])
    t = w.double() / want.double()[:, None]
    w = w.reshape(-1)
    assert torch.equal(w.half().float(), w)
    x = torch.ones(3, w.numel(), dtype=torch.float16)
    q, s = gmi.rmsnorm_quant(x.to(dev()), w.half().to(dev()), eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), want.expand(3, -1))
    codes = t.float().reshape(-1).to(ref.F8).float()  # exact quotients, nearest even
    for row in q.cpu().float():
        bad = (row != codes).nonzero().flatten().tolist()
        assert not bad, f"{len(bad)} codes are not e4m3(v / s), first at {bad[0]}"
