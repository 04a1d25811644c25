"""GPU: roundings of the fp8 mixture-of-experts calls where one step too many shows.

The norm's codes: with h = 1 everywhere, eps = 0 and power-of-two sums, v is the weight itself.  Each block's largest
value is 448 s with s a small odd multiple of a power of two, so s is exact, and the others are s times a midpoint of two
fp8 codes: v / s is that midpoint and goes to the even code.  A reciprocal's rounding on the way moves it to either side.

The router's exponentials: logits are multiples of 2^-4 that fp32 subtracts exactly, so what is left, in units of
u = 2^-24: an exponential 2 u (one step of fp32), a sum of 16 values over 16 lanes 4 u (four exchanges) on top of
its terms' 2 u, a quotient 1 u: 9 u for a weight."""
import pytest
import torch

import moe_ref as ref
from helpers import dev

U = 2.0 ** -24


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


def _spread_logits(gen, T, E):
    return (torch.randn(T, E, generator=gen) * 160).round().clamp(-640, 640) / 16.0


@pytest.mark.gpu
@pytest.mark.parametrize("renorm", [False, True])
def test_route_weights_of_far_logits(gmi, renorm):
    T, E = 4096, 16
    x = _spread_logits(torch.Generator().manual_seed(40), T, E)
    got = gmi.moe_route(x.to(dev()), E, renormalize=renorm)
    torch.cuda.synchronize()
    p, order = torch.sort(torch.softmax(x.double(), 1), dim=1, descending=True, stable=True)
    w = got.weights.cpu().double()
    assert torch.equal(torch.gather(x, 1, got.indices.cpu().long()), torch.gather(x, 1, order))
    normal = p > 2.0 ** -120
    err = ((w - p).abs() / p)[normal]
    assert (err <= 9 * U).all(), f"largest error {float(err.max()) / U:.1f} u"
    assert (w[~normal] <= 2.0 ** -119).all()


@pytest.mark.gpu
def test_route_bwd_of_far_logits(gmi):
    # p, by a reciprocal of the sum: 2 + 6 + 1 + 1 = 10 u; sum of p dw: 10 + 1 (product) + 4 (exchanges) u of the sum of
    # magnitudes; difference 1 u; product with p 10 + 1: at most 27 u of p (|dw| + sum p |dw|)
    T, E = 4096, 16
    gen = torch.Generator().manual_seed(41)
    x = _spread_logits(gen, T, E)
    dw = torch.randn(T, E, generator=gen)
    r = gmi.moe_route(x.to(dev()), E, renormalize=False)
    d = gmi.moe_route_bwd(x.to(dev()), r.indices, r.weights, r.offsets, r.live, dw.to(dev()), torch.zeros(1, device=dev()),
                          renormalize=False).cpu().double()
    p = torch.softmax(x.double(), 1)
    g = torch.zeros(T, E, dtype=torch.float64).scatter_(1, r.indices.cpu().long(), dw.double())
    dot, mag = (p * g).sum(1, keepdim=True), (p * g.abs()).sum(1, keepdim=True)
    err, allowed = (d - p * (g - dot)).abs(), 27 * U * p * (g.abs() + mag) + 1e-36
    assert (err <= allowed).all(), f"largest error {float((err / allowed).max()) * 27:.1f} u"
