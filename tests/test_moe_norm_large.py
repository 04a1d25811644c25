"""GPU: the norm and its backward over tensors large enough that inputs pass the caches (2^25 elements and more)."""
import pytest
import torch

import moe_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
F32 = 2e-5  # fp32 row sums: a few dozen roundings of 2^-24


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(8195, 4096), (65541, 520), (4099, 8200)])
def test_norm_and_backward(gmi, dtype, rows, K):
    assert rows * K >= 1 << 25
    gen = torch.Generator().manual_seed(rows)
    x, res, dy, dres = (torch.randn(rows, K, generator=gen).to(dtype) for _ in range(4))
    w = (1 + 0.2 * torch.randn(K, generator=gen)).to(dtype)
    xd, rd, dyd, drd, wd = (t.to(dev()) for t in (x, res, dy, dres, w))
    h, y = torch.empty_like(xd), torch.empty_like(xd)
    q, s = gmi.rmsnorm_quant(xd, wd, residual=rd, eps=1e-5, h=h, y=y)
    dh, dw = gmi.rmsnorm_bwd(dyd, h, wd, dres=drd, eps=1e-5)
    torch.cuda.synchronize()
    h, y, q, s, dh, dw = h.cpu(), y.cpu(), q.cpu().view(torch.uint8), s.cpu(), dh.cpu().double(), dw.cpu().double()
    hs, tiny = ref.half_step(dtype), torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    at = torch.cat([torch.arange(0, rows, 97), torch.arange(rows - 5, rows)])
    rh, rv, rs, rt = ref.norm(x[at], w, res[at], 1e-5)
    assert ((h[at].double() - rh).abs() <= (hs + 2.0 ** -23) * rh.abs() + tiny).all()
    assert ((y[at].double() - rv).abs() <= (hs + F32) * rv.abs() + tiny).all()
    assert ((s[at].double() - rs).abs() <= F32 * rs).all()
    assert ((q[at].view(ref.F8).double() - rt).abs() <= (2.0 ** -4 + 2 * F32) * rt.abs() + 2.0 ** -10).all()
    rdh, _, mag, _ = ref.norm_bwd(dy[at], h[at], w, dres[at], 1e-5)
    assert ((dh[at] - rdh).abs() <= hs * rdh.abs() + F32 * mag + tiny).all()
    rdw, wmag = torch.zeros(K, dtype=torch.float64), torch.zeros(K, dtype=torch.float64)
    for i in range(0, rows, 4096):
        _, a, _, b = ref.norm_bwd(dy[i:i + 4096], h[i:i + 4096], w, None, 1e-5)
        rdw, wmag = rdw + a, wmag + b
    # the rows that a team adds one after another (rows over 512 workgroups of 1 to 4 teams), then 512 partials over 32
    # threads: fewer than 160 roundings of 2^-24, and the terms' own
    assert ((dw - rdw).abs() <= (F32 + 160 * 2.0 ** -24) * wmag).all()
