"""GPU: the gated activation and its gradient over more blocks than one launch takes (2^27): what the second launch writes,
and what it leaves."""
import pytest
import torch

import rows_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
ROWS = (1 << 27) + 300  # one block each with N = 8; the second launch begins 300 rows before the end


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.fixture(scope="module")
def data():
    """a and dact, zeros but for the last 400 rows, of which the last 100 are not in use."""
    gen = torch.Generator().manual_seed(1)
    a = torch.zeros(ROWS, 16, dtype=torch.bfloat16, device=dev())
    dact = torch.zeros(ROWS, 8, dtype=torch.bfloat16, device=dev())
    a[-400:] = torch.randn(400, 16, generator=gen).to(torch.bfloat16).to(dev())
    dact[-400:] = torch.randn(400, 8, generator=gen).to(torch.bfloat16).to(dev())
    return a, dact, torch.tensor([ROWS - 100], dtype=torch.int32, device=dev())


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_gate_codes(gmi, data):
    a, _, live = data
    q = torch.full((ROWS, 8), 0x55, dtype=torch.uint8, device=dev())
    s = torch.full((ROWS, 1), 7.0, device=dev())
    gmi.swiglu_quant(a, live=live, q=q.view(ref.F8), scales=s)
    wq, ws = gmi.swiglu_quant(a[-400:-100].clone())
    assert same(q[-400:-100], wq) and same(s[-400:-100], ws)
    assert (q[-100:] == 0x55).all() and (s[-100:] == 7.0).all()
    assert not q[:-400].any() and int((s[:-400] != ref.TINY / 448.0).sum()) == 0


def test_gate_gradient_codes(gmi, data):
    a, dact, live = data
    q = torch.full((ROWS, 16), 0x55, dtype=torch.uint8, device=dev())
    s = torch.full((ROWS, 1), 7.0, device=dev())
    gmi.swiglu_bwd(dact, a, live=live, da=q.view(ref.F8), scales=s, quantize=True)
    wq, ws = gmi.swiglu_bwd(dact[-400:-100].clone(), a[-400:-100].clone(), quantize=True)
    assert bool(wq.view(torch.uint8).any()) and same(q[-400:-100], wq) and same(s[-400:-100], ws)
    assert (q[-100:] == 0x55).all() and (s[-100:] == 7.0).all()
    assert not q[:-400].any() and int((s[:-400] != ref.TINY / 448.0).sum()) == 0


def test_gate_gradient_in_place(gmi, data):  # last: it writes over a
    a, dact, live = data
    old = a[-400:].clone()
    want = gmi.swiglu_bwd(dact[-400:-100].clone(), old[:300].clone())
    wide = ref.swiglu_bwd(dact[-400:-100].cpu(), old[:300].cpu())
    assert ((want.cpu().double() - wide).abs() <= 2.0 ** -8 * wide.abs() + 2.0 ** -18).all()
    assert gmi.swiglu_bwd(dact, a, live=live, da=a) is a
    assert same(a[-400:-100], want) and not same(a[-400:-100], old[:300])
    assert same(a[-100:], old[300:]) and not a[:-400].any()
