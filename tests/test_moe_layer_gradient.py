"""GPU: the example layer's whole data gradient against float64 autograd on the decoded weights."""
import importlib.util
import pathlib

import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "moe_layer_f8.py"
    spec = importlib.util.spec_from_file_location("moe_layer_f8", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 256, 128, 8, 2), (96, 512, 192, 16, 4),
                                                            (700, 384, 256, 5, 3)])
def test_gradient_through_every_path(example, tokens, hidden, inner, experts, top):
    layer = example.Layer(hidden, inner, experts, top, seed=tokens)
    gen = torch.Generator().manual_seed(tokens + 2)
    x, res, dout, dh_out = (torch.randn(tokens, hidden, generator=gen).bfloat16() for _ in range(4))
    mask = torch.rand(tokens, generator=gen) > 0.1 if tokens > 1 else None
    dl = 0.3
    _, h, saved = layer.forward(x.cuda(), res.cuda(), None if mask is None else mask.cuda())
    args = dout.cuda(), torch.tensor([dl], device="cuda"), saved
    dh, dnorm, _ = layer.backward(*args, dh_out=dh_out.cuda(), through_experts=True)
    without, _, _ = layer.backward(*args, dh_out=dh_out.cuda())
    torch.cuda.synchronize()
    r = saved[3]
    idx = r.indices.cpu().long()
    live = idx >= 0
    up, down = (torch.stack([ref.spread(q[e].cpu(), s[e].cpu(), 128) for e in range(experts)])
                for q, s in (layer.up, layer.down))
    hh = h.cpu().double().requires_grad_(True)
    w = layer.norm.cpu().double().requires_grad_(True)
    v = w * hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-6)
    # the layer's own logits carry the values, v the derivative
    z = v @ layer.router.cpu().double().t()
    z = z + (saved[2].cpu().double() - z).detach()
    p = torch.softmax(z, 1)
    share = torch.where(live, p.gather(1, idx.clamp_min(0)), 0.0)
    share = share / share.sum(1, keepdim=True).clamp_min(1e-300)
    out = torch.zeros(tokens, hidden, dtype=torch.float64)
    for e in range(experts):
        t, i = ((idx == e) & live).nonzero(as_tuple=True)
        a = v[t] @ up[e].t()
        y = (torch.nn.functional.silu(a[:, :inner]) * a[:, inner:]) @ down[e].t()
        out = out.index_add(0, t, y * share[t, i][:, None])
    alive = live.any(1)
    loss = experts * (r.counts.cpu().double() / max(int(r.offsets[-1]), 1) * (p * alive[:, None]).sum(0)).sum() / max(
        int(r.live), 1)
    ((out * dout.double()).sum() + dl * loss + (hh * dh_out.double()).sum()).backward()
    # what comes through the layer, the part past the norm taken off: two products of fp8 operands (2^-4 of a value at
    # most, a few per cent of a sum of independent terms) on the way there and two on the way back, a tenth for each
    # way; bf16 everywhere else
    want, got, part = (g.cpu().double() - dh_out.double() for g in (hh.grad, dh, without))
    norm = want.pow(2).mean().sqrt()
    assert (got - want).pow(2).mean().sqrt() <= 0.2 * norm
    assert (part - want).pow(2).mean().sqrt() > 0.5 * norm, "the experts' path is the larger one"
    assert (dnorm.cpu().double() - w.grad).pow(2).mean().sqrt() <= 0.2 * w.grad.pow(2).mean().sqrt()
