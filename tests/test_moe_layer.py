"""GPU: the example layer (norm, router, experts, and back) against float64 on the decoded weights.

Each stage is held to the stage before it as the layer itself computed it, so a rounding is counted once; the
tolerances are those of the stages."""
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
def test_layer(example, tokens, hidden, inner, experts, top):
    layer = example.Layer(hidden, inner, experts, top, seed=tokens)
    gen = torch.Generator().manual_seed(tokens + 1)
    x, res, dout, dh_out = (torch.randn(tokens, hidden, generator=gen).bfloat16() for _ in range(4))
    mask = torch.rand(tokens, generator=gen) > 0.1 if tokens > 1 else None
    out, h, saved = layer.forward(x.cuda(), res.cuda(), None if mask is None else mask.cuda())
    _, y, logits, r, expert_out, _ = saved
    torch.cuda.synchronize()
    # routing of the layer's own logits
    want = ref.route(logits.cpu(), top, mask, True)
    assert (r.indices.cpu().numpy() == want["indices"]).all() and (r.slot_row.cpu().numpy() == want["slot_row"]).all()
    # experts: the float64 layer on decoded fp8 weights from the unquantised norm.  Errors: fp8 rounding of two
    # operands (2^-4 of a value at most, in sums of many independent terms: a tenth of the result's own size is ten
    # times what they leave), bf16 rounding of the first product.
    _, v, _, _ = ref.norm(x, layer.norm.cpu(), res, 1e-6)
    up, down = (torch.stack([ref.spread(q[e].cpu(), s[e].cpu(), 128) for e in range(experts)])
                for q, s in (layer.up, layer.down))
    idx = torch.from_numpy(want["indices"]).long()
    live = idx >= 0
    full = torch.zeros(tokens, top, hidden, dtype=torch.float64)
    for e in range(experts):
        t, i = ((idx == e) & live).nonzero(as_tuple=True)
        a = v[t] @ up[e].t()
        full[t, i] = (torch.nn.functional.silu(a[:, :inner]) * a[:, inner:]) @ down[e].t()
    err = (expert_out.cpu().double() - full).pow(2).mean().sqrt()
    assert err <= 0.1 * full.pow(2).mean().sqrt(), float(err)
    assert (expert_out[~live.cuda()] == 0).all()
    w = torch.from_numpy(want["weights"])
    mix = (expert_out.cpu().double() * w[..., None]).sum(1)
    mag = (expert_out.cpu().double() * w[..., None]).abs().sum(1)
    assert ((out.cpu().double() - mix).abs() <= 2.0 ** -8 * mix.abs() + 1e-4 * mag).all()

    # backward: routing weights, balance loss, norm
    dl = 0.3
    dh, dnorm, drouter = layer.backward(dout.cuda(), torch.tensor([dl], device="cuda"), saved, dh_out=dh_out.cuda())
    torch.cuda.synchronize()
    dw = (expert_out.cpu().double() * dout.double()[:, None]).sum(2)
    z = logits.cpu().double().requires_grad_(True)
    ref.route_objective(z, want, top, mask, True, dw, dl).backward()
    dlogits = torch.nan_to_num(z.grad)
    # bf16 gradients through two bf16 products: a few steps of 2^-8 of the magnitudes' sums
    got = drouter.cpu().double()
    exact, mag = dlogits.t() @ y.cpu().double(), dlogits.abs().t() @ y.cpu().double().abs()
    scale = dw.abs().amax() + dl * experts
    assert ((got - exact).abs() <= 2.0 ** -7 * mag + 2e-5 * scale * y.cpu().double().abs().sum(0)).all()
    dy = dlogits @ layer.router.cpu().double()
    rdh, rdw, hm, wm = ref.norm_bwd(dy, h.cpu(), layer.norm.cpu(), dh_out, 1e-6)
    dym = dlogits.abs() @ layer.router.cpu().double().abs() + 2e-5 * scale * layer.router.cpu().double().abs().sum(0)
    _, _, hm2, wm2 = ref.norm_bwd(dym, h.cpu().abs(), layer.norm.cpu().abs(), None, 1e-6)
    assert ((dh.cpu().double() - rdh).abs() <= 2.0 ** -8 * rdh.abs() + 2.0 ** -6 * hm2 + 2e-5 * hm).all()
    assert ((dnorm.cpu().double() - rdw).abs() <= 2.0 ** -6 * wm2 + 1e-4 * wm).all()
