"""GPU: expert routing and its backward against float64 (moe_ref.route).
Whole numbers are equal; weights, loss and gradients are fp32 sums of at most
1024 terms and exponentials of arguments up to 40 (their rounding, 40 * 2^-24,
enters the result): 2e-5 relative, and half a step of a 16-bit output."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
TOL = 2e-5


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def _logits(gen, T, E, dtype, ld=None, closed=0.0):
    x = 2.0 * torch.randn(T, ld or E, generator=gen)
    if closed:
        x[torch.rand(T, ld or E, generator=gen) < closed] = -float("inf")
        x[torch.rand(T, generator=gen) < 0.05] = -float("inf")
    return x.to(dtype)[:, :E]


def _check(got, want):
    for name in ("indices", "counts", "offsets", "slot_row", "row_slot"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert int(got.live) == want["live"]
    np.testing.assert_allclose(got.weights.cpu().numpy(), want["weights"], rtol=TOL, atol=1e-30)
    np.testing.assert_allclose(float(got.loss), want["loss"], rtol=TOL)


SIZES = [(1, 1, 1), (1, 4, 2), (3, 8, 8), (63, 60, 4), (64, 128, 8), (65, 16, 1), (129, 64, 6), (777, 60, 4),
         (300, 200, 16), (257, 256, 8), (70, 300, 5), (200, 512, 8), (130, 1024, 16), (17000, 12, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_route(gmi, dtype, T, E, k):
    gen = torch.Generator().manual_seed(T + E + k)
    x = _logits(gen, T, E, dtype, ld=E + 5)
    mask = torch.rand(T, generator=gen) > 0.1 if T > 2 else None
    for renorm in (False, True):
        got = gmi.moe_route(x.to(dev())[:, :E], k, mask=None if mask is None else mask.to(dev()), renormalize=renorm)
        _check(got, ref.route(x, k, mask, renorm))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_route_ties_and_closed_experts(gmi, dtype):
    gen = torch.Generator().manual_seed(9)
    x = torch.randint(-2, 3, (500, 40), generator=gen).float()  # many equal logits
    x[x == 0] = -0.0
    x[::3][x[::3] == 0] = 0.0
    x[torch.rand(500, 40, generator=gen) < 0.3] = -float("inf")
    x[::17] = -float("inf")  # no expert open
    x[5, 1:] = -float("inf")  # fewer than k open
    x[6] = torch.finfo(dtype).min  # the type's lowest value is an ordinary logit
    x = x.to(dtype)
    for renorm in (False, True):
        _check(gmi.moe_route(x.to(dev()), 6, renormalize=renorm), ref.route(x, 6, None, renorm))


def test_route_nothing_live(gmi):
    x = torch.zeros(70, 8)
    got = gmi.moe_route(x.to(dev()), 2, mask=torch.zeros(70, dtype=torch.uint8, device=dev()))
    assert (got.indices == -1).all() and (got.weights == 0).all() and (got.counts == 0).all()
    assert (got.offsets == 0).all() and (got.row_slot == -1).all() and (got.slot_row == -1).all()
    assert float(got.loss) == 0.0 and int(got.live) == 0
    got = gmi.moe_route(torch.empty(0, 8, device=dev()), 2)
    assert (got.counts == 0).all() and (got.offsets == 0).all() and float(got.loss) == 0.0 and int(got.live) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_not_a_number(gmi, dtype):
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(100, 20, generator=gen)
    x[3, 4] = float("nan")
    x[8] = float("nan")  # no logit above -infinity
    x[9, 0] = float("nan")
    x = x.to(dtype)
    mask = torch.ones(100, dtype=torch.bool)
    mask[9] = False
    for renorm in (False, True):
        got = gmi.moe_route(x.to(dev()), 3, mask=mask.to(dev()), renormalize=renorm)
        want = ref.route(x, 3, mask, renorm)
        assert np.array_equal(got.indices.cpu().numpy(), want["indices"])
        assert np.array_equal(got.slot_row.cpu().numpy(), want["slot_row"])
        w = got.weights.cpu().numpy()
        assert np.isnan(w[3]).all() and np.isfinite(np.delete(w, 3, 0)).all() and np.isnan(float(got.loss))
    mask[3] = False  # masked out, the value does not matter
    got = gmi.moe_route(x.to(dev()), 3, mask=mask.to(dev()))
    assert np.isfinite(float(got.loss)) and torch.isfinite(got.weights).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (63, 60, 4), (129, 64, 6), (777, 60, 4), (300, 200, 16), (200, 512, 8),
                                   (130, 1024, 16), (17000, 12, 3)])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd(gmi, dtype, T, E, k, renorm):
    gen = torch.Generator().manual_seed(T + 3 * E + k)
    x = _logits(gen, T, E, dtype, ld=E + 3, closed=0.2 if T > 2 else 0.0)
    mask = torch.rand(T, generator=gen) > 0.1 if T > 2 else None
    dw, dl = torch.randn(T, k, generator=gen), 0.5 * T
    xd, md = x.to(dev())[:, :E], None if mask is None else mask.to(dev())
    r = gmi.moe_route(xd, k, mask=md, renormalize=renorm)
    buf = torch.full((T, E + 2), 9.0, dtype=dtype, device=dev())
    gmi.moe_route_bwd(xd, r.indices, r.weights, r.offsets, r.live, dw.to(dev()),
                      torch.tensor([dl], dtype=torch.float32, device=dev()), mask=md, renormalize=renorm,
                      dlogits=buf[:, :E])
    torch.cuda.synchronize()
    want = ref.route(x, k, mask, renorm)
    z = x.double().requires_grad_(True)
    ref.route_objective(z, want, k, mask, renorm, dw, dl).backward()
    g = torch.nan_to_num(z.grad)  # closed experts: 0
    # the gradient is a difference of terms up to |dw| + E f dl / live: their rounding is absolute
    f = torch.from_numpy(want["counts"].astype(np.float64)) / max(int(want["offsets"][-1]), 1)
    scale = dw.abs().double().amax(1, keepdim=True) + float(E * f.max()) * dl / max(want["live"], 1)
    hs = 0.0 if dtype == torch.float32 else ref.half_step(dtype)
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = (buf[:, :E].cpu().double() - g).abs()
    assert (err <= hs * g.abs() + TOL * scale + tiny).all(), float((err - hs * g.abs() - TOL * scale).max())
    assert (buf[:, E:] == 9.0).all(), "padding columns written"


@pytest.mark.parametrize("renorm", [False, True])
def test_route_bwd_against_differences(gmi, renorm):
    gen = torch.Generator().manual_seed(21)
    T, E, k = 40, 12, 3
    x = torch.randn(T, E, generator=gen)
    dw, dl = torch.randn(T, k, generator=gen), 3.0
    r = gmi.moe_route(x.to(dev()), k, renormalize=renorm)
    d = gmi.moe_route_bwd(x.to(dev()), r.indices, r.weights, r.offsets, r.live, dw.to(dev()),
                          torch.tensor([dl], device=dev()), renormalize=renorm).cpu().double()
    want = ref.route(x, k, None, renorm)
    for _ in range(4):
        u = torch.randn(T, E, generator=gen).double()
        eps = 1e-6
        hi = ref.route_objective(x.double() + eps * u, want, k, None, renorm, dw, dl)
        lo = ref.route_objective(x.double() - eps * u, want, k, None, renorm, dw, dl)
        assert abs(float((hi - lo) / (2 * eps) - (d * u).sum())) <= TOL * float((d * u).abs().sum()) + 1e-6


def test_route_feeds_the_grouped_gemm_on_a_side_stream_and_in_a_graph(gmi):
    # the layer's calls on a stream of their own, then captured and replayed with eager work in between
    gen = torch.Generator().manual_seed(30)
    T, K, N, E, k = 96, 256, 192, 8, 2
    x, res = (torch.randn(T, K, generator=gen).to(torch.bfloat16).to(dev()) for _ in range(2))
    w = torch.ones(K, dtype=torch.bfloat16, device=dev())
    logits = torch.randn(T, E, generator=gen).to(dev())
    W = (torch.randn(E, N, K, generator=gen) * 100).clamp(-448, 448).to(ref.F8).to(dev())
    ws = torch.full((E, 2, 2), 0.01, device=dev())

    def layer(stream=None):
        q, s = gmi.rmsnorm_quant(x, w, residual=res, stream=stream)
        r = gmi.moe_route(logits, k, stream=stream)
        tok = torch.div(r.row_slot, k, rounding_mode="floor").long()
        Y = gmi.gemm_f8_block_grouped(r.offsets, q.view(torch.uint8)[tok].view(ref.F8), s[tok], W, ws, stream=stream)
        d = gmi.moe_route_bwd(logits, r.indices, r.weights, r.offsets, r.live, torch.ones(T, k, device=dev()),
                              torch.ones(1, device=dev()), stream=stream)
        dh, dwt = gmi.rmsnorm_bwd(x, res, w, stream=stream)
        return r, Y, d, dh, dwt

    base = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer()
    torch.cuda.synchronize()
    flat = [t for a in (base, other) for t in (*a[0], *a[1:])]
    n = len(flat) // 2
    assert all(torch.equal(p, q) for p, q in zip(flat[:n], flat[n:]))
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = layer()
    held = [*held[0], *held[1:]]
    for step in range(3):
        x.copy_(torch.randn(T, K, generator=gen).to(torch.bfloat16))
        logits.copy_(torch.randn(T, E, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        eager = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, [*eager[0], *eager[1:]])), f"replay {step}"
