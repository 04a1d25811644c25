"""GPU: RMS norm with the residual's addition and block-scaled fp8 output, and
its backward, against float64.  Tolerances: half a step of each rounding, plus
2e-5 relative for the fp32 row sums (a few dozen roundings of 2^-24 each)."""
import pytest
import torch

import moe_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
F32 = 2e-5


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def _rand(gen, rows, cols, dt, ld=None, std=1.0):
    buf = (torch.randn(rows, ld or cols, generator=gen) * std).to(dt)
    return buf[:, :cols]


def _dev_like(t, ld=None):
    """The CPU matrix on the device with leading dimension `ld` and NaN in the padding."""
    ld = ld or t.shape[1]
    buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=dev())
    buf[:, : t.shape[1]] = t.to(dev())
    return buf[:, : t.shape[1]]


def _check_norm(x, w, res, eps, h, y, q, s):
    dt = x.dtype
    rh, rv, rs, rt = ref.norm(x, w, res, eps)
    hs = ref.half_step(dt)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # half a subnormal step and more
    if h is not None:
        assert ((h.cpu().double() - rh).abs() <= hs * rh.abs() + 2.0 ** -23 * rh.abs() + tiny).all()
    if y is not None:
        assert ((y.cpu().double() - rv).abs() <= (hs + F32) * rv.abs() + tiny).all()
    if q is not None:
        assert ((s.cpu().double() - rs).abs() <= F32 * rs).all()
        err = (q.cpu().float().double() - rt).abs()
        assert (err <= (2.0 ** -4 + 2 * F32) * rt.abs() + 2.0 ** -10).all(), float(err.max())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,K,pad", [(1, 8, 0), (1, 4096, 0), (3, 128, 16), (5, 136, 8), (17, 1000, 24),
                                        (9, 2064, 0), (1100, 2048, 16), (1030, 4096, 0), (7, 8192, 0), (3, 16384, 0),
                                        (2, 20000, 16), (1, 32768, 0), (1029, 520, 0)])
def test_norm_shapes(gmi, dtype, rows, K, pad):
    gen = torch.Generator().manual_seed(rows * 7 + K)
    x, res = _rand(gen, rows, K, dtype), _rand(gen, rows, K, dtype, std=3.0)
    w = (1 + 0.2 * torch.randn(K, generator=gen)).to(dtype)
    ld = K + pad if pad else K
    h, y = (torch.zeros(rows, ld, dtype=dtype, device=dev())[:, :K] for _ in range(2))
    q = torch.zeros(rows, ld, dtype=torch.uint8, device=dev()).view(ref.F8)[:, :K]
    s = torch.full((rows, ref.blocks(K) + 1), -1.0, device=dev())
    got = gmi.rmsnorm_quant(_dev_like(x, ld), w.to(dev()), residual=_dev_like(res, ld), eps=1e-5, h=h, y=y, q=q,
                            scales=s[:, :-1])
    torch.cuda.synchronize()
    assert got[0] is q
    _check_norm(x, w, res, 1e-5, h, y, q, s[:, :-1])
    assert (s[:, -1] == -1.0).all(), "padding of the scales written"
    if pad:
        for t in (h, y):
            assert (t._base[:, K:] == 0).all(), "padding columns written"
        assert (q._base.view(torch.uint8)[:, K:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_norm_without_residual_and_single_outputs(gmi, dtype):
    gen = torch.Generator().manual_seed(3)
    x = _rand(gen, 33, 768, dtype)
    w = torch.ones(768, dtype=dtype)
    q, s = gmi.rmsnorm_quant(x.to(dev()), w.to(dev()))
    y = gmi.rmsnorm_quant(x.to(dev()), w.to(dev()), quantize=False)
    torch.cuda.synchronize()
    _check_norm(x, w, None, 1e-6, None, y, q, s)


def test_norm_in_place_residual(gmi):
    gen = torch.Generator().manual_seed(4)
    x, res = _rand(gen, 40, 512, torch.bfloat16), _rand(gen, 40, 512, torch.bfloat16)
    w = torch.ones(512, dtype=torch.bfloat16)
    stream = res.to(dev())
    q, s = gmi.rmsnorm_quant(x.to(dev()), w.to(dev()), residual=stream, h=stream)
    torch.cuda.synchronize()
    _check_norm(x, w, res, 1e-6, stream, None, q, s)


def test_norm_zero_rows_and_special_values(gmi):
    K = 384
    x = torch.zeros(6, K)
    x[1] = 1.0
    x[1, 128:256] = 0.0  # an all-zero block
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 3e-39  # subnormal squares
    x[5] = 3.0
    x = x.to(torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16)
    q, s = gmi.rmsnorm_quant(x.to(dev()), w.to(dev()), eps=1e-6)
    torch.cuda.synchronize()
    qf, s = q.cpu().float(), s.cpu()
    assert (qf[0] == 0).all() and torch.isfinite(s[0]).all() and (s[0] > 0).all()
    assert (qf[1, 128:256] == 0).all() and (qf[1, :128] == 448).all()
    assert torch.isnan(qf[2]).all()
    # an infinity: 1 / inf scales the row to zero, the infinity itself to NaN
    assert torch.isnan(qf[3, 200]) and (qf[3, :128] == 0).all()
    assert torch.isfinite(qf[4]).all() and (qf[5] == 448).all()
    q0, s0 = gmi.rmsnorm_quant(torch.empty(0, K, dtype=torch.bfloat16, device=dev()), w.to(dev()))
    assert q0.shape == (0, K) and s0.shape == (0, 3)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,K,with_res", [(1, 8, True), (1, 4096, True), (5, 136, False), (333, 2000, True),
                                             (2100, 2048, True), (4200, 1024, True), (1500, 4096, False),
                                             (600, 4104, True), (9, 16384, True), (3, 32768, True)])
def test_norm_bwd(gmi, dtype, rows, K, with_res):
    gen = torch.Generator().manual_seed(rows + K)
    h, dy = _rand(gen, rows, K, dtype, std=2.0), _rand(gen, rows, K, dtype)
    dres = _rand(gen, rows, K, dtype) if with_res else None
    w = (1 + 0.2 * torch.randn(K, generator=gen)).to(dtype)
    ld = K + 8
    dh, dw = gmi.rmsnorm_bwd(_dev_like(dy, ld), _dev_like(h, ld), w.to(dev()),
                             dres=_dev_like(dres, ld) if with_res else None, eps=1e-5)
    torch.cuda.synchronize()
    rdh, rdw, mag, wmag = ref.norm_bwd(dy, h, w, dres, 1e-5)
    hs, tiny = ref.half_step(dtype), torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert ((dh.cpu().double() - rdh).abs() <= hs * rdh.abs() + F32 * mag + tiny).all()
    # sums over rows: each partial adds at most rows / parts + parts + 16 roundings of 2^-24 on terms of F32 / 4
    assert ((dw.cpu().double() - rdw).abs() <= (F32 + 64 * 2.0 ** -24) * wmag + 1e-30).all()
    again = gmi.rmsnorm_bwd(_dev_like(dy, ld), _dev_like(h, ld), w.to(dev()),
                            dres=_dev_like(dres, ld) if with_res else None, eps=1e-5)
    assert torch.equal(again[1], dw) and torch.equal(again[0], dh)


def test_norm_bwd_against_differences(gmi):
    # directional differences of the float64 forward (the norm itself, unquantised) in 4 random directions
    gen = torch.Generator().manual_seed(11)
    rows, K, eps = 6, 256, 1e-5
    h, dy = _rand(gen, rows, K, torch.float16), _rand(gen, rows, K, torch.float16)
    w = (1 + 0.2 * torch.randn(K, generator=gen)).to(torch.float16)
    dh, dw = gmi.rmsnorm_bwd(dy.to(dev()), h.to(dev()), w.to(dev()), eps=eps)
    torch.cuda.synchronize()

    def f(hh, ww):
        return (dy.double() * ww * hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps)).sum()

    for _ in range(4):
        dirh, dirw = torch.randn(rows, K, generator=gen).double(), torch.randn(K, generator=gen).double()
        d = 1e-5
        num = (f(h.double() + d * dirh, w.double() + d * dirw) - f(h.double() - d * dirh, w.double() - d * dirw)) / (2 * d)
        got = (dh.cpu().double() * dirh).sum() + (dw.cpu().double() * dirw).sum()
        mag = (dh.cpu().double() * dirh).abs().sum() + (dw.cpu().double() * dirw).abs().sum()
        assert abs(float(num - got)) <= 2.0 ** -11 * float(mag) + 1e-6 * float(mag)


def test_norm_bwd_eps_zero_and_no_rows(gmi):
    gen = torch.Generator().manual_seed(12)
    h, dy = _rand(gen, 5, 64, torch.bfloat16), _rand(gen, 5, 64, torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    dh, dw = gmi.rmsnorm_bwd(dy.to(dev()), h.to(dev()), w.to(dev()), eps=0.0)
    rdh, rdw, mag, wmag = ref.norm_bwd(dy, h, w, None, 0.0)
    assert ((dw.cpu().double() - rdw).abs() <= F32 * wmag).all()
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=dev())
    dw = torch.full((64,), 7.0, device=dev())
    gmi.rmsnorm_bwd(none, none, w.to(dev()), dweight=dw)
    assert (dw == 0).all()


def test_norm_more_rows_than_one_launch(gmi):
    rows, K = (1 << 22) + 5, 8
    gen = torch.Generator().manual_seed(15)
    x, res = (torch.randn(rows, K, generator=gen).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(K, dtype=torch.bfloat16)
    h = torch.zeros(rows, K, dtype=torch.bfloat16, device=dev())
    q, s = gmi.rmsnorm_quant(x.to(dev()), w.to(dev()), residual=res.to(dev()), eps=1e-5, h=h)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(0, rows, 9973), torch.arange((1 << 22) - 4, rows)])
    _check_norm(x[at], w, res[at], 1e-5, h[at.to(dev())], None, q.view(torch.uint8)[at.to(dev())].view(ref.F8),
                s[at.to(dev())])
