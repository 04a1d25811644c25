"""GPU: rows between the products of a mixture-of-experts layer against float64."""
import math

import pytest
import torch

import rows_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


# ---------------------------------------------------------------- group_rows
@pytest.mark.parametrize("n,groups", [(0, 3), (1, 1), (2, 7), (63, 5), (64, 16), (65, 1024), (1023, 60), (1024, 2),
                                      (1025, 128), (2048, 300), (2049, 300), (4096, 1023), (4097, 9), (5000, 1024), (40000, 128), (300001, 37)])
def test_group_rows(gmi, n, groups):
    gen = torch.Generator().manual_seed(n + groups)
    index = torch.randint(-2, groups + 2, (n,), generator=gen).to(torch.int32)
    got = gmi.group_rows(index.to(dev()), groups)
    torch.cuda.synchronize()
    for g, w in zip(got, ref.group(index, groups)):
        assert torch.equal(g.cpu(), w)


@pytest.mark.parametrize("n", [100, 5000, 70000])
@pytest.mark.parametrize("value", [0, 4, -1, 5, 2 ** 31 - 1, -2 ** 31])
def test_group_rows_all_in_one_or_in_none(gmi, n, value):
    index = torch.full((n,), value, dtype=torch.int32)
    got = gmi.group_rows(index.to(dev()), 5)
    for g, w in zip(got, ref.group(index, 5)):
        assert torch.equal(g.cpu(), w)


def test_group_rows_stands_in_for_the_routers_order(gmi):
    logits = torch.randn(700, 24, generator=torch.Generator().manual_seed(5)).to(dev())
    mask = torch.rand(700, generator=torch.Generator().manual_seed(6)).to(dev()) > 0.1
    r = gmi.moe_route(logits, 3, mask=mask)
    g = gmi.group_rows(r.indices, 24)
    total = int(r.offsets[-1])
    assert torch.equal(g.offsets, r.offsets) and torch.equal(g.place, r.slot_row)
    assert torch.equal(g.order[:total], r.row_slot[:total]) and g.place.shape == (700, 3)
    assert total < 2100 and (torch.sort(g.order)[0].cpu() == torch.arange(2100)).all()


# ---------------------------------------------------------------- permute
@pytest.mark.parametrize("dtype", [ref.F8, *DTYPES])
@pytest.mark.parametrize("tokens,k,cols,spare", [(1, 1, 16, 0), (1, 16, 4096, 3), (5, 3, 2000, 7), (300, 8, 144, 0),
                                                 (3000, 2, 1040, 1), (17, 9, 8208, 40)])
def test_permute(gmi, dtype, tokens, k, cols, spare):
    gen = torch.Generator().manual_seed(cols)
    x = torch.randint(0, 256, (tokens, cols * (1 if dtype == ref.F8 else 2)), generator=gen, dtype=torch.uint8)
    slot_row = ref.slots(gen, tokens, k, spare)
    rows = tokens * k + spare
    scales = torch.rand(tokens, ref.blocks(cols), generator=gen) if dtype == ref.F8 else None
    out = torch.full((rows, x.shape[1]), 0x3c, dtype=torch.uint8, device=dev())
    out_scales = torch.full((rows, ref.blocks(cols)), 7.0, device=dev()) if scales is not None else None
    gmi.moe_permute(x.to(dev()).view(dtype), slot_row.to(dev()), scales=None if scales is None else scales.to(dev()),
                    out=out.view(dtype), out_scales=out_scales)
    want = torch.full((rows, x.shape[1]), 0x3c, dtype=torch.uint8)
    want_s = torch.full((rows, ref.blocks(cols)), 7.0)
    for t in range(tokens):
        for i in range(k):
            if slot_row[t, i] >= 0:
                want[slot_row[t, i]] = x[t]
                if scales is not None:
                    want_s[slot_row[t, i]] = scales[t]
    assert torch.equal(out.cpu(), want)
    assert scales is None or torch.equal(out_scales.cpu(), want_s)


def test_permute_strided_and_row_numbers_past_the_end(gmi):
    # rows of wider buffers; row numbers outside the output are no rows, whatever they are
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(6, 272, generator=gen).to(torch.bfloat16).to(dev())[:, 8:264]
    out = torch.zeros(20, 512, dtype=torch.bfloat16, device=dev())
    slot_row = torch.tensor([[0, 9], [10, 1], [2 ** 31 - 1, 3], [-2 ** 31, 4], [-1, -5], [5, 1000]], dtype=torch.int32)
    gmi.moe_permute(x, slot_row.to(dev()), out=out[:10, 256:])
    want = torch.zeros(20, 512, dtype=torch.bfloat16)
    for t, i, r in ((0, 0, 0), (0, 1, 9), (1, 1, 1), (2, 1, 3), (3, 1, 4), (5, 0, 5)):
        want[r, 256:] = x[t].cpu()
    assert torch.equal(out.cpu(), want)
    assert gmi.moe_permute(x[:0], slot_row[:0].to(dev())).shape == (0, 256)


# ---------------------------------------------------------------- unpermute and its gradient
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 8), (1, 8, 4096), (3, 2, 2000), (16, 8, 4096), (333, 5, 264),
                                           (3000, 3, 1032), (40, 16, 8200)])
@pytest.mark.parametrize("weighted,add", [(True, True), (True, False), (False, False), (False, True)])
def test_unpermute(gmi, dtype, tokens, k, cols, weighted, add):
    gen = torch.Generator().manual_seed(tokens + cols)
    slot_row = ref.slots(gen, tokens, k, 5)
    y = torch.randn(tokens * k + 5, cols, generator=gen).to(dtype)
    w = torch.rand(tokens, k, generator=gen) if weighted else None
    plus = torch.randn(tokens, cols, generator=gen).to(dtype) if add else None
    got = gmi.moe_unpermute(y.to(dev()), slot_row.to(dev()), weights=None if w is None else w.to(dev()),
                            add=None if plus is None else plus.to(dev())).cpu()
    out, mag = ref.unpermute(y, slot_row, w, plus)
    # one rounding; k + 1 fp32 steps
    assert ((got.double() - out).abs() <= ref.STEP[dtype] * out.abs() + ref.FLOOR[dtype] + (k + 2) * 2.0 ** -24 * mag).all()


def test_unpermute_slots_without_a_row_add_nothing(gmi):
    # neither weights nor rows of dead slots are seen; a token without any slot gets `add`, or zero
    y = torch.full((4, 64), math.nan, dtype=torch.bfloat16, device=dev())
    y[1] = 2.0
    slot_row = torch.tensor([[-1, 1], [-1, -1], [4, 2 ** 31 - 1]], dtype=torch.int32, device=dev())
    w = torch.tensor([[math.nan, 3.0], [math.inf, math.nan], [math.nan, 1.0]], device=dev())
    out = gmi.moe_unpermute(y, slot_row, weights=w).cpu()
    assert (out[0] == 6.0).all() and (out[1:] == 0.0).all()
    plus = torch.full((3, 64), 0.5, dtype=torch.bfloat16, device=dev())
    again = gmi.moe_unpermute(y, slot_row, weights=w, add=plus, out=plus)
    assert again is plus and (plus[0] == 6.5).all() and (plus[1:] == 0.5).all()
    assert (gmi.moe_unpermute(y[:0], slot_row).cpu() == 0.0).all()


def test_unpermute_passes_on_what_is_not_finite(gmi):
    y = torch.ones(3, 8, dtype=torch.float16)
    y[0, 0], y[1, 1], y[2, 2], y[0, 3], y[1, 3] = math.nan, math.inf, -math.inf, math.inf, -math.inf
    y[:, 4] = 60000.0
    slot_row = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    out = gmi.moe_unpermute(y.to(dev()), slot_row.to(dev()))[0].cpu()
    assert out[0].isnan() and out[1] == math.inf and out[2] == -math.inf and out[3].isnan()
    assert out[4] == math.inf and (out[5:] == 3.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 8), (1, 8, 4096), (3, 2, 2000), (70, 5, 264), (2100, 2, 512),
                                           (2100, 1, 648), (9, 16, 1032)])
@pytest.mark.parametrize("quant", [False, True])
def test_unpermute_bwd(gmi, dtype, tokens, k, cols, quant):
    gen = torch.Generator().manual_seed(tokens + cols)
    slot_row = ref.slots(gen, tokens, k, 5)
    rows = tokens * k + 5
    y, dout = (torch.randn(n, cols, generator=gen).to(dtype) for n in (rows, tokens))
    dout[:, : min(cols, 128)][tokens // 2] = 0.0  # a block of zeros
    w = torch.randn(tokens, k, generator=gen)
    drows = torch.full((rows, cols), 3.0, device=dev()).to(ref.F8 if quant else dtype)
    scales = torch.full((rows, ref.blocks(cols)), 5.0, device=dev()) if quant else None
    got = gmi.moe_unpermute_bwd(dout.to(dev()), slot_row.to(dev()), weights=w.to(dev()), rows=y.to(dev()), drows=drows,
                                scales=scales, quantize=quant)
    d, dw, mag = ref.unpermute_bwd(dout, slot_row, w, y, rows)
    used = ~d.isnan().any(1)
    # a lane's sum, six lane exchanges, the waves
    assert ((got[-1].cpu().double() - dw).abs() <= (cols / 64 + 24) * 2.0 ** -24 * mag).all()
    if quant:
        ref.check_codes(drows.cpu()[used], scales.cpu()[used], d[used], 2.0 ** -24)
        assert (scales.cpu()[~used] == 5.0).all()
    else:
        v = drows.cpu()[used].double()
        assert ((v - d[used]).abs() <= (ref.STEP[dtype] + 2.0 ** -24) * d[used].abs() + ref.FLOOR[dtype]).all()
    assert (drows.cpu()[~used].float() == 3.0).all()


@pytest.mark.parametrize("quant", [False, True])
def test_unpermute_bwd_without_weights_or_rows(gmi, quant):
    gen = torch.Generator().manual_seed(8)
    slot_row = ref.slots(gen, 20, 3, 0, dead=0.0)
    dout = torch.randn(20, 264, generator=gen).to(torch.bfloat16)
    got = gmi.moe_unpermute_bwd(dout.to(dev()), slot_row.to(dev()), quantize=quant)
    assert got[-1] is None
    d, _, _ = ref.unpermute_bwd(dout, slot_row, None, None, 60)
    if quant:
        ref.check_codes(got[0].cpu(), got[1].cpu(), d, 0.0)
    else:
        assert torch.equal(got[0].cpu().double(), d)


def test_unpermute_bwd_of_the_weights_alone(gmi):
    gen = torch.Generator().manual_seed(11)
    slot_row = ref.slots(gen, 300, 4, 3).to(dev())
    y, dout = (torch.randn(n, 520, generator=gen).to(torch.bfloat16).to(dev()) for n in (1203, 300))
    keep = y.clone()
    drows, dw = gmi.moe_unpermute_bwd(dout, slot_row, rows=y, row_grad=False)
    _, want = gmi.moe_unpermute_bwd(dout, slot_row, rows=y)
    assert drows is None and same(dw, want) and same(y, keep)


def test_unpermute_bwd_over_the_rows_it_reads(gmi):
    # the rows' gradient in the place of the rows
    gen = torch.Generator().manual_seed(9)
    slot_row = ref.slots(gen, 50, 4, 0, dead=0.0).to(dev())
    y, dout = (torch.randn(n, 520, generator=gen).to(torch.float16).to(dev()) for n in (200, 50))
    w = torch.rand(50, 4, generator=gen).to(dev())
    want = gmi.moe_unpermute_bwd(dout, slot_row, weights=w, rows=y)
    got = gmi.moe_unpermute_bwd(dout, slot_row, weights=w, rows=y, drows=y)
    assert got[0] is y and same(got[0], want[0]) and same(got[1], want[1])


def test_unpermute_bwd_codes_of_what_is_not_finite(gmi):
    dout = torch.ones(1, 256, dtype=torch.bfloat16)
    dout[0, 3], dout[0, 130] = math.nan, 4.0
    w = torch.tensor([[2.0, math.nan, 0.0]])
    slot_row = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    q, s, _ = gmi.moe_unpermute_bwd(dout.to(dev()), slot_row.to(dev()), weights=w.to(dev()), quantize=True)
    q, s = q.float().cpu(), s.cpu()
    assert q[0, 3].isnan() and (q[0, 4:128] == 448.0).all() and q[0, 130] == 448.0 and (q[0, 131:] == 112.0).all()
    assert s[0, 0] == 2.0 / 448.0 and s[0, 1] == 8.0 / 448.0
    assert q[1].isnan().all() and q[2, 3].isnan() and (q[2, 4:] == 0.0).all() and (s[2] == ref.TINY / 448.0).all()


def test_permute_and_unpermute_are_each_others_gradients(gmi):
    # <permute(x), g> = <x, unpermute(g)> and differences of the weighted sum along random directions
    gen = torch.Generator().manual_seed(10)
    T, k, K = 60, 4, 256
    slot_row = ref.slots(gen, T, k, 0).to(dev())
    x = torch.randint(-8, 9, (T, K), generator=gen).to(torch.bfloat16).to(dev())
    g = torch.randint(-8, 9, (T * k, K), generator=gen).to(torch.bfloat16).to(dev())
    out = torch.zeros(T * k, K, dtype=torch.bfloat16, device=dev())
    gmi.moe_permute(x, slot_row, out=out)
    left = (out.double() * g.double()).sum()
    right = (x.double() * gmi.moe_unpermute(g, slot_row).double()).sum()  # sums of four such integers are bf16 numbers
    assert left == right
    # f(w, y) = <unpermute(y, w), dout> is linear in each: a difference is the gradient's product with the step, to the
    # rounding of outputs of a few units (2^-8 each, 15360 of them with random signs: six of their deviations)
    w = torch.rand(T, k, generator=gen).to(dev())
    dw, dy = torch.randn(T, k, generator=gen).to(dev()), torch.randn(T * k, K, generator=gen).to(torch.bfloat16).to(dev())
    dout = torch.randn(T, K, generator=gen).to(torch.bfloat16).to(dev())

    def f(w, y):
        o = gmi.moe_unpermute(y, slot_row, weights=w)
        return (o.double() * dout.double()).sum(), 2.0 ** -8 * (o.double() * dout.double()).pow(2).sum().sqrt()

    drows, dweights = gmi.moe_unpermute_bwd(dout, slot_row, weights=w, rows=g)
    used = torch.zeros(T * k, dtype=torch.bool, device=dev())
    used[slot_row[slot_row >= 0].long()] = True
    (f0, e0), (f1, e1) = f(w, g), f(w + dw, g)
    assert (f1 - f0 - (dweights.double() * dw.double()).sum()).abs() <= 6 * (e0 + e1)
    f2, e2 = f(w, (g + dy).to(torch.bfloat16))
    step = torch.where(used[:, None], drows.double(), 0.0) * ((g + dy).to(torch.bfloat16).double() - g.double())
    assert (f2 - f0 - step.sum()).abs() <= 6 * (e0 + e2 + 2.0 ** -8 * step.pow(2).sum().sqrt())


# ---------------------------------------------------------------- gated activation
def gated(gen, rows, N, dtype):
    a = torch.randn(rows, 2 * N, generator=gen) * 3
    a[:, 0] = torch.linspace(-30, 30, rows) if rows > 1 else 30.0
    return a.to(dtype)


def rel(a):
    """What the gate's value is off, relative: g log2 e is rounded before the exponential (|g| 2^-24 of e^-g: half a step
    of |g| log2 e, times ln 2), which reaches 1 / (1 + e^-g) with the factor e^-g / (1 + e^-g) <= 1; two fp32 steps
    (2^-23 each) of exponential and reciprocal, half steps of the constant, the sum and three products."""
    g = a.double()[:, : a.shape[1] // 2].abs().nan_to_num()
    return float((g * 2.0 ** -24).max()) + 8 * 2.0 ** -24


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,N", [(1, 8), (1, 1024), (3, 120), (64, 128), (333, 200), (1000, 1032), (5, 4096)])
def test_swiglu(gmi, dtype, rows, N):
    a = gated(torch.Generator().manual_seed(N), rows, N, dtype)
    v = ref.swiglu(a)
    y = torch.empty(rows, N, dtype=dtype, device=dev())
    q, s = gmi.swiglu_quant(a.to(dev()), y=y)
    ref.check_codes(q.cpu(), s.cpu(), v, rel(a))
    near = (ref.STEP[dtype] + rel(a)) * v.abs() + ref.FLOOR[dtype]
    assert ((y.cpu().double() - v).abs() <= near).all()
    only = gmi.swiglu_quant(a.to(dev()), quantize=False)
    assert same(only, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,N", [(1, 8), (1, 1024), (3, 120), (64, 128), (333, 200), (1000, 1032), (5, 4096)])
@pytest.mark.parametrize("quant", [False, True])
def test_swiglu_bwd(gmi, dtype, rows, N, quant):
    gen = torch.Generator().manual_seed(N)
    a, dact = gated(gen, rows, N, dtype), torch.randn(rows, N, generator=gen).to(dtype)
    v = ref.swiglu_bwd(dact, a)
    # 1 + g (1 - s) loses what its terms' sum cancels (near g = -1.28 it is zero), and 1 - s what s is off, |g| times
    # that in all: steps of the terms with the term g s in the place of g s (1 - s)
    g, u = a.double().chunk(2, 1)
    sg = torch.sigmoid(g)
    off = rel(a) * torch.cat([dact.double().abs() * u.abs() * sg * (1 + g.abs()), v[:, N:].abs()], 1)
    if quant:
        q, s = gmi.swiglu_bwd(dact.to(dev()), a.to(dev()), quantize=True)
        q, s = q.cpu().float().double(), s.cpu().double()
        pad = torch.nn.functional.pad(v, (0, ref.blocks(2 * N) * 128 - 2 * N)).view(rows, -1, 128)
        want = pad.abs().amax(2).clamp_min(ref.TINY) / 448.0
        worst = torch.nn.functional.pad(off, (0, ref.blocks(2 * N) * 128 - 2 * N)).view(rows, -1, 128).amax(2)
        assert ((s - want).abs() <= 2.0 ** -22 * want + worst / 448.0).all()
        # half a step of the code (2^-4 of it, or half the smallest), and what the value is off
        spread = s.repeat_interleave(128, 1)[:, : 2 * N]
        assert ((q * spread - v).abs() <= (2.0 ** -4 + 2.0 ** -20) * v.abs() + 2.0 ** -10 * spread + 2 * off).all()
    else:
        got = gmi.swiglu_bwd(dact.to(dev()), a.to(dev())).cpu().double()
        assert ((got - v).abs() <= (ref.STEP[dtype] + 2.0 ** -22) * v.abs() + ref.FLOOR[dtype] + off).all()
        held = a.to(dev())
        again = gmi.swiglu_bwd(dact.to(dev()), held, da=held)
        assert again is held and torch.equal(again.cpu().double(), got)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("N", [120, 256])
@pytest.mark.parametrize("used", [-3, 0, 1, 37, 50, 60])
def test_swiglu_rows_behind_the_last(gmi, quant, N, used):
    # rows from `live` on are neither read nor written; more than there are is all of them
    gen = torch.Generator().manual_seed(N)
    a, dact = gated(gen, 50, N, torch.bfloat16).to(dev()), torch.randn(50, N, generator=gen).to(torch.bfloat16).to(dev())
    live = torch.tensor([0, used], dtype=torch.int32, device=dev())[1:]
    n = max(0, min(50, used))
    a[n:] = math.nan

    def full(cols, dt):
        return torch.full((50, cols), 3.0, device=dev()).to(dt)

    if quant:
        q, s = full(N, ref.F8), full(ref.blocks(N), torch.float32)
        gmi.swiglu_quant(a, live=live, q=q, scales=s)
        dq, ds = full(2 * N, ref.F8), full(ref.blocks(2 * N), torch.float32)
        gmi.swiglu_bwd(dact, a, live=live, da=dq, scales=ds, quantize=True)
        parts = [(q, gmi.swiglu_quant(a)[0]), (s, gmi.swiglu_quant(a)[1]),
                 (dq, gmi.swiglu_bwd(dact, a, quantize=True)[0]), (ds, gmi.swiglu_bwd(dact, a, quantize=True)[1])]
    else:
        y, da = full(N, torch.bfloat16), full(2 * N, torch.bfloat16)
        gmi.swiglu_quant(a, live=live, y=y, quantize=False)
        gmi.swiglu_bwd(dact, a, live=live, da=da)
        parts = [(y, gmi.swiglu_quant(a, quantize=False)), (da, gmi.swiglu_bwd(dact, a))]
    for got, whole in parts:
        assert same(got[:n], whole[:n]) and (got[n:].float() == 3.0).all()


def test_swiglu_at_the_ends_of_the_range(gmi):
    big = torch.finfo(torch.bfloat16).max
    g = torch.tensor([big, -big, 1000.0, -1000.0, 0.0, -0.0, math.inf, math.nan], dtype=torch.bfloat16)
    a = torch.cat([g, torch.ones(8, dtype=torch.bfloat16)])[None].to(dev())
    y = gmi.swiglu_quant(a, quantize=False)[0].cpu()
    assert y[0] == big and y[1] == 0 and y[2] == 1000.0 and y[3] == 0 and y[4] == 0 and y[5] == 0
    assert y[6] == math.inf and y[7].isnan()
    d = gmi.swiglu_bwd(torch.ones(1, 8, dtype=torch.bfloat16, device=dev()), a)[0].cpu()
    assert d[0] == 1 and d[1] == 0 and d[2] == 1 and d[3] == 0 and d[4] == 0.5 and d[5] == 0.5 and d[7].isnan()
    assert d[8] == big and d[9] == 0 and d[10] == 1000.0 and d[11] == 0 and d[14] == math.inf and d[15].isnan()


def test_swiglu_gradient_against_differences(gmi):
    gen = torch.Generator().manual_seed(4)
    a = torch.randn(20, 2 * 64, generator=gen).to(torch.float16)
    dact = torch.randn(20, 64, generator=gen).to(torch.float16)
    da = gmi.swiglu_bwd(dact.to(dev()), a.to(dev())).cpu().double()
    step = torch.randn(20, 128, generator=gen).double() * 1e-4

    def f(x):
        g, u = x.chunk(2, 1)
        return (g / (1 + torch.exp(-g)) * u * dact.double()).sum()

    slope = (f(a.double() + step) - f(a.double() - step)) / 2
    # each gradient is off by 2^-11 of itself at most
    assert (slope - (da * step).sum()).abs() <= 2.0 ** -11 * (da.abs() * step.abs()).sum() * 1.01 + 1e-9


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows(gmi, dtype):
    # every operand a part of a wider buffer, the last row at its end
    gen = torch.Generator().manual_seed(12)
    T, k, N = 33, 3, 136

    def wide(rows, cols, dt, fill=None):
        b = torch.randn(rows, cols + 24, generator=gen).to(dt) if fill is None else torch.full((rows, cols + 24), fill).to(dt)
        return b.to(dev())[:, 16:16 + cols]

    slot_row = ref.slots(gen, T, k, 0).to(dev())
    w = torch.rand(T, k, generator=gen).to(dev())
    y, plus, dout, a = wide(T * k, N, dtype), wide(T, N, dtype), wide(T, N, dtype), wide(T * k, 2 * N, dtype)
    out, drows, da = wide(T, N, dtype, 0.0), wide(T * k, N, dtype, 0.0), wide(T * k, 2 * N, dtype, 0.0)
    act, q, s = wide(T * k, N, dtype, 0.0), wide(T * k, N, ref.F8, 0.0), wide(T * k, 2, torch.float32, 0.0)
    gmi.moe_unpermute(y, slot_row, weights=w, add=plus, out=out)
    assert same(out, gmi.moe_unpermute(y.contiguous(), slot_row, weights=w, add=plus.contiguous()))
    _, dw = gmi.moe_unpermute_bwd(dout, slot_row, weights=w, rows=y, drows=drows)
    zero = torch.zeros_like(y.contiguous())
    d2, dw2 = gmi.moe_unpermute_bwd(dout.contiguous(), slot_row, weights=w, rows=y.contiguous(), drows=zero)
    assert same(drows, d2) and same(dw, dw2)
    gmi.swiglu_quant(a, y=act, q=q, scales=s)
    y2 = torch.empty(T * k, N, dtype=dtype, device=dev())
    q2, s2 = gmi.swiglu_quant(a.contiguous(), y=y2)
    assert same(act, y2) and same(q, q2) and same(s, s2)
    gmi.swiglu_bwd(act, a, da=da)
    assert same(da, gmi.swiglu_bwd(act.contiguous(), a.contiguous()))
    for b in (out, drows, da, act, q):
        whole = b._base if b._base is not None else b
        assert (whole[:, :16].float() == 0).all() and (whole[:, 16 + b.shape[1]:].float() == 0).all()
