"""GPU: the adapters' product from 512 rows on, whose runs go through shared memory: values that must not reach other rows,
odd orders, strides and fp16's range, against float64."""
import math

import pytest
import torch

import rows_ref as ref
from helpers import dev
from test_lora import case, check, up

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [8, 16, 24, 72])
@pytest.mark.parametrize("run", [1, 37, 90])
def test_rows_see_their_own_adapter_alone(gmi, dtype, rank, run):
    # not-a-number and infinity in other rows, other adapters and in adapters nobody asks for reach nothing
    X, A, B, index, scales, base = case(700, 136, 264, rank, 5, dtype, none=0.2, run=run)
    zero = index == 0
    want = ref.lora(torch.where(zero[:, None], X, torch.zeros_like(X)), A[:1], B[:1], index, scales, base)
    tol = ref.lora_tolerance(*want, dtype, 264, rank)
    X[index == 1], A[2], B[3, 7] = math.nan, math.inf, math.nan
    A[4], B[4] = math.nan, math.inf
    index[index == 4] = -1
    X[index < 0] = math.inf
    d = up(X, A, B, index, scales, base)
    for order in (None, gmi.group_rows(d[3], 5).order):
        got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], order=order).cpu()
        assert ((got.double() - want[0]).abs() <= tol)[zero].all()
        assert torch.equal(got[index < 0], base[index < 0])
        assert got[index == 1].isnan().all() and not got[index == 2].isfinite().any()
        three = got[index == 3]
        assert three[:, 7].isnan().all() and three[:, :7].isfinite().all() and three[:, 8:].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [8, 40, 104])
@pytest.mark.parametrize("based", [False, True])
def test_parts_of_wider_buffers(gmi, dtype, rank, based):
    # what lies beside the operands' columns, and what stood in the result, is not-a-number
    M, N, K = 600, 200, 328
    X, A, B, index, scales, base = case(M, N, K, rank, 3, dtype, run=70)
    bx, ba, bb, bz, by = (torch.full(s, math.nan, dtype=dtype, device=dev()) for s in (
        (M, K + 64), (5, rank + 16, K + 24), (5, N + 10, rank + 24), (M, N + 16), (M, N + 32)))
    x, a, b, z, y = (bx[:, 16:16 + K], ba[1:4, 8:8 + rank, 8:8 + K], bb[1:4, :N, 16:16 + rank], bz[:, 8:8 + N],
                     by[:, 24:24 + N])
    for v, s in ((x, X), (a, A), (b, B), (z, base)):
        v.copy_(s)
    i, s = up(index, scales)
    for order in (None, gmi.group_rows(i, 3).order):
        by.fill_(math.nan)
        got = gmi.gemm_lora(x, a, b, i, scales=s, base=z if based else None, Y=y, order=order)
        check(got, X, A, B, index, scales, base if based else None)
        assert by[:, :24].isnan().all() and by[:, 24 + N:].isnan().all()


@pytest.mark.parametrize("sx,sa", [(2.0 ** 12, 2.0 ** 6), (2.0 ** -6, 2.0 ** -12)])
@pytest.mark.parametrize("rank", [16, 32, 128])
def test_fp16_products_past_its_range(gmi, sx, sa, rank):
    X, A, B, index, _, _ = case(600, 64, 256, rank, 3, torch.float16, none=0.0, run=50)
    X, A = (X.float() * sx).half(), (A.float() * sa).half()
    scales = torch.full((3,), 1.0 / (sx * sa))
    d = up(X, A, B, index, scales, None)
    check(gmi.gemm_lora(*d[:4], scales=d[4]), X, A, B, index, scales, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_odd_orders(gmi, dtype):
    # rows left out of the order, entries that are no rows, adapters past the last: base, or as they were
    M = 650
    X, A, B, index, scales, base = case(M, 72, 128, 8, 4, dtype, none=0.0, run=40)
    index[5], index[6], index[7] = 4, 2 ** 31 - 1, -2 ** 31
    order = torch.arange(M, dtype=torch.int32).flip(0)
    out = [3, 9, 64, 127, 128, 500, 649]
    order[out] = torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31, -7, M + 1, -1], dtype=torch.int32)
    left = M - 1 - torch.tensor(out)
    d = up(X, A, B, index, scales, base)
    Y = torch.full((M, 72), 9.0, dtype=dtype, device=dev())
    got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], order=order.to(dev()), Y=Y).cpu()
    assert (got[left] == 9.0).all() and torch.equal(got[5:8], base[5:8])
    keep = torch.ones(M, dtype=torch.bool)
    keep[left] = False
    want = ref.lora(X, A, B, index, scales, base)
    assert ((got.double() - want[0]).abs() <= ref.lora_tolerance(*want, dtype, 128, 8))[keep].all()


def test_no_order_of_some_thousand_rows(gmi):
    # none of the entries is a row: nothing is written
    X, A, B, index, scales, base = case(1300, 72, 128, 8, 4, torch.bfloat16)
    d = up(X, A, B, index, scales, base)
    Y = torch.full((1300, 72), 9.0, dtype=torch.bfloat16, device=dev())
    gmi.gemm_lora(*d[:4], base=d[5], order=torch.full((1300,), -1, dtype=torch.int32, device=dev()), Y=Y)
    assert (Y == 9.0).all()
