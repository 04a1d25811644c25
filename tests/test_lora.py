"""GPU: the adapters' product against float64."""
import math

import pytest
import torch

import rows_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def case(M, N, K, rank, adapters, dtype, seed=0, none=0.1, run=1):
    gen = torch.Generator().manual_seed(seed + M + N + K + rank)
    X, base = (torch.randn(M, c, generator=gen).to(dtype) for c in (K, N))
    A = (torch.randn(adapters, rank, K, generator=gen) * K ** -0.5).to(dtype)
    B = (torch.randn(adapters, N, rank, generator=gen) * rank ** -0.5).to(dtype)
    scales = torch.rand(adapters, generator=gen) + 0.5
    index = torch.randint(0, adapters, (M,), generator=gen)
    index[torch.rand(M, generator=gen) < none] = -1
    if run > 1:
        index = index.repeat_interleave(run)[:M]
    return X, A, B, index.to(torch.int32), scales, base


def check(got, X, A, B, index, scales, base):
    want = ref.lora(X, A, B, index, scales, base)
    tol = ref.lora_tolerance(*want, X.dtype, X.shape[1], A.shape[1])
    off = (got.cpu().double() - want[0]).abs() - tol
    assert (off <= 0).all(), (int(off.argmax()), float(off.max()))


def up(*tensors):
    return [None if t is None else t.to(dev()) for t in tensors]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,rank,adapters,run", [
    (1, 8, 8, 8, 1, 1), (1, 512, 512, 16, 3, 1), (2, 64, 40, 8, 2, 1), (16, 1032, 2056, 16, 16, 1),
    (17, 264, 328, 24, 5, 1), (64, 256, 1024, 32, 64, 1), (65, 200, 264, 40, 4, 7), (100, 72, 520, 64, 3, 33),
    (128, 520, 256, 72, 2, 64), (200, 136, 300 // 8 * 8, 128, 3, 20), (333, 2000, 2056, 40, 12, 7),
    (1000, 256, 768, 16, 300, 1), (700, 128, 4096, 48, 2, 350), (511, 264, 1032, 64, 6, 40),
    (512, 72, 40, 8, 3, 100), (513, 8, 8, 64, 5, 9), (900, 200, 2056, 72, 4, 130), (1500, 1032, 264, 128, 3, 200),
    (640, 136, 1000, 32, 700, 1), (2048, 520, 4096, 24, 8, 300), (777, 328, 648, 96, 2, 64),
    # X A^T in more than eight runs of K: short runs of up to 16, 32 and 64 rows, long ones up to rank 16
    (3, 200, 4104, 48, 2, 1), (9, 264, 8192, 16, 4, 1), (15, 72, 4352, 128, 1, 15), (30, 136, 4096, 24, 1, 30),
    (50, 72, 4360, 128, 2, 25), (60, 200, 6000, 40, 1, 60), (64, 136, 4096, 16, 1, 64), (600, 72, 4608, 16, 3, 100)])
def test_lora(gmi, dtype, M, N, K, rank, adapters, run):
    X, A, B, index, scales, base = case(M, N, K, rank, adapters, dtype, run=run)
    d = up(X, A, B, index, scales, base)
    order = gmi.group_rows(d[3], adapters).order
    sorted_ = gmi.gemm_lora(*d[:4], scales=d[4], order=order, base=d[5])
    check(sorted_, X, A, B, index, scales, base)
    plain = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5])
    assert torch.equal(plain, sorted_), "the order of the rows changes no result"
    alone = gmi.gemm_lora(*d[:4])
    check(alone, X, A, B, index, None, None)
    assert (alone.cpu()[index < 0] == 0).all()


def test_lora_in_the_place_of_the_dense_product(gmi):
    X, A, B, index, scales, base = case(150, 264, 512, 16, 6, torch.bfloat16)
    d = up(X, A, B, index, scales, base)
    want = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5])
    got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], Y=d[5])
    assert got is d[5] and torch.equal(got, want)


def test_lora_rows_see_their_own_adapter_alone(gmi):
    # not-a-number and infinity in other rows, other adapters and in adapters nobody asks for reach nothing
    X, A, B, index, scales, base = case(90, 136, 264, 16, 5, torch.bfloat16, none=0.2)
    clean = ref.lora(X, A, B, index, scales, base)
    X[index == 1], A[2], B[3, 7] = math.nan, math.inf, math.nan
    A[4], B[4] = math.nan, math.inf
    index[index == 4] = -1
    X[index < 0] = math.inf
    clean = ref.lora(torch.where((index == 0)[:, None], X, torch.zeros_like(X)), A[:1], B[:1], index, scales, base)
    d = up(X, A, B, index, scales, base)
    for order in (None, gmi.group_rows(d[3], 5).order):
        got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], order=order).cpu()
        tol = ref.lora_tolerance(*clean, torch.bfloat16, 264, 16)
        rows = index == 0
        assert ((got.double() - clean[0]).abs() <= tol)[rows].all()
        assert torch.equal(got[index < 0], base[index < 0])
        assert got[index == 1].isnan().all() and not got[index == 2].isfinite().any()
        three = index == 3
        assert got[three][:, 7].isnan().all() and got[three][:, :7].isfinite().all() and got[three][:, 8:].isfinite().all()


@pytest.mark.parametrize("sx,sa", [(2.0 ** 12, 2.0 ** 6), (2.0 ** -6, 2.0 ** -12), (1.0, 1.0)])
def test_lora_fp16_holds_products_past_its_range(gmi, sx, sa):
    # X A^T around 2^18 and 2^-18 between the two products: past the largest fp16 and below its normal numbers
    X, A, B, index, _, _ = case(40, 64, 256, 32, 3, torch.float16, none=0.0)
    X, A = (X.float() * sx).half(), (A.float() * sa).half()
    scales = torch.full((3,), 1.0 / (sx * sa))
    d = up(X, A, B, index, scales, None)
    check(gmi.gemm_lora(*d[:4], scales=d[4]), X, A, B, index, scales, None)


@pytest.mark.parametrize("M", [40, 600])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_lora_infinity_beside_products_past_the_type(gmi, dtype, M):
    # one row of A holds an infinity: X A^T is infinite in that column and about 2^20 in the others, whose sums of
    # either sign leave the infinity as it is
    rank, K, N = 24, 128, 72
    X, A = torch.full((M, K), 64.0), torch.full((1, rank, K), 128.0)
    A[0, 3, 5] = math.inf
    B = torch.where(torch.arange(rank) % 2 == 0, -1.0, 1.0).expand(1, N, rank).clone()
    B[0, 7::2] *= -1
    index = torch.zeros(M, dtype=torch.int32)
    got = gmi.gemm_lora(*up(X.to(dtype), A.to(dtype), B.to(dtype), index)).cpu().float()
    assert torch.equal(got, (B[0, :, 3] * math.inf).expand(M, N))


def test_lora_odd_orders(gmi):
    # rows left out of the order, entries that are no rows, adapters past the last: base, or as they were
    X, A, B, index, scales, base = case(70, 72, 128, 8, 4, torch.float16, none=0.0)
    index[5], index[6], index[7] = 4, 2 ** 31 - 1, -2 ** 31
    order = torch.arange(70, dtype=torch.int32).flip(0)
    order[3], order[9] = -1, 70  # rows 66 and 60 are left out
    d = up(X, A, B, index, scales, base)
    Y = torch.full((70, 72), 9.0, dtype=torch.float16, device=dev())
    got = gmi.gemm_lora(*d[:4], scales=d[4], base=d[5], order=order.to(dev()), Y=Y).cpu()
    assert (got[66] == 9.0).all() and (got[60] == 9.0).all() and torch.equal(got[5:8], base[5:8])
    keep = torch.ones(70, dtype=torch.bool)
    keep[[60, 66]] = False
    want = ref.lora(X, A, B, index, scales, base)
    tol = ref.lora_tolerance(*want, torch.float16, 128, 8)
    assert ((got.double() - want[0]).abs() <= tol)[keep].all()


def test_lora_without_adapters_or_rows(gmi):
    X, A, B, index, scales, base = case(20, 64, 64, 8, 2, torch.bfloat16)
    d = up(X, A[:0], B[:0], index, scales[:0], base)
    assert torch.equal(gmi.gemm_lora(*d[:4], base=d[5]).cpu(), base)
    assert (gmi.gemm_lora(*d[:4]) == 0).all()
    d = up(X[:0], A, B, index[:0], scales, base[:0])
    assert gmi.gemm_lora(*d[:4], base=d[5]).shape == (0, 64)


def test_lora_strided(gmi):
    # operands that are parts of wider buffers, adapters apart by more than their data
    X, A, B, index, scales, base = case(75, 120, 136, 24, 3, torch.bfloat16, run=10)
    bx, ba, bb, bz, by = (torch.full(s, math.nan, dtype=torch.bfloat16, device=dev()) for s in (
        (75, 200), (5, 40, 160), (5, 130, 48), (75, 136), (75, 152)))
    x, a, b, z, y = bx[:, 16:152], ba[1:4, 8:32, 8:144], bb[1:4, :120, 16:40], bz[:, 8:128], by[:, 24:144]
    for v, s in ((x, X), (a, A), (b, B), (z, base)):
        v.copy_(s)
    i, s = up(index, scales)
    got = gmi.gemm_lora(x, a, b, i, scales=s, base=z, Y=y)
    check(got, X, A, B, index, scales, base)
    assert by[:, :24].isnan().all() and by[:, 144:].isnan().all()
