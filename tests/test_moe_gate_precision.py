"""GPU: the gated activation and its gradient to the last bits of fp32.  A block with a single value other than zero has
that value over 448 as its scale, in float32, which shows what a 16-bit output would round away."""
import pytest
import torch

import rows_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
U = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    g.lib()
    return g


def one_a_row(dtype, N, at, seed):
    """a [rows][2 N] and dact [rows][N], zeros but for column `at`: every sign and size of the gate whose sigmoid is a
    normal fp32 number, and where the gate's derivative crosses zero."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.cat([torch.linspace(-87.25, 87.25, 1400), torch.linspace(-2.0, 2.0, 200), torch.linspace(-1.3, -1.26, 40),
                   torch.tensor([100.0, 127.0, 129.0, 1000.0, 2.0 ** -14, -2.0 ** -14])]).to(dtype)
    a, d = torch.zeros(len(g), 2 * N, dtype=dtype), torch.zeros(len(g), N, dtype=dtype)

    def factors():
        return ((torch.rand(len(g), generator=gen) + 1) * torch.where(torch.rand(len(g), generator=gen) < 0.5, -16.0, 16.0)).to(dtype)

    a[:, at], a[:, N + at], d[:, at] = g, factors(), factors()
    return a, d


def held(got, want, off):
    """Scales `got` of single values `want` that may be off by `off`: the division by 448 adds half a step."""
    want = want.abs()
    want, off = want.clamp_min(ref.TINY), torch.where(want + off < ref.TINY, 0.0, off)
    miss = (got.cpu().double() * 448.0 - want).abs() - off - 1.001 * U * (want + off)
    assert (miss <= 0).all(), (int(miss.argmax()), float((miss / want).max()) / U)


# e^-g: two half steps of the exponential (a step of it, whichever way), one of the factor that takes the rounding of g
# log2 e back, and |g| 2^-28 of that factor's ln 2 in fp32.  1 / (1 + e^-g): one of the sum, two of the reciprocal.
def sigmoid_steps(g):
    return 6 + g.abs().clamp_max(128.0) / 16


@pytest.mark.parametrize("dtype", DTYPES)
def test_gate_to_fp32(gmi, dtype):
    a, _ = one_a_row(dtype, 128, 5, 1)
    g = a[:, 5].double()
    v = ref.swiglu(a)[:, 5]
    _, s = gmi.swiglu_quant(a.to(dev()))
    held(s[:, 0], v, (sigmoid_steps(g) + 2) * U * v.abs())  # two products


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,at", [(128, 5), (120, 64)])
def test_gate_gradient_to_fp32(gmi, dtype, N, at):
    a, d = one_a_row(dtype, N, at, 2)
    g, u, dv = a[:, at].double(), a[:, N + at].double(), d[:, at].double()
    want = ref.swiglu_bwd(d, a)
    dg, du = want[:, at], want[:, N + at]
    _, s = gmi.swiglu_bwd(d.to(dev()), a.to(dev()), quantize=True)
    held(s[:, 1], du, (sigmoid_steps(g) + 2) * U * du.abs())
    # the sum 1 + g (1 - s) loses what its terms cancel: what 1 - s is off (the exponential's and the sigmoid's half
    # steps, one of their product) stands beside the half steps of the sum, of s and of three products
    term = (dv * u * g).abs() * torch.sigmoid(g) * torch.sigmoid(-g)
    held(s[:, 0], dg, U * ((sigmoid_steps(g) + 4) * dg.abs() + (sigmoid_steps(g) + 4 + g.abs().clamp_max(128.0) / 16) * term))
