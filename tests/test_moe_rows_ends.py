"""GPU: the rows' calls at the ends of their ranges of sizes."""
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


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("n,groups", [(17_000_001, 1024), (40_000_000, 3)])
def test_group_rows_past_256_workgroups(gmi, n, groups):
    # a workgroup counts at most 64512 rows, so that there are more than 256
    index = torch.randint(-1, groups + 1, (n,), dtype=torch.int32, device=dev())
    got = gmi.group_rows(index, groups)
    none = (index < 0) | (index >= groups)
    key = torch.where(none, groups, index)
    counts = torch.bincount(key, minlength=groups + 1)
    order = torch.argsort(key, stable=True)
    assert torch.equal(got.offsets.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)[:groups]]))
    assert torch.equal(got.order.long(), order)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(n, device=dev()))
    assert torch.equal(got.place.long(), torch.where(none, -1, place))


@pytest.mark.parametrize("N", [1 << 22, (1 << 22) - 8, (1 << 21) + 136])
def test_gate_of_the_widest_rows(gmi, N):
    gen = torch.Generator(device=dev()).manual_seed(N)
    a = torch.randn(3, 2 * N, generator=gen, device=dev()).to(torch.bfloat16)
    dact = torch.randn(3, N, generator=gen, device=dev()).to(torch.bfloat16)
    cut = torch.cat([torch.arange(0, 4096), torch.arange(N - N % 128 - 4096, N)]).to(dev())  # whole blocks at both ends
    y = torch.empty(3, N, dtype=torch.bfloat16, device=dev())
    q, s = gmi.swiglu_quant(a, y=y)
    part = torch.cat([a[:, cut], a[:, N + cut]], 1)
    py = torch.empty(3, len(cut), dtype=torch.bfloat16, device=dev())
    pq, ps = gmi.swiglu_quant(part, y=py)
    assert same(y[:, cut], py) and same(q.view(torch.uint8)[:, cut], pq) and same(s[:, cut[::128] // 128], ps)
    da, pda = gmi.swiglu_bwd(dact, a), gmi.swiglu_bwd(dact[:, cut].contiguous(), part)
    assert same(torch.cat([da[:, cut], da[:, N + cut]], 1), pda)
    # codes: the 16-bit gradient is off by half its step, a code by half a code's
    dq, ds = gmi.swiglu_bwd(dact, a, quantize=True)
    spread = ds.repeat_interleave(128, 1)[:, : 2 * N]
    got, want = dq.float() * spread, da.float()
    assert ((got - want).abs() <= (2.0 ** -4 + 2.0 ** -7) * want.abs() + 2.0 ** -10 * spread).all()
    top = torch.nn.functional.pad(want.abs(), (0, ds.shape[1] * 128 - 2 * N)).view(3, -1, 128).amax(2) / 448.0
    assert ((ds - top).abs() <= 2.0 ** -7 * top).all()


@pytest.mark.parametrize("quant", [False, True])
def test_weights_gradient_of_more_tokens_than_workgroups(gmi, quant):
    # four waves a token, 2^20 workgroups a launch: the first ones take a second token
    T, K = (1 << 20) + 5, 520
    y = torch.randint(-4, 5, (T, K), device=dev(), dtype=torch.int8).to(torch.bfloat16)
    dout = torch.randint(-4, 5, (T, K), device=dev(), dtype=torch.int8).to(torch.bfloat16)
    slots = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev()).view(T, 1)
    w = torch.full((T, 1), -2.0, device=dev())
    got = gmi.moe_unpermute_bwd(dout, slots, weights=w, rows=y, quantize=quant)
    want = torch.cat([(dout[i:i + 65536].float() * y.flip(0)[i:i + 65536].float()).sum(1) for i in range(0, T, 65536)])
    assert torch.equal(got[-1][:, 0], want)  # whole numbers
    if not quant:
        assert torch.equal(got[0], -2 * dout.flip(0))
    else:
        for i in list(range(0, T, 1 << 17)) + [T - 7]:
            d = -2.0 * dout.flip(0)[i:i + 7].double().cpu()
            ref.check_codes(got[0][i:i + 7].cpu(), got[1][i:i + 7].cpu(), d, 0.0)


@pytest.mark.parametrize("N", [136, 256])
def test_gate_gradient_codes_into_parts_of_wider_buffers(gmi, N):
    gen = torch.Generator().manual_seed(N)
    a, dact = (torch.randn(50, c, generator=gen).to(torch.bfloat16).to(dev()) for c in (2 * N, N))
    wq = torch.full((50, 2 * N + 24), 0x55, dtype=torch.uint8, device=dev())
    ws = torch.full((50, ref.blocks(2 * N) + 3), 7.0, device=dev())
    q, s = wq[:, 8:8 + 2 * N].view(ref.F8), ws[:, 1:1 + ref.blocks(2 * N)]
    gmi.swiglu_bwd(dact, a, da=q, scales=s, quantize=True)
    q2, s2 = gmi.swiglu_bwd(dact, a, quantize=True)
    assert same(wq[:, 8:8 + 2 * N], q2) and same(s, s2)
    assert (wq[:, :8] == 0x55).all() and (wq[:, 8 + 2 * N:] == 0x55).all()
    assert (ws[:, 0] == 7.0).all() and (ws[:, 1 + ref.blocks(2 * N):] == 7.0).all()


def test_permute_codes_without_scales(gmi):
    x = torch.randint(0, 256, (40, 272), dtype=torch.uint8, device=dev())
    slots = ref.slots(torch.Generator().manual_seed(1), 40, 3, 0, dead=0.0).to(dev())
    out = gmi.moe_permute(x.view(ref.F8), slots)
    assert torch.equal(out.view(torch.uint8)[slots.long()], x[:, None].expand(40, 3, 272))
