"""GPU: the calls that move and shape rows and the adapters' product on other streams, in captured graphs, at the ends of
their size ranges, and one after another as a layer uses them."""
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


class Case:
    """Inputs of every call; `calls(stream)` runs them and returns their outputs, all made by the calls."""

    def __init__(self, gmi, seed, rows=700):
        gen = torch.Generator().manual_seed(seed)
        self.gmi, self.gen = gmi, gen
        T, k, K, L, r = 600, 3, 520, 5, 24
        self.index = torch.randint(-1, L, (6000,), generator=gen).to(torch.int32).to(dev())
        self.slots = ref.slots(gen, T, k, 0, dead=0.0).to(dev())
        self.x = self.randn(T, K)
        self.y, self.a = self.randn(T * k, K), self.randn(T * k, 2 * 264)
        self.dact = self.randn(T * k, 264)
        self.w = torch.rand(T, k, generator=gen).to(dev())
        self.X, self.base = self.randn(rows, K), self.randn(rows, 328)
        self.A, self.B = self.randn(L, r, K), self.randn(L, 328, r)
        self.adapter = torch.randint(-1, L, (rows,), generator=gen).to(torch.int32).to(dev())

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(torch.bfloat16).to(dev())

    def calls(self, st):
        g = self.gmi
        order = g.group_rows(self.adapter, 5, stream=st).order
        out = [*g.group_rows(self.index, 5, stream=st), order, g.moe_permute(self.x, self.slots, stream=st),
               g.moe_unpermute(self.y, self.slots, weights=self.w, add=self.x, stream=st),
               *g.moe_unpermute_bwd(self.x, self.slots, weights=self.w, rows=self.y, quantize=True, stream=st),
               *g.moe_unpermute_bwd(self.x, self.slots, weights=self.w, rows=self.y, stream=st),
               *g.swiglu_quant(self.a, stream=st), g.swiglu_quant(self.a, quantize=False, stream=st),
               g.swiglu_bwd(self.dact, self.a, stream=st), *g.swiglu_bwd(self.dact, self.a, quantize=True, stream=st),
               g.gemm_lora(self.X, self.A, self.B, self.adapter, order=order, base=self.base, stream=st)]
        return out

    def renew(self):
        for t in (self.x, self.y, self.a, self.dact, self.X, self.base):
            t.copy_(torch.randn(t.shape, generator=self.gen))
        self.adapter.copy_(torch.randint(-1, 5, self.adapter.shape, generator=self.gen))
        self.index.copy_(torch.randint(-1, 5, self.index.shape, generator=self.gen))


@pytest.mark.parametrize("rows", [100, 700])
@pytest.mark.parametrize("as_handle", [False, True])
def test_on_another_stream_beside_queued_work(gmi, as_handle, rows):
    # the current stream holds freed blocks of the outputs' sizes that queued kernels have yet to write
    c = Case(gmi, 1, rows)
    want = [t.clone() for t in c.calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    for t in want:
        torch.empty(t.untyped_storage().nbytes(), dtype=torch.uint8, device=dev()).fill_(0x55)
    got = c.calls(side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(want, got)):
        assert same(a, b), i


@pytest.mark.parametrize("rows", [100, 700])
def test_in_a_graph_on_a_forked_stream(gmi, rows):
    c = Case(gmi, 2, rows)
    c.calls(None)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        held = c.calls(side)
        torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        c.renew()
        graph.replay()
        torch.cuda.synchronize()
        eager = c.calls(None)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, eager)):
            assert same(a, b), (step, i)


def test_two_graphs_and_eager_calls_share_a_workspace(gmi):
    cases = [Case(gmi, 3, 700), Case(gmi, 4, 90)]
    ws = torch.empty(8 << 20, dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()

    def run(c, out):
        gmi.group_rows(c.index, 5, out=out[0], workspace=ws)
        gmi.gemm_lora(c.X, c.A, c.B, c.adapter, base=c.base, Y=out[1], workspace=ws)

    held, graphs = [], []
    for c in cases:
        i32 = dict(dtype=torch.int32, device=dev())
        out = gmi.Grouping(torch.empty(6, **i32), torch.empty(6000, **i32), torch.empty(6000, **i32)), torch.empty_like(c.base)
        run(c, out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run(c, out)
        held.append(out)
        graphs.append(g)
    for step in range(3):
        for c in cases:
            c.renew()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, (group, Y) in zip(cases, held):
            for a, b in zip(group, gmi.group_rows(c.index, 5)):
                assert torch.equal(a, b), step
            assert same(Y, gmi.gemm_lora(c.X, c.A, c.B, c.adapter, base=c.base)), step


def test_two_streams_at_once(gmi):
    cases = [Case(gmi, 5), Case(gmi, 6)]
    want = [[t.clone() for t in c.calls(None)] for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [c.calls(s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(same(a, b) for a, b in zip(w, g))


def test_rows_more_than_4_gb_apart(gmi):
    # leading dimensions that put rows past 32-bit byte offsets
    rows, ld, K = 40, 1 << 27, 256
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device=dev())  # 10 GB
    gen = torch.Generator().manual_seed(7)

    def far(n, cols, at, fill=True):
        v = torch.as_strided(big, (n, cols), (ld, 1), at)
        near = torch.randn(n, cols, generator=gen).to(torch.bfloat16).to(dev())
        v.copy_(near if fill else torch.zeros_like(near))
        return v, near

    slots = ref.slots(gen, 20, 2, 0, dead=0.0).to(dev())
    w = torch.rand(20, 2, generator=gen).to(dev())
    (y, yn), (x, xn), (a, an) = far(40, K, 0), far(20, K, 1024), far(40, 2 * K, 2048)
    out, _ = far(40, K, 4096, fill=False)
    gmi.moe_permute(x, slots, out=out)
    assert same(out, gmi.moe_permute(xn, slots))
    back, _ = far(20, K, 8192, fill=False)
    gmi.moe_unpermute(y, slots, weights=w, add=x, out=back)
    assert same(back, gmi.moe_unpermute(yn, slots, weights=w, add=xn))
    _, dw = gmi.moe_unpermute_bwd(x, slots, weights=w, rows=y, drows=out)
    dn, dwn = gmi.moe_unpermute_bwd(xn, slots, weights=w, rows=yn)
    assert same(out, dn) and same(dw, dwn)
    gmi.swiglu_quant(a, y=out, quantize=False)
    assert same(out, gmi.swiglu_quant(an, quantize=False))
    da, _ = far(40, 2 * K, 16384, fill=False)
    gmi.swiglu_bwd(y, a, da=da)
    assert same(da, gmi.swiglu_bwd(yn, an))
    A, B = (torch.randn(3, n, c, generator=gen).to(torch.bfloat16).to(dev()) for n, c in ((16, K), (K, 16)))
    idx = torch.randint(0, 3, (40,), generator=gen).to(torch.int32).to(dev())
    gmi.gemm_lora(y, A, B, idx, base=a[:, :K], Y=out)
    assert same(out, gmi.gemm_lora(yn, A, B, idx, base=an[:, :K].contiguous()))
    # adapters as far apart
    Af, Bf = (torch.as_strided(big, (3, n, c), (ld * 12, c, 1), at) for n, c, at in ((16, K, 65536), (K, 16, 131072)))
    Af.copy_(A), Bf.copy_(B)
    assert same(out, gmi.gemm_lora(yn, Af, Bf, idx, base=an[:, :K].contiguous()))


def test_lora_long_runs_with_rows_4_gb_apart(gmi):
    M, ld, K, N = 520, 1 << 23, 128, 72
    big = torch.empty(M * ld, dtype=torch.float16, device=dev())  # 8.7 GB
    gen = torch.Generator().manual_seed(8)
    near = [torch.randn(M, c, generator=gen).half().to(dev()) for c in (K, N)]
    X, base = (torch.as_strided(big, (M, c), (ld, 1), at) for c, at in ((K, 0), (N, 4096)))
    X.copy_(near[0]), base.copy_(near[1])
    A, B = (torch.randn(2, n, c, generator=gen).half().to(dev()) for n, c in ((8, K), (N, 8)))
    idx = (torch.arange(M) // 300).to(torch.int32).to(dev())
    gmi.gemm_lora(X, A, B, idx, base=base, Y=base)
    assert same(base, gmi.gemm_lora(near[0], A, B, idx, base=near[1]))


def test_more_tokens_than_waves_of_a_launch(gmi):
    # a launch has 2^22 waves; the rest of the tokens is walked to
    T = (1 << 22) + 77
    x = torch.randint(0, 256, (T, 16), dtype=torch.uint8, device=dev())
    slots = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev()).view(T, 1)
    assert torch.equal(gmi.moe_permute(x.view(ref.F8), slots).view(torch.uint8), x.flip(0))
    y = torch.randint(-8, 8, (T, 8), device=dev()).to(torch.bfloat16)
    assert torch.equal(gmi.moe_unpermute(y, slots), y.flip(0))
    w = torch.full((T, 1), 2.0, device=dev())
    drows, dw = gmi.moe_unpermute_bwd(y, slots, weights=w, rows=y)
    assert torch.equal(drows, 2 * y.flip(0)) and torch.equal(dw, (y.float() * y.flip(0).float()).sum(1, keepdim=True))


def test_gate_over_several_launches(gmi):
    # 2^27 blocks a launch; the rows in use end in the second
    rows = (1 << 27) + 300
    a = torch.zeros(rows, 16, dtype=torch.bfloat16, device=dev())
    a[-400:] = torch.randn(400, 16, device=dev()).to(torch.bfloat16)
    y = torch.full((rows, 8), 3.0, dtype=torch.bfloat16, device=dev())
    live = torch.tensor([rows - 100], dtype=torch.int32, device=dev())
    gmi.swiglu_quant(a, live=live, y=y, quantize=False)
    assert same(y[-400:-100], gmi.swiglu_quant(a[-400:-100].contiguous(), quantize=False))
    assert (y[-100:] == 3.0).all() and int((y[:-400] != 0).sum()) == 0
    dact = torch.ones(rows, 8, dtype=torch.bfloat16, device=dev())
    da = gmi.swiglu_bwd(dact, a, live=live, da=a)  # in place
    want = gmi.swiglu_bwd(dact[:300].contiguous(), a[-100:].new_zeros(300, 16))
    assert da is a and same(a[1000:1300], want)


def test_chain_in_16_bits(gmi):
    # routing, rows out, two grouped products with the gate between them, rows back beside a shared expert, an adapter on
    # top: each stage against float64 on what the stage before left
    gen = torch.Generator().manual_seed(9)
    T, k, E, H, N = 300, 2, 6, 256, 136

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).to(dev())

    x, shared = randn(T, H), randn(T, H)
    Wu, Wd = randn(E, 2 * N, H, std=H ** -0.5), randn(E, H, N, std=N ** -0.5)
    mask = (torch.rand(T, generator=gen) > 0.1).to(dev())
    r = gmi.moe_route(torch.randn(T, E, generator=gen).to(dev()), k, mask=mask)
    used = int(r.offsets[-1])
    rows = gmi.moe_permute(x, r.slot_row)
    token = (r.row_slot[:used] // k).long()
    assert torch.equal(rows[:used], x[token])
    a = torch.zeros(T * k, 2 * N, dtype=torch.bfloat16, device=dev())
    gmi.gemm_grouped_offsets(r.offsets, rows, Wu, a)
    expert = torch.repeat_interleave(torch.arange(E, device=dev()), r.counts.long())
    want = torch.stack([rows[i].double() @ Wu[expert[i]].double().t() for i in range(used)])
    assert ((a[:used].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10).all()
    act = gmi.swiglu_quant(a, live=r.offsets[-1:], quantize=False)
    v = ref.swiglu(a[:used].cpu())
    assert ((act[:used].cpu().double() - v).abs() <= (2.0 ** -8 + 2.0 ** -18) * v.abs() + ref.FLOOR[torch.bfloat16]).all()
    d = torch.zeros(T * k, H, dtype=torch.bfloat16, device=dev())
    gmi.gemm_grouped_offsets(r.offsets, act, Wd, d)
    out = gmi.moe_unpermute(d, r.slot_row, weights=r.weights, add=shared)
    o, mag = ref.unpermute(d.cpu(), r.slot_row.cpu(), r.weights.cpu(), shared.cpu())
    assert ((out.cpu().double() - o).abs() <= 2.0 ** -8 * o.abs() + 4 * 2.0 ** -24 * mag).all()
    A, B = randn(3, 16, H, std=H ** -0.5), randn(3, H, 16, std=0.25)
    adapter = torch.randint(-1, 3, (T,), generator=gen).to(torch.int32)
    keep = out.clone()
    gmi.gemm_lora(x, A, B, adapter.to(dev()), order=gmi.group_rows(adapter.to(dev()), 3).order, base=out, Y=out)
    want = ref.lora(x.cpu(), A.cpu(), B.cpu(), adapter, None, keep.cpu())
    assert ((out.cpu().double() - want[0]).abs() <= ref.lora_tolerance(*want, torch.bfloat16, H, 16)).all()
    assert torch.equal(out[adapter.to(dev()) < 0], keep[adapter.to(dev()) < 0])
