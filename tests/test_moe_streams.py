"""The fp8 mixture-of-experts calls on a stream that is not the current one: what they allocate belongs to that
stream, so that neither work still queued on the current one nor later reuse can touch it."""
import contextlib

import pytest
import torch

import moe_ref as ref
from helpers import dev


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    return g


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_new_tensors_come_from_the_stream_of_the_call(gmi, monkeypatch):
    # CPU: who is current when the allocator is asked, and whom it is told of
    current = [_Stream(5)]
    asked, told = [], []

    @contextlib.contextmanager
    def under(s):
        current.append(s)
        yield
        current.pop()

    class Made:
        def record_stream(self, s):
            told.append(s.cuda_stream)

    def empty(*a, **k):
        asked.append(current[-1].cuda_stream)
        return Made()

    monkeypatch.setattr(gmi, "_stream", lambda s: current[-1].cuda_stream if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(torch, "empty", empty)
    for stream, where, whom in ((None, 5, []), (_Stream(5), 5, []), (5, 5, []), (_Stream(9), 9, [5]), (9, 9, [5])):
        asked.clear(), told.clear()
        gmi._new((4,), torch.float32, "cpu", stream)
        assert asked == [where] and told == whom, stream
        asked.clear(), told.clear()
        gmi._scratch(16, "cpu", stream)
        assert asked == [where] and told == [], stream


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_calls_on_another_stream_beside_queued_work(gmi, as_handle):
    # the current stream holds freed blocks of the outputs' sizes that queued kernels have yet to write
    gen = torch.Generator().manual_seed(50)
    T, K, N, E, k = 320, 512, 384, 4, 2
    x, res, dy = (torch.randn(T, K, generator=gen).to(torch.bfloat16).to(dev()) for _ in range(3))
    w = torch.ones(K, dtype=torch.bfloat16, device=dev())
    logits = torch.randn(T, E, generator=gen).to(dev())
    W = (torch.randn(E, N, K, generator=gen) * 100).clamp(-448, 448).to(ref.F8).to(dev())
    ws = torch.full((E, 3, 4), 0.01, device=dev())
    off = torch.tensor([0, 100, 100, 290, T], dtype=torch.int32, device=dev())
    ones, one = torch.ones(T, k, device=dev()), torch.ones(1, device=dev())
    q0, s0 = gmi.rmsnorm_quant(x, w, residual=res)
    r0 = gmi.moe_route(logits, k)
    torch.cuda.synchronize()
    calls = [lambda st: gmi.rmsnorm_quant(x, w, residual=res, stream=st),
             lambda st: (gmi.rmsnorm_quant(x, w, residual=res, quantize=False, stream=st),),
             lambda st: gmi.rmsnorm_bwd(dy, x, w, stream=st),
             lambda st: (gmi.gemm_f8_block(q0, s0, W[1], ws[1], stream=st),),
             lambda st: (gmi.gemm_f8_block_grouped(off, q0, s0, W, ws, stream=st),),
             lambda st: gmi.moe_route(logits, k, stream=st),
             lambda st: (gmi.moe_route_bwd(logits, r0.indices, r0.weights, r0.offsets, r0.live, ones, one, stream=st),)]
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = [t.clone() for t in call(None)]
        sizes = [t.untyped_storage().nbytes() for t in want] + [1 << 20]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for n in sizes:  # written after the sleep, free for the allocator now
            torch.empty(n, dtype=torch.uint8, device=dev()).fill_(0x55)
        got = call(side.cuda_stream if as_handle else side)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(want, got)), i


@pytest.mark.gpu
def test_calls_on_a_forked_stream_in_a_graph(gmi):
    # captured on one stream, run on another that joins the capture: outputs and workspaces from the graph's memory
    gen = torch.Generator().manual_seed(51)
    T, K, N, E, k = 200, 2048, 256, 8, 2
    x, dy = (torch.randn(T, K, generator=gen).to(torch.bfloat16).to(dev()) for _ in range(2))
    w = torch.ones(K, dtype=torch.bfloat16, device=dev())
    logits = torch.randn(T, E, generator=gen).to(dev())
    W = (torch.randn(N, K, generator=gen) * 100).clamp(-448, 448).to(ref.F8).to(dev())
    ws = torch.full((2, 16), 0.01, device=dev())
    assert gmi.lib().gmi_gemm_f8_block_workspace_bytes(T, N, K) > 0

    def calls(st):
        q, s = gmi.rmsnorm_quant(x, w, stream=st)
        return [gmi.gemm_f8_block(q, s, W, ws, stream=st), *gmi.moe_route(logits, k, stream=st),
                *gmi.rmsnorm_bwd(dy, x, w, stream=st)]

    calls(None)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        held = calls(side)
        torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        x.copy_(torch.randn(T, K, generator=gen).to(torch.bfloat16))
        logits.copy_(torch.randn(T, E, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        eager = calls(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), f"replay {step}"
