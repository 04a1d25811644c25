"""One mixture-of-experts layer over block-scaled fp8 operands, as a program runs it.

  forward   residual add + RMS norm -> fp8 rows with scales; router -> experts, weights, row order, balance loss;
            rows to their experts; up and gate projection per expert; gated activation in fp8; down projection per
            expert; weighted sum of each token's experts
  backward  of the routing weights, the balance loss and the norm, and with through_experts of the experts' input, the
            layer's whole data gradient: the same grouped products with the transposed weights, on gradients that are
            quantised as activations are (the experts' weights are frozen)

    python examples/moe_layer_f8.py [--tokens 4096] [--hidden 4096] [--inner 1024] [--experts 128] [--top 8]
"""
import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))
import grouped_mixed_input_amd as gmi  # noqa: E402

F8 = torch.float8_e4m3fn


def quantize_weight(w):
    """fp8 codes and scales of [experts][N][K] weights, per 128 x 128 block."""
    E, N, K = w.shape
    nb, kb = -(-N // gmi.BLOCK), -(-K // gmi.BLOCK)
    b = torch.nn.functional.pad(w.float(), (0, kb * gmi.BLOCK - K, 0, nb * gmi.BLOCK - N))
    b = b.view(E, nb, gmi.BLOCK, kb, gmi.BLOCK)
    s = b.abs().amax((2, 4)).clamp_min(1e-30) / 448.0
    q = (b / s[:, :, None, :, None]).view(E, nb * gmi.BLOCK, kb * gmi.BLOCK)[:, :N, :K].contiguous()
    return q.to(F8), s


def transposed(w, s):
    """The weights of the data gradient: codes and block scales of [experts][N][K] as those of [experts][K][N]."""
    return w.view(torch.uint8).transpose(1, 2).contiguous().view(F8), s.transpose(1, 2).contiguous()


class Layer:
    """Weights of one layer: norm [hidden], router [experts][hidden], gate + up [experts][2 inner][hidden], down
    [experts][hidden][inner]."""

    def __init__(self, hidden, inner, experts, top, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def randn(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device)

        self.top, self.inner = top, inner
        self.norm = (1.0 + randn(hidden, std=0.1)).bfloat16()
        self.router = randn(experts, hidden, std=hidden ** -0.5).bfloat16()
        self.up = quantize_weight(randn(experts, 2 * inner, hidden, std=hidden ** -0.5))
        self.down = quantize_weight(randn(experts, hidden, inner, std=inner ** -0.5))
        self.up_t, self.down_t = transposed(*self.up), transposed(*self.down)

    def forward(self, x, residual, mask=None, per_slot=True):
        """Returns the layer's output, the new residual stream and what the backward pass needs; with it, for
        inspection, the experts' output of each slot in float32 (None without per_slot)."""
        h, y = torch.empty_like(x), torch.empty_like(x)
        q, s = gmi.rmsnorm_quant(x, self.norm, residual=residual, h=h, y=y)
        logits = y @ self.router.t()
        r = gmi.moe_route(logits, self.top, mask=mask)
        # rows past the last routed one belong to no expert: nothing reads or writes them
        a = gmi.gemm_f8_block_grouped(r.offsets, *gmi.moe_permute(q, r.slot_row, scales=s), *self.up)
        d = gmi.gemm_f8_block_grouped(r.offsets, *gmi.swiglu_quant(a, live=r.offsets[-1:]), *self.down)
        out = gmi.moe_unpermute(d, r.slot_row, weights=r.weights)
        expert_out = None
        if per_slot:
            expert_out = torch.where(r.slot_row[..., None] >= 0, d[r.slot_row.clamp_min(0).long()].float(), 0.0)
        return out, h, (h, y, logits, r, expert_out, (mask, a, d))

    def backward(self, dout, dloss, saved, dh_out=None, through_experts=False):
        """Gradients of the sum before the norm (through the routing weights and the balance loss, past the norm:
        dh_out, and through the experts if asked), of the norm's and of the router's weight."""
        h, y, logits, r, _, (mask, a, d) = saved
        if through_experts:
            q, s, dweights = gmi.moe_unpermute_bwd(dout, r.slot_row, weights=r.weights, rows=d, quantize=True)
        else:
            _, dweights = gmi.moe_unpermute_bwd(dout, r.slot_row, weights=r.weights, rows=d, row_grad=False)
        dlogits = gmi.moe_route_bwd(logits, r.indices, r.weights, r.offsets, r.live, dweights, dloss, mask=mask)
        dy = dlogits @ self.router
        if through_experts:
            # the experts' data gradient: the transposed products (the roundings to fp8 have no derivative)
            dact = gmi.gemm_f8_block_grouped(r.offsets, q, s, *self.down_t)
            q, s = gmi.swiglu_bwd(dact, a, live=r.offsets[-1:], quantize=True)
            dy = gmi.moe_unpermute(gmi.gemm_f8_block_grouped(r.offsets, q, s, *self.up_t), r.slot_row, add=dy, out=dy)
        dh, dnorm = gmi.rmsnorm_bwd(dy, h, self.norm, dres=dh_out)
        return dh, dnorm, dlogits.t().contiguous() @ y


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4096), ("hidden", 4096), ("inner", 1024), ("experts", 128), ("top", 8)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    layer = Layer(a.hidden, a.inner, a.experts, a.top)
    gen = torch.Generator().manual_seed(1)
    x, res, dout = (torch.randn(a.tokens, a.hidden, generator=gen).bfloat16().cuda() for _ in range(3))
    dloss = torch.tensor([0.01], device="cuda")

    def step():
        out, h, saved = layer.forward(x, res, per_slot=False)
        return saved[3], layer.backward(dout, dloss, saved, dh_out=dout, through_experts=True)

    for _ in range(3):
        r, _ = step()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        step()
    stop.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.experts} experts, top {a.top}: {start.elapsed_time(stop) / 10:.3f} ms forward and "
          f"backward; balance loss {float(r.loss):.3f}, rows per expert {int(r.counts.min())} .. {int(r.counts.max())}")


if __name__ == "__main__":
    main()
