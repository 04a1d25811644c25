"""One mixture-of-experts layer over block-scaled fp8 operands, as a program runs it.

  forward   residual add + RMS norm -> fp8 rows with scales; router -> experts, weights, row order, balance loss;
            rows gathered by expert; up and gate projection per expert; SiLU; down projection per expert;
            weighted sum of each token's experts
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


def quantize(v):
    """fp8 codes and scales of a [rows][K] matrix, per row and 128 columns (plain torch: weights, once)."""
    rows, K = v.shape
    nb = -(-K // gmi.BLOCK)
    b = torch.nn.functional.pad(v.float(), (0, nb * gmi.BLOCK - K)).view(rows, nb, gmi.BLOCK)
    s = b.abs().amax(2).clamp_min(1e-30) / 448.0
    return (b / s[:, :, None]).view(rows, -1)[:, :K].to(F8), s


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

    def forward(self, x, residual, mask=None):
        """Returns the layer's output, the new residual stream and what the backward pass needs."""
        h, y = torch.empty_like(x), torch.empty_like(x)
        q, s = gmi.rmsnorm_quant(x, self.norm, residual=residual, h=h, y=y)
        logits = y @ self.router.t()
        r = gmi.moe_route(logits, self.top, mask=mask)
        # rows past the last routed one hold -1: they belong to no expert, any token will do
        token = torch.div(r.row_slot, self.top, rounding_mode="floor").clamp_min(0).long()
        a = gmi.gemm_f8_block_grouped(r.offsets, q.view(torch.uint8)[token].view(F8), s[token], *self.up)
        routed = torch.arange(len(token), device=x.device) < r.offsets[-1]
        act = torch.nn.functional.silu(a[:, : self.inner].float()) * a[:, self.inner:].float()
        aq, a_scales = quantize(torch.where(routed[:, None], act, 0.0))
        d = gmi.gemm_f8_block_grouped(r.offsets, aq, a_scales, *self.down)
        expert_out = torch.where(r.slot_row[..., None] >= 0, d[r.slot_row.clamp_min(0).long()].float(), 0.0)
        out = (expert_out * r.weights[..., None]).sum(1).to(x.dtype)
        return out, h, (h, y, logits, r, expert_out, (mask, token, routed, a))

    def backward(self, dout, dloss, saved, dh_out=None, through_experts=False):
        """Gradients of the sum before the norm (through the routing weights and the balance loss, past the norm:
        dh_out, and through the experts if asked), of the norm's and of the router's weight."""
        h, y, logits, r, expert_out, rows = saved
        dweights = (expert_out * dout[:, None].float()).sum(2)
        dlogits = gmi.moe_route_bwd(logits, r.indices, r.weights, r.offsets, r.live, dweights, dloss, mask=rows[0])
        dy = dlogits @ self.router
        if through_experts:
            dy = (dy.float() + self.experts_backward(dout, r, rows)).to(dy.dtype)
        dh, dnorm = gmi.rmsnorm_bwd(dy, h, self.norm, dres=dh_out)
        return dh, dnorm, dlogits.t().contiguous() @ y

    def experts_backward(self, dout, r, rows):
        """Gradient of the experts' input, float32 [tokens][hidden] (the roundings to fp8 have no derivative)."""
        _, token, routed, a = rows
        share = torch.where(routed, r.weights.view(-1)[r.row_slot.clamp_min(0).long()], 0.0)
        q, s = quantize(dout[token].float() * share[:, None])
        dact = gmi.gemm_f8_block_grouped(r.offsets, q, s, *self.down_t).float()
        gate, up = a[:, : self.inner].float(), a[:, self.inner:].float()
        sig = torch.sigmoid(gate)
        da = torch.cat([dact * up * sig * (1.0 + gate * (1.0 - sig)), dact * gate * sig], 1)
        q, s = quantize(torch.where(routed[:, None], da, 0.0))
        dx = gmi.gemm_f8_block_grouped(r.offsets, q, s, *self.up_t)
        return torch.where(r.slot_row[..., None] >= 0, dx[r.slot_row.clamp_min(0).long()].float(), 0.0).sum(1)


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
        out, h, saved = layer.forward(x, res)
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
