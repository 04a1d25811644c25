"""64-bit definitions of the block-scaled fp8 mixture-of-experts operators, on the CPU, for the tests."""
import numpy as np
import torch

F8 = torch.float8_e4m3fn
TINY = 448.0 * 2.0 ** -126


def blocks(n):
    return (n + 127) // 128


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm(x, weight, residual, eps):
    """h, v, s, v / s in float64."""
    h = x.double() + (residual.double() if residual is not None else 0.0)
    v = weight.double() * h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    K = x.shape[1]
    pad = torch.nn.functional.pad(v, (0, blocks(K) * 128 - K)).view(x.shape[0], blocks(K), 128)
    s = pad.abs().amax(2).clamp_min(TINY) / 448.0
    t = (pad / s[:, :, None]).view(x.shape[0], -1)[:, :K]
    return h, v, s, t


def norm_bwd(dy, h, weight, dres, eps):
    """dh, dweight, and the sums of magnitudes their roundings grow with."""
    dy, h, w = dy.double(), h.double(), weight.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    n, g = h * r, dy * w
    dh = r * (g - n * (g * n).mean(1, keepdim=True))
    mag = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    return dh, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def spread(q, s, rows_per_scale):
    v = q.float().double() * s.double().repeat_interleave(rows_per_scale, 0)[: q.shape[0]].repeat_interleave(
        128, 1)[:, : q.shape[1]]
    return v


def gemm(X, xs, W, ws):
    """The product and the sum of the terms' magnitudes."""
    x, w = spread(X, xs, 1), spread(W, ws, 128)
    return x @ w.t(), x.abs() @ w.abs().t()


def gemm_tolerance(ref, mag, K):
    """Half a bf16 step, and fp32 sums of 128 terms in a block and of the blocks (2^-23 per addition, whichever way
    it rounds, and the products with the scales)."""
    return 2.0 ** -8 * ref.abs() + (128 + blocks(K) + 16) * 2.0 ** -23 * mag


def route(logits, k, mask, renorm):
    """Everything moe_route writes, by an insertion over numpy rows."""
    x = logits.double().numpy()
    T, E = x.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    psum, live_n = np.zeros(E), 0
    for t in range(T):
        row = x[t]
        ok = [e for e in range(E) if row[e] > -np.inf]
        if (mask is not None and not bool(mask[t])) or not ok:
            continue
        live_n += 1
        take = sorted(ok, key=lambda e: (-row[e], e))[:k]
        with np.errstate(invalid="ignore"):
            ex = np.exp(row - row[take[0]])
            p = ex / ex.sum()
        psum += p
        idx[t, : len(take)] = take
        w[t, : len(take)] = p[take] / (p[take].sum() if renorm else 1.0)
        if renorm and np.isnan(p).any():
            w[t, : len(take)] = np.nan
    flat = idx.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)], np.int64)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    row_slot = np.full(T * k, -1, np.int64)
    order = [s for e in range(E) for s in np.flatnonzero(flat == e)]
    row_slot[: len(order)] = order
    slot_row = np.full(T * k, -1, np.int64)
    slot_row[order] = np.arange(len(order))
    total = offsets[-1]
    loss = E * (counts / total * psum).sum() / live_n if live_n else 0.0
    return dict(indices=idx, weights=w, counts=counts, offsets=offsets, slot_row=slot_row.reshape(T, k),
                row_slot=row_slot, loss=loss, live=live_n)


def route_objective(x, ref, k, mask, renorm, dweights, dloss):
    """sum(dweights * weights) + dloss * loss as a function of the float64 logits, the selection held fixed."""
    T, E = x.shape
    live = torch.isfinite(x).any(1) | (x == np.inf).any(1)
    if mask is not None:
        live = live & mask.bool()
    p = torch.where(live[:, None], torch.softmax(torch.where(live[:, None], x, torch.zeros_like(x)), 1), 0.0)
    idx = torch.from_numpy(ref["indices"].astype(np.int64))
    w = torch.where(idx >= 0, p.gather(1, idx.clamp_min(0)), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    f = torch.from_numpy(ref["counts"].astype(np.float64)) / max(int(ref["offsets"][-1]), 1)
    loss = E * (f * p.sum(0)).sum() / max(ref["live"], 1)
    return (torch.where(idx >= 0, dweights.double(), 0.0) * w).sum() + dloss * loss
