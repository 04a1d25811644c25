"""Cases and plain forms of the block-scaled fp8 mixture-of-experts operators.

Three operators that one layer runs after another, each in the directions a user calls:

  norm        h = x + residual; y = weight * h / rms(h); y in fp8 E4M3 with one fp32 scale per row and 128 columns
  norm_bwd    gradients of h and of the weight, with the gradient that the residual stream brings
  gemm        Y = X W^T, X and W in fp8 with scales per 1 x 128 (X) and 128 x 128 (W) block, Y bf16
  grouped     the same per expert, the experts' row ranges in device memory
  route       top-k experts of each token, their weights, counts, row offsets and order, and the balance loss
  route_bwd   gradient of the logits from those of the weights and of the loss

`own` selects who computes: False, elementary torch operations in fp32; True, grouped_mixed_input_amd.
"""
import math

import torch

own = False

BLOCK = 128
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY_AMAX = F8_MAX * 2.0**-126  # keeps the scale of an all-zero block a normal number
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of a decode step: latency of a single row
        dict(name="norm token", op="norm", rows=1, cols=4096, dtype="bf16"),
        # the prompt tokens of the mixture-of-experts layer
        dict(name="norm prefill", op="norm", rows=16384, cols=4096, dtype="bf16"),
        # a short fine-tuning batch in fp16, last block partial
        dict(name="norm bwd ragged", op="norm_bwd", rows=333, cols=2000, dtype="fp16"),
        # a training step's backward over the same layer
        dict(name="norm bwd train", op="norm_bwd", rows=16384, cols=4096, dtype="bf16"),
        # a decode step of 16 sequences through one dense projection: weights are read once
        dict(name="gemm decode", op="gemm", rows=16, n=8192, k=8192),
        # a prompt chunk through the same kind of projection: matrix-bound
        dict(name="gemm prefill", op="gemm", rows=4096, n=8192, k=8192),
        # 16 tokens routed to 8 of 128 experts each: most experts see one or two rows
        dict(name="experts decode", op="grouped", groups=128, rows=128, n=2048, k=4096),
        # the full mixture-of-experts layer, skewed experts, some without rows
        dict(name="experts prefill", op="grouped", groups=128, rows=16384, n=2048, k=4096),
        # routing of one decode step
        dict(name="route decode", op="route", tokens=16, experts=128, top=8, dtype="fp32", renorm=True, blocked=False),
        # routing of a prompt; padding tokens masked out
        dict(name="route prefill", op="route", tokens=16384, experts=128, top=8, dtype="bf16", renorm=True, blocked=False),
        # backward of a short batch: odd sizes, some experts closed to some tokens
        dict(name="route bwd ragged", op="route_bwd", tokens=777, experts=60, top=4, dtype="fp32", renorm=False, blocked=True),
        # backward of a training step
        dict(name="route bwd train", op="route_bwd", tokens=16384, experts=128, top=8, dtype="bf16", renorm=True, blocked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gemm", "grouped", "route", "route_bwd"])
    if op in ("norm", "norm_bwd"):
        return dict(op=op, rows=_log(rng, 1, 16384), cols=16 * _log(rng, 8, 512), dtype=rng.choice(["bf16", "fp16"]))
    if op == "gemm":
        return dict(op=op, rows=_log(rng, 1, 4096), n=_log(rng, 64, 8192), k=16 * _log(rng, 8, 512))
    if op == "grouped":
        return dict(op=op, groups=_log(rng, 1, 128), rows=_log(rng, 1, 16384), n=_log(rng, 64, 2048), k=16 * _log(rng, 8, 256))
    experts = _log(rng, 4, 256)
    return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, top=rng.randint(1, min(8, experts)),
                dtype=rng.choice(["bf16", "fp16", "fp32"]), renorm=rng.random() < 0.5, blocked=rng.random() < 0.5)


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- inputs
def _f8_blocks(gen, *shape):
    """Codes as a quantiser leaves them: every block of 128 reaches far up the format's range."""
    q = torch.randn(shape, generator=gen, device="cuda")
    return q.mul_(120.0).clamp_(-F8_MAX, F8_MAX).to(F8)


def _scales(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").mul_(0.3).exp_().mul_(2.0**-8)


def _offsets(seed, groups, rows):
    """Row ranges of the experts: Zipf-skewed counts, one expert in sixteen without rows."""
    g = torch.Generator().manual_seed(seed)
    p = (torch.randperm(groups, generator=g) + 1).double() ** -1.1
    p[torch.randperm(groups, generator=g)[: groups // 16]] = 0.0
    pick = torch.multinomial(p, rows, replacement=True, generator=g)
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(pick, minlength=groups).cumsum(0)]).to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        spread = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 12.0, 1.0)  # outlier channels
        s["weight"] = (1.0 + 0.1 * randn(cols)).to(dt)
        if op == "norm":
            s["x"] = randn(rows, cols).to(dt)
            s["residual"] = (randn(rows, cols) * spread).to(dt)
            s["h"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            s["q"] = torch.empty(rows, cols, dtype=F8, device="cuda")
            s["scale"] = torch.empty(rows, _blocks(cols), device="cuda")
        else:
            s["h"] = (randn(rows, cols) * spread).to(dt)
            s["dy"] = randn(rows, cols).to(dt)
            s["dres"] = randn(rows, cols).to(dt)
            s["dh"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            s["dweight"] = torch.empty(cols, device="cuda")
    elif op in ("gemm", "grouped"):
        rows, n, k = case["rows"], case["n"], case["k"]
        lead = () if op == "gemm" else (case["groups"],)
        s["X"], s["xs"] = _f8_blocks(gen, rows, k), _scales(gen, rows, _blocks(k))
        s["W"], s["ws"] = _f8_blocks(gen, *lead, n, k), _scales(gen, *lead, _blocks(n), _blocks(k))
        s["Y"] = torch.empty(rows, -(-n // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :n]
        if op == "grouped":
            s["offsets"] = _offsets(seed, case["groups"], rows)
    else:
        t, e = case["tokens"], case["experts"]
        logits = randn(t, e) + 0.5 * randn(e)
        if case["blocked"]:  # experts closed to a token (capacity or placement); some tokens find all closed
            logits.masked_fill_(torch.rand(t, e, generator=gen, device="cuda") < 0.1, -math.inf)
            logits.masked_fill_(torch.rand(t, 1, generator=gen, device="cuda") < 0.01, -math.inf)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["mask"] = torch.rand(t, generator=gen, device="cuda") >= 0.03  # padding tokens are False
        if t < 32:
            s["mask"].fill_(True)
        if op == "route":
            k = case["top"]
            i32 = dict(dtype=torch.int32, device="cuda")
            s["out"] = (torch.empty(t, k, **i32), torch.empty(t, k, device="cuda"), torch.empty(e, **i32), torch.empty(e + 1, **i32),
                        torch.empty(t, k, **i32), torch.empty(t * k, **i32), torch.empty(1, device="cuda"), torch.empty(1, **i32))
        else:
            s["routed"] = _route_plain(s["logits"], s["mask"], case["top"], case["renorm"])
            s["dweights"] = randn(t, case["top"])
            s["dloss"] = torch.full((1,), 0.01 * t, device="cuda")  # the training loss is summed over tokens
            s["dlogits"] = torch.empty_like(s["logits"])
    # scratch that a program keeps for its calls
    s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _norm_plain(s):
    rows, cols, dt = s["rows"], s["cols"], DTYPES[s["dtype"]]
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    nb = _blocks(cols)
    yb = torch.nn.functional.pad(y, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    scale = yb.abs().amax(2).clamp_min(TINY_AMAX) / F8_MAX
    q = (yb / scale[:, :, None]).view(rows, nb * BLOCK)[:, :cols].to(F8)
    return {"h": h.to(dt), "q": q, "scale": scale}


def _norm_bwd_plain(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * r
    g = dy * w
    dh = s["dres"].float() + r * (g - n * (g * n).mean(1, keepdim=True))
    return {"dh": dh.to(s["h"].dtype), "dweight": (dy * n).sum(0)}


def _spread(q, scale, rows_per_scale):
    """Blocks of codes times their scales."""
    s = scale.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[: q.shape[0]]
    return q.to(scale.dtype) * s


def _gemm_plain(s):
    return {"Y": (_spread(s["X"], s["xs"], 1) @ _spread(s["W"], s["ws"], BLOCK).t()).to(torch.bfloat16)}


def _grouped_plain(s):
    x = _spread(s["X"], s["xs"], 1)
    off = s["offsets"].tolist()
    parts = [x[off[g]:off[g + 1]] @ _spread(s["W"][g], s["ws"][g], BLOCK).t() for g in range(s["groups"]) if off[g + 1] > off[g]]
    return {"Y": torch.cat(parts).to(torch.bfloat16)}


def _route_plain(logits, mask, top, renorm):
    t, e = logits.shape
    x = logits.float()
    best = x.amax(1)
    live = mask & (best > -math.inf)
    ex = torch.where(live[:, None], torch.exp(x - torch.where(live, best, 0.0)[:, None]), 0.0)
    prob = ex / ex.sum(1, keepdim=True).clamp_min(1e-30)
    value, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits: lowest expert first
    taken = live[:, None] & (value[:, :top] > -math.inf)
    index = torch.where(taken, order[:, :top], -1)
    weight = torch.where(taken, prob.gather(1, order[:, :top]), 0.0)
    if renorm:
        weight = weight / weight.sum(1, keepdim=True).clamp_min(1e-30)
    key = torch.where(taken, order[:, :top], e).reshape(-1)
    counts = torch.bincount(key, minlength=e + 1)[:e]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rank = torch.argsort(key, stable=True)  # slots by expert, tokens in order within one
    place = torch.arange(t * top, device=x.device)
    row_slot = torch.where(place < offsets[-1], rank, -1)
    slot_row = torch.empty_like(rank).scatter_(0, rank, torch.where(place < offsets[-1], place, -1))
    n_live = live.sum()
    share = counts.float() / offsets[-1].clamp_min(1)
    loss = e * (share * prob.sum(0)).sum() / n_live.clamp_min(1)
    i32 = torch.int32
    return {"indices": index.to(i32), "weights": weight, "counts": counts.to(i32), "offsets": offsets.to(i32),
            "slot_row": slot_row.view(t, top).to(i32), "row_slot": row_slot.to(i32), "loss": loss.view(1),
            "live": n_live.view(1).to(i32)}


def _route_bwd_plain(s):
    e, r = s["experts"], s["routed"]
    x = s["logits"].float()
    best = x.amax(1)
    live = s["mask"] & (best > -math.inf)
    ex = torch.where(live[:, None], torch.exp(x - torch.where(live, best, 0.0)[:, None]), 0.0)
    prob = ex / ex.sum(1, keepdim=True).clamp_min(1e-30)
    share = r["counts"].float() / r["offsets"][-1].clamp_min(1)
    dprob = (s["dloss"] * e / r["live"].clamp_min(1) * share).expand(x.shape)
    at = r["indices"].clamp_min(0).long()
    dw = torch.where(r["indices"] >= 0, s["dweights"], 0.0)
    if s["renorm"]:
        dsel = r["weights"] * (dw - (r["weights"] * dw).sum(1, keepdim=True))
        dx = prob * (dprob - (prob * dprob).sum(1, keepdim=True))
        dx = dx.scatter_add(1, at, dsel)
    else:
        dprob = dprob.scatter_add(1, at, dw)
        dx = prob * (dprob - (prob * dprob).sum(1, keepdim=True))
    return {"dlogits": torch.where(live[:, None], dx, 0.0).to(s["logits"].dtype)}


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["op"]
    if own:
        import grouped_mixed_input_amd as gmi

        if op == "norm":
            gmi.rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS, h=s["h"], q=s["q"], scales=s["scale"])
            return {"h": s["h"], "q": s["q"], "scale": s["scale"]}
        if op == "norm_bwd":
            gmi.rmsnorm_bwd(s["dy"], s["h"], s["weight"], dres=s["dres"], eps=EPS, dh=s["dh"], dweight=s["dweight"],
                            workspace=s["workspace"])
            return {"dh": s["dh"], "dweight": s["dweight"]}
        if op == "gemm":
            return {"Y": gmi.gemm_f8_block(s["X"], s["xs"], s["W"], s["ws"], Y=s["Y"], workspace=s["workspace"])}
        if op == "grouped":
            return {"Y": gmi.gemm_f8_block_grouped(s["offsets"], s["X"], s["xs"], s["W"], s["ws"], Y=s["Y"],
                                                   workspace=s["workspace"])}
        if op == "route":
            return dict(gmi.moe_route(s["logits"], s["top"], mask=s["mask"], renormalize=s["renorm"],
                                      out=gmi.Routing(*s["out"]), workspace=s["workspace"])._asdict())
        gmi.moe_route_bwd(s["logits"], s["routed"]["indices"], s["routed"]["weights"], s["routed"]["offsets"],
                          s["routed"]["live"], s["dweights"], s["dloss"], mask=s["mask"], renormalize=s["renorm"],
                          dlogits=s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_bwd":
        return _norm_bwd_plain(s)
    if op == "gemm":
        return _gemm_plain(s)
    if op == "grouped":
        return _grouped_plain(s)
    if op == "route":
        return _route_plain(s["logits"], s["mask"], s["top"], s["renorm"])
    return _route_bwd_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without
def _experts_with_rows(groups, rows):
    """How many experts the skewed draw of _offsets leaves with rows, on average: only their weights are read."""
    p = [r ** -1.1 for r in range(1, groups - groups // 16 + 1)]
    return sum(1.0 - (1.0 - q / sum(p)) ** rows for q in p)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        if op == "norm":  # x, residual, h in 16 bits, q in 8, the weight, the scales
            return {"bytes": 7 * n + 2 * cols + 4 * case["rows"] * _blocks(cols), "flops": 8 * n}
        return {"bytes": 8 * n + 6 * cols, "flops": 14 * n}
    if op in ("gemm", "grouped"):
        m, n, k = case["rows"], case["n"], case["k"]
        g = 1 if op == "gemm" else _experts_with_rows(case["groups"], m)
        b = m * k + 4 * m * _blocks(k) + g * (n * k + 4 * _blocks(n) * _blocks(k)) + 2 * m * n
        return {"bytes": b, "flops": 2 * m * n * k}
    t, e, k = case["tokens"], case["experts"], case["top"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "route":  # logits and mask in; indices, weights and both orders out
        return {"bytes": t * (e * size + 1 + 16 * k) + 8 * e, "flops": t * e * 6}
    return {"bytes": t * (2 * e * size + 1 + 12 * k) + 4 * e, "flops": t * e * 8}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        y = h / ((h**2).sum(1, keepdim=True) / case["cols"] + EPS).sqrt() * s["weight"].double()
        # a block at a time; the codes' values before their rounding to 8 bits
        cuts = torch.split(y, BLOCK, 1)
        scale = torch.stack([c.abs().max(1).values.clamp_min(TINY_AMAX) / F8_MAX for c in cuts], 1)
        return {"h": h, "q": torch.cat([c / scale[:, i:i + 1] for i, c in enumerate(cuts)], 1), "scale": scale}
    if op == "norm_bwd":
        h, dy, w = s["h"].double(), s["dy"].double(), s["weight"].double()
        ms = (h**2).sum(1, keepdim=True) / case["cols"] + EPS
        # the quotient rule on h / sqrt(ms)
        dh = dy * w / ms.sqrt() - h * (dy * w * h).sum(1, keepdim=True) / (case["cols"] * ms**1.5)
        return {"dh": dh + s["dres"].double(), "dweight": (dy * h / ms.sqrt()).sum(0)}
    if op in ("gemm", "grouped"):
        m, n, k = case["rows"], case["n"], case["k"]
        y = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        off = [0, m] if op == "gemm" else s["offsets"].tolist()
        ww, wss = (s["W"][None], s["ws"][None]) if op == "gemm" else (s["W"], s["ws"])
        for g in range(len(off) - 1):
            a, b = off[g], off[g + 1]
            if a == b:
                continue
            w = ww[g].double()
            for c in range(_blocks(n)):
                for d in range(_blocks(k)):
                    w[c * BLOCK:(c + 1) * BLOCK, d * BLOCK:(d + 1) * BLOCK] *= wss[g, c, d].double()
            x = s["X"][a:b].double()
            for d in range(_blocks(k)):
                x[:, d * BLOCK:(d + 1) * BLOCK] *= s["xs"][a:b, d:d + 1].double()
            y[a:b] = x @ w.t().contiguous()
        return {"Y": y}
    t, e, k = case["tokens"], case["experts"], case["top"]
    x = s["logits"].double()
    live = s["mask"] & torch.isfinite(x).any(1)
    x = torch.where(live[:, None], x, 0.0)
    prob = torch.softmax(x, 1) * live[:, None]
    if op == "route":
        left, index, weight = x.clone(), [], []
        for _ in range(k):
            v = left.max(1, keepdim=True).values
            j = (left == v).to(torch.uint8).argmax(1, keepdim=True)  # the first expert that has the maximum
            ok = live[:, None] & (v > -math.inf)
            index.append(torch.where(ok, j, -1))
            weight.append(torch.where(ok, prob.gather(1, j), 0.0))
            left.scatter_(1, j, -math.inf)
        index, weight = torch.cat(index, 1), torch.cat(weight, 1)
        if case["renorm"]:
            weight = torch.where(live[:, None], weight / weight.sum(1, keepdim=True), 0.0)
        counts = torch.stack([(index == j).sum() for j in range(e)])
        total, n_live = int(counts.sum()), int(live.sum())
        loss = e * (counts.double() / max(total, 1) * prob.sum(0)).sum() / max(n_live, 1)
        # whole numbers are held to the plain form's
        return {"indices": None, "weights": weight, "counts": None, "offsets": None, "slot_row": None,
                "row_slot": None, "loss": loss.view(1), "live": None}
    r = s["routed"]
    dw = torch.where(r["indices"] >= 0, s["dweights"], 0.0).double()
    at = r["indices"].clamp_min(0).long()
    total, n_live = max(int(r["offsets"][-1]), 1), max(int(r["live"]), 1)
    x.requires_grad_(True)
    with torch.enable_grad():
        p = torch.softmax(x, 1)
        sel = torch.where(r["indices"] >= 0, p.gather(1, at), 0.0)
        if case["renorm"]:
            sel = sel / sel.sum(1, keepdim=True).clamp_min(1e-300)
        loss = e * (r["counts"].double() / total * (p * live[:, None]).sum(0)).sum() / n_live
        ((sel * dw).sum() + s["dloss"].double() * loss).backward()
    return {"dlogits": x.grad * live[:, None]}
