"""Cases and plain forms of the operators around the products of a mixture-of-experts layer and beside a dense one.

  group          rows ordered by a number that each carries (its expert, its adapter), with the row offsets of the groups
  permute        each token's row copied to the rows of its experts: fp8 codes with their scales, or 16-bit values
  unpermute      the experts' rows back to the tokens, weighted and summed, onto what a shared expert left
  unpermute_bwd  its gradients: of the experts' rows (16-bit, or fp8 with scales for the next product) and of the weights
  gate           v = silu(gate) * up between the experts' two products, fp8 with one scale per row and 128 columns
  gate_bwd       its gradient, gate and up side by side, 16-bit or fp8 with scales
  lora           Y = base + s (X A^T) B^T with each row's own adapter: requests of many adapters beside one projection

`own` selects who computes: False, elementary torch operations in fp32; True, grouped_mixed_input_amd.
"""
import math

import torch

own = False

BLOCK = 128
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY_AMAX = F8_MAX * 2.0**-126  # keeps the scale of an all-zero block a normal number
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": F8}


def listed():
    return [
        # a decode step's rows brought into the order of their adapters, once for all projections of the step
        dict(name="group decode", op="group", rows=64, groups=32, top=1),
        # the slots of a prompt, 8 experts a token, from a router of the user's own
        dict(name="group prefill", op="group", rows=16384, groups=128, top=8),
        # a decode step of 16 sequences, fp8 rows as the norm leaves them: latency
        dict(name="sort decode", op="permute", tokens=16, top=8, experts=128, cols=4096, dtype="fp8", blocked=False),
        # a prompt's fp8 rows to their experts
        dict(name="sort prefill", op="permute", tokens=16384, top=8, experts=128, cols=4096, dtype="fp8", blocked=False),
        # the experts' rows of a prompt back to the tokens, beside a shared expert
        dict(name="back prefill", op="unpermute", tokens=16384, top=8, experts=128, cols=4096, dtype="bf16", blocked=False,
             weighted=True, add=True),
        # a short fine-tuning batch in fp16, last block partial, experts closed to some tokens
        dict(name="back bwd ragged", op="unpermute_bwd", tokens=777, top=4, experts=60, cols=2000, dtype="fp16",
             blocked=True, quant=False),
        # a training step: the gradient leaves as the fp8 operand of the data gradient's product
        dict(name="back bwd train", op="unpermute_bwd", tokens=16384, top=8, experts=128, cols=4096, dtype="bf16",
             blocked=False, quant=True),
        # between the two products of a prompt's experts
        dict(name="gate prefill", op="gate", rows=131072, inner=1024, dtype="bf16", live=1.0),
        # a training step's backward through it
        dict(name="gate bwd train", op="gate_bwd", rows=131072, inner=1024, dtype="bf16", live=0.97, quant=True),
        # a decode step of 16 requests, each with an adapter of its own, beside the 8192 x 8192 projection
        dict(name="lora decode", op="lora", rows=16, n=8192, k=8192, rank=16, adapters=16, dtype="bf16", run=1),
        # a mixed batch: short prompt pieces and single tokens, odd sizes, some rows without an adapter
        dict(name="lora ragged", op="lora", rows=333, n=2000, k=2056, rank=40, adapters=12, dtype="fp16", run=7),
        # prompts of a few requests
        dict(name="lora prefill", op="lora", rows=4096, n=8192, k=8192, rank=64, adapters=8, dtype="bf16", run=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group", "permute", "unpermute", "unpermute_bwd", "gate", "gate_bwd", "lora"])
    if op == "group":
        return dict(op=op, rows=_log(rng, 1, 16384), groups=_log(rng, 1, 256), top=rng.randint(1, 8))
    if op in ("gate", "gate_bwd"):
        c = dict(op=op, rows=_log(rng, 1, 65536), inner=8 * _log(rng, 16, 256), dtype=rng.choice(["bf16", "fp16"]),
                 live=rng.choice([1.0, 0.97, 0.5]))
        return dict(c, quant=rng.random() < 0.5) if op == "gate_bwd" else c
    if op == "lora":
        return dict(op=op, rows=_log(rng, 1, 4096), n=8 * _log(rng, 16, 1024), k=8 * _log(rng, 16, 1024),
                    rank=8 * rng.choice([1, 2, 3, 4, 5, 6, 8]), adapters=_log(rng, 1, 8) if rng.random() < 0.5 else _log(rng, 1, 32),
                    dtype=rng.choice(["bf16", "fp16"]), run=_log(rng, 1, 512))
    experts = _log(rng, 4, 256)
    top = rng.randint(1, min(8, experts))
    cols = 16 * _log(rng, 8, 256)
    c = dict(op=op, tokens=min(_log(rng, 1, 16384), 3 * 2**27 // (top * cols)), top=top, experts=experts, cols=cols,
             dtype=rng.choice(["fp8", "bf16", "fp16"] if op == "permute" else ["bf16", "fp16"]), blocked=rng.random() < 0.5)
    if op == "unpermute":
        c.update(weighted=rng.random() < 0.7, add=rng.random() < 0.5)
    elif op == "unpermute_bwd":
        c.update(quant=rng.random() < 0.5)
    return c


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- inputs
def _routed(gen, tokens, top, experts, blocked):
    """Skewed top-k choice: experts of each slot (-1 where all are closed), weights, the row of each slot, rows in use."""
    x = torch.randn(tokens, experts, generator=gen, device="cuda") + 0.5 * torch.randn(experts, generator=gen, device="cuda")
    if blocked:  # padding tokens, and experts closed to a token by capacity or placement
        x.masked_fill_(torch.rand(tokens, experts, generator=gen, device="cuda") < 0.3, -math.inf)
        x.masked_fill_(torch.rand(tokens, 1, generator=gen, device="cuda") < 0.03, -math.inf)
    value, pick = x.topk(top, dim=1)
    pick = torch.where(value > -math.inf, pick, -1)
    w = torch.where(value > -math.inf, torch.exp(value - value[:, :1]), 0.0)
    w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    key = torch.where(pick >= 0, pick, experts).reshape(-1)
    rank = torch.argsort(key, stable=True)
    used = int((key < experts).sum())
    slot_row = torch.empty_like(rank).scatter_(0, rank, torch.arange(len(rank), device="cuda"))
    slot_row = torch.where(key < experts, slot_row, -1).view(tokens, top)
    return w, slot_row.to(torch.int32), used


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case)
    op = case["op"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "group":
        n, g = case["rows"], case["groups"]
        p = (torch.arange(1, g + 1, device="cuda", dtype=torch.float32) ** -0.7)[torch.randperm(g, generator=gen, device="cuda")]
        index = torch.multinomial(p, n * case["top"], replacement=True, generator=gen).view(n, case["top"])
        lost = torch.rand(n, case["top"], generator=gen, device="cuda") < 0.05  # rows of no group
        s["index"] = torch.where(lost, -1, index).to(torch.int32)
        s["out"] = (torch.empty(g + 1, **i32), torch.empty(n * case["top"], **i32), torch.empty(n, case["top"], **i32))
    elif op in ("permute", "unpermute", "unpermute_bwd"):
        t, k, cols, dt = case["tokens"], case["top"], case["cols"], DTYPES[case["dtype"]]
        w, s["slot_row"], used = _routed(gen, t, k, case["experts"], case["blocked"])
        rows = t * k
        quant = case["dtype"] == "fp8" or case.get("quant", False)
        if op == "permute":
            s["x"] = randn(t, cols).mul_(120.0).clamp_(-F8_MAX, F8_MAX).to(F8) if quant else randn(t, cols).to(dt)
            s["scales"] = randn(t, _blocks(cols)).mul_(0.3).exp_().mul_(2.0**-8) if quant else None
        else:
            s["weights"] = w if case.get("weighted", True) else None
            s["rows"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            for part in s["rows"].split(1 << 15):
                part.copy_(randn(*part.shape))
            if op == "unpermute":
                s["add"] = randn(t, cols).to(dt) if case["add"] else None
            else:
                s["dout"] = (randn(t, cols) * torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 12.0, 1.0)).to(dt)
                s["dweights"] = torch.empty(t, k, device="cuda")
        # rows behind the last one in use stay as they are: zero here
        if op == "unpermute":
            s["out"] = torch.empty(t, cols, dtype=dt, device="cuda")
        else:
            s["out"] = torch.zeros(rows, cols, dtype=F8 if quant else dt, device="cuda")
            s["out_scales"] = torch.zeros(rows, _blocks(cols), device="cuda") if quant else None
    elif op in ("gate", "gate_bwd"):
        r, n, dt = case["rows"], case["inner"], DTYPES[case["dtype"]]
        s["a"] = randn(r, 2 * n).mul_(1.5).to(dt)
        s["used"] = torch.full((1,), max(1, int(r * case["live"])), **i32)
        quant, cols = (True, n) if op == "gate" else (case["quant"], 2 * n)
        if op == "gate_bwd":
            s["dact"] = randn(r, n).to(dt)
        s["out"] = torch.zeros(r, cols, dtype=F8 if quant else dt, device="cuda")
        s["out_scales"] = torch.zeros(r, _blocks(cols), device="cuda") if quant else None
    else:
        m, n, k, r, l, dt = (case[v] for v in ("rows", "n", "k", "rank", "adapters", "dtype"))
        dt = DTYPES[dt]
        s["X"], s["base"] = randn(m, k).to(dt), randn(m, n).to(dt)
        s["A"], s["B"] = (randn(l, r, k) * k**-0.5).to(dt), (randn(l, n, r) * r**-0.5).to(dt)
        s["scales"] = torch.rand(l, generator=gen, device="cuda") + 0.5
        # runs of rows of one request; one request in nine uses the projection alone
        g = torch.Generator().manual_seed(seed)
        pick = torch.randint(0, l, (m,), generator=g) if case["run"] > 1 else torch.randperm(m, generator=g) % l
        pick[torch.rand(m, generator=g) < 1 / 9] = -1
        first = torch.cumsum(torch.rand(m, generator=g) < 1 / case["run"], 0)
        s["index"] = pick[first.clamp_max(m - 1)].to(torch.int32).cuda()
        key = torch.where(s["index"] >= 0, s["index"], l)
        s["order"] = torch.argsort(key, stable=True).to(torch.int32)
        s["Y"] = torch.empty(m, n, dtype=dt, device="cuda")
    # scratch that a program keeps for its calls
    s["workspace"] = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _group_plain(s):
    g, index = s["groups"], s["index"].reshape(-1)
    ok = (index >= 0) & (index < g)
    key = torch.where(ok, index, g)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=g + 1)[:g]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=order.device))
    place = torch.where(ok, place, -1).view(s["index"].shape)
    return {"offsets": offsets.to(torch.int32), "order": order.to(torch.int32), "place": place.to(torch.int32)}


def _tokens_of_rows(s):
    """Slot of each row and whether the row is in use."""
    flat = s["slot_row"].reshape(-1).long()
    ok = flat >= 0
    slot = torch.zeros_like(flat).scatter_(0, torch.where(ok, flat, len(flat) - 1), torch.arange(len(flat), device=flat.device) * ok)
    return slot, torch.arange(len(flat), device=flat.device) < ok.sum()


def _quantized(v):
    """Codes and scales of fp32 rows, a block of 128 columns at a time."""
    rows, cols = v.shape
    nb = _blocks(cols)
    b = torch.nn.functional.pad(v, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    scale = b.abs().amax(2).clamp_min(TINY_AMAX) / F8_MAX
    return (b / scale[:, :, None]).view(rows, nb * BLOCK)[:, :cols].to(F8), scale


def _left(v, scale, keep):
    """What is written for the rows in use; zeros behind them."""
    v = torch.where(keep[:, None], v.view(torch.uint8), 0).view(F8) if scale is not None else torch.where(keep[:, None], v, 0.0)
    return {"out": v} if scale is None else {"out": v, "scales": torch.where(keep[:, None], scale, 0.0)}


def _permute_plain(s):
    slot, used = _tokens_of_rows(s)
    token = torch.div(slot, s["top"], rounding_mode="floor")
    if s["scales"] is None:
        return _left(s["x"][token], None, used)
    return _left(s["x"].view(torch.uint8)[token].view(F8), s["scales"][token], used)


def _slots(s):
    """The experts' rows of each slot in fp32, zero where there is none."""
    at = s["slot_row"].long()
    return torch.where(at[..., None] >= 0, s["rows"][at.clamp_min(0)].float(), 0.0)


def _unpermute_plain(s):
    v = _slots(s)
    if s["weights"] is not None:
        v = v * s["weights"][..., None]
    v = v.sum(1)
    if s["add"] is not None:
        v = v + s["add"].float()
    return {"out": v.to(s["out"].dtype)}


def _unpermute_bwd_plain(s):
    slot, used = _tokens_of_rows(s)
    token = torch.div(slot, s["top"], rounding_mode="floor")
    d = s["dout"].float()[token] * s["weights"].reshape(-1)[slot][:, None]
    out = _left(*_quantized(d), used) if s["quant"] else _left(d.to(s["out"].dtype), None, used)
    return dict(out, dweights=(_slots(s) * s["dout"].float()[:, None]).sum(2))


def _gate_plain(s):
    n = s["inner"]
    g, u = s["a"][:, :n].float(), s["a"][:, n:].float()
    keep = torch.arange(s["rows"], device=g.device) < s["used"]
    return _left(*_quantized(g / (1.0 + torch.exp(-g)) * u), keep)


def _gate_bwd_plain(s):
    n = s["inner"]
    g, u, d = s["a"][:, :n].float(), s["a"][:, n:].float(), s["dact"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    da = torch.cat([d * u * sig * (1.0 + g * (1.0 - sig)), d * g * sig], 1)
    keep = torch.arange(s["rows"], device=g.device) < s["used"]
    return _left(*_quantized(da), keep) if s["quant"] else _left(da.to(s["out"].dtype), None, keep)


def _lora_plain(s):
    l, r, n, k = s["adapters"], s["rank"], s["n"], s["k"]
    # every adapter's first product, all but the row's own struck out, then one product with all the second factors
    t = (s["X"].float() @ s["A"].float().reshape(l * r, k).t()).view(-1, l, r)
    mine = s["index"][:, None] == torch.arange(l, device=t.device)
    t = torch.where(mine[..., None], t * s["scales"][:, None], 0.0)
    return {"Y": (s["base"].float() + t.reshape(-1, l * r) @ s["B"].float().transpose(1, 2).reshape(l * r, n)).to(s["Y"].dtype)}


PLAIN = {"group": _group_plain, "permute": _permute_plain, "unpermute": _unpermute_plain,
         "unpermute_bwd": _unpermute_bwd_plain, "gate": _gate_plain, "gate_bwd": _gate_bwd_plain, "lora": _lora_plain}


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return PLAIN[s["op"]](s)
    import grouped_mixed_input_amd as gmi

    op = s["op"]
    if op == "group":
        return dict(gmi.group_rows(s["index"], s["groups"], out=gmi.Grouping(*s["out"]), workspace=s["workspace"])._asdict())
    if op == "permute":
        gmi.moe_permute(s["x"], s["slot_row"], scales=s["scales"], out=s["out"], out_scales=s["out_scales"])
    elif op == "unpermute":
        gmi.moe_unpermute(s["rows"], s["slot_row"], weights=s["weights"], add=s["add"], out=s["out"])
        return {"out": s["out"]}
    elif op == "unpermute_bwd":
        gmi.moe_unpermute_bwd(s["dout"], s["slot_row"], weights=s["weights"], rows=s["rows"], drows=s["out"],
                              scales=s["out_scales"], dweights=s["dweights"], quantize=s["quant"])
    elif op == "gate":
        gmi.swiglu_quant(s["a"], live=s["used"], q=s["out"], scales=s["out_scales"])
    elif op == "gate_bwd":
        gmi.swiglu_bwd(s["dact"], s["a"], live=s["used"], da=s["out"], scales=s["out_scales"], quantize=s["quant"])
    else:
        return {"Y": gmi.gemm_lora(s["X"], s["A"], s["B"], s["index"], order=s["order"], scales=s["scales"],
                                   base=s["base"], Y=s["Y"], workspace=s["workspace"])}
    out = {"out": s["out"]}
    if s["out_scales"] is not None:
        out["scales"] = s["out_scales"]
    if op == "unpermute_bwd":
        out["dweights"] = s["dweights"]
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "group":
        n = case["rows"] * case["top"]
        return {"bytes": 12 * n + 4 * case["groups"] + 4, "flops": n}
    if op in ("permute", "unpermute", "unpermute_bwd"):
        t, k, cols = case["tokens"], case["top"], case["cols"]
        slots = t * k
        used = slots if not case["blocked"] else int(0.97 * slots)  # the skewed choice finds nearly all slots filled
        wide = 1 if case["dtype"] == "fp8" else 2
        if op == "permute":
            row = cols * wide + (4 * _blocks(cols) if wide == 1 else 0)
            return {"bytes": (t + used) * row + 4 * slots, "flops": 0}
        b = 2 * used * cols + 2 * t * cols + 4 * slots
        if op == "unpermute":
            b += 4 * slots * case["weighted"] + 2 * t * cols * case["add"]
            return {"bytes": b, "flops": (1 + case["weighted"]) * used * cols}
        b += used * (cols + 4 * _blocks(cols) if case["quant"] else 2 * cols) + 8 * slots
        return {"bytes": b, "flops": (3 + 2 * case["quant"]) * used * cols}
    if op in ("gate", "gate_bwd"):
        r, n = max(1, int(case["rows"] * case["live"])), case["inner"]
        if op == "gate":
            return {"bytes": r * (5 * n + 4 * _blocks(n)) + 4, "flops": 8 * r * n}
        return {"bytes": r * (6 * n + (2 * n + 4 * _blocks(2 * n) if case["quant"] else 4 * n)) + 4, "flops": 16 * r * n}
    m, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
    with_one = m * 8 / 9  # rows that have an adapter
    chosen = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** max(1.0, with_one / case["run"]))
    return {"bytes": int(2 * with_one * k + 4 * m * n + 2 * chosen * r * (n + k) + 8 * m), "flops": int(2 * with_one * r * (n + k))}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_codes(v, keep):
    """Values over their block's scale before they are rounded to 8 bits, and the scales."""
    cuts = torch.split(v, BLOCK, 1)
    scale = torch.stack([c.abs().max(1).values.clamp_min(TINY_AMAX) / F8_MAX for c in cuts], 1)
    q = torch.cat([c / scale[:, i:i + 1] for i, c in enumerate(cuts)], 1)
    return {"out": q * keep[:, None], "scales": scale * keep[:, None]}


def exact(case, seed):
    op = case["op"]
    if op == "group":  # whole numbers are held to the plain form's
        return None
    s = prepare(case, seed)
    if op in ("permute", "unpermute", "unpermute_bwd"):
        t, k, cols = case["tokens"], case["top"], case["cols"]
        place = s["slot_row"].long()
        if op == "unpermute":
            out = torch.zeros(t, cols, dtype=torch.float64, device="cuda")
            for i in range(k):
                has = place[:, i] >= 0
                v = s["rows"][place[has, i]].double()
                out[has] += v if s["weights"] is None else v * s["weights"][has, i:i + 1].double()
            return {"out": out if s["add"] is None else out + s["add"].double()}
        wide = torch.zeros(t * k, cols, dtype=torch.float64, device="cuda")
        keep = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        scale = torch.zeros(t * k, _blocks(cols), dtype=torch.float64, device="cuda")
        dw = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for i in range(k):
            has = place[:, i] >= 0
            to = place[has, i]
            keep[to] = 1.0
            if op == "permute":
                wide[to] = s["x"][has].double()
                if s["scales"] is not None:
                    scale[to] = s["scales"][has].double()
            else:
                d = s["dout"][has].double()
                wide[to] = d * s["weights"][has, i:i + 1].double()
                dw[has, i] = (d * s["rows"][to].double()).sum(1)
        if op == "permute":
            return {"out": wide} if s["scales"] is None else {"out": wide, "scales": scale}
        return dict(_exact_codes(wide, keep) if case["quant"] else {"out": wide}, dweights=dw)
    if op in ("gate", "gate_bwd"):
        r, n = case["rows"], case["inner"]
        g, u = s["a"].double().split(n, 1)
        keep = (torch.arange(r, device="cuda") < s["used"]).double()
        if op == "gate":
            return _exact_codes(torch.sigmoid(g) * g * u, keep)
        d = s["dact"].double()
        # the derivative of g sigmoid(g) is sigmoid(g) + g sigmoid(g) sigmoid(-g)
        da = torch.cat([d * u * (torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)), d * g * torch.sigmoid(g)], 1)
        return _exact_codes(da, keep) if case["quant"] else {"out": da * keep[:, None]}
    y = s["base"].double()
    for a in range(case["adapters"]):
        mine = (s["index"] == a).nonzero()[:, 0]
        if len(mine):
            t = s["X"][mine].double() @ s["A"][a].double().t().contiguous()
            y[mine] += s["scales"][a].double() * (t @ s["B"][a].double().t().contiguous())
    return {"Y": y}
