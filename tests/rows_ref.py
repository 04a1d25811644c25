"""64-bit definitions of the calls that move and shape rows between products, and of the adapters' product, on the CPU."""
import torch

F8 = torch.float8_e4m3fn
TINY = 448.0 * 2.0 ** -126
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest subnormal's step


def blocks(n):
    return (n + 127) // 128


def group(index, groups):
    """offsets, order, place by a walk over the rows."""
    flat = index.reshape(-1).tolist()
    lists = [[] for _ in range(groups + 1)]
    for i, g in enumerate(flat):
        lists[g if 0 <= g < groups else groups].append(i)
    order = [i for rows in lists for i in rows]
    offsets = [0]
    for rows in lists[:groups]:
        offsets.append(offsets[-1] + len(rows))
    place = [-1] * len(flat)
    for r, i in enumerate(order[: offsets[-1]]):
        place[i] = r
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32),
            torch.tensor(place, dtype=i32).view(index.shape))


def slots(gen, tokens, k, spare=0, dead=0.1):
    """Random slot rows: a permutation of tokens * k + spare rows, some slots without one."""
    perm = torch.randperm(tokens * k + spare, generator=gen)[: tokens * k].view(tokens, k)
    return torch.where(torch.rand(tokens, k, generator=gen) < dead, -1, perm).to(torch.int32)


def unpermute(y, slot_row, weights, add):
    """The sum and the sum of its terms' magnitudes."""
    at = slot_row.long()
    ok = (at >= 0) & (at < len(y))
    v = torch.where(ok[..., None], y.double()[torch.where(ok, at, 0)] if len(y) else torch.zeros(1, dtype=torch.float64), 0.0)
    if weights is not None:
        v = v * torch.where(ok, weights.double(), 0.0)[..., None]
    out, mag = v.sum(1), v.abs().sum(1)
    if add is not None:
        out, mag = out + add.double(), mag + add.double().abs()
    return out, mag


def unpermute_bwd(dout, slot_row, weights, y, rows):
    """Row gradients (nan where no slot has the row), dweights and the magnitudes of their terms."""
    T, k = slot_row.shape
    d = torch.full((rows, dout.shape[1]), float("nan"), dtype=torch.float64)
    dw, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for i in range(k):
            r = int(slot_row[t, i])
            if 0 <= r < rows:
                d[r] = dout[t].double() * (weights[t, i].double() if weights is not None else 1.0)
                if y is not None:
                    p = dout[t].double() * y[r].double()
                    dw[t, i], mag[t, i] = p.sum(), p.abs().sum()
    return d, dw, mag


def swiglu(a):
    g, u = a.double().chunk(2, 1)
    return g * torch.sigmoid(g) * u


def swiglu_bwd(dact, a):
    g, u = a.double().chunk(2, 1)
    d, s = dact.double(), torch.sigmoid(g)
    return torch.cat([d * u * (s + g * s * torch.sigmoid(-g)), d * g * s], 1)


def check_codes(q, s, v, rel):
    """q and s are codes and scales of values that lie within `rel` of v: the scale is amax / 448 to that and one fp32
    step, and the code is that of a quotient inside the interval that leaves."""
    rows, cols = v.shape
    pad = torch.nn.functional.pad(v, (0, blocks(cols) * 128 - cols)).view(rows, -1, 128)
    want = pad.abs().amax(2).clamp_min(TINY) / 448.0
    assert ((s.double() - want).abs() <= (rel + 2.0 ** -22) * want).all(), "scales"
    t = v / s.double().repeat_interleave(128, 1)[:, :cols]
    slack = 2 * rel + 2.0 ** -22
    lo, hi = (t * (1 - slack)).float(), (t * (1 + slack)).float()
    lo, hi = torch.minimum(lo, hi).clamp(-448, 448).to(F8).float(), torch.maximum(lo, hi).clamp(-448, 448).to(F8).float()
    got = q.float()
    assert ((got >= lo) & (got <= hi)).all(), "codes"


def lora(X, A, B, index, scales, base):
    """Y, and the magnitudes with which its errors grow: of the second product's terms, of both products' terms, and
    of the largest of X A^T in a row times the row sums of |B|."""
    M, N = X.shape[0], B.shape[1]
    y = base.double().clone() if base is not None else torch.zeros(M, N, dtype=torch.float64)
    second, both, top = (torch.zeros(M, N, dtype=torch.float64) for _ in range(3))
    for a in range(A.shape[0]):
        m = (index == a).nonzero()[:, 0]
        if len(m) == 0:
            continue
        s = scales[a].double() if scales is not None else 1.0
        x, fa, fb = X[m].double(), A[a].double(), B[a].double()
        t = x @ fa.t()
        y[m] += s * (t @ fb.t())
        second[m] = s * (t.abs() @ fb.abs().t())
        both[m] = s * (x.abs() @ fa.abs().t()) @ fb.abs().t()
        top[m] = s * t.abs().amax(1, keepdim=True) * fb.abs().sum(1)
    return y, second, both, top


def lora_tolerance(y, second, both, top, dtype, K, rank):
    """Half a step of the result; fp32 sums of K and of 2 * rank + 2 terms (2^-23 an addition, whichever way it
    rounds); X A^T as two terms of the type (2^-17 of each for bf16, of a row's largest 2^-22 for fp16)."""
    split = 2.0 ** -17 * second if dtype == torch.bfloat16 else 2.0 ** -22 * top
    return STEP[dtype] * y.abs() + FLOOR[dtype] + split + (K + 2 * rank + 4) * 2.0 ** -23 * both
