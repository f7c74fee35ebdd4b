"""Plain fp64 forms (torch on the CPU) of the operators around the indexer's gradient, with the
error bounds that their fp32 kernels have to stay in. Test infrastructure; shares no code with the
CUDA path."""

import torch

U = 2.0 ** -24           # half a unit in the last place of fp32, relative

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}   # half the smallest step of fp16

# Roundings of fp32 that meet in one value. A head's sum of D = 128 terms is 16 additions in a
# thread, 3 across threads: 19, on products of one rounding each; the reciprocal square root adds
# 2 units (4 half units) to half of that, the products by r, gain, cos and sin and their sum 5,
# the bias 1. 32 covers the forward, and the backward has a second sum (20), xhat again (20) and
# four products: 64.
FORWARD, BACKWARD = 32, 64


def angles(cos_sin, pos, R):
    """cos, sin [T, 1, R / 2] of each row, and which rows take part."""
    live = (pos >= 0) & (pos < cos_sin.shape[0]) if R else pos >= 0
    t = cos_sin.double()[torch.where(live, pos, 0).long()] if R else None
    return (t[:, None, : R // 2], t[:, None, R // 2:], live) if R else (None, None, live)


def halves(y, R, pairs):
    return (y[..., 0:R:2], y[..., 1:R:2]) if pairs else (y[..., : R // 2], y[..., R // 2: R])


def join(a, b, y, R, pairs):
    first = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([first, y[..., R:]], -1)


def turned(y, cos, sin, R, pairs):
    if not R:
        return y
    a, b = halves(y, R, pairs)
    return join(a * cos - b * sin, b * cos + a * sin, y, R, pairs)


def mixed(y, R, pairs):
    """Bound of a turned vector's entries: the sum of both entries' sizes."""
    if not R:
        return y
    a, b = halves(y, R, pairs)
    return join(a + b, a + b, y, R, pairs)


def normed(x, kind, eps):
    """xhat, r, and the size that xhat's fp32 error is relative to: the mean of a layer norm is off
    by units of mean |x|, which r carries into xhat."""
    if kind == "none":
        return x, torch.ones_like(x[..., :1]), x.abs()
    scale = x.abs().mean(-1, keepdim=True)
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    size = (x * r).abs()
    return x * r, r, size + r * scale if kind == "layer" else size


def norm_rope(x, kind, gain, bias, cos_sin, pos, R, pairs, eps, dtype):
    """x [T, N, D] fp64 -> (y, bound of |kernel - y|), padding rows zero."""
    cos, sin, live = angles(cos_sin, pos, R)
    xhat, _, size = normed(x, kind, eps)
    if gain is not None:
        xhat, size = xhat * gain.double(), size * gain.double().abs()
    if bias is not None:
        xhat, size = xhat + bias.double(), size + bias.double().abs()
    y = turned(xhat, cos, sin, R, pairs)
    y = torch.where(live[:, None, None], y, 0.0)
    err = FORWARD * U * mixed(size, R, pairs)
    return y, HALF[dtype] * (y.abs() + err) + err + TINY[dtype]


def norm_rope_grad(dy, x, kind, gain, cos_sin, pos, R, pairs, eps, dtype):
    """dy, x [T, N, D] fp64 -> dict of (value, bound) of dx, dgain, dbias (the last two None where
    the norm has none)."""
    cos, sin, live = angles(cos_sin, pos, R)
    take = live[:, None, None]
    g = torch.where(take, turned(dy, cos, -sin if R else None, R, pairs), 0.0)
    gs = torch.where(take, mixed(dy.abs(), R, pairs), 0.0)
    out = dict(dgain=None, dbias=None)
    if kind != "none":
        xhat, r, size = normed(x, kind, eps)
        adds = BACKWARD + x.shape[0] * x.shape[1] // 32     # in a row of one thread's running sum
        out["dgain"] = (g * xhat).sum((0, 1)), adds * U * (gs * size).sum((0, 1)) + 1e-30
        if kind == "layer":
            out["dbias"] = g.sum((0, 1)), adds * U * gs.sum((0, 1)) + 1e-30
        if gain is not None:
            g, gs = g * gain.double(), gs * gain.double().abs()
        g = r * (g - xhat * (g * xhat).mean(-1, keepdim=True)
                 - (g.mean(-1, keepdim=True) if kind == "layer" else 0.0))
        gs = r * (gs + size * (gs * size).mean(-1, keepdim=True) + gs.mean(-1, keepdim=True))
    g = torch.where(take, g, 0.0)
    err = BACKWARD * U * gs
    out["dx"] = g, HALF[dtype] * (g.abs() + err) + err + TINY[dtype]
    return out


def key_weights(weights, idx, batch_rows, batch_keys, scores, decay, used_q=None, used_k=None):
    """Sums per key row; batch_rows / batch_keys: (first, count) of each batch's query and key rows."""
    out = decay * scores.double()
    for b, ((q0, qn), (k0, kn)) in enumerate(zip(batch_rows, batch_keys)):
        qn = qn if used_q is None else min(max(used_q[b], 0), qn)
        kn = kn if used_k is None else min(max(used_k[b], 0), kn)
        i, w = idx[q0: q0 + qn].reshape(-1).long(), weights[q0: q0 + qn].reshape(-1).double()
        ok = (i >= 0) & (i < kn)
        out[k0: k0 + kn] += torch.bincount(i[ok], weights=w[ok], minlength=kn)[:kn]
    return out


def evict(scores, n, budget, sinks, recent):
    """Kept local indices, ascending, of one sequence whose scores are `scores[:n]`."""
    if n <= budget:
        return list(range(n))
    key = [(1, 0.0) if s != s else (0, -s) for s in scores[:n].tolist()]   # NaN below -inf
    middle = sorted(range(sinks, n - recent), key=lambda j: (key[j], j))
    return sorted(list(range(sinks)) + middle[: budget - sinks - recent] + list(range(n - recent, n)))
