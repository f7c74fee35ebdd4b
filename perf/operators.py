"""What stands around the indexer's gradient in a training step and beside its key cache, as cases that can be timed.

Four operators, each in a plain form (elementary torch operations in 32 bits, one rounding at the end) and, where `own` is
true, as a user calls it in this library:

  norm_rope       q and k from the outputs of the projections: norm of each head, then the rotation of the first dims by the
                  row's position; from 16-bit projections or from an 8-bit checkpoint of them, which it can also write
  norm_rope_grad  dq, dk back to the projections and to the norms' gains, at the projections or at their checkpoint
  key_weights     the weight that the query rows of a call put on each key row, added to what it had before
  evict           which key rows stay in a cache of limited size, and the caches with only those rows
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# --- cases -----------------------------------------------------------------------------------

def _rope_case(op, name, **kw):
    """T1 / T2 rows of q / k in B batches (T1 a multiple of B for BSND); rot: rotated dims; pairs: neighbours are rotated
    together (else the two halves); norm: of q and of k; packed: q and k are views of one projection's output; far:
    positions up to 131071 in any order (else 0, 1, .. in each batch); source: what is read; keep: a checkpoint is written."""
    c = dict(name=name, op=op, dtype="bf16", layout="BSND", B=1, T1=0, T2=0, N=64, D=128, rot=64, pairs=False,
             norm_q="rms", norm_k="rms", packed=False, far=False, source="x", keep=False)
    c.update(kw)
    return c


def _weights_case(name, **kw):
    """T1 query rows in B sequences of a cache of S2 key rows each; every row names topk keys it sees; skew: keys that are
    recent or low come up much more often, some twice in a row, and three in ten slots are empty."""
    c = dict(name=name, op="key_weights", layout="BSND", B=1, T1=0, S2=0, topk=2048, start=0, skew=False, decay=1.0)
    c.update(kw)
    return c


def _evict_case(name, **kw):
    """B sequences of up to S2 key rows (ragged: of many lengths), of which `budget` stay; heads: cache rows of [1, D] for
    the indexer's keys and of [heads, D] for the attention's keys and values."""
    c = dict(name=name, op="evict", B=1, S2=0, budget=0, sinks=4, recent=32, D=128, heads=1, ragged=False, layout="BSND")
    c.update(kw)
    return c


def listed():
    return [
        # one new token of each of eight sequences far into their context: latency is all there is
        _rope_case("norm_rope", "rope_decode_8", B=8, T1=8, T2=8, norm_k="layer", far=True),
        # the causal training workload of the benchmark, with the checkpoint that its backward will read
        _rope_case("norm_rope", "rope_causal_4096_keep", T1=4096, T2=4096, norm_k="layer", keep=True),
        # sequences of many lengths behind one another, q and k still in the output of one projection
        _rope_case("norm_rope", "rope_varlen_fp16_packed", dtype="fp16", layout="TND", B=8, T1=34117, T2=34117, N=32,
                   rot=128, pairs=True, packed=True),
        # the queries and keys of the long-context workload formed again from the checkpoint
        _rope_case("norm_rope", "rope_longctx_from_8bit", T1=8192, T2=131072, far=True, source="x8"),
        # the tiny training workload
        _rope_case("norm_rope_grad", "rope_grad_tiny_256", T1=256, T2=256, N=8, D=64, rot=32),
        # the causal training workload's way back
        _rope_case("norm_rope_grad", "rope_grad_causal_4096", T1=4096, T2=4096, norm_k="layer"),
        # few heads, four long batches, at the 8-bit checkpoint
        _rope_case("norm_rope_grad", "rope_grad_4x8192_from_8bit", B=4, T1=32768, T2=32768, N=16, norm_q="layer", pairs=True,
                   rot=128, source="x8"),
        # one decoding step of 32 sequences
        _weights_case("weights_decode_32x8192", B=32, T1=32, S2=8192, start=8191, decay=0.99),
        # the whole causal prefill
        _weights_case("weights_causal_4096", T1=4096, S2=4096),
        # 8192 queries at the end of a long context: the keys' sums do not fit one multiprocessor
        _weights_case("weights_longctx_131072", T1=8192, S2=131072, start=122880),
        # a short cache cut to a quarter: latency
        _evict_case("evict_601_to_150", S2=601, budget=150, D=64),
        # eight long caches of many lengths, the attention's keys and values beside the indexer's keys
        _evict_case("evict_8x131072_to_16384", B=8, S2=131072, budget=16384, heads=2, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "key_weights", "evict"])
    if op in ("norm_rope", "norm_rope_grad"):
        D = rng.choice([64, 128])
        N = rng.choice([1, _log_int(rng, 2, 128), rng.choice([8, 16, 32, 64, 128])])
        B = _log_int(rng, 1, 16)
        most = (60 if op == "norm_rope" else 30) * 1000 * 1000 // (D * (N + 1))
        S = _log_int(rng, 1, max(1, min(8192, most // B)))
        packed = rng.random() < 0.3
        layout = rng.choice(["BSND", "TND"])
        source = rng.choice(["x", "x", "x8"]) if not packed else "x"
        c = _rope_case(op, "", dtype=rng.choice(["bf16", "fp16"]), layout=layout, B=B, T1=B * S, N=N, D=D,
                       rot=16 * rng.randint(0, D // 16), pairs=rng.random() < 0.5,
                       norm_q=rng.choice(["rms", "layer", "none"]), norm_k=rng.choice(["rms", "layer", "none"]),
                       packed=packed, far=rng.random() < 0.5, source=source,
                       keep=op == "norm_rope" and source == "x" and rng.random() < 0.5)
        c["T2"] = c["T1"] if packed else B * _log_int(rng, 1, max(1, min(16384, most // B)))
        if layout == "TND":
            c["T1"] = max(B, c["T1"] - rng.randint(0, B))
            c["T2"] = c["T1"] if packed else max(B, c["T2"] - rng.randint(0, B))
    elif op == "key_weights":
        B = _log_int(rng, 1, 32)
        topk = _log_int(rng, 1, 2048)
        S1 = _log_int(rng, 1, max(1, min(8192, 16000000 // (B * topk))))
        S2 = S1 + _log_int(rng, 1, max(1, min(131072 - S1, 4000000 // B)))
        c = _weights_case("", layout=rng.choice(["BSND", "TND"]), B=B, T1=B * S1, S2=S2, topk=topk, start=S2 - S1,
                          skew=rng.random() < 0.5, decay=rng.choice([1.0, 0.0, round(rng.uniform(0.5, 1.0), 3)]))
    else:
        B = _log_int(rng, 1, 16)
        S2 = _log_int(rng, 16, 131072 // (1 if B <= 8 else 2))
        budget = _log_int(rng, 8, max(8, min(16384, S2, 120000 // B)))
        sinks = rng.randint(0, min(8, budget // 2))
        c = _evict_case("", B=B, S2=S2, budget=budget, sinks=sinks, recent=rng.randint(0, budget - sinks),
                        D=rng.choice([64, 128]), heads=rng.randint(1, 2), ragged=rng.random() < 0.6,
                        layout=rng.choice(["BSND", "TND"]))
    del c["name"]
    return c


# --- inputs ----------------------------------------------------------------------------------

def _lengths(total, B, salt):
    """B lengths of many sizes, each at least 1, that sum to `total`: a matter of the case alone."""
    r = random.Random(total * 131 + B * 7 + salt)
    parts = [r.uniform(0.1, 1.0) for _ in range(B)]
    lens = [1 + int((total - B) * p / sum(parts)) for p in parts]
    lens[-1] += total - sum(lens)
    return lens


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _positions(c, T, salt, gen):
    """Position of each row; None where they are 0, 1, .. in equal batches and the call knows them without."""
    if c["far"]:
        return torch.randint(0, 131072, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if c["layout"] == "BSND":
        return None
    return torch.cat([torch.arange(n, dtype=torch.int32) for n in _lengths(T, c["B"], salt)]).cuda()


def _to_8bit(x):
    """(values, scale): e4m3 values and one fp32 scale for each head of each row."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, (top / E4M3_MAX).clamp_min(torch.finfo(torch.float32).tiny), torch.zeros_like(top))
    inv = torch.where(top > 0, 1.0 / scale, torch.zeros_like(top))
    return (x * inv[..., None]).to(torch.float8_e4m3fn), scale


def _prepare_rope(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, N, D = DTYPES[c["dtype"]], c["N"], c["D"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def shape(T, heads):
        return (c["B"], T // c["B"], heads, D) if c["layout"] == "BSND" else (T, heads, D)

    s = dict(case=c)
    spread = torch.exp(0.5 * normal(N + 1, D))  # some channels of a projection's output are much larger than others
    if c["packed"]:
        x = normal(c["T1"], N + 1, D).mul_(spread).to(dt)
        s["x_q"], s["x_k"] = (v.reshape(shape(c["T1"], -1)) if c["layout"] == "TND" else
                              v.unflatten(0, (c["B"], -1)) for v in (x[:, :N], x[:, N:]))
    else:
        s["x_q"] = normal(*shape(c["T1"], N)).mul_(spread[:N]).to(dt)
        s["x_k"] = normal(*shape(c["T2"], 1)).mul_(spread[N:]).to(dt)
    if c["source"] == "x8":
        for side in ("q", "k"):
            s["x8_" + side] = _to_8bit(s.pop("x_" + side))
    for side, T in (("q", c["T1"]), ("k", c["T2"])):
        kind = c["norm_" + side]
        s["pos_" + side] = _positions(c, T, 3, gen)
        s["gain_" + side] = 1 + 0.2 * normal(D) if kind != "none" else None
        s["bias_" + side] = 0.2 * normal(D) if kind == "layer" else None
        if c["op"] == "norm_rope_grad":
            s["d" + side] = normal(*shape(T, N if side == "q" else 1)).mul_(1e-2).to(dt)
    if c["rot"]:
        rows = 131072 if c["far"] else max(c["T1"], c["T2"])
        freq = 10000.0 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / c["rot"])
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    else:
        s["cos_sin"] = None
    return s


def _prepare_weights(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, S1, K, S2 = c["B"], c["T1"] // c["B"], c["topk"], c["S2"]
    T1 = B * S1

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    sees = (torch.arange(S1, device="cuda") + c["start"] + 1).clamp_max(S2).repeat(B).double()[:, None]  # keys a row sees
    slot = torch.arange(K, device="cuda").double()
    if c["skew"]:
        reach = torch.exp(uniform(T1, K).double() * torch.log(sees + 1)) - 1  # small much more often than large
        idx = torch.where(uniform(T1, K) < 0.5, reach, sees - 1 - reach).floor().clamp_min(0).clamp(max=sees - 1)
        valid = (slot < sees) & (uniform(T1, K) >= 0.3)
    else:
        named = sees.clamp_max(K)  # one key of each of `named` equal parts of what the row sees, in order
        idx = ((slot + uniform(T1, K).double()) * sees / named).floor().clamp(max=sees - 1)
        valid = slot < named
    idx = torch.where(valid, idx, -1.0).to(torch.int32)
    p = torch.exp(torch.randn(T1, K, generator=gen, device="cuda")) * valid
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    bsnd = c["layout"] == "BSND"
    scores = 4 * uniform(B, S2) * (c["start"] + 1) / S2
    return dict(case=c, weights=p.reshape((B, S1, 1, K) if bsnd else (T1, 1, K)),
                idx=idx.reshape((B, S1, 1, K) if bsnd else (T1, 1, K)), scores=scores if bsnd else scores.reshape(-1),
                cu_q=None if bsnd else _cu([S1] * B), cu_k=None if bsnd else _cu([S2] * B),
                out=torch.zeros_like(scores if bsnd else scores.reshape(-1)))


def _prepare_evict(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, S2, D = c["B"], c["S2"], c["D"]
    bsnd = c["layout"] == "BSND"
    lens = [max(1, int(S2 * f)) for f in _fractions(c)]
    rows = (B, S2) if bsnd else (sum(lens),)
    scores = torch.randn(*rows, generator=gen, device="cuda").exp()
    scores = torch.where(torch.rand(*rows, generator=gen, device="cuda") < 0.3, (scores * 8).round() / 8, scores)  # ties
    shapes = [(1, D)] + [(c["heads"], D)] * 2
    caches = [torch.randn(*rows, *h, generator=gen, device="cuda", dtype=torch.bfloat16) for h in shapes]
    return dict(case=c, scores=scores, caches=caches, lens=lens,
                cu_k=None if bsnd else _cu(lens), used=torch.tensor(lens, dtype=torch.int32, device="cuda") if bsnd else None,
                out=[torch.zeros(B, c["budget"], *h, device="cuda", dtype=torch.bfloat16) for h in shapes])


def _fractions(c):
    """Share of S2 that each sequence fills."""
    if not c["ragged"]:
        return [1.0] * c["B"]
    r = random.Random(c["S2"] * 17 + c["B"])
    return [r.uniform(0.02, 1.0) for _ in range(c["B"])]


def prepare(case, seed):
    kind = {"norm_rope": _prepare_rope, "norm_rope_grad": _prepare_rope, "key_weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]]
    return kind(dict(case), seed)


# --- plain forms -------------------------------------------------------------------------------

def _angles(s, side, T):
    c = s["case"]
    pos = s["pos_" + side]
    if pos is None:
        pos = torch.arange(T, device="cuda") % (T // c["B"])
    t = s["cos_sin"][pos.long()]
    return t[:, None, : c["rot"] // 2], t[:, None, c["rot"] // 2:]


def _rotate(y, cos, sin, R, pairs):
    """The first R dims of y [T, N, D] turned by the angles; with -sin, back."""
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if pairs else (y[..., : R // 2], y[..., R // 2: R])
    u, v = a * cos - b * sin, b * cos + a * sin
    first = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([first, y[..., R:]], -1)


def _source(s, side):
    """x [T, N, D] in 32 bits."""
    D = s["case"]["D"]
    if s["case"]["source"] == "x8":
        v, scale = s["x8_" + side]
        return (v.float() * scale[..., None]).reshape(-1, v.shape[-2], D)
    x = s["x_" + side]
    return x.float().reshape(-1, x.shape[-2], D)


def _shape_of(s, side):
    return (s["x8_" + side][0] if s["case"]["source"] == "x8" else s["x_" + side]).shape


def _normed(x, kind):
    """(xhat, r): the row's values less their mean (layer only), times r = 1 / sqrt(mean square + eps)."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_rope(s):
    c, out = s["case"], {}
    for side in ("q", "k"):
        x = _source(s, side)
        y = _normed(x, c["norm_" + side])[0]
        if s["gain_" + side] is not None:
            y = y * s["gain_" + side]
        if s["bias_" + side] is not None:
            y = y + s["bias_" + side]
        if c["rot"]:
            y = _rotate(y, *_angles(s, side, x.shape[0]), c["rot"], c["pairs"])
        out[side] = y.to(DTYPES[c["dtype"]]).reshape(_shape_of(s, side))
        if c["keep"]:
            v, scale = _to_8bit(s["x_" + side])
            out["kept_" + side] = [v, scale]
    return out


def _plain_rope_grad(s):
    c, out = s["case"], {}
    for side in ("q", "k"):
        kind = c["norm_" + side]
        x = _source(s, side)
        g = s["d" + side].float().reshape(x.shape)
        if c["rot"]:
            cos, sin = _angles(s, side, x.shape[0])
            g = _rotate(g, cos, -sin, c["rot"], c["pairs"])
        if kind != "none":
            xhat, r = _normed(x, kind)
            out["dgain_" + side] = (g * xhat).sum((0, 1))
            if kind == "layer":
                out["dbias_" + side] = g.sum((0, 1))
            g = g * s["gain_" + side]
            m = xhat * (g * xhat).mean(-1, keepdim=True)
            g = r * (g - m - g.mean(-1, keepdim=True)) if kind == "layer" else r * (g - m)
        out["dx_" + side] = g.to(DTYPES[c["dtype"]]).reshape(_shape_of(s, side))
    return out


def _plain_weights(s):
    c = s["case"]
    B, S2 = c["B"], c["S2"]
    idx = s["idx"].reshape(B, -1).long()
    row = idx + S2 * torch.arange(B, device="cuda")[:, None]
    valid = (idx >= 0) & (idx < S2)
    w = torch.where(valid, s["weights"].reshape(B, -1), 0.0).double()  # thousands of small weights meet in one sum
    total = torch.zeros(B * S2, dtype=torch.float64, device="cuda")
    total.index_add_(0, torch.where(valid, row, 0).reshape(-1), w.reshape(-1))
    return (c["decay"] * s["scores"].double().reshape(-1) + total).float().reshape(s["scores"].shape)


def _plain_evict(s):
    c = s["case"]
    B, S2, budget = c["B"], c["S2"], c["budget"]
    n = torch.tensor(s["lens"], device="cuda")[:, None]
    first = S2 * torch.arange(B, device="cuda")[:, None] if c["layout"] == "BSND" else n.cumsum(0) - n
    j = torch.arange(S2, device="cuda")
    inside = j < n
    row = torch.where(inside, first + j, 0)  # of sequence b's key j
    # the order in which keys stay: what always stays, then by score, then what is not there; ties by their place
    order = s["scores"].reshape(-1)[row].double().nan_to_num(nan=-math.inf, posinf=1e300, neginf=-math.inf)
    order = torch.where((j < c["sinks"]) | (j >= n - c["recent"]), math.inf, order)
    order = torch.where(inside, order, -math.inf)
    keep = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :budget].sort(1).values
    keep = torch.nn.functional.pad(keep, (0, budget - keep.shape[1]), value=S2)
    there = keep < n
    at = torch.where(there, first + keep, 0)
    scores = torch.where(there, s["scores"].reshape(-1)[at], 0.0)
    caches = [torch.where(there[..., None, None], x.reshape(-1, *o.shape[2:])[at], 0.0) for x, o in zip(s["caches"], s["out"])]
    return dict(kept=torch.where(there, keep, -1).int(), lengths=there.sum(1).int(), scores=scores, caches=caches)


# --- the library's calls -------------------------------------------------------------------------

def _own_rope_args(s):
    c = s["case"]
    return dict(pos_q=s["pos_q"], pos_k=s["pos_k"], gain_q=s["gain_q"], gain_k=s["gain_k"], norm_q=c["norm_q"],
                norm_k=c["norm_k"], rot_layout="pairs" if c["pairs"] else "halves", eps=EPS, layout_q=c["layout"],
                layout_k=c["layout"])


def _own_sources(s):
    import sparse_lightning_indexer_b200 as sli
    if s["case"]["source"] == "x8":
        return [sli.Checkpoint(*s["x8_" + side], DTYPES[s["case"]["dtype"]]) for side in ("q", "k")]
    return [s["x_q"], s["x_k"]]


def _own_rope(s):
    import sparse_lightning_indexer_b200 as sli
    r = sli.qk_norm_rope(*_own_sources(s), s["cos_sin"], bias_q=s["bias_q"], bias_k=s["bias_k"],
                         checkpoint=s["case"]["keep"], **_own_rope_args(s))
    out = dict(q=r["q"], k=r["k"])
    if s["case"]["keep"]:
        out["kept_q"], out["kept_k"] = (list(r["checkpoint_" + side][:2]) for side in ("q", "k"))
    return out


def _own_rope_grad(s):
    import sparse_lightning_indexer_b200 as sli
    r = sli.qk_norm_rope_grad(s["dq"], s["dk"], *_own_sources(s), s["cos_sin"], **_own_rope_args(s))
    return {n: r[n] for n in sorted(r) if n != "workspace" and r[n] is not None}


def _own_weights(s):
    import sparse_lightning_indexer_b200 as sli
    c = s["case"]
    return sli.key_weights(s["weights"], s["idx"], s["scores"], decay=c["decay"], layout_q=c["layout"], layout_k=c["layout"],
                           cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], key_range_bound=c["S2"], out=s["out"])["scores"]


def _own_evict(s):
    import sparse_lightning_indexer_b200 as sli
    c = s["case"]
    r = sli.evict(s["scores"], s["caches"], c["budget"], sinks=c["sinks"], recent=c["recent"], layout_k=c["layout"],
                  cu_seqlens_k=s["cu_k"], seq_used_k=s["used"], key_range_bound=c["S2"], out=dict(caches=s["out"]))
    return {n: r[n] for n in ("kept", "lengths", "scores", "caches")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_rope": _own_rope, "norm_rope_grad": _own_rope_grad, "key_weights": _own_weights,
                "evict": _own_evict}[op](state)
    return {"norm_rope": _plain_rope, "norm_rope_grad": _plain_rope_grad, "key_weights": _plain_weights,
            "evict": _plain_evict}[op](state)


# --- what a pass cannot do without ------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        n = 0
        for T, N in ((c["T1"], c["N"]), (c["T2"], 1)):
            e = T * N * c["D"]
            src = e * 2 if c["source"] == "x" else e + 4 * T * N
            n += src + 2 * e + (2 * e if c["op"] == "norm_rope_grad" else 0) + (e + 4 * T * N if c["keep"] else 0)
            n += min(T, 131072 if c["far"] else max(1, T // c["B"])) * c["rot"] * 4 + 4 * T * c["far"]
        e = (c["T1"] * c["N"] + c["T2"]) * c["D"]
        return {"bytes": n, "flops": e * (8 if c["op"] == "norm_rope" else 14)}
    if c["op"] == "key_weights":
        return {"bytes": c["T1"] * c["topk"] * 8 + 8 * c["B"] * c["S2"], "flops": c["T1"] * c["topk"] + 2 * c["B"] * c["S2"]}
    lens = [max(1, int(c["S2"] * f)) for f in _fractions(c)]
    kept = sum(min(n, c["budget"]) for n in lens)
    row = 2 * c["D"] * (1 + 2 * c["heads"])
    return {"bytes": 4 * sum(lens) + 2 * kept * row + 8 * c["B"] * c["budget"], "flops": sum(lens)}


# --- the definition in 64 bits ---------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_rope, "norm_rope_grad": _exact_rope_grad, "key_weights": _exact_weights,
            "evict": lambda s: None}[case["op"]](s)


def _exact_input(s, side):
    """x as [rows of one head, D] in 64 bits, and the matrix entries of each row's rotation as cos, sin [rows, R / 2]."""
    c = s["case"]
    if c["source"] == "x8":
        v, scale = s["x8_" + side]
        x = v.double() * scale.double().unsqueeze(-1)
    else:
        x = s["x_" + side].double()
    N = x.shape[-2]
    x = x.reshape(-1, c["D"])
    if not c["rot"]:
        return x, None, None
    T = x.shape[0] // N
    pos = s["pos_" + side]
    if pos is None:
        pos = torch.arange(T // c["B"], device="cuda").repeat(c["B"])
    table = s["cos_sin"].double().index_select(0, pos.to(torch.int64)).repeat_interleave(N, 0)
    return x, table[:, : c["rot"] // 2], table[:, c["rot"] // 2:]


def _exact_turn(y, cos, sin, c, back=False):
    """In place: as numbers of the complex plane, times cos + i sin (its conjugate on the way back)."""
    if cos is None:
        return y
    R = c["rot"]
    re, im = (slice(0, R, 2), slice(1, R, 2)) if c["pairs"] else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(y[:, re].contiguous(), y[:, im].contiguous())
    w = torch.complex(cos.contiguous(), (-sin if back else sin).contiguous())
    z *= w
    y[:, re], y[:, im] = z.real, z.imag
    return y


def _exact_stats(x, kind):
    """(mean, 1 / deviation) of each row."""
    mean = x.sum(1, keepdim=True) / x.shape[1] if kind == "layer" else torch.zeros_like(x[:, :1])
    var = (x - mean).square().sum(1, keepdim=True) / x.shape[1]
    return mean, (var + EPS).rsqrt() if kind != "none" else torch.ones_like(var)


def _exact_rope(s):
    c, out = s["case"], {}
    for side in ("q", "k"):
        x, cos, sin = _exact_input(s, side)
        mean, r = _exact_stats(x, c["norm_" + side])
        y = (x - mean) * r
        if s["gain_" + side] is not None:
            y *= s["gain_" + side].double()
        if s["bias_" + side] is not None:
            y += s["bias_" + side].double()
        out[side] = _exact_turn(y, cos, sin, c).reshape(_shape_of(s, side))
        if c["keep"]:
            scale = x.abs().max(1).values / E4M3_MAX
            shape = _shape_of(s, side)
            out["kept_" + side] = [(x / scale[:, None]).reshape(shape), scale.reshape(shape[:-1])]
    return out


def _exact_rope_grad(s):
    c, out = s["case"], {}
    for side in ("q", "k"):
        kind = c["norm_" + side]
        x, cos, sin = _exact_input(s, side)
        g = _exact_turn(s["d" + side].double().reshape(x.shape), cos, sin, c, back=True)
        if kind != "none":
            mean, r = _exact_stats(x, kind)
            xhat = (x - mean) * r
            out["dgain_" + side] = torch.einsum("td,td->d", g, xhat)
            if kind == "layer":
                out["dbias_" + side] = g.sum(0)
            g = g * s["gain_" + side].double()
            # the Jacobian of a norm is r (1 - projection on xhat [- projection on 1]) / D
            along = torch.einsum("td,td->t", g, xhat)[:, None] / c["D"]
            lift = g.mean(1, keepdim=True) if kind == "layer" else 0.0
            g = (g - lift - xhat * along) * r
        out["dx_" + side] = g.reshape(_shape_of(s, side))
    return out


def _exact_weights(s):
    c = s["case"]
    B, S2 = c["B"], c["S2"]
    idx, w = s["idx"].reshape(B, -1), s["weights"].reshape(B, -1)
    rows = []
    for b in range(B):
        ok = idx[b] >= 0
        rows.append(torch.bincount(idx[b][ok].long(), weights=w[b][ok].double(), minlength=S2))
    total = torch.stack(rows) + c["decay"] * s["scores"].double().reshape(B, S2)
    return total.reshape(s["scores"].shape)
