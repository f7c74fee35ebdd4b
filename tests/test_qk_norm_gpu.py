"""GPU tests of the norm and rotation of q and k, their 8-bit checkpoints, and the gradient back to
the projections, against plain fp64 forms with derived bounds (operators_reference.py)."""

import pytest
import torch

import oracle
import slikl_inputs as si
import sparse_lightning_indexer_b200 as sli
import operators_reference as ref

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
EPS = 1e-6


def table(P, R, seed=0):
    a = torch.rand(P, max(R, 2) // 2, generator=torch.Generator().manual_seed(seed),
                   dtype=torch.float64) * 400 - 200
    return torch.cat([a.cos(), a.sin()], 1).float() if R else None


def inside(name, got, want):
    value, bound = want
    got = got.double().cpu().reshape(value.shape)
    assert torch.isfinite(got).all(), name
    over = (got - value).abs() > bound
    assert not over.any(), (name, int(over.sum()), (got - value).abs().max(), bound[over][0])


def make(seed, T, N, D, R, dtype, kind, gain=True, bias=True, mean=0.0):
    """One side's inputs, on the CPU: x with channels of very different sizes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, N, D, generator=g) * torch.exp(torch.randn(N, D, generator=g)) + mean
    return dict(x=x.to(dtype), kind=kind, dtype=dtype, R=R,
                gain=1 + 0.3 * torch.randn(D, generator=g) if gain and kind != "none" else None,
                bias=torch.randn(D, generator=g) if bias and kind == "layer" else None,
                dy=(torch.randn(T, N, D, generator=g) * 0.05).to(dtype))


def dev(t):
    return None if t is None else t.cuda()


def dequant(c):
    return c.values.cpu().double() * c.scale.cpu().double()[..., None]


# (T1, N1, T2, D, R, pairs, dtype, norm_q, norm_k): one row to several blocks, heads that do not
# divide a warp's rows, rotations of none, some and all dims, every norm on either side
CASES = [
    (1, 1, 1, 64, 16, False, BF, "rms", "layer"),
    (1, 64, 1, 128, 64, False, BF, "rms", "layer"),
    (5, 3, 7, 128, 48, True, BF, "layer", "rms"),
    (33, 7, 129, 64, 48, False, FP, "rms", "rms"),
    (64, 128, 64, 128, 128, True, FP, "layer", "layer"),
    (37, 8, 1000, 128, 96, False, BF, "none", "rms"),
    (300, 16, 300, 64, 64, True, BF, "rms", "none"),
    (200, 64, 131, 128, 64, False, FP, "none", "none"),
    (129, 32, 1, 128, 0, False, BF, "rms", "layer"),
    (1500, 32, 4000, 128, 64, False, BF, "rms", "layer"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).split(".")[-1] for v in c))
@pytest.mark.parametrize("source", ["x", "x8"])
def test_forward_and_gradient(case, source):
    T1, N1, T2, D, R, pairs, dtype, nq, nk = case
    sides = dict(q=make(1, T1, N1, D, R, dtype, nq), k=make(2, T2, 1, D, R, dtype, nk))
    P = 500
    cs = table(P, R)
    g = torch.Generator().manual_seed(9)
    pos = {}
    for n, s in sides.items():
        p = torch.randint(0, P, (s["x"].shape[0],), generator=g, dtype=torch.int32)
        if len(p) > 4:
            p[1], p[-1] = -1, -1                     # padding rows, the last one among them
        pos[n] = p
    x = {n: s["x"].cuda() for n, s in sides.items()}
    given = x
    if source == "x8":
        given = {n: sli.checkpoint_pack(v) for n, v in x.items()}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    common = dict(pos_q=dev(pos["q"]), pos_k=dev(pos["k"]), gain_q=dev(sides["q"]["gain"]),
                  gain_k=dev(sides["k"]["gain"]), norm_q=nq, norm_k=nk, layout_q="TND",
                  layout_k="TND", rot_layout="pairs" if pairs else "halves", eps=EPS, status=status)
    fwd = sli.qk_norm_rope(given["q"], given["k"], dev(cs), bias_q=dev(sides["q"]["bias"]),
                           bias_k=dev(sides["k"]["bias"]), checkpoint=source == "x", **common)
    bwd = sli.qk_norm_rope_grad(dev(sides["q"]["dy"]), dev(sides["k"]["dy"]), given["q"],
                                given["k"], dev(cs), **common)
    again = sli.qk_norm_rope_grad(dev(sides["q"]["dy"]), dev(sides["k"]["dy"]), given["q"],
                                  given["k"], dev(cs), **common)
    torch.cuda.synchronize()
    assert int(status) == 0
    for n, s in sides.items():
        at = dequant(given[n]) if source == "x8" else s["x"].double()
        inside(n, fwd[n], ref.norm_rope(at, s["kind"], s["gain"], s["bias"], cs, pos[n], R, pairs,
                                        EPS, dtype))
        want = ref.norm_rope_grad(s["dy"].double(), at, s["kind"], s["gain"], cs, pos[n], R, pairs,
                                  EPS, dtype)
        for what in ("dx", "dgain", "dbias"):
            got = bwd[f"{what}_{n}"]
            assert (got is None) == (want[what] is None), what
            if got is not None:
                inside(f"{what}_{n}", got, want[what])
                assert torch.equal(got, again[f"{what}_{n}"]), what   # the same bits each call
        if source == "x":                  # the checkpoint of the same pass: padding rows are zero
            check_checkpoint(fwd["checkpoint_" + n], s["x"], pos[n])


@pytest.mark.parametrize("T1,N1,T2", [(6, 1, 24717), (4, 5, 63928), (40000, 1, 3), (700, 64, 1), (0, 4, 30000)])
@pytest.mark.parametrize("source", ["x", "x8"])
def test_sides_of_very_different_sizes(T1, N1, T2, source):
    """A side of a few rows beside one of many gets its rows done, with the same bits as alone."""
    D, R = 64, 32
    q, k = make(21, T1, N1, D, R, BF, "layer"), make(22, T2, 1, D, R, BF, "rms")
    cs = dev(table(300, R))
    pos = {n: dev(torch.arange(t, dtype=torch.int32) % 300) for n, t in (("q", T1), ("k", T2))}
    xq, xk = dev(q["x"]), dev(k["x"])
    if source == "x8":
        xq, xk = sli.checkpoint_pack(xq), sli.checkpoint_pack(xk)
    kw = dict(norm_q="layer", norm_k="rms", layout_q="TND", layout_k="TND")
    keep = source == "x"

    def fill(*shape):
        return torch.full(shape, float("nan"), dtype=BF, device="cuda")

    both = sli.qk_norm_rope(xq, xk, cs, pos_q=pos["q"], pos_k=pos["k"], checkpoint=keep,
                            out=dict(q=fill(T1, N1, D), k=fill(T2, 1, D)), **kw)
    one = sli.qk_norm_rope(xq, None, cs, pos_q=pos["q"], checkpoint=keep, **kw)
    two = sli.qk_norm_rope(None, xk, cs, pos_k=pos["k"], checkpoint=keep, **kw)
    assert torch.equal(both["q"], one["q"]) and torch.equal(both["k"], two["k"])
    if keep:
        for n, alone in (("q", one), ("k", two)):
            c, d = both["checkpoint_" + n], alone["checkpoint_" + n]
            assert torch.equal(c.values.view(torch.uint8), d.values.view(torch.uint8)) and torch.equal(c.scale, d.scale)
    dq, dk = dev(q["dy"]), dev(k["dy"])
    both = sli.qk_norm_rope_grad(dq, dk, xq, xk, cs, pos_q=pos["q"], pos_k=pos["k"],
                                 out=dict(dx_q=fill(T1, N1, D), dx_k=fill(T2, 1, D)), **kw)
    at = {n: dequant(x) if source == "x8" else s["x"].double() for n, x, s in (("q", xq, q), ("k", xk, k))}
    for n, s, kind in (("q", q, "layer"), ("k", k, "rms")):
        want = ref.norm_rope_grad(s["dy"].double(), at[n], kind, None, cs.cpu(), pos[n].cpu(), R, False, EPS, BF)
        for what in ("dx", "dgain", "dbias"):
            if want[what] is not None and both[f"{what}_{n}"].numel():
                inside(f"{what}_{n}", both[f"{what}_{n}"], want[what])


@pytest.mark.parametrize("D,T", [(128, 1800), (64, 3600)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("source", ["x", "x8", "slices"])
def test_two_rows_a_step(D, T, pairs, kind, source):
    """Calls large enough for two rows of a token a step in both directions (16 heads; 28416 rows of 128 values
    forward, 56832 of 64, half of that backward), from dense rows, checkpoints and slices of one
    projection; padding rows with NaN among them; beside them keys of one head."""
    N, R, dtype = 16, 48, FP if pairs else BF
    assert T * N >= 2 * (512 // D) * 4 * 148 * 6
    q, k = make(41, T, N, D, R, dtype, kind), make(42, T, 1, D, R, dtype, "rms")
    g = torch.Generator().manual_seed(43)
    cs, pos = table(700, R), torch.randint(0, 700, (T,), generator=g, dtype=torch.int32)
    pos[[0, 17, T // 2, T - 1]] = -1
    xq, xk, dq, dk = dev(q["x"]), dev(k["x"]), dev(q["dy"]), dev(k["dy"])
    out = None
    at = {"q": q["x"].double(), "k": k["x"].double()}
    if source == "x8":
        xq, xk = sli.checkpoint_pack(xq), sli.checkpoint_pack(xk)
        at = {"q": dequant(xq), "k": dequant(xk)}
        xq.values.view(torch.uint8)[dev(pos < 0)] = 0x7f                # NaN
    else:
        xq[dev(pos < 0)] = float("nan")
    dq[dev(pos < 0)] = float("inf")
    if source == "slices":
        W = (N + 1) * D + 24
        proj = torch.full((T, W), 5.0, dtype=dtype, device="cuda")
        grads = torch.full((T, W), 7.0, dtype=dtype, device="cuda")

        def cut(p):
            return p[:, 8: 8 + N * D].unflatten(1, (N, D)), p[:, 16 + N * D: 16 + (N + 1) * D].unflatten(1, (1, D))

        for to, v in zip(cut(proj), (xq, xk)):
            to.copy_(v)
        xq, xk = cut(proj)
        out = dict(zip(("dx_q", "dx_k"), cut(grads)))
    kw = dict(pos_q=dev(pos), pos_k=dev(pos), gain_q=dev(q["gain"]), gain_k=dev(k["gain"]), norm_q=kind,
              layout_q="TND", layout_k="TND", rot_layout="pairs" if pairs else "halves", eps=EPS)
    f = sli.qk_norm_rope(xq, xk, dev(cs), bias_q=dev(q["bias"]), checkpoint=source != "x8", **kw)
    b = sli.qk_norm_rope_grad(dq, dk, xq, xk, dev(cs), out=out, **kw)
    for n, s in (("q", q), ("k", k)):
        inside(n, f[n], ref.norm_rope(at[n], s["kind"], s["gain"], s["bias"], cs, pos, R, pairs, EPS, dtype))
        want = ref.norm_rope_grad(s["dy"].double(), at[n], s["kind"], s["gain"], cs, pos, R, pairs, EPS, dtype)
        for what in ("dx", "dgain", "dbias"):
            assert (b[f"{what}_{n}"] is None) == (want[what] is None)
            if want[what] is not None:
                inside(f"{what}_{n}", b[f"{what}_{n}"], want[what])
        if source != "x8":
            check_checkpoint(f["checkpoint_" + n], s["x"], pos)
    if source == "slices":
        for sl in (slice(0, 8), slice(8 + N * D, 16 + N * D), slice(16 + (N + 1) * D, W)):
            assert (grads[:, sl] == 7).all()


def check_checkpoint(c, x, pos=None):
    live = (pos >= 0)[:, None] if pos is not None else torch.ones(x.shape[:-1], dtype=torch.bool)
    x = torch.where(live[..., None], x.double(), 0.0)
    scale = c.scale.cpu().double()
    want = x.abs().amax(-1) / 448
    normal = want >= 2.0 ** -126
    assert ((scale - want).abs() <= 2.0 ** -23 * want)[normal].all()
    assert (scale[want == 0] == 0).all()
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 of the scale below; the quotient's own
    # three roundings move a value by less than 2^-21 of itself
    bound = torch.maximum(x.abs() * 2.0 ** -4, scale[..., None] * 2.0 ** -10) * (1 + 2.0 ** -14)
    assert ((dequant(c) - x).abs() <= bound + 1e-300).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
def test_checkpoint_values(dtype, D):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(7, 11, D, generator=g) * torch.exp(4 * torch.randn(7, 11, 1, generator=g))).to(dtype)
    x[0, 0] = 0
    x[0, 1] = torch.finfo(dtype).max
    x[0, 2] = torch.finfo(dtype).smallest_normal * 2.0 ** -5       # a row of subnormal values
    x[0, 3, 1:] = 0
    x[0, 4, 5] = float("nan")
    x[0, 5, 5] = float("inf")
    c = sli.checkpoint_pack(x.cuda())
    back = sli.checkpoint_unpack(c)
    v = dequant(c)
    assert torch.isnan(v[0, 4, 5]) and torch.isnan(v[0, 5]).all()
    keep = torch.isfinite(x).all(-1)            # (a row drawn above fp16's range is infinite too)
    check_checkpoint(sli.Checkpoint(c.values[keep.cuda()][None], c.scale[keep.cuda()][None], dtype), x[keep][None])
    b = back.cpu().double()[keep]
    want = v[keep]
    tiny = torch.finfo(dtype).smallest_normal * 2.0 ** (-8 if dtype == BF else -11)
    # one fp32 rounding of the product, one of the 16-bit type (below its normal range: half a step)
    lim = torch.finfo(dtype).max
    ok = want.abs() <= lim
    assert ((b - want).abs() <= want.abs() * (2.0 ** -24 + ref.HALF[dtype]) + tiny)[ok].all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_checkpoint_scale_and_codes_by_the_definition(dtype):
    """The scale is max|x| / 448 rounded to fp32, bit by bit, and every code the one that x / scale rounds to
    in whichever way the quotient's own error may lead: a reciprocal to 2 units (2^-22 of itself) and a
    product's rounding (2^-24), less than 2^-21 together."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(400, 16, 128, generator=g) * torch.exp(2 * torch.randn(400, 16, 1, generator=g))).to(dtype)
    c = sli.checkpoint_pack(x.cuda())
    scale, codes = c.scale.cpu(), c.values.cpu().float()
    assert torch.equal(scale, x.float().abs().amax(-1) / 448)
    quotient = x.double() / scale.double()[..., None]
    either = [(quotient * (1 + f * 2.0 ** -21)).float().clamp(-448, 448).to(torch.float8_e4m3fn).float() for f in (-1, 1)]
    assert ((codes == either[0]) | (codes == either[1])).all()
    # that leaves most codes no choice: 448 x / max is a middle between codes only where 7 X = O M 2^l, X and M
    # the significands and O one of the eight odd numbers from 17 to 31, so for at most 8 of the 128 (bf16)
    # or 1024 X to a given M, and no significand is more than twice as likely as the average one
    assert ((either[0] == either[1]).double().mean()) > 7 / 8
    # every positive finite maximum
    bits = torch.arange(1, 0x7c00 if dtype == FP else 0x7f80, dtype=torch.int16)
    x = torch.zeros(len(bits), 1, 64, dtype=dtype)
    x[:, 0, 17] = bits.view(dtype)
    c = sli.checkpoint_pack(x.cuda())
    want = (x[:, :, 17].float() / 448).clamp_min(2.0 ** -126)
    assert torch.equal(c.scale.cpu(), want)


def test_default_positions_and_batches():
    B, S, N, D, R = 3, 21, 4, 64, 32
    s = make(5, B * S, N, D, R, BF, "rms")
    k = make(6, B * S, 1, D, R, BF, "layer")
    cs = table(S, R)
    r = sli.qk_norm_rope(s["x"].cuda().view(B, S, N, D), k["x"].cuda().view(B, S, 1, D), dev(cs),
                         gain_q=dev(s["gain"]), gain_k=dev(k["gain"]), bias_k=dev(k["bias"]),
                         norm_k="layer")
    pos = torch.arange(S, dtype=torch.int32).repeat(B)
    assert r["q"].shape == (B, S, N, D) and r["k"].shape == (B, S, 1, D)
    inside("q", r["q"], ref.norm_rope(s["x"].double(), "rms", s["gain"], None, cs, pos, R, False, EPS, BF))
    inside("k", r["k"], ref.norm_rope(k["x"].double(), "layer", k["gain"], k["bias"], cs, pos, R, False, EPS, BF))


@pytest.mark.parametrize("layout", ["BSND", "TND"])
def test_slices_of_one_projection(layout):
    """x and dx as slices of [T, N D + D + 40]: the columns between and behind stay as they were."""
    B, S, N, D, R = 2, 37, 5, 128, 64
    T, W = B * S, N * D + D + 40
    g = torch.Generator().manual_seed(8)
    proj = torch.randn(T, W, generator=g).to(BF)
    lead = (B, S) if layout == "BSND" else (T,)

    def cut(p):
        p = p.view(*lead, W)
        return p[..., 8: 8 + N * D].unflatten(-1, (N, D)), p[..., 16 + N * D: 16 + N * D + D].unflatten(-1, (1, D))

    pos = torch.randint(0, 60, (T,), generator=g, dtype=torch.int32)
    cs = table(60, R)
    xq, xk = cut(proj.cuda())
    kw = dict(pos_q=dev(pos), pos_k=dev(pos), norm_k="layer", layout_q=layout, layout_k=layout)
    r = sli.qk_norm_rope(xq, xk, dev(cs), **kw)
    cq, ck = (t.reshape(T, -1, D).double() for t in cut(proj))
    inside("q", r["q"], ref.norm_rope(cq, "rms", None, None, cs, pos, R, False, EPS, BF))
    inside("k", r["k"], ref.norm_rope(ck, "layer", None, None, cs, pos, R, False, EPS, BF))
    dproj = torch.full((T, W), 7.0, dtype=BF, device="cuda")
    dq, dk = torch.randn_like(r["q"]), torch.randn_like(r["k"])
    gq, gk = cut(dproj)
    b = sli.qk_norm_rope_grad(dq, dk, xq, xk, dev(cs), out=dict(dx_q=gq, dx_k=gk), **kw)
    for n, dy, x, kind, got in (("q", dq, cq, "rms", gq), ("k", dk, ck, "layer", gk)):
        want = ref.norm_rope_grad(dy.cpu().double().reshape(x.shape), x, kind, None, cs, pos, R, False, EPS, BF)
        inside("dx_" + n, got, want["dx"])
        inside("dgain_" + n, b["dgain_" + n], want["dgain"])
    for sl in (slice(0, 8), slice(8 + N * D, 16 + N * D), slice(16 + N * D + D, W)):
        assert (dproj[:, sl] == 7).all()


def test_one_side_alone_and_empty_sides():
    cs = table(10, 64)
    s = make(11, 9, 4, 64, 64, BF, "rms")
    pos = torch.arange(9, dtype=torch.int32)
    kw = dict(layout_q="TND", layout_k="TND")
    r = sli.qk_norm_rope(None, dev(s["x"]), dev(cs), pos_k=dev(pos), gain_k=dev(s["gain"]), **kw)
    assert r["q"] is None
    inside("k", r["k"], ref.norm_rope(s["x"].double(), "rms", s["gain"], None, cs, pos, 64, False, EPS, BF))
    none = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    nopos = torch.empty(0, dtype=torch.int32, device="cuda")
    r = sli.qk_norm_rope(none, none, dev(cs), pos_q=nopos, pos_k=nopos, checkpoint=True, **kw)
    assert r["q"].shape == (0, 4, 64) and r["checkpoint_q"].scale.shape == (0, 4)
    b = sli.qk_norm_rope_grad(none, dev(s["dy"]), none, dev(s["x"]), dev(cs), pos_q=nopos,
                              pos_k=dev(pos), norm_q="layer", **kw)
    torch.cuda.synchronize()
    assert (b["dgain_q"] == 0).all() and (b["dbias_q"] == 0).all() and b["dgain_k"].abs().sum() > 0


def test_positions_outside_the_table():
    cs = table(16, 64)
    s = make(12, 6, 4, 64, 64, BF, "rms")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(layout_q="TND", layout_k="TND", status=status)
    for bad in (16, -2, 2 ** 31 - 1, -2 ** 31):
        pos = torch.tensor([0, bad, 15, -1, 3, 4], dtype=torch.int32)
        status.zero_()
        r = sli.qk_norm_rope(dev(s["x"]), None, dev(cs), pos_q=dev(pos), **kw)
        assert int(status) == sli.SLIKL_DEV_BAD_POSITION
        inside("q", r["q"], ref.norm_rope(s["x"].double(), "rms", None, None, cs, pos, 64, False, EPS, BF))
        status.zero_()
        b = sli.qk_norm_rope_grad(dev(s["dy"]), None, dev(s["x"]), None, dev(cs), pos_q=dev(pos), **kw)
        assert int(status) == sli.SLIKL_DEV_BAD_POSITION
        want = ref.norm_rope_grad(s["dy"].double(), s["x"].double(), "rms", None, cs, pos, 64, False, EPS, BF)
        inside("dx", b["dx_q"], want["dx"])
        inside("dgain", b["dgain_q"], want["dgain"])
    # a batch longer than the table, without positions
    status.zero_()
    x = torch.randn(1, 17, 1, 64, device="cuda").to(BF)
    r = sli.qk_norm_rope(x, None, dev(cs), status=status)
    assert int(status) == sli.SLIKL_DEV_BAD_POSITION and (r["q"][:, 16] == 0).all()


def test_padding_rows_may_hold_anything():
    """NaN and infinities in a padding row reach neither outputs nor the gains' gradients."""
    cs = table(16, 64)
    s = make(13, 40, 8, 128, 64, FP, "layer")
    x, dy = s["x"].clone(), s["dy"].clone()
    pos = torch.arange(40, dtype=torch.int32) % 16
    pos[5] = pos[39] = -1
    x[5], dy[5], x[39], dy[39] = float("nan"), float("inf"), float("-inf"), float("nan")
    kw = dict(pos_q=dev(pos), layout_q="TND", norm_q="layer")
    r = sli.qk_norm_rope(dev(x), None, dev(cs), bias_q=dev(s["bias"]), checkpoint=True, **kw)
    b = sli.qk_norm_rope_grad(dev(dy), None, dev(x), None, dev(cs), **kw)
    for t in (r["q"], r["checkpoint_q"].values.float(), r["checkpoint_q"].scale, b["dx_q"]):
        assert (t[5] == 0).all() and (t[39] == 0).all() and torch.isfinite(t).all()
    want = ref.norm_rope_grad(s["dy"].double(), s["x"].double(), "layer", None, cs, pos, 64, False, EPS, FP)
    inside("dgain", b["dgain_q"], want["dgain"])
    inside("dbias", b["dbias_q"], want["dbias"])


def test_a_mean_far_above_the_deviation():
    s = make(14, 50, 4, 128, 0, BF, "layer", mean=200.0)
    pos = torch.zeros(50, dtype=torch.int32)
    r = sli.qk_norm_rope(dev(s["x"]), None, None, norm_q="layer", gain_q=dev(s["gain"]),
                         bias_q=dev(s["bias"]), layout_q="TND")
    inside("q", r["q"], ref.norm_rope(s["x"].double(), "layer", s["gain"], s["bias"], None, pos, 0,
                                      False, EPS, BF))


def test_zero_rows_have_finite_results():
    x = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    for kind in ("rms", "layer"):
        r = sli.qk_norm_rope(x, None, None, norm_q=kind, layout_q="TND")
        b = sli.qk_norm_rope_grad(torch.ones_like(x), None, x, None, None, norm_q=kind, layout_q="TND")
        assert (r["q"] == 0).all() and torch.isfinite(b["dx_q"]).all() and (b["dgain_q"] == 0).all()


def test_smallest_eps():
    """Rows of zeros and padding rows with r up to 1e19, whose cube is beyond fp32."""
    s = make(21, 12, 8, 128, 64, BF, "rms")
    x, cs = s["x"].clone(), table(12, 64)
    x[3] = 0
    pos = torch.arange(12, dtype=torch.int32)
    pos[7] = -1
    for kind in ("rms", "layer"):
        kw = dict(pos_q=dev(pos), layout_q="TND", norm_q=kind, gain_q=dev(s["gain"]), eps=1e-38)
        b = sli.qk_norm_rope_grad(dev(s["dy"]), None, dev(x), None, dev(cs), **kw)
        want = ref.norm_rope_grad(s["dy"].double(), x.double(), kind, s["gain"], cs, pos, 64, False, 1e-38, BF)
        inside("dx", b["dx_q"], want["dx"])
        inside("dgain", b["dgain_q"], want["dgain"])
        assert (b["dx_q"][7] == 0).all()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("N", [1, 16])
def test_dims_behind_the_rotated_ones_do_not_meet(pairs, N):
    """Without a norm an infinity or NaN in a dim that is not turned stays there."""
    s = make(22, 4000, N, 128, 64, FP, "none")
    x, cs = s["x"].clone(), table(50, 64)
    x[5, 0, 70], x[9, N - 1, 127], x[3990, 0, 64] = float("inf"), float("nan"), float("-inf")
    kw = dict(pos_q=dev(torch.arange(4000, dtype=torch.int32) % 50), layout_q="TND", norm_q="none",
              rot_layout="pairs" if pairs else "halves")
    y = sli.qk_norm_rope(dev(x), None, dev(cs), **kw)["q"].cpu()
    dx = sli.qk_norm_rope_grad(dev(x), None, dev(x), None, dev(cs), **kw)["dx_q"].cpu()
    for got in (y, dx):
        assert torch.equal(torch.isfinite(got), torch.isfinite(x))
        assert torch.equal(got[..., 64:][torch.isfinite(x[..., 64:])], x[..., 64:][torch.isfinite(x[..., 64:])])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("N", [1, 16])
def test_gains_of_dims_behind_the_rotated_ones_do_not_meet(kind, pairs, N):
    """An infinite or NaN gain of a dim that is not turned spoils that dim alone."""
    s = make(24, 4000, N, 128, 64, FP, kind)
    cs, gain = table(50, 64), s["gain"].clone()
    pos = torch.arange(4000, dtype=torch.int32) % 50
    spoilt = (65, 90, 127)
    for d, v in zip(spoilt, (float("inf"), float("nan"), float("-inf"))):
        gain[d] = v
    y = sli.qk_norm_rope(dev(s["x"]), None, dev(cs), pos_q=dev(pos), layout_q="TND", norm_q=kind, gain_q=dev(gain),
                         rot_layout="pairs" if pairs else "halves")["q"].cpu().double()
    value, bound = ref.norm_rope(s["x"].double(), kind, s["gain"], None, cs, pos, 64, pairs, EPS, FP)
    rest = [d for d in range(128) if d not in spoilt]
    inside("q", y[..., rest], (value[..., rest], bound[..., rest]))
    assert not torch.isfinite(y[..., list(spoilt)]).any()


def test_in_place():
    s = make(15, 100, 16, 128, 64, BF, "rms")
    cs = table(100, 64)
    pos = dev(torch.arange(100, dtype=torch.int32))
    kw = dict(pos_q=pos, layout_q="TND")
    x = dev(s["x"])
    want = sli.qk_norm_rope(x, None, dev(cs), **kw)["q"]
    dwant = sli.qk_norm_rope_grad(dev(s["dy"]), None, x, None, dev(cs), **kw)
    dy, xc = dev(s["dy"]), x.clone()
    got = sli.qk_norm_rope_grad(dy, None, x, None, dev(cs), out=dict(dx_q=dy), **kw)
    assert torch.equal(dy, dwant["dx_q"]) and torch.equal(got["dgain_q"], dwant["dgain_q"])
    sli.qk_norm_rope_grad(dev(s["dy"]), None, xc, None, dev(cs), out=dict(dx_q=xc), **kw)
    assert torch.equal(xc, dwant["dx_q"])
    sli.qk_norm_rope(x, None, dev(cs), out=dict(q=x), **kw)
    assert torch.equal(x, want)


def test_gradient_against_differences():
    """dgain, dbias and dx along random directions against the forward's own central differences:
    the loss <dy, y> moves by <dx, d> h + O(h^3); its two evaluations carry y's 16-bit rounding, at
    most 2^-11 (fp16) of sum |dy y| in all and a random walk of that in practice, so the fp64 form of
    the forward, which the kernel is within its bound of, is what is differenced."""
    s = make(16, 12, 3, 64, 32, FP, "layer")
    cs, pos = table(50, 32), torch.randint(0, 50, (12,), dtype=torch.int32)
    x, dy = s["x"].double(), s["dy"].double()
    b = sli.qk_norm_rope_grad(dev(s["dy"]), None, dev(s["x"]), None, dev(cs), pos_q=dev(pos),
                              norm_q="layer", gain_q=dev(s["gain"]), rot_layout="pairs", layout_q="TND")

    def loss(x, gain, bias):
        return (ref.norm_rope(x, "layer", gain, bias, cs, pos, 32, True, EPS, FP)[0] * dy).sum()

    g = torch.Generator().manual_seed(1)
    h = 1e-4
    for what, at in (("dx_q", x), ("dgain_q", s["gain"].double()), ("dbias_q", s["bias"].double())):
        d = torch.randn(at.shape, generator=g, dtype=torch.float64)
        args = [[x, s["gain"].double(), s["bias"].double()] for _ in range(2)]
        i = ("dx_q", "dgain_q", "dbias_q").index(what)
        args[0][i], args[1][i] = at + h * d, at - h * d
        want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        got = (b[what].cpu().double() * d).sum()
        # dx: 2^-11 of each entry; the sums: 2^-24 of each term times their count; h^2 terms 1e-7
        room = (b[what].cpu().double() * d).abs().sum() * (2.0 ** -11 if what == "dx_q" else 1e-5)
        assert abs(want - got) <= room + 1e-6 * abs(want), what


def test_graph_other_stream_and_shared_workspace():
    s = make(17, 700, 16, 128, 64, BF, "layer")
    k = make(18, 700, 1, 128, 64, BF, "rms")
    cs = dev(table(700, 64))
    pos = dev(torch.arange(700, dtype=torch.int32))
    kw = dict(pos_q=pos, pos_k=pos, norm_q="layer", layout_q="TND", layout_k="TND")
    xq, xk, dq, dk = dev(s["x"]), dev(k["x"]), dev(s["dy"]), dev(k["dy"])
    want = sli.qk_norm_rope(xq, xk, cs, **kw), sli.qk_norm_rope_grad(dq, dk, xq, xk, cs, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = sli.qk_norm_rope(xq, xk, cs, stream=st, **kw), sli.qk_norm_rope_grad(dq, dk, xq, xk, cs, stream=st, **kw)
    st.synchronize()
    for w, v in zip(want, got):
        assert all(torch.equal(w[n], v[n]) for n in w if n != "workspace" and w[n] is not None)
    ws = torch.zeros(want[1]["workspace"].numel(), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for i in range(2):                       # two graphs that share one workspace, replayed in turn
        x2 = xq if i == 0 else xq.flip(0).contiguous()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f = sli.qk_norm_rope(x2, xk, cs, **kw)
            b = sli.qk_norm_rope_grad(dq, dk, x2, xk, cs, workspace=ws, **kw)
        graphs.append(g)
        outs.append((f, b, x2))
    for i in (0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for f, b, x2 in outs:
        w = sli.qk_norm_rope(x2, xk, cs, **kw), sli.qk_norm_rope_grad(dq, dk, x2, xk, cs, **kw)
        torch.cuda.synchronize()
        for u, v in zip(w, (f, b)):
            assert all(torch.equal(u[n], v[n]) for n in u if n != "workspace" and u[n] is not None)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows against the same rows alone."""
    T, N, D, R = 262200, 64, 128, 64
    x = torch.empty(T, N, D, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    pos = (torch.arange(T, device="cuda") % 100).int()
    cs = dev(table(100, R))
    r = sli.qk_norm_rope(x, None, cs, pos_q=pos, layout_q="TND", checkpoint=True)
    tail = sli.qk_norm_rope(x[-70:].contiguous(), None, cs, pos_q=pos[-70:].contiguous(),
                            layout_q="TND", checkpoint=True)
    assert torch.equal(r["q"][-70:], tail["q"])
    c, ct = r["checkpoint_q"], tail["checkpoint_q"]
    assert torch.equal(c.values[-70:].view(torch.uint8), ct.values.view(torch.uint8))
    assert torch.equal(c.scale[-70:], ct.scale)
    del r
    b = sli.qk_norm_rope_grad(x, None, x, None, cs, pos_q=pos, layout_q="TND", norm_q="layer")
    bt = sli.qk_norm_rope_grad(x[-70:].contiguous(), None, x[-70:].contiguous(), None, cs,
                               pos_q=pos[-70:].contiguous(), layout_q="TND", norm_q="layer")
    assert torch.equal(b["dx_q"][-70:], bt["dx_q"])
    b8 = sli.qk_norm_rope_grad(x, None, c, None, cs, pos_q=pos, layout_q="TND", norm_q="layer")
    bt = sli.qk_norm_rope_grad(x[-70:].contiguous(), None, ct, None, cs,
                               pos_q=pos[-70:].contiguous(), layout_q="TND", norm_q="layer")
    assert torch.equal(b8["dx_q"][-70:], bt["dx_q"])


# --- together: projections -> q, k -> the indexer's gradient -> projections -------------------------

@pytest.mark.parametrize("layout", ["BSND", "TND"])
@pytest.mark.parametrize("source", ["x", "x8"])
@pytest.mark.parametrize("mode", [("auto", False), ("scatter", False), ("auto", True)])
def test_projected_gradient(layout, source, mode):
    """grad_projected against the oracle run on the q and k that the forward call forms, and its
    dq, dk taken back in fp64; and, bit by bit, against the three calls made one by one where the
    middle one is deterministic."""
    path, det = mode
    wl = si.small(seed=71, layout=layout, B=2, S1=40, S2=300, N1=16, D=128, K=96, pattern="causal")
    R, dtype = 64, wl.q.dtype
    T1, T2, N1, D = wl.T1, wl.T2, wl.N1, wl.D
    q, k = make(72, T1, N1, D, R, dtype, "rms"), make(73, T2, 1, D, R, dtype, "layer")
    g = torch.Generator().manual_seed(74)
    pos = {n: torch.randint(0, 400, (T,), generator=g, dtype=torch.int32) for n, T in (("q", T1), ("k", T2))}
    cs = table(400, R)
    xq, xk = (dev(s["x"]).reshape(w.shape) for s, w in ((q, wl.q), (k, wl.k)))
    if source == "x8":
        xq, xk = sli.checkpoint_pack(xq), sli.checkpoint_pack(xk)
    # q of the workload's size, so that the softmax is not a single slot
    gain_q = q["gain"] * 0.1
    qk = dict(pos_q=dev(pos["q"]), pos_k=dev(pos["k"]), gain_q=dev(gain_q), gain_k=dev(k["gain"]),
              norm_k="layer", layout_q=layout, layout_k=layout)
    idx = dict(cu_seqlens_q=dev(wl.cu_seqlens_q), cu_seqlens_k=dev(wl.cu_seqlens_k),
               deterministic=det, dk_path=path, key_range_bound=sli.key_range_bound_of(wl))
    res = sli.grad_projected(xq, xk, dev(wl.w), dev(wl.p), dev(wl.idx), dev(cs), bias_k=dev(k["bias"]),
                             loss=True, **qk, **idx)
    fwd = sli.qk_norm_rope(xq, xk, dev(cs), bias_k=dev(k["bias"]), **qk)
    mid = sli.grad(fwd["q"], fwd["k"], dev(wl.w), dev(wl.p), dev(wl.idx), layout, layout, loss=True, **idx)
    bwd = sli.qk_norm_rope_grad(mid["dq"], mid["dk"], xq, xk, dev(cs), **qk)
    torch.cuda.synchronize()
    assert sli.slikl_read_device_status(res["workspace"].data_ptr()) == 0
    for n in ("dw", "softmax_out", "loss"):
        assert torch.equal(res[n], mid[n]), n
    assert torch.equal(res["dx_q"], bwd["dx_q"]) and torch.equal(res["dgain_q"], bwd["dgain_q"])
    if det:
        assert all(torch.equal(res[n], bwd[n]) for n in ("dx_k", "dgain_k", "dbias_k"))
    wl.q, wl.k = fwd["q"].cpu(), fwd["k"].cpu()
    want = oracle.grad(wl)
    for n, s, N, gain, kind in (("q", q, N1, gain_q, "rms"), ("k", k, 1, k["gain"], "layer")):
        x = dequant(xq if n == "q" else xk).reshape(-1, N, D) if source == "x8" else s["x"].double()
        dy = torch.from_numpy(want["d" + n]).reshape(-1, N, D)
        r = ref.norm_rope_grad(dy, x, kind, gain, cs, pos[n], R, False, EPS, dtype)
        # dq and dk come within 5e-3 (relative 2-norm) of the oracle's. The way back is linear in
        # them: a rotation, the gain, and r times a projection, so an error of norm e becomes one
        # of at most e max|gain| max r in dx; its sum with xhat over the rows is at most e times
        # the largest norm of a column of xhat (Cauchy-Schwarz), and dx itself is rounded
        e = 5e-3 * dy.norm()
        xhat, rr, _ = ref.normed(x, kind, EPS)
        far = (res["dx_" + n].cpu().double().reshape(x.shape) - r["dx"][0]).norm()
        assert far <= e * gain.abs().max() * rr.max() + ref.HALF[dtype] * r["dx"][0].norm() + r["dx"][1].norm(), n
        far = (res["dgain_" + n].cpu().double() - r["dgain"][0]).norm()
        assert far <= e * xhat.reshape(-1, D).norm(dim=0).max() + r["dgain"][1].norm(), n
    # a bad position reaches the status word that grad's own flags are in
    qk["pos_k"] = qk["pos_k"].clone()
    qk["pos_k"][0] = 400
    res = sli.grad_projected(xq, xk, dev(wl.w), dev(wl.p), dev(wl.idx), dev(cs), **qk, **idx)
    assert sli.slikl_read_device_status(res["workspace"].data_ptr()) == sli.SLIKL_DEV_BAD_POSITION


def test_structs_and_addresses_instead_of_tensors():
    """The functions that take the C structs, for memory that is not torch's, do what those for tensors do."""
    wl = si.small(seed=78, B=1, S1=40, S2=300, N1=16, D=128, K=96)
    T1, T2, N1, D, R, dtype = wl.T1, wl.T2, wl.N1, wl.D, 64, wl.q.dtype
    q, k = make(79, T1, N1, D, R, dtype, "rms"), make(80, T2, 1, D, R, dtype, "layer")
    cs, pos = dev(table(400, R)), {n: torch.arange(T, dtype=torch.int32, device="cuda") for n, T in (("q", T1), ("k", T2))}
    t = {n: {m: dev(s[m]) for m in ("x", "dy", "gain", "bias")} for n, s in (("q", q), ("k", k))}
    xq, xk = t["q"]["x"].reshape(wl.q.shape), t["k"]["x"].reshape(wl.k.shape)
    w, p, idx = dev(wl.w), dev(wl.p), dev(wl.idx)
    kw = dict(pos_q=pos["q"], pos_k=pos["k"], gain_q=t["q"]["gain"], gain_k=t["k"]["gain"], norm_k="layer", eps=EPS)
    fwd = sli.qk_norm_rope(xq, xk, cs, bias_k=t["k"]["bias"], checkpoint=True, **kw)
    bwd = sli.qk_norm_rope_grad(t["q"]["dy"].view(wl.q.shape), t["k"]["dy"].view(wl.k.shape), xq, xk, cs, **kw)
    both = sli.grad_projected(xq, xk, w, p, idx, cs, bias_k=t["k"]["bias"], deterministic=True, **kw)
    qk = sli.slikl_qk_problem(dtype=sli.SLIKL_BF16 if dtype == BF else sli.SLIKL_FP16, rot_layout=sli.SLIKL_ROT_HALVES, D=D,
                              rot_dim=R, table_rows=400, eps=EPS,
                              q=sli.slikl_qk_side(T=T1, N=N1, norm=sli.SLIKL_NORM_RMS),
                              k=sli.slikl_qk_side(T=T2, N=1, norm=sli.SLIKL_NORM_LAYER))
    tn, held = sli.slikl_qk_tensors(cos_sin=cs.data_ptr()), {}
    for n, side in (("q", tn.q), ("k", tn.k)):
        x = t[n]["x"]
        held[n] = dict(y=torch.empty_like(x), keep8=torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"),
                       keep8_scale=torch.empty(x.shape[:-1], device="cuda"), dx=torch.empty_like(x),
                       dgain=torch.empty(D, device="cuda"))
        if n == "k":
            held[n]["dbias"] = torch.empty(D, device="cuda")
            side.bias = t[n]["bias"].data_ptr()
        for name, v in (*held[n].items(), ("x", x), ("dy", t[n]["dy"]), ("gain", t[n]["gain"]), ("positions", pos[n])):
            setattr(side, name, v.data_ptr())
    st = torch.cuda.current_stream().cuda_stream
    sli.slikl_qk_norm_rope(qk, tn, st)
    n_grad = sli.slikl_qk_norm_rope_grad_workspace_size(qk)
    ws = torch.empty(n_grad, dtype=torch.uint8, device="cuda")
    sli.slikl_qk_norm_rope_grad(qk, tn, ws.data_ptr(), n_grad, st)

    def same(a, b):
        return torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))

    for n in "qk":
        assert same(held[n]["y"], fwd[n]) and same(held[n]["keep8"], fwd["checkpoint_" + n].values)
        assert same(held[n]["keep8_scale"], fwd["checkpoint_" + n].scale) and same(held[n]["dx"], bwd["dx_" + n])
        assert same(held[n]["dgain"], bwd["dgain_" + n])
    assert same(held["k"]["dbias"], bwd["dbias_k"])
    pr = sli.make_problem(xq, xk, idx, deterministic=True)
    n_all = sli.slikl_grad_projected_workspace_size(pr, qk)
    ws, dw, y = torch.empty(n_all, dtype=torch.uint8, device="cuda"), torch.empty_like(w), torch.empty_like(p)
    main = sli.slikl_tensors(w=w.data_ptr(), attn_softmax_l1norm=p.data_ptr(), sparse_indices=idx.data_ptr(),
                             dw=dw.data_ptr(), softmax_out=y.data_ptr())
    sli.slikl_grad_projected(pr, qk, main, tn, ws.data_ptr(), n_all, st)
    assert same(dw, both["dw"]) and same(y, both["softmax_out"]) and same(held["k"]["dbias"], both["dbias_k"])
    for n in "qk":
        assert same(held[n]["dx"], both["dx_" + n]) and same(held[n]["dgain"], both["dgain_" + n])
    for call in (lambda: sli.slikl_qk_norm_rope(qk, sli.slikl_qk_tensors(), st),
                 lambda: sli.slikl_qk_norm_rope_grad(qk, tn, ws.data_ptr(), n_grad - 1, st),
                 lambda: sli.slikl_grad_projected(pr, qk, main, tn, ws.data_ptr(), n_all - 1, st)):
        with pytest.raises(sli.SliklError):
            call()


@pytest.mark.parametrize("layout,positions", [("BSND", True), ("BSND", False), ("TND", True)])
@pytest.mark.parametrize("source", ["x", "x8"])
def test_projected_gradient_of_a_padded_batch(layout, positions, source):
    """Rows behind the used lengths hold NaN: everything is as with zeros at position -1 in their place,
    bit by bit, and their dx is 0."""
    B, S1, S2, N1, D, K, R = 3, 30, 200, 16, 128, 64, 64
    wl = si.small(seed=75, layout=layout, B=B, S1=S1, S2=S2, N1=N1, D=D, K=K)
    dtype = wl.q.dtype
    cuq, cuk = ([0, S1, 2 * S1, 3 * S1], [0, S2, 2 * S2, 3 * S2]) if layout == "BSND" else (
        wl.cu_seqlens_q.tolist(), wl.cu_seqlens_k.tolist())
    B, T1, T2 = len(cuq) - 1, wl.T1, wl.T2
    used_q = [max(0, (cuq[b + 1] - cuq[b]) * (2 - b) // 2) for b in range(B)]      # all, half, none
    used_k = [max(1, (cuk[b + 1] - cuk[b]) * (b + 1) // B) for b in range(B)]
    q, k = make(76, T1, N1, D, R, dtype, "layer"), make(77, T2, 1, D, R, dtype, "rms")
    cs, pad, pos, x = table(400, R), {}, {}, {}
    for n, s, cu, used in (("q", q, cuq, used_q), ("k", k, cuk, used_k)):
        local = torch.cat([torch.arange(cu[b + 1] - cu[b]) for b in range(B)])
        pad[n] = torch.cat([torch.arange(cu[b + 1] - cu[b]) >= used[b] for b in range(B)])
        pos[n] = (local + 100 if positions else local).to(torch.int32)
        x[n] = s["x"].clone()
        x[n][pad[n]] = 0
    assert pad["q"].any() and pad["k"].any()
    shape = dict(q=wl.q.shape, k=wl.k.shape)
    i32 = dict(dtype=torch.int32, device="cuda")
    kw = dict(gain_q=dev(q["gain"] * 0.1), gain_k=dev(k["gain"]), bias_q=dev(q["bias"]), norm_q="layer",
              layout_q=layout, layout_k=layout, deterministic=True, loss=True,
              cu_seqlens_q=dev(wl.cu_seqlens_q), cu_seqlens_k=dev(wl.cu_seqlens_k),
              key_range_bound=sli.key_range_bound_of(wl), seq_used_q=torch.tensor(used_q, **i32),
              seq_used_k=torch.tensor(used_k, **i32))

    def run(x, **pos):
        xs = [dev(x[n]).reshape(shape[n]) for n in "qk"]
        if source == "x8":
            xs = [sli.checkpoint_pack(t) for t in xs]
        r = sli.grad_projected(*xs, dev(wl.w), dev(wl.p), dev(wl.idx), dev(cs), **pos, **kw)
        torch.cuda.synchronize()
        assert sli.slikl_read_device_status(r.pop("workspace").data_ptr()) == 0
        return r

    want = run(x, **{"pos_" + n: dev(torch.where(pad[n], -1, pos[n])) for n in "qk"})
    for n in "qk":
        x[n][pad[n]] = float("nan")
        pos[n][pad[n]] = 1 << 30                 # no position either
    got = run(x, **({"pos_" + n: dev(pos[n]) for n in "qk"} if positions else {}))
    for n, v in want.items():
        assert (got[n] is None) == (v is None) and (v is None or torch.equal(got[n], v)), n
    for n in "qk":
        assert torch.isfinite(got["dgain_" + n]).all() and got["dgain_" + n].abs().sum() > 0
        dx = got["dx_" + n].reshape(-1, N1 if n == "q" else 1, D)
        assert (dx[pad[n].cuda()] == 0).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("T1,T2", [(0, 40), (30, 0)])
def test_projected_gradient_without_queries_or_keys(T1, T2):
    """Empty TND sides: what is there gets zero gradients."""
    N1, D, K = 8, 64, 16
    q, k = make(91, T1, N1, D, 32, BF, "rms"), make(92, T2, 1, D, 32, BF, "layer")
    cu = [torch.tensor([0, t], dtype=torch.int32, device="cuda") for t in (T1, T2)]
    pos = [torch.arange(t, dtype=torch.int32, device="cuda") for t in (T1, T2)]
    r = sli.grad_projected(dev(q["x"]), dev(k["x"]), torch.rand(T1, N1, device="cuda"),
                           torch.rand(T1, 1, K, device="cuda"),
                           torch.full((T1, 1, K), -1, dtype=torch.int32, device="cuda"), dev(table(50, 32)),
                           pos_q=pos[0], pos_k=pos[1], norm_k="layer", layout_q="TND", layout_k="TND",
                           cu_seqlens_q=cu[0], cu_seqlens_k=cu[1])
    torch.cuda.synchronize()
    assert sli.slikl_read_device_status(r["workspace"].data_ptr()) == 0
    for n in ("dx_q", "dx_k", "dgain_q", "dgain_k", "dbias_k"):
        assert (r[n] == 0).all(), n


def test_two_streams_at_once():
    """Calls in flight on two streams do not disturb each other."""
    cs = dev(table(2000, 64))
    sides = [(make(31 + i, 2000, 16, 128, 64, BF, "layer"), make(33 + i, 2000, 1, 128, 64, BF, "rms")) for i in range(2)]
    pos = torch.arange(2000, dtype=torch.int32, device="cuda")
    kw = dict(pos_q=pos, pos_k=pos, norm_q="layer", layout_q="TND", layout_k="TND")
    args = [tuple(dev(s[n]) for n in ("dy", "x") for s in two) for two in sides]
    want = [sli.qk_norm_rope_grad(*a, cs, **kw) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[sli.qk_norm_rope_grad(*a, cs, stream=s, **kw) for s, a in zip(streams, args)] for _ in range(20)]
    torch.cuda.synchronize()
    for turn in got:
        for w, g in zip(want, turn):
            assert all(torch.equal(w[n], g[n]) for n in w if n != "workspace" and w[n] is not None)
