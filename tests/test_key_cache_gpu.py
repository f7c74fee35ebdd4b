"""GPU tests of the weights on the keys and of the cache cut to the keys that carry most of it,
against plain fp64 forms (operators_reference.py): weights within their derived bound, kept rows and
copied caches exactly."""

import math

import pytest
import torch

import slikl_inputs as si
import sparse_lightning_indexer_b200 as sli
import operators_reference as ref

pytestmark = pytest.mark.gpu


def dev(t):
    return None if t is None else t.cuda()


def ranges(lens):
    at, out = 0, []
    for n in lens:
        out.append((at, n))
        at += n
    return out


def cu(lens):
    return torch.tensor([0] + [a + n for a, n in ranges(lens)], dtype=torch.int32)


def draw_rows(seed, lens_q, lens_k, K, invalid=0.3, dup=True):
    """Indices (any order, repeats, -1 in between) and weights normalised over the valid slots."""
    g = torch.Generator().manual_seed(seed)
    idx, w = [], []
    for qn, kn in zip(lens_q, lens_k):
        i = torch.randint(0, max(kn, 1), (qn, K), generator=g)
        if not dup and kn >= K and qn:
            i = torch.stack([torch.randperm(kn, generator=g)[:K] for _ in range(qn)])
        bad = torch.rand(qn, K, generator=g) < invalid
        i[bad | torch.tensor(kn == 0)] = -1
        idx.append(i)
        w.append(torch.exp(torch.randn(qn, K, generator=g)))
    idx, w = torch.cat(idx).to(torch.int32), torch.cat(w)
    valid = idx >= 0
    w = w / (w * valid).sum(-1, keepdim=True).clamp_min(1e-3)
    w = w.clamp_max(2.0)
    w[~valid] = float("nan")                    # never looked at
    return idx, w


def weights_bound(want, named, slots, scores):
    """Half an fp32 step of the result, and half a unit 2^-u for each slot that names the key."""
    u = min(40, 61 - math.ceil(math.log2(max(slots, 1))))
    return want.abs() * 2.0 ** -24 + named * 2.0 ** -(u + 1) + 2.0 ** -149


def check_weights(got, idx, w, br, bk, scores, decay, used_q=None, used_k=None):
    want = ref.key_weights(w, idx, br, bk, scores, decay, used_q, used_k)
    named = ref.key_weights(torch.ones_like(w), idx, br, bk, torch.zeros_like(scores), 0.0, used_q, used_k)
    got = got.cpu().double().reshape(-1)
    over = (got - want).abs() > weights_bound(want, named, idx.numel(), scores)
    assert torch.isfinite(got).all() and not over.any(), (got - want).abs().max()


# (layout, query lengths, key lengths, topk): single rows, a batch without queries, one without
# keys, ranges on both sides of what one multiprocessor holds, rows shorter than a warp
CASES = [
    ("BSND", [1] * 5, [700] * 5, 33),
    ("BSND", [40, 40], [300, 300], 200),
    ("BSND", [1], [1], 1),
    ("BSND", [513], [4096], 257),
    ("BSND", [3] * 300, [50] * 300, 16),
    ("TND", [0, 5, 3, 17], [4, 0, 6, 999], 8),
    ("TND", [130, 1, 64], [5000, 40000, 1], 100),
    ("TND", [600], [131072], 64),
    ("BSND", [4] * 2, [70000] * 2, 2048),
    ("BSND", [2000], [64], 8192),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{len(c[1])}x{max(c[1])}-{max(c[2])}-{c[3]}")
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.875])
def test_key_weights(case, decay):
    layout, lq, lk, K = case
    idx, w = draw_rows(5, lq, lk, K)
    g = torch.Generator().manual_seed(6)
    scores = torch.rand(sum(lk), generator=g) * 10
    B = len(lq)
    bsnd = layout == "BSND"
    s = scores.clone()
    if decay == 0.0:
        s[:] = float("nan")                     # not read
    args = (dev(w).reshape(B, lq[0], 1, K) if bsnd else dev(w)[:, None],
            dev(idx).reshape(B, lq[0], 1, K) if bsnd else dev(idx)[:, None],
            dev(s).reshape(B, lk[0]) if bsnd else dev(s))
    kw = dict(decay=decay, layout_q=layout, layout_k=layout, cu_seqlens_q=None if bsnd else dev(cu(lq)),
              cu_seqlens_k=None if bsnd else dev(cu(lk)), key_range_bound=max(lk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sli.key_weights(*args, status=status, **kw)
    check_weights(r["scores"], idx, w, ranges(lq), ranges(lk), scores, decay)
    assert int(status) == 0
    for _ in range(3):
        assert torch.equal(sli.key_weights(*args, **kw)["scores"], r["scores"])
    if not bsnd:                                # no promise about the longest range
        kw["key_range_bound"] = 0
        assert torch.equal(sli.key_weights(*args, **kw)["scores"], r["scores"])
    own = args[2]
    sli.key_weights(args[0], args[1], own, out=own, **kw)
    assert torch.equal(own, r["scores"])        # in place


@pytest.mark.parametrize("layout_q,layout_k", [("BSND", "TND"), ("TND", "BSND")])
def test_key_weights_mixed_layouts(layout_q, layout_k):
    lq, lk, K = [6, 6, 6], [90, 90, 90], 40
    idx, w = draw_rows(15, lq, lk, K)
    scores = torch.rand(sum(lk), generator=torch.Generator().manual_seed(1))
    r = sli.key_weights(dev(w).reshape((3, 6, 1, K) if layout_q == "BSND" else (18, 1, K)),
                        dev(idx).reshape((3, 6, 1, K) if layout_q == "BSND" else (18, 1, K)),
                        dev(scores).reshape((3, 90) if layout_k == "BSND" else (270,)),
                        layout_q=layout_q, layout_k=layout_k, cu_seqlens_q=dev(cu(lq)),
                        cu_seqlens_k=dev(cu(lk)))
    check_weights(r["scores"], idx, w, ranges(lq), ranges(lk), scores, 1.0)


def test_key_weights_used_lengths():
    lq, lk, K = [50] * 4, [400] * 4, 60
    idx, w = draw_rows(7, lq, lk, K, invalid=0.1)
    idx2 = idx.view(4, 50, K).clone()
    used_q, used_k = [50, 0, 17, 1], [400, 300, 0, 3]
    for b, u in enumerate(used_q):
        idx2[b, u:] = 1 << 30                   # padding rows are not read
    scores = torch.zeros(1600)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    r = sli.key_weights(dev(w).reshape(4, 50, 1, K), dev(idx2).reshape(4, 50, 1, K), dev(scores).reshape(4, 400),
                        seq_used_q=torch.tensor(used_q, **i32), seq_used_k=torch.tensor(used_k, **i32), status=status)
    check_weights(r["scores"], idx2.reshape(-1, K), w, ranges(lq), ranges(lk), scores, 1.0, used_q, used_k)
    assert int(status) == 0
    sli.key_weights(dev(w).reshape(4, 50, 1, K), dev(idx).reshape(4, 50, 1, K), dev(scores).reshape(4, 400),
                    seq_used_q=torch.tensor([51, 0, 0, 0], **i32), status=status)
    assert int(status) == sli.SLIKL_DEV_BAD_SEQ_USED


@pytest.mark.parametrize("lk", [300, 60000])
def test_key_weights_flags(lk):
    """Indices, weights and cu_seqlens that break the contract are flagged, and touch nothing else."""
    lq, K = [9, 4], 50
    idx, w = draw_rows(8, lq, [lk, lk], K, invalid=0.2)
    scores = torch.zeros(2 * lk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(idx, w, cq=cu(lq), ck=cu([lk, lk])):
        status.zero_()
        r = sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), layout_q="TND", layout_k="TND",
                            cu_seqlens_q=dev(cq), cu_seqlens_k=dev(ck), status=status)
        return r["scores"], int(status)

    for bad in (lk, -2, 2 ** 31 - 1, -2 ** 31):
        i2 = idx.clone()
        i2[3, 7] = bad
        got, st = run(i2, w)
        assert st == sli.SLIKL_DEV_INDEX_OUT_OF_RANGE
        i2[3, 7] = -1
        check_weights(got, i2, w, ranges(lq), ranges([lk, lk]), scores, 1.0)
    for bad, stands in ((-1.0, 0.0), (float("nan"), 0.0), (2.5, 2.0), (float("inf"), 2.0), (float("-inf"), 0.0)):
        i2, w2 = idx.clone(), w.clone()
        i2[3, 7], w2[3, 7] = 5, bad
        got, st = run(i2, w2)
        assert st == sli.SLIKL_DEV_BAD_WEIGHT
        w2[3, 7] = stands
        check_weights(got, i2, w2, ranges(lq), ranges([lk, lk]), scores, 1.0)
    i32 = torch.int32
    for cq, ck, bit in ((torch.tensor([0, 20, 13], dtype=i32), cu([lk, lk]), sli.SLIKL_DEV_BAD_CU_SEQLENS_Q),
                        (torch.tensor([0, 9, 12], dtype=i32), cu([lk, lk]), sli.SLIKL_DEV_BAD_CU_SEQLENS_Q),
                        (torch.tensor([-5, 9, 13], dtype=i32), cu([lk, lk]), sli.SLIKL_DEV_BAD_CU_SEQLENS_Q),
                        (cu(lq), torch.tensor([0, 3 * lk, 2 * lk], dtype=i32), sli.SLIKL_DEV_BAD_CU_SEQLENS_K),
                        (cu(lq), torch.tensor([-7, lk, 2 * lk], dtype=i32), sli.SLIKL_DEV_BAD_CU_SEQLENS_K)):
        got, st = run(idx, w, cq, ck)
        assert st & bit


@pytest.mark.parametrize("rows,K", [(13, 50), (1000, 300)])      # both sides of 65536 slots a batch
def test_key_weights_unusable_key_ranges(rows, K):
    """Key ranges that overlap, leave rows out or lead outside are all emptied, as for the gradient: every
    row of the result is written, as decay * scores, in place too."""
    lk = 700
    assert (rows * K > 2 * 65536) == (rows == 1000)
    idx, w = draw_rows(51, [rows - 3, 3], [lk, lk], K)
    scores = torch.rand(2 * lk, generator=torch.Generator().manual_seed(52))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ck in ([0, 2100, 1400], [-7, 700, 1400], [0, 700, 1399], [5, 700, 1400], [0, 900, 800], [1400, 700, 0]):
        status.zero_()
        out = torch.full((2 * lk,), float("nan"), device="cuda")
        kw = dict(decay=0.5, layout_q="TND", layout_k="TND", cu_seqlens_q=dev(cu([rows - 3, 3])),
                  cu_seqlens_k=torch.tensor(ck, dtype=torch.int32, device="cuda"), status=status)
        sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), out=out, **kw)
        assert int(status) & sli.SLIKL_DEV_BAD_CU_SEQLENS_K
        assert torch.equal(out.cpu(), 0.5 * scores), ck
        own = dev(scores)
        sli.key_weights(dev(w)[:, None], dev(idx)[:, None], own, out=own, **kw)
        assert torch.equal(own.cpu(), 0.5 * scores), ck


def test_key_weights_of_many_short_sequences():
    """More sequences than every block looks at, TND, with used lengths and empty ones; unusable ranges among
    them empty all."""
    B, K = 3000, 24
    lq, lk = [b % 3 for b in range(B)], [(7 * b) % 31 for b in range(B)]
    assert sum(lq) * K <= 65536 * B
    idx, w = draw_rows(54, lq, lk, K)
    scores = torch.rand(sum(lk), generator=torch.Generator().manual_seed(55))
    used_k = [max(0, n - b % 4) for b, n in enumerate(lk)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(decay=0.5, layout_q="TND", layout_k="TND", cu_seqlens_q=dev(cu(lq)), status=status)
    for bound in (0, 31, 5):
        got = sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), cu_seqlens_k=dev(cu(lk)), key_range_bound=bound,
                              seq_used_k=torch.tensor(used_k, dtype=torch.int32, device="cuda"), **kw)["scores"]
        check_weights(got, idx, w, ranges(lq), ranges(lk), scores, 0.5, None, used_k)
        assert int(status) == 0
    broken = cu(lk)
    broken[1700] += 500
    for bound in (0, 31, 5):
        got = torch.full((sum(lk),), float("nan"), device="cuda")
        sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), cu_seqlens_k=dev(broken), key_range_bound=bound,
                        out=got, **kw)
        assert int(status) & sli.SLIKL_DEV_BAD_CU_SEQLENS_K and torch.equal(got.cpu(), 0.5 * scores)


@pytest.mark.parametrize("rows,K", [(4, 33), (700, 300)])        # both sides of 65536 slots
@pytest.mark.parametrize("decay", [0.99, 1 / 3, 1e-45])
def test_key_weights_decay_in_64_bits(rows, K, decay):
    """What no slot names is the product with the decay that the caller gave, rounded once."""
    scores = torch.rand(1, 5000, generator=torch.Generator().manual_seed(53)) * 10
    idx = torch.full((1, rows, 1, K), -1, dtype=torch.int32, device="cuda")
    got = sli.key_weights(torch.zeros(1, rows, 1, K, device="cuda"), idx, dev(scores), decay=decay)["scores"].cpu()
    assert torch.equal(got, (scores.double() * decay).float())


def test_key_weights_beyond_one_pass_of_p():
    """A hot key that every row names with its whole weight: the sum is exact."""
    T, S2 = 5000, 40
    idx = torch.full((1, T, 1, 4), -1, dtype=torch.int32)
    idx[..., 2] = 17
    w = torch.full((1, T, 1, 4), 7.0)
    w[..., 2] = 1.0
    r = sli.key_weights(dev(w), dev(idx), torch.zeros(1, S2, device="cuda"))["scores"].cpu()
    assert r[0, 17] == T and r.sum() == T


def test_more_sequences_than_a_grid_dimension_holds():
    """66000 sequences of a few rows: weights over all of them, and their caches cut."""
    B, S2, K = 66000, 5, 3
    idx, w = draw_rows(31, [1] * B, [S2] * B, K)
    scores = torch.rand(B * S2, generator=torch.Generator().manual_seed(32))
    r = sli.key_weights(dev(w).view(B, 1, 1, K), dev(idx).view(B, 1, 1, K), dev(scores).view(B, S2), decay=0.5)
    rows = torch.where(idx >= 0, idx + S2 * torch.arange(B)[:, None], 0).reshape(-1).long()
    full = torch.where(idx >= 0, w, 0.0).double().reshape(-1)
    want = 0.5 * scores.double() + torch.bincount(rows, weights=full, minlength=B * S2)
    named = torch.bincount(rows, minlength=B * S2)
    got = r["scores"].cpu().double().reshape(-1)
    assert ((got - want).abs() <= weights_bound(want, named, idx.numel(), scores)).all()
    c = torch.randn(B, S2, 8, device="cuda").to(torch.bfloat16)
    cut = sli.evict(r["scores"], [c], 2, recent=1)
    order = r["scores"].clone()
    order[:, -1] = float("inf")
    keep = order.sort(dim=1, descending=True, stable=True).indices[:, :2].sort(1).values
    assert torch.equal(cut["kept"].long(), keep) and (cut["lengths"] == 2).all()
    assert torch.equal(cut["caches"][0], c.gather(1, keep[..., None].expand(-1, -1, 8)))


def test_key_weights_calls_in_flight_on_two_streams():
    """Calls of several launches each, behind one another and beside each other, with workspaces of their own."""
    sets = []
    for seed in (41, 42):
        idx, w = draw_rows(seed, [700], [9000], 300)
        sets.append((dev(w).view(1, 700, 1, 300), dev(idx).view(1, 700, 1, 300), torch.rand(1, 9000, device="cuda")))
    want = [sli.key_weights(*a)["scores"] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    ws = [sli.key_weights(*a)["workspace"] for a in sets]
    torch.cuda.synchronize()
    got = [[sli.key_weights(*a, workspace=k, stream=st)["scores"] for a, k, st in zip(sets, ws, streams)] for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, v) for turn in got for g, v in zip(turn, want))


def test_a_stream_of_another_device_is_refused():
    """It could not order the call's work, which would have gone to the tensors' own device unordered."""
    n = torch.cuda.device_count()
    if n > 1:
        other = torch.cuda.Stream(device=1)
    else:
        other = torch.Stream(stream_id=0, device_index=1, device_type=int(torch._C._autograd.DeviceType.CUDA))
    s = torch.rand(1, 30, device="cuda:0")
    w, i = torch.rand(1, 2, 1, 8, device="cuda:0"), torch.zeros(1, 2, 1, 8, dtype=torch.int32, device="cuda:0")
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda:0")
    for call in (lambda: sli.key_weights(w, i, s, stream=other), lambda: sli.evict(s, [], 4, stream=other),
                 lambda: sli.qk_norm_rope(x, None, layout_q="TND", stream=other),
                 lambda: sli.qk_norm_rope_grad(x, None, x, None, layout_q="TND", stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def slots_of(lq, K):
    """Slots of the call, which the form for many of them takes above 65536 a batch on average."""
    return sum(lq) * K, 65536 * len(lq)


# more than 65536 slots a batch: ranges of one, two and three chunks of 55296 keys, uneven sequences with empty
# ones on either side, more batches than multiprocessors can share, one long batch among short ones
LARGE = [
    ("BSND", [400], [60000], 300),
    ("BSND", [300] * 2, [70000] * 2, 500),
    ("BSND", [70] * 160, [300] * 160, 1000),
    ("TND", [600], [131072], 300),
    ("TND", [0, 700, 3, 500, 40], [40, 60000, 0, 9000, 55297], 400),
    ("TND", [1, 2500, 1, 1], [55296, 110593, 77, 1], 128),
    ("TND", [130 + 7 * (b % 5) for b in range(100)], [50 + 130 * (b % 9) for b in range(100)], 600),
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{c[0]}-{len(c[1])}x{max(c[1])}-{max(c[2])}-{c[3]}")
def test_key_weights_of_many_slots(case):
    layout, lq, lk, K = case
    slots, few = slots_of(lq, K)
    assert slots > few
    idx, w = draw_rows(61, lq, lk, K)
    scores = torch.rand(sum(lk), generator=torch.Generator().manual_seed(62)) * 10
    bsnd, B = layout == "BSND", len(lq)
    lead = (B, lq[0]) if bsnd else (sum(lq),)
    i, wd, s = dev(idx).reshape(*lead, 1, K), dev(w).reshape(*lead, 1, K), dev(scores).reshape((B, lk[0]) if bsnd else (-1,))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(decay=0.7, layout_q=layout, layout_k=layout, cu_seqlens_q=None if bsnd else dev(cu(lq)),
              cu_seqlens_k=None if bsnd else dev(cu(lk)), status=status)
    r = sli.key_weights(wd, i, s, **kw)["scores"]
    check_weights(r, idx, w, ranges(lq), ranges(lk), scores, 0.7)
    # a promise about the longest range that is right, one that is not, and the result in place
    for bound in () if bsnd else (max(lk), max(1, max(lk) // 3), 1):
        assert torch.equal(sli.key_weights(wd, i, s, key_range_bound=bound, **kw)["scores"], r), bound
    used_q = [n * (b % 4) // 3 for b, n in enumerate(lq)]
    used_k = [n * (3 - b % 4) // 3 for b, n in enumerate(lk)]
    i32 = dict(dtype=torch.int32, device="cuda")
    ur = sli.key_weights(wd, i, s, seq_used_q=torch.tensor(used_q, **i32), seq_used_k=torch.tensor(used_k, **i32), **kw)["scores"]
    check_weights(ur, idx, w, ranges(lq), ranges(lk), scores, 0.7, used_q, used_k)
    sli.key_weights(wd, i, s, out=s, **kw)
    assert torch.equal(s, r) and int(status) == 0


@pytest.mark.parametrize("layout_q,layout_k", [("BSND", "TND"), ("TND", "BSND")])
def test_key_weights_of_many_slots_in_mixed_layouts(layout_q, layout_k):
    B, S1, S2, K = 3, 300, 60000, 300
    assert B * S1 * K > 65536 * B
    idx, w = draw_rows(63, [S1] * B, [S2] * B, K)
    scores = torch.rand(B * S2, generator=torch.Generator().manual_seed(64))
    lead = (B, S1) if layout_q == "BSND" else (B * S1,)
    r = sli.key_weights(dev(w).reshape(*lead, 1, K), dev(idx).reshape(*lead, 1, K),
                        dev(scores).reshape((B, S2) if layout_k == "BSND" else (B * S2,)), layout_q=layout_q,
                        layout_k=layout_k, cu_seqlens_q=dev(cu([S1] * B)), cu_seqlens_k=dev(cu([S2] * B)))["scores"]
    check_weights(r, idx, w, ranges([S1] * B), ranges([S2] * B), scores, 1.0)


@pytest.mark.parametrize("lk", [900, 60000])
def test_key_weights_flags_of_many_slots(lk):
    """What breaks the contract in a large call is flagged, and touches nothing else."""
    lq, K = [500, 4], 300
    assert sum(lq) * K > 65536 * 2
    idx, w = draw_rows(65, lq, [lk, lk], K, invalid=0.2)
    scores = torch.zeros(2 * lk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(layout_q="TND", layout_k="TND", cu_seqlens_k=dev(cu([lk, lk])), status=status)

    def run(idx, w, cq=cu(lq)):
        status.zero_()
        r = sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), cu_seqlens_q=dev(cq), **kw)
        return r["scores"], int(status)

    for bad in (lk, -2, 2 ** 31 - 1, -2 ** 31):
        i2 = idx.clone()
        i2[3, 7] = i2[501, 299] = bad
        got, st = run(i2, w)
        assert st == sli.SLIKL_DEV_INDEX_OUT_OF_RANGE
        i2[3, 7] = i2[501, 299] = -1
        check_weights(got, i2, w, ranges(lq), ranges([lk, lk]), scores, 1.0)
    for bad, stands in ((-1.0, 0.0), (float("nan"), 0.0), (2.5, 2.0), (float("inf"), 2.0), (float("-inf"), 0.0)):
        i2, w2 = idx.clone(), w.clone()
        i2[3, 7], w2[3, 7], i2[501, 299], w2[501, 299] = 5, bad, lk - 1, bad
        got, st = run(i2, w2)
        assert st == sli.SLIKL_DEV_BAD_WEIGHT
        w2[3, 7] = w2[501, 299] = stands
        check_weights(got, i2, w2, ranges(lq), ranges([lk, lk]), scores, 1.0)
    for cq in ([0, 700, 504], [0, 500, 503], [-5, 500, 504]):
        got, st = run(idx, w, torch.tensor(cq, dtype=torch.int32))
        assert st & sli.SLIKL_DEV_BAD_CU_SEQLENS_Q and torch.isfinite(got).all()
    status.zero_()
    sli.key_weights(dev(w)[:, None], dev(idx)[:, None], dev(scores), cu_seqlens_q=dev(cu(lq)),
                    seq_used_q=torch.tensor([501, 4], dtype=torch.int32, device="cuda"), **kw)
    assert int(status) == sli.SLIKL_DEV_BAD_SEQ_USED


@pytest.mark.parametrize("rows,K", [(4, 8), (700, 300)])         # both sides of 65536 slots
def test_key_weights_smallest_unit(rows, K):
    """Units of 2^-40 up to 2^21 slots: a weight of one unit counts, half a unit (a tie, to even) does not,
    and what lies above the half counts as one."""
    w = torch.full((1, rows, 1, K), float("nan"))
    idx = torch.full((1, rows, 1, K), -1, dtype=torch.int32)
    for k, x in enumerate((2.0 ** -40, 2.0 ** -41, 2.0 ** -41 * (1 + 2.0 ** -23), 2.0 ** -42, 1.5 * 2.0 ** -40, 2.0)):
        w[0, rows - 1, 0, k], idx[0, rows - 1, 0, k] = x, k
    got = sli.key_weights(dev(w), dev(idx), torch.zeros(1, 10, device="cuda"))["scores"].cpu()[0].tolist()
    unit = 2.0 ** -40
    assert got == [unit, 0.0, unit, 0.0, 2 * unit, 2.0, 0.0, 0.0, 0.0, 0.0]


def test_key_weights_two_graphs_share_a_workspace():
    """Calls that keep their sums in the workspace, captured on one workspace and replayed in turn."""
    idx, w = draw_rows(66, [700], [9000], 300)
    i, s = dev(idx).view(1, 700, 1, 300), torch.rand(1, 9000, device="cuda")
    ws, graphs = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), []
    for scale in (1.0, 0.5):
        wd = dev(w).view(1, 700, 1, 300) * scale
        sli.key_weights(wd, i, s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sli.key_weights(wd, i, s, workspace=ws)["scores"]
        graphs.append((g, out, wd))
    for j in (0, 1, 1, 0, 1):
        graphs[j][0].replay()
    torch.cuda.synchronize()
    for _, out, wd in graphs:
        assert torch.equal(out, sli.key_weights(wd, i, s)["scores"])


def test_key_weights_without_queries_or_keys():
    e = torch.empty(0, 1, 8, device="cuda")
    s = torch.rand(30, device="cuda")
    z = dev(torch.zeros(2, dtype=torch.int32))
    r = sli.key_weights(e, e.int(), s, decay=0.5, layout_q="TND", layout_k="TND", cu_seqlens_q=z,
                        cu_seqlens_k=dev(cu([30])))
    assert torch.equal(r["scores"], s * 0.5)
    w = torch.rand(2, 1, 8, device="cuda")
    r = sli.key_weights(w, torch.full((2, 1, 8), -1, dtype=torch.int32, device="cuda"), s[:0], layout_q="TND",
                        layout_k="TND", cu_seqlens_q=dev(cu([2])), cu_seqlens_k=z)
    assert r["scores"].numel() == 0


# --- eviction ------------------------------------------------------------------------------------

def make_scores(seed, total, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "normal":
        return torch.randn(total, generator=g)
    if kind == "ties":                          # few values, both zeros among them
        return torch.randint(-2, 3, (total,), generator=g).float() * torch.where(
            torch.rand(total, generator=g) < 0.5, -1.0, 1.0)
    if kind == "same":
        return torch.full((total,), 0.25)
    if kind == "close":                         # alike in their high bits
        return 1 + torch.randint(0, 1000, (total,), generator=g).float() * 2.0 ** -23
    s = torch.randn(total, generator=g) * torch.exp(20 * torch.randn(total, generator=g))
    r = torch.rand(total, generator=g)
    for k, v in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-45, -1e-45, -float("nan"))):
        s[(r >= 0.05 * k) & (r < 0.05 * (k + 1))] = v
    return s


EVICT = [
    # layout, lengths, budget, sinks, recent
    ("BSND", [37] * 3, 12, 2, 3),
    ("BSND", [601], 150, 4, 32),
    ("BSND", [1024] * 2, 1, 0, 0),
    ("BSND", [1025] * 2, 1024, 0, 0),
    ("BSND", [5000] * 4, 700, 700, 0),
    ("BSND", [5000] * 2, 700, 0, 700),
    ("BSND", [8192] * 4, 2048, 4, 64),
    ("BSND", [20000] * 2, 19999, 1, 1),
    ("BSND", [131072], 16384, 4, 32),
    ("TND", [0, 1, 5, 900, 40, 33000], 40, 3, 5),
    ("TND", [50] * 200, 33, 0, 1),
    ("TND", [140000, 3], 5000, 0, 0),
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"{c[0]}-{len(c[1])}x{max(c[1])}-{c[2]}-{c[3]}-{c[4]}")
@pytest.mark.parametrize("kind", ["normal", "ties", "same", "close", "strange"])
def test_evict(case, kind):
    layout, lens, budget, sinks, recent = case
    B, total = len(lens), sum(lens)
    scores = make_scores(11, total, kind)
    g = torch.Generator().manual_seed(12)
    bsnd = layout == "BSND"
    used = [max(0, n - 7 * b) for b, n in enumerate(lens)] if bsnd and B > 2 else None
    caches = [torch.randn(total, 1, 64, generator=g).to(torch.bfloat16), torch.randn(total, 2, 2, generator=g),
              torch.randint(0, 255, (total, 48), generator=g).to(torch.uint8)]
    lead = (B, lens[0]) if bsnd else (total,)
    outs = [torch.full((B, budget, *c.shape[1:]), 3, dtype=c.dtype, device="cuda") for c in caches]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sli.evict(dev(scores).reshape(lead), [dev(c).reshape(*lead, *c.shape[1:]) for c in caches], budget,
                  sinks=sinks, recent=recent, layout_k=layout, cu_seqlens_k=None if bsnd else dev(cu(lens)),
                  seq_used_k=None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda"),
                  out=dict(caches=outs), status=status)
    assert int(status) == 0
    for b, (at, n) in enumerate(ranges(lens)):
        n = n if used is None else used[b]
        keep = ref.evict(scores[at: at + n], n, budget, sinks, recent)
        m = len(keep)
        assert int(r["lengths"][b]) == m
        assert r["kept"][b].tolist() == keep + [-1] * (budget - m)
        rows = at + torch.tensor(keep, dtype=torch.long)
        got = r["scores"][b].cpu()
        assert torch.equal(got[:m].view(torch.int32), scores[rows].view(torch.int32)) and (got[m:] == 0).all()
        for c, o in zip(caches, r["caches"]):
            assert torch.equal(o[b, :m].cpu(), c[rows]) and (o[b, m:] == 3).all()


@pytest.mark.parametrize("bound", [20, 8192, 9001, 40000])
@pytest.mark.parametrize("kind", ["normal", "same", "strange"])
def test_evict_with_a_promise_about_the_longest_sequence(bound, kind):
    """key_range_bound only chooses how many multiprocessors share a sequence; one that the lengths break
    costs time, not rows."""
    lens, budget, sinks, recent = [3000, 40000, 0, 20, 8192, 700, 9001], 600, 3, 50
    scores = make_scores(14, sum(lens), kind)
    c = torch.arange(4 * sum(lens), dtype=torch.int32).reshape(-1, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sli.evict(dev(scores), [dev(c)], budget, sinks=sinks, recent=recent, layout_k="TND", cu_seqlens_k=dev(cu(lens)),
                  key_range_bound=bound, status=status)
    assert int(status) == 0
    for b, (at, n) in enumerate(ranges(lens)):
        keep = ref.evict(scores[at: at + n], n, budget, sinks, recent)
        m = len(keep)
        assert int(r["lengths"][b]) == m and r["kept"][b].tolist() == keep + [-1] * (budget - m)
        rows = at + torch.tensor(keep, dtype=torch.long)
        assert torch.equal(r["scores"][b, :m].cpu().view(torch.int32), scores[rows].view(torch.int32))
        assert torch.equal(r["caches"][0][b, :m].cpu(), c[rows]) and (r["caches"][0][b, m:] == 0).all()


def test_evict_without_caches_and_default_outputs():
    s = torch.rand(2, 100, device="cuda")
    r = sli.evict(s, [], 10)
    assert r["caches"] == [] and (r["lengths"] == 10).all()
    c = torch.rand(2, 100, 4, device="cuda")
    used = torch.tensor([3, 100], dtype=torch.int32, device="cuda")
    r = sli.evict(s, [c], 10, seq_used_k=used)
    assert torch.equal(r["caches"][0][0, :3], c[0, :3]) and (r["caches"][0][0, 3:] == 0).all()


@pytest.mark.parametrize("S2", [60, 3000, 20000])
def test_evict_lengths_in_place(S2):
    """The used lengths may become the kept ones in place."""
    s = torch.rand(4, S2, device="cuda")
    used = torch.tensor([0, 7, S2, S2 // 2], dtype=torch.int32, device="cuda")
    want = sli.evict(s, [], 20, sinks=1, recent=2, seq_used_k=used.clone())
    got = sli.evict(s, [], 20, sinks=1, recent=2, seq_used_k=used, out=dict(lengths=used))
    assert used.tolist() == [0, 7, 20, 20] and torch.equal(got["kept"], want["kept"])
    assert torch.equal(got["scores"], want["scores"])


def test_evict_flags():
    s = torch.rand(3, 20, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sli.evict(s, [], 30, seq_used_k=torch.tensor([21, -1, 20], dtype=torch.int32, device="cuda"), status=status)
    assert int(status) == sli.SLIKL_DEV_BAD_SEQ_USED and r["lengths"].tolist() == [20, 0, 20]
    c = torch.rand(60, 4, device="cuda")
    for bad in ([0, 70, 60], [0, 30, 20], [-4, 30, 60], [0, 30, 59]):
        status.zero_()
        r = sli.evict(s.reshape(-1), [c], 5, layout_k="TND", cu_seqlens_k=torch.tensor(bad, dtype=torch.int32, device="cuda"),
                      status=status)
        torch.cuda.synchronize()
        assert int(status) & sli.SLIKL_DEV_BAD_CU_SEQLENS_K


def test_evict_beyond_32_bits():
    """A cache of more than 2^32 bytes whose last rows stay."""
    S2, row = 1 << 20, 4352 // 2
    c = torch.zeros(2, S2, row, dtype=torch.bfloat16, device="cuda")
    c[1, -3:] = torch.arange(3, device="cuda")[:, None].to(torch.bfloat16) + 1
    s = torch.zeros(2, S2, device="cuda")
    s[1, -3:] = 1
    r = sli.evict(s, [c], 4)
    assert r["kept"].tolist() == [[0, 1, 2, 3], [0, S2 - 3, S2 - 2, S2 - 1]]
    assert torch.equal(r["caches"][0][1, 1:], c[1, -3:])


# --- together ------------------------------------------------------------------------------------

def test_weights_then_eviction_then_the_gradient_on_the_smaller_cache():
    """p of grad_recompute_p -> key_weights -> evict -> grad on the smaller cache, whose slots are the
    kept keys' new places and whose lengths are its used lengths, against the gradient on the full
    cache with the same keys named."""
    B, S1, S2, K = 2, 24, 300, 64
    wl = si.small(seed=81, layout="BSND", B=B, S1=S1, S2=S2, N1=16, D=128, K=K)
    main = si.main_attention(wl, 16, 128, seed=82)
    first = sli.grad_recompute_p_workload(wl, main)
    scores = sli.key_weights(first["p"], dev(wl.idx), torch.zeros(B, S2, device="cuda"))["scores"]
    want = ref.key_weights(first["p"].cpu().reshape(-1, K), wl.idx.reshape(-1, K), ranges([S1] * B), ranges([S2] * B),
                           torch.zeros(B * S2), 0.0)
    assert ((scores.cpu().double().reshape(-1) - want).abs() <= want * 2.0 ** -24 + S1 * 2.0 ** -41).all()
    assert abs(float(scores.double().sum()) - B * S1) < 1e-2 * B * S1    # each row's p sums to one
    budget = 100
    k = dev(wl.k)
    cut = sli.evict(scores, [k], budget, sinks=2, recent=10)
    place = torch.full((B, S2), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        place[b, cut["kept"][b].long()] = torch.arange(budget, dtype=torch.int32, device="cuda")
    idx = dev(wl.idx).reshape(B, -1)
    new = torch.where(idx >= 0, place.gather(1, idx.clamp_min(0).long()), -1).reshape(wl.idx.shape)
    full = torch.where(new >= 0, dev(wl.idx), -1)
    p = torch.where(new >= 0, first["p"], 0.0)
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    args = dev(wl.w), p
    small = sli.grad(dev(wl.q), cut["caches"][0], *args, new, deterministic=True, seq_used_k=cut["lengths"])
    big = sli.grad(dev(wl.q), k, *args, full, deterministic=True)
    torch.cuda.synchronize()
    assert sli.slikl_read_device_status(small["workspace"].data_ptr()) == 0
    for n in ("dq", "dw", "softmax_out"):
        assert torch.equal(small[n], big[n]), n
    # dk's sums run over other blocks of keys: the same terms, at most S1 * 16 of |w| |q|, in another
    # order in fp32, then one rounding to 16 bits on either side
    terms = S1 * 16 * float(wl.w.abs().max()) * float(wl.q.float().abs().max())
    for b in range(B):
        x, y = small["dk"][b].float(), big["dk"][b, cut["kept"][b].long()].float()
        assert ((x - y).abs() <= 2 * 2.0 ** -8 * y.abs() + 2 * S1 * 16 * 2.0 ** -24 * terms).all()


def test_structs_and_addresses_instead_of_tensors():
    """The functions that take the C structs, for memory that is not torch's, do what those for tensors do."""
    S1, S2, K, budget, D = 60, 3000, 128, 500, 64
    idx, w = draw_rows(71, [S1], [S2], K)
    i, w, s = dev(idx).reshape(1, S1, 1, K), dev(w).reshape(1, S1, 1, K), torch.rand(1, S2, device="cuda")
    c = torch.randn(1, S2, D, device="cuda")
    want = sli.key_weights(w, i, s, decay=0.9)["scores"]
    cut = sli.evict(want, [c], budget, sinks=4, recent=8)
    st = torch.cuda.current_stream().cuda_stream
    pr = sli.slikl_problem(layout_q=sli.SLIKL_BSND, layout_k=sli.SLIKL_BSND, B=1, S1=S1, S2=S2, topk=K)
    n = sli.slikl_key_weights_workspace_size(pr)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(s)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tn = sli.slikl_key_weights_tensors(sparse_indices=i.data_ptr(), weights=w.data_ptr(), scores=s.data_ptr(),
                                       out=out.data_ptr(), status=status.data_ptr())
    sli.slikl_key_weights(pr, tn, 0.9, ws.data_ptr(), n, st)
    assert torch.equal(out, want)
    kept, lengths = torch.empty(1, budget, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    best, small = torch.empty(1, budget, device="cuda"), torch.empty(1, budget, D, device="cuda")
    pr = sli.slikl_evict_problem(layout_k=sli.SLIKL_BSND, n_caches=1, B=1, S2=S2, budget=budget, sinks=4, recent=8)
    tn = sli.slikl_evict_tensors(scores=out.data_ptr(), kept=kept.data_ptr(), lengths=lengths.data_ptr(),
                                 scores_out=best.data_ptr(), status=status.data_ptr())
    tn.caches[0] = (c.data_ptr(), small.data_ptr(), D * 4)
    sli.slikl_evict(pr, tn, st)
    assert torch.equal(kept, cut["kept"]) and torch.equal(lengths, cut["lengths"]) and torch.equal(best, cut["scores"])
    assert torch.equal(small, cut["caches"][0]) and int(status) == 0
    tn.caches[0] = (c.data_ptr(), kept.data_ptr() // 16 * 16, D * 4)
    with pytest.raises(sli.SliklError):
        sli.slikl_evict(pr, tn, st)
    pr = sli.slikl_problem(layout_q=sli.SLIKL_BSND, layout_k=sli.SLIKL_BSND, B=1, S1=S1, S2=S2, topk=0)
    with pytest.raises(sli.SliklError):
        sli.slikl_key_weights(pr, sli.slikl_key_weights_tensors(), 1.0, ws.data_ptr(), n, st)


def test_graph_and_other_stream():
    lq, lk, K = [64], [3000], 128
    idx, w = draw_rows(21, lq, lk, K)
    i, w, s = dev(idx).reshape(1, 64, 1, K), dev(w).reshape(1, 64, 1, K), torch.rand(1, 3000, device="cuda")
    c = torch.randn(1, 3000, 64, device="cuda")
    want = sli.key_weights(w, i, s)["scores"]
    cut = sli.evict(want, [c], 500, sinks=4, recent=8)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = sli.key_weights(w, i, s, stream=st)["scores"]
    b = sli.evict(a, [c], 500, sinks=4, recent=8, stream=st)
    st.synchronize()
    assert torch.equal(a, want) and torch.equal(b["kept"], cut["kept"]) and torch.equal(b["caches"][0], cut["caches"][0])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graphs = []
    for scale in (1.0, 0.5):                    # two graphs that share one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a = sli.key_weights(w * scale, i, s, workspace=ws)["scores"]
            b = sli.evict(a, [c], 500, sinks=4, recent=8)
        graphs.append((g, a, b, scale))
    for j in (0, 1, 1, 0):
        graphs[j][0].replay()
    torch.cuda.synchronize()
    for _, a, b, scale in graphs:
        want = sli.key_weights(w * scale, i, s)["scores"]
        cut = sli.evict(want, [c], 500, sinks=4, recent=8)
        assert torch.equal(a, want) and torch.equal(b["kept"], cut["kept"])
        assert torch.equal(b["caches"][0], cut["caches"][0])
