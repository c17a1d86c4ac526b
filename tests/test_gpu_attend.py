"""Attention of the new rows over the paged cache, against the fp64 oracle.

Tolerance of an output, from its own sums (A the softmax-weighted mean of |v|, E the largest
scale * sum |q k| a row meets):
  * a score is a sum of d exact products in fp32, then one fused multiply-add in the exponent: its
    error is at most 2^-24 (d + 4) E, and the running maximum may lie 8 ln 2 off the largest score,
    which costs one more rounding of 2^-24 (E + 6); the exponential itself 2^-22.  A weight is then
    off by that much of itself, and so is the normaliser: twice the sum of these, times A;
  * sums of T terms in fp32: 2^-24 T each for the output and the normaliser;
  * bf16 rows: weights rounded to bf16 (half a step, 2^-8 of each at most) and the output rounded once
    (2^-8 of it);
  * fp32 rows: weights in three bf16 parts (2^-24), the output rounded to fp32 (2^-24)."""
import numpy as np
import pytest
import torch

from oracle import target_oracle as T
from tests.test_gpu_kv_cache import DT, i32, tables

pytestmark = pytest.mark.gpu


def tolerance(mean, big, d, length, rows_kind):
    u = 2.0 ** -24
    weight = u * ((d + 4) * big + big + 6) + 4 * u
    rel = 2 * weight[..., None] + 2 * u * (length + 8) + (2 * 2.0 ** -8 if rows_kind == "bf16" else 4 * u)
    return mean * rel + 1e-30


def random_trees(B, R, gen, depth=16):
    anc = np.zeros((B, R), np.int64)
    for b in range(B):
        de = [0]
        for t in range(1, R):
            open_ = [s for s in range(t) if de[s] < depth]
            p = open_[int(torch.randint(0, len(open_), (1,), generator=gen))] if t > 2 else t - 1
            de.append(de[p] + 1)
            anc[b, t] = np.int64(np.uint64(int(anc[b, p]) & (2 ** 64 - 1) | 1 << (t - 1)).astype(np.int64))
    return anc


def setup(g, B, R, Hq, H, d, page, kind, rows_kind, ctx, n, mask, seed, scale_v=1.0):
    """A cache holding every request's ctx + n rows (written by the library), everything else in it
    NaN; the rows' values as the cache holds them, in fp64."""
    gen = torch.Generator().manual_seed(seed)
    width = max(1, -(-(max(ctx) + R) // page))
    kv = g.KVCache.empty(1, B * width + 1, H, page, d, DT[kind])
    for x in (kv.k, kv.v):
        x.view(torch.uint8).fill_(0x7f if kind == "e4m3" else 0xff)
    if kind == "e4m3":
        kv.k_scale.fill_(127), kv.v_scale.fill_(127)
    table = tables(B, width, B * width + 1, gen)
    total = max(c + m for c, m in zip(ctx, n))
    k, v = (torch.randn(B, total, H, d, generator=gen).cuda() for _ in range(2))
    v = v * scale_v
    count = i32([c + m for c, m in zip(ctx, n)])
    g.gdntree_cache_write(kv, 0, table, i32([0] * B), k, v, count=count)
    vals = [x.double().cpu().numpy() for x in g.gdntree_cache_read(kv, 0, table, i32([0] * B), total, out_dtype=torch.float32)]
    q = torch.randn(B, R, Hq, d, generator=gen).to(DT[rows_kind]).cuda()
    anc = random_trees(B, R, gen) if mask == "tree" else None
    return kv, table, vals, q, anc


def as_tree(g, anc, n):
    B, R = anc.shape
    t = g.Tree.empty(B, R - 1, "cuda")
    t.anc.copy_(torch.from_numpy(anc))
    t.n_nodes.copy_(torch.tensor(n, dtype=torch.int32))
    return t


def call(g, kv, table, q, ctx, n, anc, o=None, **kw):
    if anc is not None:
        return g.gdntree_attend(q, kv, 0, table, i32(ctx), tree=as_tree(g, anc, n), o=o, **kw)
    return g.gdntree_attend(q, kv, 0, table, i32(ctx), n_rows=i32(n), o=o, **kw)


def check(o, q, vals, ctx, n, anc, rows_kind, scale=None):
    """Every used row against the oracle; rows not in use still hold 7."""
    R, d = q.shape[1], q.shape[3]
    got, qn = o.double().cpu().numpy(), q.double().cpu().numpy()
    worst = 0.0
    for b, (c, m) in enumerate(zip(ctx, n)):
        used = m if 1 <= m <= R else 0
        assert (got[b, used:] == 7.0).all(), f"request {b}: rows not in use were written"
        if not used:
            continue
        see = T.visible(m, c, None if anc is None else anc[b].view(np.uint64))
        want, mean, big = T.attend(qn[b, :m], vals[0][b, :c + m], vals[1][b, :c + m], see, scale or d ** -0.5)
        err = np.abs(got[b, :m] - want) / tolerance(mean, big, d, c + m, rows_kind)
        assert np.isfinite(err).all(), f"request {b}: not finite"
        worst = max(worst, float(err.max()))
    assert worst <= 1.0, f"{worst:.3f} of the tolerance"
    return worst


CASES = [  # B, R, Hq, H, d, page, cache, rows, contexts, rows in use, mask
    (1, 1, 1, 1, 64, 16, "bf16", "bf16", [0], [1], "chain"),
    (1, 1, 4, 2, 128, 16, "bf16", "f32", [1], [1], "chain"),
    (6, 1, 8, 2, 128, 16, "e4m3", "bf16", [0, 14, 15, 16, 30, 31], [1] * 6, "chain"),
    (5, 1, 8, 8, 64, 32, "e4m3", "f32", [32, 33, 63, 127, 128], [1] * 5, "chain"),
    (4, 1, 48, 3, 128, 64, "bf16", "bf16", [129, 255, 1000, 2047], [1] * 4, "chain"),
    (2, 1, 5, 1, 64, 256, "bf16", "f32", [700, 5000], [1, 1], "chain"),
    (3, 2, 6, 2, 128, 16, "bf16", "bf16", [0, 31, 77], [2, 1, 2], "chain"),
    (3, 9, 8, 2, 64, 16, "e4m3", "bf16", [0, 100, 250], [9, 5, 1], "tree"),
    (4, 25, 8, 2, 128, 32, "bf16", "bf16", [0, 7, 40, 600], [25, 24, 1, 13], "tree"),
    (3, 25, 4, 1, 128, 16, "e4m3", "f32", [3, 300, 31], [25, 20, 2], "tree"),
    (3, 65, 8, 2, 128, 64, "bf16", "bf16", [0, 65, 513], [65, 64, 33], "tree"),
    (2, 65, 12, 4, 64, 16, "bf16", "f32", [15, 200], [65, 50], "tree"),
    (2, 65, 16, 1, 64, 32, "e4m3", "bf16", [1, 320], [65, 64], "chain"),
    (2, 64, 4, 4, 128, 128, "e4m3", "bf16", [129, 1025], [64, 63], "tree"),
    (5, 3, 4, 2, 64, 16, "bf16", "bf16", [5, 6, 7, 8, 9], [3, 0, 4, -1, 2], "chain"),   # bad row counts
    (70, 1, 2, 1, 64, 16, "bf16", "bf16", [(17 * b) % 90 for b in range(70)], [1] * 70, "chain"),
    (130, 4, 4, 2, 64, 16, "e4m3", "bf16", [(29 * b) % 200 for b in range(130)], [1 + b % 4 for b in range(130)], "tree"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend_matches_the_oracle(case):
    import gdn_draft_tree_amd as g
    B, R, Hq, H, d, page, kind, rows_kind, ctx, n, mask = CASES[case]
    n_ok = [m if 1 <= m <= R else 1 for m in n]
    kv, table, vals, q, anc = setup(g, B, R, Hq, H, d, page, kind, rows_kind, ctx, n_ok, mask, case)
    o = torch.full_like(q, 7.0)
    call(g, kv, table, q, ctx, n, anc, o=o)
    check(o, q, vals, ctx, n, anc, rows_kind)


@pytest.mark.parametrize("kind,rows_kind,R", [("bf16", "bf16", 1), ("e4m3", "f32", 1), ("bf16", "bf16", 25)])
def test_long_and_ragged_contexts(kind, rows_kind, R):
    """One request of 40,000 positions beside short ones: split, joined and not split in one launch."""
    import gdn_draft_tree_amd as g
    ctx = [3, 40001, 0, 700]
    kv, table, vals, q, anc = setup(g, 4, R, 4, 1, 64, 64, kind, rows_kind, ctx, [R] * 4, "tree" if R > 1 else "chain", 5)
    o = torch.full_like(q, 7.0)
    call(g, kv, table, q, ctx, [R] * 4, anc, o=o)
    check(o, q, vals, ctx, [R] * 4, anc, rows_kind)


@pytest.mark.parametrize("kind,rows_kind,R,Hq,H,d,ctx", [
    ("bf16", "bf16", 65, 8, 2, 128, 2999), ("e4m3", "bf16", 33, 4, 2, 64, 1501), ("bf16", "f32", 25, 2, 1, 128, 4100),
    ("bf16", "bf16", 16, 2, 2, 64, 9001), ("e4m3", "f32", 5, 3, 1, 128, 6007)])
def test_one_request_over_a_long_context(kind, rows_kind, R, Hq, H, d, ctx):
    """A single request's many rows, each joined from many parts."""
    import gdn_draft_tree_amd as g
    kv, table, vals, q, anc = setup(g, 1, R, Hq, H, d, 64, kind, rows_kind, [ctx], [R], "tree", R)
    o = torch.full_like(q, 7.0)
    call(g, kv, table, q, [ctx], [R], anc, o=o)
    check(o, q, vals, [ctx], [R], anc, rows_kind)


@pytest.mark.parametrize("rows_kind", ["bf16", "f32"])
def test_large_scores_and_growing_maxima(rows_kind):
    """Scores of some hundreds that grow along the context (the running maximum moves all the way),
    and a scale of its own."""
    import gdn_draft_tree_amd as g
    ctx, n = [513], [2]
    kv, table, vals, q, anc = setup(g, 1, 2, 2, 1, 64, 16, "bf16", rows_kind, ctx, n, "chain", 9)
    grow = torch.linspace(0.0, 6.0, 515, device="cuda")[:, None] * torch.sign(q[0, 0, 0].float())[None]
    k = grow[None, :, None].to(torch.bfloat16)
    v = torch.from_numpy(vals[1]).to("cuda", torch.bfloat16)
    g.gdntree_cache_write(kv, 0, table, i32([0]), k.contiguous(), v.contiguous())
    vals = [k.double().cpu().numpy(), v.double().cpu().numpy()]
    o = torch.full_like(q, 7.0)
    call(g, kv, table, q, ctx, n, anc, o=o, scale=0.7)
    check(o, q, vals, ctx, n, anc, rows_kind, scale=0.7)


@pytest.mark.parametrize("R,Hq,kind", [(9, 4, "bf16"), (65, 8, "bf16"), (33, 2, "e4m3")])
def test_what_a_row_does_not_see_has_no_effect(R, Hq, kind):
    """NaN and infinities in some tree rows' keys and values: rows that do not descend from them equal
    the clean run's bit for bit, their descendants are not finite."""
    import gdn_draft_tree_amd as g
    ctx = [37, 0]
    kv, table, vals, q, anc = setup(g, 2, R, Hq, 2, 64, 16, kind, "bf16", ctx, [R, R], "tree", 21)
    clean = call(g, kv, table, q, ctx, [R, R], anc).clone()
    bad_slots = [R - 1, R // 2]
    rows = torch.zeros(2, 1, 2, 64, device="cuda")
    for i, s in enumerate(bad_slots):
        kr, vr = rows.clone(), rows.clone()
        if i == 0:
            vr[..., 3] = float("inf")
        else:
            kr[..., 1] = float("nan")
            vr[..., 5] = float("nan")
        g.gdntree_cache_write(kv, 0, table, i32([c + s for c in ctx]), kr, vr)
    got = call(g, kv, table, q, ctx, [R, R], anc)
    for b in range(2):
        for t in range(R):
            touched = [s for s in bad_slots if (int(anc[b, t]) >> (s - 1)) & 1]
            if not touched:
                if kind == "bf16":   # the values product runs term by term there: the same to fp32 sums
                    assert torch.allclose(got[b, t].float(), clean[b, t].float(), rtol=2 ** -7, atol=2 ** -9), (b, t)
                assert torch.isfinite(got[b, t]).all(), (b, t)
            else:
                assert not torch.isfinite(got[b, t]).all(), (b, t)


def test_bad_requests_get_nan_and_spare_the_others():
    import gdn_draft_tree_amd as g
    ctx = [40, 40, 40, 40, 40, 3000]
    n = [3] * 6
    kv, table, vals, q, anc = setup(g, 6, 3, 4, 2, 64, 16, "bf16", "bf16", ctx, n, "chain", 2)
    table[0, 1] = -1
    table[1, 2] = kv.k.shape[1]
    table[5, 120] = -7                           # in the middle of a request that is split
    call_ctx = [40, 40, -1, table.shape[1] * 16 - 2, 40, 3000]
    o = torch.full_like(q, 7.0)
    call(g, kv, table, q, call_ctx, n, None, o=o)
    assert torch.isnan(o[[0, 1, 2, 3, 5]]).all()
    check(o[4:5], q[4:5], [x[4:5] for x in vals], [40], [3], None, "bf16")


def test_all_scores_minus_infinity_is_nan_like_the_formula():
    import gdn_draft_tree_amd as g
    kv, table, vals, q, _ = setup(g, 1, 1, 1, 1, 64, 16, "bf16", "f32", [4], [1], "chain", 3)
    k = torch.full((1, 5, 1, 64), -3.0e38, device="cuda")
    q = torch.full_like(q, 3.0e38)
    g.gdntree_cache_write(kv, 0, table, i32([0]), k, torch.ones_like(k))
    assert torch.isnan(g.gdntree_attend(q, kv, 0, table, i32([4]))).all()


def test_repeatable_and_prepared_and_other_streams():
    import gdn_draft_tree_amd as g
    ctx, n = [3000, 70], [25, 25]
    kv, table, vals, q, anc = setup(g, 2, 25, 8, 2, 128, 32, "e4m3", "bf16", ctx, n, "tree", 4)
    first = call(g, kv, table, q, ctx, n, anc)
    again = call(g, kv, table, q, ctx, n, anc)
    assert torch.equal(first, again)
    prep = call(g, kv, table, q, ctx, n, anc, prepare=True)
    prep.result.zero_()
    assert torch.equal(prep(), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [call(g, kv, table, q, ctx, n, anc, stream=s) for _ in range(20)]    # scratch of earlier calls is not reused early
    handle = call(g, kv, table, q, ctx, n, anc, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(x, first) for x in outs + [handle])


def test_captured_graph_serves_new_lengths():
    import gdn_draft_tree_amd as g
    kv, table, vals, q, _ = setup(g, 3, 1, 8, 2, 128, 16, "bf16", "bf16", [900, 20, 300], [1] * 3, "chain", 6)
    ctx = i32([900, 20, 300])
    o = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.gdntree_attend(q, kv, 0, table, ctx, o=o)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gdntree_attend(q, kv, 0, table, ctx, o=o)
    for lens in ([900, 20, 300], [5, 20, 0], [450, 1, 299], [900, 20, 300]):
        ctx.copy_(i32(lens))
        want = g.gdntree_attend(q, kv, 0, table, ctx)
        o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_binding_refusals():
    import gdn_draft_tree_amd as g
    kv, table, vals, q, anc = setup(g, 2, 3, 4, 2, 64, 16, "bf16", "bf16", [5, 6], [3, 3], "tree", 1)
    ctx = i32([5, 6])
    tree = as_tree(g, anc, [3, 3])
    for bad in (dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(q=q[:, :, :, :32]), dict(ctx=ctx.long()),
                dict(table=table[:1]), dict(n_rows=i32([3, 3]), tree=tree), dict(o=q.float()),
                dict(workspace=torch.empty(64, dtype=torch.uint8)), dict(layer=1), dict(layer=-1), dict(scale=0.0),
                # contexts that may be long need the whole workspace (short ones, as above, need none)
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"), table=table.repeat(1, 80))):
        a = dict(q=q, ctx=ctx, table=table, layer=0, tree=None, n_rows=None, scale=None, o=None, workspace=None)
        a.update(bad)
        with pytest.raises((ValueError, g.GdnTreeError)):
            g.gdntree_attend(a["q"], kv, a["layer"], a["table"], a["ctx"], tree=a["tree"], n_rows=a["n_rows"],
                             scale=a["scale"], o=a["o"], workspace=a["workspace"])


def test_two_calls_at_once():
    """Calls on two streams, each with scratch memory of its own, beside each other."""
    import gdn_draft_tree_amd as g
    ctx = [5001, 1203]
    one = setup(g, 2, 33, 4, 2, 128, 64, "bf16", "bf16", ctx, [33, 33], "tree", 3)
    two = setup(g, 2, 1, 4, 2, 128, 64, "e4m3", "bf16", ctx, [1, 1], "chain", 4)
    alone = [call(g, x[0], x[1], x[3], ctx, [r, r], x[4]) for x, r in ((one, 33), (two, 1))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for s, x, r in zip(streams, (one, two), (33, 1)):
            with torch.cuda.stream(s):
                got.append(call(g, x[0], x[1], x[3], ctx, [r, r], x[4]))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a, b)
