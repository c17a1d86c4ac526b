"""Timed cases of the operators around the hybrid target's attention layers and of sampled
acceptance: the paged key-value cache (write, read back, accepted-path commit), attention of the
new rows over it, and acceptance at a temperature.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the package's
entry points.  A case's context lengths and path lengths follow from the case alone; its values
come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 151936      # the vocabulary of this repository's workloads
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one request, one new token, a short conversation: launch latency; fp32 rows, d = 64
        dict(name="attend_short", op="attend", B=1, R=1, mask="chain", hq=16, hkv=4, d=64, page=16, cache="bf16",
             dtype="f32", lo=200, hi=517),
        # one request, one new token behind a very long context: the cache's bytes
        dict(name="attend_long", op="attend", B=1, R=1, mask="chain", hq=32, hkv=8, d=128, page=64, cache="bf16",
             dtype="bf16", lo=131000, hi=131000),
        # a decoding batch of ragged lengths over an 8-bit cache
        dict(name="attend_batch_e4m3", op="attend", B=32, R=1, mask="chain", hq=32, hkv=8, d=128, page=32,
             cache="e4m3", dtype="bf16", lo=1, hi=16001),
        # the ragged batch's trees (64 drafts and the root) over ragged contexts: the verify step
        dict(name="attend_tree", op="attend", B=32, R=65, mask="tree", hq=32, hkv=8, d=128, page=64, cache="bf16",
             dtype="bf16", lo=100, hi=4099),
        # the cache rows of one new token each of a batch
        dict(name="write_decode", op="write", B=32, R=1, hkv=8, d=128, page=32, cache="e4m3", dtype="bf16", lo=0,
             hi=2000),
        # prompts written as they are prefilled, of ragged lengths
        dict(name="write_prompt", op="write", B=8, R=4093, hkv=8, d=128, page=64, cache="e4m3", dtype="bf16", lo=0,
             hi=300),
        # a short prefix read back from a bf16 cache, fp32 out
        dict(name="read_prefix", op="read", B=1, R=333, hkv=4, d=64, page=16, cache="bf16", dtype="f32", lo=0, hi=64),
        # whole contexts read back from an 8-bit cache (to hand a cache on)
        dict(name="read_contexts", op="read", B=8, R=4093, hkv=8, d=128, page=64, cache="e4m3", dtype="bf16", lo=0,
             hi=300),
        # the accepted path of one request, a few layers
        dict(name="commit_one", op="commit", B=1, L=4, N=24, P=8, hkv=8, d=128, page=16, cache="bf16", lo=90, hi=101),
        # the accepted paths of the ragged batch, every attention layer of a 64-layer hybrid
        dict(name="commit_batch", op="commit", B=32, L=16, N=64, P=16, hkv=8, d=128, page=32, cache="e4m3", lo=5,
             hi=200),
        # one request's tree, sampled
        dict(name="accept_one", op="accept", B=1, N=24, P=8, V=VOCAB, dtype="f32", greedy=0),
        # the ragged batch's trees, sampled, every fourth request greedy
        dict(name="accept_batch", op="accept", B=32, N=64, P=16, V=VOCAB, dtype="bf16", greedy=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read", "commit", "accept"])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "attend":
        B = _log_int(rng, 1, 40)
        R = rng.choice([1, 1, 1, 9, 25, 65, rng.randint(1, 65)])
        group = rng.choice([1, 2, 4, 5, 8])
        # at most the positions of the listed tree case in multiplications, of the long one in bytes
        most = min(131000, 500_000 // (B * max(1, hkv // 4)), 4_000_000 // (B * R * max(1, group * hkv // 16)))
        hi = _log_int(rng, 1, max(1, most))
        return dict(op=op, B=B, R=R, mask=rng.choice(["tree", "chain"]) if R > 1 else "chain", hq=hkv * group,
                    hkv=hkv, d=d, page=page, cache=cache, dtype=dtype, lo=rng.choice([0, 1, hi // 2, hi]) if hi else 0,
                    hi=hi)
    if op in ("write", "read"):
        B = _log_int(rng, 1, 32)
        R = _log_int(rng, 1, 32000 // B)
        return dict(op=op, B=B, R=R, hkv=hkv, d=d, page=page, cache=cache, dtype=dtype, lo=0,
                    hi=_log_int(rng, 1, 500))
    if op == "commit":
        P = rng.choice([4, 8, 16])
        return dict(op=op, B=_log_int(rng, 1, 32), L=_log_int(rng, 1, 16), N=rng.randint(P, 64), P=P, hkv=hkv, d=d,
                    page=page, cache=cache, lo=0, hi=_log_int(rng, 1, 200))
    V = rng.choice([VOCAB, 32000, _log_int(rng, 50, 200000)])
    P = rng.choice([4, 8, 16])
    N = rng.randint(P, 64)
    elem = 2 if dtype == "bf16" else 4
    most = max(1, 32 * 65 * VOCAB * 2 // ((N + 1) * V * elem))
    return dict(op=op, B=_log_int(rng, 1, min(48, most)), N=N, P=P, V=V, dtype=dtype, greedy=rng.choice([0, 2, 4]))


# ------------------------------------------------------------------------------------------------
# sizes that follow from the case


def _spread(case, lo, hi):
    """One length per request in [lo, hi], the last request at hi, spread evenly but out of order."""
    B = case["B"]
    return [hi if b == B - 1 else lo + int((hi - lo + 1) * ((b * GOLDEN + 0.31) % 1.0)) for b in range(B)]


def _starts(case):
    return _spread(case, case["lo"], case["hi"])


def _counts(case):
    """Rows in use per request: all of them, or for every third request fewer."""
    R = case["R"]
    return [R if b % 3 != 1 else max(1, R - 1 - (b * 7) % max(1, R // 2)) for b in range(case["B"])]


def _taus(case):
    return [1 + (case["P"] - 3 * b) % (case["P"] + 1) for b in range(case["B"])]


def _row_bytes(case):
    """Bytes of one token's keys (or values) of one head in the cache."""
    return case["d"] * 2 if case["cache"] == "bf16" else case["d"] + 1


def work(case):
    op = case["op"]
    elem = 4 if case.get("dtype") == "f32" else 2
    if op == "attend":
        lens = [c + n for c, n in zip(_starts(case), _counts(case))]
        rows = sum(_counts(case))
        return {"bytes": 2 * sum(lens) * case["hkv"] * _row_bytes(case) + 2 * rows * case["hq"] * case["d"] * elem,
                "flops": 4 * sum(length * n for length, n in zip(lens, _counts(case))) * case["hq"] * case["d"]}
    if op in ("write", "read"):
        rows = sum(_counts(case)) * case["hkv"]
        return {"bytes": 2 * rows * (case["d"] * elem + _row_bytes(case)), "flops": 2 * rows * case["d"]}
    if op == "commit":
        moved = sum(t - 1 for t in _taus(case)) * case["L"] * case["hkv"]
        return {"bytes": 4 * moved * _row_bytes(case) + 8 * case["B"] * (case["P"] + 2), "flops": 0}
    rows = sum(_counts(dict(case, R=case["N"] + 1)))
    return {"bytes": rows * case["V"] * elem, "flops": 4 * rows * case["V"]}


# ------------------------------------------------------------------------------------------------
# what a program has in hand


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(case, gen, capacity, L=1):
    """A paged cache that holds capacity[b] positions of every request on pages in random order,
    filled with rows of unit scale."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    need = [-(-c // page) for c in capacity]
    pages, width = sum(need) + 3, max(need) + 1
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    slots = torch.full((case["B"], width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        slots[b, :n] = perm[at:at + n]
        at += n
    shape = (L, pages, hkv, page, d)
    if case["cache"] == "bf16":
        k, v = (torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        ks = vs = None
    else:
        k, v = (torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(100).clamp_(-448, 448)
                .to(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.randint(119, 122, shape[:-1], generator=gen, device=DEV, dtype=torch.uint8) for _ in range(2))
    return dict(k=k, v=v, k_scale=ks, v_scale=vs), slots


def _trees(case, gen, N, P, V=1 << 17):
    """Random draft trees in insertion order, depth at most P, siblings with distinct tokens."""
    B, R = case["B"], N + 1
    pick = torch.rand((B, R), generator=gen, device=DEV).tolist()
    parent, depth, anc = [], [], []
    for b in range(B):
        pa, de, an, open_ = [-1], [0], [0], [0]
        for t in range(1, R):
            # the first P slots are a chain, so that the deepest path exists; then any open slot
            p = t - 1 if t <= P else open_[int(pick[b][t] * len(open_))]
            pa.append(p)
            de.append(de[p] + 1)
            an.append(an[p] | (1 << (t - 1)))
            if de[t] < P:
                open_.append(t)
        parent.append(pa)
        depth.append(de)
        anc.append([a - (1 << 64) if a >= 1 << 63 else a for a in an])
    # odd steps through the vocabulary: siblings (and all slots) differ while R < V
    first = torch.randint(0, V, (B, 1), generator=gen, device=DEV)
    stride = 1 if V < 5 * R else V // R
    token = (first + stride * torch.arange(R, device=DEV)) % V
    n = _i32(_counts(dict(case, R=R)))
    return dict(parent=_i32(parent), depth=_i32(depth), rank=torch.zeros(B, R, dtype=torch.int32, device=DEV),
                token=token.to(torch.int32), score=torch.zeros(B, R, dtype=torch.float64, device=DEV),
                anc=torch.tensor(anc, dtype=torch.int64, device=DEV), n_nodes=n)


def prepare(case, seed):
    gen = _gen(seed)
    op, B = case["op"], case["B"]
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    s = dict(case=case)
    if op == "accept":
        N, P, V = case["N"], case["P"], case["V"]
        s["tree"] = t = _trees(case, gen, N, P, V)
        logits = torch.randn((B, N + 1, V), generator=gen, device=DEV, dtype=torch.float32).mul_(2.0)
        # a drafted token is the target's choice with probability 0.3 to 0.9 of what is left
        level = math.log(V) + 2.0
        share = torch.rand((B, N), generator=gen, device=DEV) * 0.6 + 0.3
        rows = torch.arange(B, device=DEV)[:, None].expand(B, N)
        logits[rows, t["parent"][:, 1:].long(), t["token"][:, 1:].long()] = level + torch.log(share / (1 - share))
        s["logits"] = logits.to(dt)
        s["temperature"] = torch.rand(B, generator=gen, device=DEV) * 0.5 + 0.8
        if case["greedy"]:
            s["temperature"][case["greedy"] - 1::case["greedy"]] = 0.0
        s["uniform"] = torch.rand((B, N + 1), generator=gen, device=DEV, dtype=torch.float64)
        return s
    starts = _starts(case)
    if op == "commit":
        N, P, taus = case["N"], case["P"], _taus(case)
        s["cache"], s["table"] = _cache(case, gen, [c + N + 1 for c in starts], case["L"])
        order = torch.rand((B, N), generator=gen, device=DEV).argsort(-1).tolist()
        path = [[0] + sorted(x + 1 for x in order[b][:t - 1]) + [-1] * (P + 1 - t) for b, t in enumerate(taus)]
        s["ctx"], s["acc_len"], s["acc_node"] = _i32(starts), _i32(taus), _i32(path)
        return s
    R, d = case["R"], case["d"]
    s["cache"], s["table"] = _cache(case, gen, [c + R for c in starts])
    s["start"], s["count"] = _i32(starts), _i32(_counts(case))
    if op == "attend":
        s["length"] = max(starts) + R
        s["q"] = torch.randn((B, R, case["hq"], d), generator=gen, device=DEV).to(dt)
        s["o"] = torch.zeros((B, R, case["hq"], d), dtype=dt, device=DEV)
        if case["mask"] == "tree":
            s["tree"] = _trees(case, gen, R - 1, 16)
    elif op == "write":
        s["rows"] = tuple(torch.randn((B, R, case["hkv"], d), generator=gen, device=DEV).to(dt) for _ in range(2))
    else:
        s["out"] = tuple(torch.zeros((B, R, case["hkv"], d), dtype=dt, device=DEV) for _ in range(2))
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms


def _places(table, pos, page):
    """Page and slot of positions pos [B][T]."""
    return table.gather(1, pos // page).long().clamp_min(0), pos % page


def _power(biased):
    """2^(biased - 127) in fp32, exactly, from int32 in [1, 254]."""
    return (biased << 23).view(torch.float32)


def _values(codes, scale, page, slot):
    """fp32 rows [B][T][H][d] of one layer's cache."""
    x = codes[page, :, slot] if codes.dtype == torch.bfloat16 else \
        codes.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    x = x.float()
    return x if scale is None else x * _power(scale[page, :, slot].int())[..., None]


def _visible(s, T):
    """[B][R][T]: which positions row t attends to."""
    case, B, R = s["case"], s["case"]["B"], s["case"]["R"]
    pos = torch.arange(T, device=DEV)
    slot = pos[None] - s["start"][:, None].long()                       # [B][T]
    if case["mask"] == "chain":
        new = slot[:, None] <= torch.arange(R, device=DEV)[None, :, None]
    else:
        bits = (s["tree"]["anc"][:, :, None] >> (slot[:, None] - 1).clamp(0, 63)) & 1
        new = (slot[:, None] == 0) | (bits == 1)
    return (slot[:, None] < 0) | (new & (slot[:, None] < s["count"][:, None, None]) & (slot[:, None] >= 0))


def _plain_attend(s):
    case, T = s["case"], s["length"]
    B, R, hq, hkv, d = (case[x] for x in ("B", "R", "hq", "hkv", "d"))
    c = s["cache"]
    pos = torch.arange(T, device=DEV)[None].expand(B, T)
    used = pos < (s["start"] + s["count"])[:, None]
    page, slot = _places(s["table"], torch.where(used, pos, 0), case["page"])
    k, v = (_values(c[x][0], None if c[x + "_scale"] is None else c[x + "_scale"][0], page, slot) for x in "kv")
    k = k.permute(0, 2, 3, 1).contiguous()                              # [B][H][d][T]
    v = torch.where(used[:, :, None, None], v, 0.0).permute(0, 2, 1, 3).contiguous()
    q = s["q"].float().view(B, R, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    score = torch.matmul(q, k).view(B, hkv, hq // hkv, R, T) * d ** -0.5
    score = score.masked_fill(~_visible(s, T)[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, -1, T), v).view(B, hkv, hq // hkv, R, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, R, hq, d)
    keep = torch.arange(R, device=DEV)[None] < s["count"][:, None]
    return torch.where(keep[..., None, None], o, 0.0).to(s["q"].dtype)


def _quantised(x):
    """e4m3 codes and biased scale exponents of fp32 rows."""
    amax = x.abs().amax(-1)
    frac, exp = torch.frexp(amax)                                       # amax = frac 2^exp, frac in [1/2, 1)
    e = torch.where(frac <= 0.875, exp - 9, exp - 8).clamp_min(-117)
    e = torch.where(amax > 0, e, -117)
    return (x * _power(127 - e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_write(s):
    case, c = s["case"], s["cache"]
    t = torch.arange(case["R"], device=DEV)[None]
    page, slot = _places(s["table"], s["start"][:, None].long() + t, case["page"])
    used = (t < s["count"][:, None])[..., None]
    for x, rows in zip("kv", s["rows"]):
        if case["cache"] == "bf16":
            at = c[x][0]
            at[page, :, slot] = torch.where(used[..., None], rows.to(torch.bfloat16), at[page, :, slot])
        else:
            codes, scale = _quantised(rows.float())
            at = c[x][0].view(torch.uint8)
            at[page, :, slot] = torch.where(used[..., None], codes.view(torch.uint8), at[page, :, slot])
            at = c[x + "_scale"][0]
            at[page, :, slot] = torch.where(used, scale, at[page, :, slot])
    return c


def _plain_read(s):
    case, c = s["case"], s["cache"]
    t = torch.arange(case["R"], device=DEV)[None]
    page, slot = _places(s["table"], s["start"][:, None].long() + t, case["page"])
    used = (t < s["count"][:, None])[..., None, None]
    return tuple(torch.where(used, _values(c[x][0], None if c[x + "_scale"] is None else c[x + "_scale"][0], page,
                                           slot), 0.0).to(s["out"][0].dtype) for x in "kv")


def _plain_commit(s):
    case, c = s["case"], s["cache"]
    i = torch.arange(case["P"] + 1, device=DEV)[None]
    used = i < s["acc_len"][:, None]
    ctx = s["ctx"][:, None].long()
    to = ctx + i
    # a place past the path keeps its own row
    src = _places(s["table"], torch.where(used, ctx + s["acc_node"], to), case["page"])
    dst = _places(s["table"], to, case["page"])
    for x in "kv":
        at = c[x].view(torch.int16 if case["cache"] == "bf16" else torch.uint8)
        at[:, dst[0], :, dst[1]] = at[:, src[0], :, src[1]]
        if c[x + "_scale"] is not None:
            at = c[x + "_scale"]
            at[:, dst[0], :, dst[1]] = at[:, src[0], :, src[1]]
    return c


def _plain_accept(s):
    case, tree = s["case"], s["tree"]
    B, R, P, V = case["B"], case["N"] + 1, case["P"], case["V"]
    greedy = s["temperature"] == 0.0
    row = torch.arange(R, device=DEV)
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    best = torch.where(x == top, torch.arange(V, device=DEV), V).amin(-1)            # lowest index on a tie
    w = torch.exp((x - top) / torch.where(greedy, 1.0, s["temperature"]).double()[:, None, None])
    del x
    total = w.sum(-1)
    parent, token = tree["parent"].long().clamp_min(0), tree["token"].long()
    is_node = (row >= 1) & (row < tree["n_nodes"][:, None])
    pick = w.view(B, -1).gather(1, parent * V + token) / total.gather(1, parent)      # p(token | parent)
    pick = torch.where(is_node, pick, 0.0)
    sibling = (parent[:, :, None] == parent[:, None]) & (row[:, None] > row[None]) & is_node[:, None]
    before = (sibling * pick[:, None]).sum(-1)
    u = s["uniform"].gather(1, parent)
    chosen = torch.where(greedy[:, None], best.gather(1, parent) == token, (u >= before) & (u < before + pick))
    chosen = chosen & is_node
    onto = ((tree["anc"][:, :, None] >> (row - 1).clamp_min(0)) & 1).bool() & (row >= 1)   # ancestor-or-self slots
    taken = ((chosen[:, None] | ~onto).all(-1) & is_node) | (row == 0)                # on the accepted path
    length = taken.sum(-1)
    depth = tree["depth"].long()
    last = torch.where(taken, depth, -1).argmax(-1, keepdim=True)
    place = torch.where(taken, depth, P + 1)
    node = torch.full((B, P + 2), -1, dtype=torch.int64, device=DEV).scatter_(1, place, row.expand(B, R))[:, :P + 1]
    # the bonus token from what the last node's children leave
    wl = w.gather(1, last[:, :, None].expand(B, 1, V))[:, 0].clone()
    child = is_node & (parent == last)
    mass = torch.where(child, pick, 0.0).sum(-1)
    gone = torch.zeros((B, V + 1), dtype=torch.bool, device=DEV).scatter_(1, torch.where(child, token, V), True)[:, :V]
    wl.masked_fill_(gone, 0.0)
    cdf = wl.cumsum(-1)
    rest = (s["uniform"].gather(1, last)[:, 0] - mass) * total.gather(1, last)[:, 0]
    drawn = torch.searchsorted(cdf, rest[:, None], right=True)[:, 0]
    final = torch.where(wl > 0, torch.arange(V, device=DEV), 0).amax(-1)              # last token with any mass
    bonus = torch.where(greedy, best.gather(1, last)[:, 0], torch.minimum(drawn, final))
    tok = torch.cat([token.gather(1, node[:, 1:].clamp_min(0)), token[:, :1]], 1)
    step = torch.arange(P + 1, device=DEV)
    tok = torch.where(step < length[:, None] - 1, tok, torch.where(step == length[:, None] - 1, bonus[:, None], -1))
    return length.int(), tok.int(), node.int()


# ------------------------------------------------------------------------------------------------
# the package's entry points


def _own(s):
    import gdn_draft_tree_amd as g
    case = s["case"]
    op = case["op"]
    if op == "accept":
        return g.gdntree_accept_sample(g.Tree(**s["tree"]), s["logits"], s["temperature"], s["uniform"], case["P"])
    cache = g.KVCache(**s["cache"])
    if op == "commit":
        g.gdntree_cache_commit(cache, s["table"], s["ctx"], s["acc_len"], s["acc_node"], case["N"])
        return s["cache"]
    if op == "write":
        g.gdntree_cache_write(cache, 0, s["table"], s["start"], *s["rows"], count=s["count"])
        return s["cache"]
    if op == "read":
        return g.gdntree_cache_read(cache, 0, s["table"], s["start"], case["R"], count=s["count"], out=s["out"])
    if case["mask"] == "tree":
        return g.gdntree_attend(s["q"], cache, 0, s["table"], s["start"], tree=g.Tree(**s["tree"]), o=s["o"])
    return g.gdntree_attend(s["q"], cache, 0, s["table"], s["start"], n_rows=s["count"], o=s["o"])


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read, "commit": _plain_commit,
            "accept": _plain_accept}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# 64-bit results, request by request from the definitions


def _two_to(e):
    """2^e in fp64, exactly, from whole numbers held in fp64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rows64(case, cache, x, table_row, first, n):
    """Positions first .. first + n - 1 of one request, fp64 [n][H][d]."""
    at = torch.arange(first, first + n, device=DEV)
    ids, slot = table_row[at // case["page"]].long(), at % case["page"]
    codes = cache[x][0]
    raw = codes.view(torch.int16 if case["cache"] == "bf16" else torch.uint8)[ids, :, slot]
    got = raw.view(codes.dtype).double()
    if cache[x + "_scale"] is not None:
        got = got * _two_to(cache[x + "_scale"][0][ids, :, slot].double() - 127)[..., None]
    return got


def _exact_attend(s):
    case = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = case["hq"] // case["hkv"]
    for b, (ctx, n) in enumerate(zip(_starts(case), _counts(case))):
        k, v = (_rows64(case, s["cache"], x, s["table"][b], 0, ctx + n) for x in "kv")
        see = torch.ones((n, ctx + n), dtype=torch.bool, device=DEV)
        for t in range(n):
            word = (1 << t) - 1 if case["mask"] == "chain" else int(s["tree"]["anc"][b, t]) & ((1 << 64) - 1)
            see[t, ctx:] = torch.tensor([j == 0 or (word >> (j - 1)) & 1 == 1 for j in range(n)], device=DEV) \
                if case["mask"] == "tree" else torch.arange(n, device=DEV) <= t
        for h in range(case["hq"]):
            a = s["q"][b, :n, h].double() @ k[:, h // group].t().contiguous() / math.sqrt(case["d"])
            out[b, :n, h] = torch.softmax(torch.where(see, a, -math.inf), -1) @ v[:, h // group].contiguous()
    return out


def _nearest_e4m3(y):
    """The e4m3 number nearest to y (|y| <= 448), ties to the even one."""
    step = _two_to(torch.frexp(y)[1].double().sub(1).clamp_min(-6.0) - 3.0)
    return torch.round(y / step) * step


def _exact_write(s):
    case, c = s["case"], {x: t for x, t in s["cache"].items()}
    out = {x: (c[x].double() if x in "kv" else (None if c[x] is None else c[x].long())) for x in c}
    for x, rows in zip("kv", s["rows"]):
        for b, (start, n) in enumerate(zip(_starts(case), _counts(case))):
            at = torch.arange(start, start + n, device=DEV)
            ids, slot = s["table"][b][at // case["page"]].long(), at % case["page"]
            r = rows[b, :n].double()
            if case["cache"] == "bf16":
                out[x][0][ids, :, slot] = r.float().to(torch.bfloat16).double()
            else:
                e = torch.ceil(torch.log2(r.abs().amax(-1) / 448.0)).clamp_min(-117.0)
                e = torch.where(r.abs().amax(-1) > 448.0 * _two_to(e), e + 1, e)
                out[x][0][ids, :, slot] = _nearest_e4m3(r / _two_to(e)[..., None])
                out[x + "_scale"][0][ids, :, slot] = (e + 127).long()
    return out


def _exact_read(s):
    case = s["case"]
    out = []
    for x, o in zip("kv", s["out"]):
        full = torch.zeros(o.shape, dtype=torch.float64, device=DEV)
        for b, (start, n) in enumerate(zip(_starts(case), _counts(case))):
            full[b, :n] = _rows64(case, s["cache"], x, s["table"][b], start, n)
        out.append(full)
    return tuple(out)


def _exact_commit(s):
    case, c = s["case"], s["cache"]
    out = {x: None if t is None else (t.double() if x in "kv" else t.long()) for x, t in c.items()}
    path = s["acc_node"].tolist()
    for b, (ctx, tau) in enumerate(zip(_starts(case), _taus(case))):
        ids = s["table"][b].tolist()
        for i in range(tau):
            src, dst = ctx + path[b][i], ctx + i
            for x in out:
                if out[x] is not None:
                    out[x][:, ids[dst // case["page"]], :, dst % case["page"]] = \
                        out[x][:, ids[src // case["page"]], :, src % case["page"]]
    return out


def exact(case, seed):
    if case["op"] == "accept":      # whole numbers only
        return None
    return {"attend": _exact_attend, "write": _exact_write, "read": _exact_read,
            "commit": _exact_commit}[case["op"]](prepare(case, seed))
