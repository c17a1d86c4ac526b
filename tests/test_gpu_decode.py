"""The operators together, as a decode loop of a hybrid target uses them: a prompt written into the
cache, then steps of build -> verify (Gated-DeltaNet layers) and cache_write + attend (attention
layers) over the tree's rows -> accept_sample -> commit and cache_commit.

The target is a toy: a token's rows are looked up from (token, position) tables, and the logits are
a projection of every layer's outputs plus a bias that the drafter's candidates come from.  Each
step is held to what decoding token by token computes: the Gated-DeltaNet outputs and states by the
fp64 recurrence along the node's path from the state before the step (2e-3 of the state's norm, for
queries of norm at most 1), the attention outputs by fp64 attention over the rows of all emitted tokens
and the node's path (the tolerance of the attention tests), the acceptance by the fp64 rule (exactly),
and the cache at the end by the rows of the emitted tokens (exactly)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import target_oracle as T
from tests.gpu_harness import TOL
from tests.test_gpu_attend import tolerance
from tests.test_gpu_kv_cache import DT, i32, stored, tables

pytestmark = pytest.mark.gpu

B, N, P, K, V = 3, 16, 5, 6, 48
HG, DG = 2, 128                    # Gated-DeltaNet heads
LA, HKV, HQ, D = 2, 2, 8, 64       # attention layers and heads
PAGE, WIDTH, STEPS = 16, 10, 6
PROMPT = [37, 16, 0]


class Toy:
    """Tables on the CPU (bf16), copied to the device; the rows of (tokens, positions)."""

    def __init__(self, seed):
        gen = torch.Generator().manual_seed(seed)
        top = PAGE * WIDTH
        t = {}
        for name, shape in (("gq", (HG, DG)), ("gk", (HG, DG)), ("gv", (HG, DG)), ("ak", (LA, HKV, D)), ("av", (LA, HKV, D)),
                            ("aq", (LA, HQ, D))):
            tok, pos = torch.randn(V, *shape, generator=gen), 0.3 * torch.randn(top, *shape, generator=gen)
            if name in ("gk", "gq"):       # rows of norm at most 1
                tok, pos = 0.7 * tok / tok.norm(dim=-1, keepdim=True), 0.25 * pos / pos.norm(dim=-1, keepdim=True)
            t[name] = (tok.to(torch.bfloat16), pos.to(torch.bfloat16))
        self.alpha = (0.9 + 0.1 * torch.rand(V, HG, generator=gen)).to(torch.bfloat16)
        self.beta = (0.1 + 0.8 * torch.rand(V, HG, generator=gen)).to(torch.bfloat16)
        self.cpu = t
        self.dev = {k: tuple(x.cuda() for x in v) for k, v in t.items()}
        self.dev_alpha, self.dev_beta = self.alpha.cuda(), self.beta.cuda()
        self.proj = (torch.randn(HG * DG + LA * HQ * D, V, generator=gen) * 0.08).cuda()
        self.bias = torch.randn(V, generator=gen) * 2
        self.dev_bias = self.bias.cuda()

    def rows(self, name, tok, pos, dev=True):
        a, b = (self.dev if dev else self.cpu)[name]
        return (a[tok].float() + b[pos].float()).to(torch.bfloat16)

    def lattice(self, gen):
        """Candidates of every position: the likeliest tokens of a disturbed bias, best first."""
        x = torch.log_softmax(self.bias + 0.5 * torch.randn(B, P, V, generator=gen), -1)
        p, t = x.topk(K, -1)
        return p.contiguous().cuda(), t.to(torch.int32).contiguous().cuda()


class Step:
    """The buffers of one decode step and its two halves (the logits come between)."""

    def __init__(self, g, toy, kind):
        R = N + 1
        self.g, self.toy = g, toy
        self.kv = g.KVCache.empty(LA, B * WIDTH, HKV, PAGE, D, DT[kind])
        for x in (self.kv.k, self.kv.v):
            x.view(torch.uint8).fill_(0x7f if kind == "e4m3" else 0xff)     # NaN until written
        if kind == "e4m3":
            self.kv.k_scale.fill_(127), self.kv.v_scale.fill_(127)
        self.table = tables(B, WIDTH, B * WIDTH, torch.Generator().manual_seed(5))
        self.tree = g.Tree.empty(B, N, "cuda")
        self.ctx = i32(PROMPT)
        self.lat = (torch.zeros(B, P, K, device="cuda"), torch.zeros(B, P, K, dtype=torch.int32, device="cuda"))
        self.root = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.state = torch.zeros(1, B, HG, DG, DG, device="cuda")
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.og, self.oa = z(1, B, R, HG, DG), z(LA, B, R, HQ, D)
        self.logits = torch.zeros(B, R, V, device="cuda")
        self.uniform = torch.zeros(B, R, dtype=torch.float64, device="cuda")
        self.temperature = torch.tensor([0.7, 1.0, 0.0], device="cuda")
        self.acc = tuple(torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, P + 1), (B, P + 1)))

    def prompt(self, tok):
        """tok [B][most]: the prompts' rows into every attention layer (request b's first PROMPT[b])."""
        pos = torch.arange(tok.shape[1], device="cuda").expand(B, -1)
        k, v = (self.toy.rows(x, tok, pos) for x in ("ak", "av"))
        for layer in range(LA):
            self.g.gdntree_cache_write(self.kv, layer, self.table, i32([0] * B), k[:, :, layer].contiguous(),
                                       v[:, :, layer].contiguous(), count=i32(PROMPT))

    def first(self):
        g, toy = self.g, self.toy
        g.gdntree_build(*self.lat, self.root, N, out=self.tree)
        used = torch.arange(N + 1, device="cuda")[None] < self.tree.n_nodes[:, None]
        tok = torch.where(used, self.tree.token, 0).long()
        self.tok, pos = tok, torch.where(used, self.ctx[:, None] + self.tree.depth, 0).long()
        rows = {x: toy.rows(x, tok, pos) for x in toy.dev}
        self.gk, self.gv = rows["gk"][None].contiguous(), rows["gv"][None].contiguous()
        self.alpha, self.beta = toy.dev_alpha[tok][None].contiguous(), toy.dev_beta[tok][None].contiguous()
        g.gdntree_verify(self.tree, rows["gq"][None].contiguous(), self.gk, self.gv, self.alpha, self.beta, self.state,
                         o=self.og)
        for layer in range(LA):
            k, v, q = (rows[x][:, :, layer].contiguous() for x in ("ak", "av", "aq"))
            g.gdntree_cache_write(self.kv, layer, self.table, self.ctx, k, v, count=self.tree.n_nodes)
            g.gdntree_attend(q, self.kv, layer, self.table, self.ctx, tree=self.tree, o=self.oa[layer])

    def heads(self):
        x = torch.cat([self.og[0].float().flatten(2), self.oa.float().permute(1, 2, 0, 3, 4).reshape(B, N + 1, -1)], -1)
        self.logits.copy_(x @ self.toy.proj + self.toy.dev_bias)

    def second(self):
        g = self.g
        g.gdntree_accept_sample(self.tree, self.logits, self.temperature, self.uniform, P, acc=self.acc)
        g.gdntree_commit(self.tree, self.acc[0], self.acc[2], self.gk, self.gv, self.alpha, self.beta, self.state, P)
        g.gdntree_cache_commit(self.kv, self.table, self.ctx, self.acc[0], self.acc[2], N)
        self.root.copy_(self.acc[1].gather(1, self.acc[0][:, None].long() - 1)[:, 0])
        self.ctx.add_(self.acc[0])


def captured(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    return graph.replay


def run(kind, graphs):
    import gdn_draft_tree_amd as g
    toy = Toy(11)
    st = Step(g, toy, kind)
    gen, rng = torch.Generator().manual_seed(3), np.random.default_rng(4)
    prompts = torch.randint(0, V, (B, max(PROMPT)), generator=gen)
    st.prompt(prompts.cuda())
    seq = [prompts[b, :PROMPT[b]].tolist() for b in range(B)]        # tokens whose rows are in the cache
    st.root.copy_(i32([7, 8, 9]))
    first, second = st.first, st.second
    if graphs:                                                       # (a capture does not run anything)
        first, second = captured(st.first), captured(st.second)
    taken = 0
    f64 = lambda x: x.double().numpy()  # noqa: E731
    for step in range(STEPS):
        for dst, src in zip(st.lat, toy.lattice(gen)):
            dst.copy_(src)
        uni = rng.random((B, N + 1))
        st.uniform.copy_(torch.from_numpy(uni))
        root, state = st.root.cpu().tolist(), st.state[0].double().cpu().numpy()
        first()
        st.heads()
        second()
        torch.cuda.synchronize()
        tree = {f: getattr(st.tree, f).cpu().numpy() for f in ("parent", "depth", "token", "n_nodes")}
        acc = [x.cpu().numpy() for x in st.acc]
        og, oa, logits = st.og[0].double().cpu().numpy(), st.oa.double().cpu().numpy(), st.logits.double().cpu().numpy()
        for b in range(B):
            n, ctx = int(tree["n_nodes"][b]), len(seq[b])
            par, tok = tree["parent"][b], tree["token"][b]
            assert tok[0] == root[b]
            states = {-1: state[b]}
            for t in range(n):
                path = [t]
                while path[0] != 0:
                    path.insert(0, int(par[path[0]]))
                toks = torch.tensor(seq[b] + [int(tok[i]) for i in path])
                pos = torch.arange(len(toks))
                here = (toks[-1:], pos[-1:])
                gk, gv, gq = (f64(toy.rows(x, *here, dev=False))[0] for x in ("gk", "gv", "gq"))
                up = states[-1] if t == 0 else states[int(par[t])]
                states[t], want = oracle.gdn_step(up, gq, gk, gv, f64(toy.alpha[here[0]])[0], f64(toy.beta[here[0]])[0])
                norm = np.sqrt((states[t] ** 2).sum((-2, -1)))
                assert (np.abs(og[b, t] - want) <= TOL * norm[:, None]).all(), ("gdn", step, b, t)
                for layer in range(LA):
                    k, v = (stored(toy.rows(x, toks, pos, dev=False)[None, :, layer].cuda(), kind) for x in ("ak", "av"))
                    k, v = k[0][0], v[0][0]
                    q = f64(toy.rows("aq", *here, dev=False))[:, layer]
                    o, mean, big = T.attend(q, k, v, np.ones((1, len(toks)), bool), D ** -0.5)
                    assert (np.abs(oa[layer, b, t] - o[0]) <= tolerance(mean, big, D, len(toks), "bf16")[0]).all(), \
                        ("attend", step, b, t, layer)
            temp = float(st.temperature[b].item())
            path, toks = T.accept_sample(par, tok, n, logits[b], temp, uni[b], P)
            assert acc[0][b] == len(path) and acc[2][b, :len(path)].tolist() == path, ("accept", step, b)
            assert acc[1][b, :len(toks)].tolist() == toks, ("accept", step, b)
            taken += len(path) - 1
            seq[b] += [int(tok[i]) for i in path]
            want, got = states[path[-1]], st.state[0, b].double().cpu().numpy()
            assert (np.abs(got - want).max((-2, -1)) <= TOL * np.sqrt((want ** 2).sum((-2, -1)))).all(), ("state", step, b)
        assert st.ctx.cpu().tolist() == [len(s) for s in seq]
    assert taken > 0
    # the cache holds the rows of the emitted tokens, in order
    most = max(len(s) for s in seq)
    for layer in range(LA):
        got = g.gdntree_cache_read(st.kv, layer, st.table, i32([0] * B), most, out_dtype=torch.float32)
        for x, have in zip(("ak", "av"), got):
            for b in range(B):
                t = torch.tensor(seq[b])
                want, _ = stored(toy.rows(x, t, torch.arange(len(t)), dev=False)[None, :, layer].cuda(), kind)
                np.testing.assert_array_equal(have[b, :len(t)].double().cpu().numpy(), want[0])
    return seq


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_decode_loop_equals_decoding_token_by_token(kind):
    eager = run(kind, graphs=False)
    assert run(kind, graphs=True) == eager
