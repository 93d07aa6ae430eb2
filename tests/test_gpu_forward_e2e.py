"""The forward-pass operators as a caller runs them: prompts into the cache,
then speculative rounds -- trees staged and committed, chains in place, a
ragged pool -- each with the library's verification and realignment.  The
model is a small attention-only transformer with random weights; what the
rounds commit has to be, token for token, what it generates greedily one
token at a time in 64 bits without a cache."""
import numpy as np
import pytest
import torch

import forward_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu

LAYERS, HQ, H, D, V, EPS = 2, 4, 2, 64, 101, 1e-6
DIM = HQ * D
GENERATED = 24


class Model:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
        self.embed = r(V, DIM)
        self.qkv = [r(DIM, (HQ + 2 * H) * D) / DIM ** 0.5 for _ in range(LAYERS)]
        self.out = [r(DIM, DIM) / DIM ** 0.5 for _ in range(LAYERS)]
        self.qw = [(1 + 0.1 * r(D)).float() for _ in range(LAYERS)]
        self.kw = [(1 + 0.1 * r(D)).float() for _ in range(LAYERS)]
        self.inv_freq = (1.0 / 1e4 ** (torch.arange(0, D, 2).double() / D)).float()

    def logits(self, tokens):
        """Last row's logits of a token list, in 64 bits, no cache."""
        x = self.embed[torch.tensor(tokens)]
        n = len(tokens)
        for i in range(LAYERS):
            qkv = (x @ self.qkv[i]).view(n, HQ + 2 * H, D)
            pos = torch.arange(n)
            q = ref.turned(ref.normed(qkv[:, :HQ], self.qw[i], EPS), pos, self.inv_freq, False)
            k = ref.turned(ref.normed(qkv[:, HQ:HQ + H], self.kw[i], EPS), pos, self.inv_freq, False)
            v = qkv[:, HQ + H:]
            k, v = k.repeat_interleave(HQ // H, 1), v.repeat_interleave(HQ // H, 1)
            s = torch.einsum("thd,shd->hts", q, k) * D ** -0.5
            s = s.masked_fill(torch.ones(n, n).triu(1).bool(), float("-inf"))
            o = torch.einsum("hts,shd->thd", torch.softmax(s, -1), v).reshape(n, DIM)
            x = x + o @ self.out[i]
        return x[-1] @ self.embed.T / DIM ** 0.5

    def greedy(self, tokens, steps):
        """(continuation, smallest margin of the choices)"""
        tokens, out, margin = list(tokens), [], 1e9
        for _ in range(steps):
            top = torch.topk(self.logits(tokens), 2)
            margin = min(margin, float(top.values[0] - top.values[1]))
            out.append(int(top.indices[0]))
            tokens.append(out[-1])
        return out, margin

    def to(self, dtype):
        d = lambda t: t.to(device="cuda", dtype=dtype)  # noqa: E731
        self.dev = dict(embed=d(self.embed), qkv=[d(w) for w in self.qkv], out=[d(w) for w in self.out],
                        qw=[d(w) for w in self.qw], kw=[d(w) for w in self.kw], inv=self.inv_freq.cuda())
        return self

    def run(self, tokens, append, attend):
        """tokens [..] on the device through every layer; append(layer, qkv,
        norms) -> q, attend(layer, q) -> out.  -> logits [.., V]"""
        m = self.dev
        x = m["embed"][tokens.long()]
        for i in range(LAYERS):
            qkv = (x @ m["qkv"][i]).view(*tokens.shape, HQ + 2 * H, D)
            q, flags = append(i, qkv, dict(inv_freq=m["inv"], q_weight=m["qw"][i], k_weight=m["kw"][i], eps=EPS))
            assert (flags == 0).all()
            o, flags = attend(i, q)
            assert (flags == 0).all()
            x = x + o.reshape(*tokens.shape, DIM) @ m["out"][i]
        return x @ m["embed"].T / DIM ** 0.5


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def world():
    """Prompts and what follows them; seeds whose choices are no near ties."""
    for seed in range(50):
        m = Model(seed)
        rng = np.random.default_rng(seed)
        prompts = [rng.integers(0, V, n).tolist() for n in (1, 17, 40)]
        both = [m.greedy(p, GENERATED) for p in prompts]
        if min(b[1] for b in both) > 0.02:
            return m, prompts, [b[0] for b in both]
    raise AssertionError("no seed without near ties")


def prefill(m, prompts, kv, pad, idx=None):
    """The prompts' keys and values, and each one's first token."""
    cu = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
    tokens = i32(sum(prompts, []))
    logits = m.run(tokens, lambda i, x, w: sv.spec_append_prompt(x, kv, i, i32(cu), pad, idx=idx, **w),
                   lambda i, q: sv.spec_attend_prompt(q, kv, i, i32(cu), pad, idx=idx))
    return logits[torch.tensor(cu[1:] - 1, device="cuda")].argmax(-1).int()


def propose(rng, truth, parent, n):
    """Tokens of a tree's nodes: the true continuation on some path, else anything."""
    T = len(parent)
    tok, on, depth = rng.integers(0, V, T), [True] + [False] * (T - 1), [0] * T
    for i in range(1, n):
        p = parent[i]
        depth[i] = depth[p] + 1
        if on[p] and depth[i] <= len(truth) and rng.random() < 0.6:
            tok[i], on[i] = truth[depth[i] - 1], True
    return tok


@pytest.mark.parametrize("form", ["tree", "chain", "pool"])
def test_rounds_generate_what_the_model_generates_alone(world, form):
    m, prompts, truth = world
    m.to(torch.float32)
    B, T, S, rng = len(prompts), 7, 96, np.random.default_rng(3)
    N = B + 2 if form == "pool" else B
    rows = [4, 0, 2] if form == "pool" else list(range(B))
    idx = i32(rows) if form == "pool" else None
    kv = torch.full((LAYERS, 2, N, H, S, D), float("nan"), device="cuda")
    lens = np.array([len(p) for p in prompts])
    pad = None if form == "pool" else i32(lens.max() - lens)
    first = prefill(m, prompts, kv, pad, idx)
    done = [[int(t)] for t in first]
    length = i32(lens + 1)
    pool_len = None
    if form == "pool":
        pool_len = i32(np.ones(N, np.int64))
        pool_len[idx.long()] = length
    pos = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    mask = torch.zeros((B, S), dtype=torch.uint8, device="cuda")
    if pad is not None:
        sv.spec_rebuild_pos_mask(pad, pos, mask)
    staged = torch.full((LAYERS, 2, B, H, T, D), float("nan"), device="cuda")
    accepted = 0
    while min(len(x) for x in done) < GENERATED:
        if form == "chain":
            parent, n = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1)), np.full(B, T, np.int32)
        else:
            parent, n = ref.random_trees(rng, B, T)
        left = [GENERATED - len(x) for x in done]
        tokens = np.stack([propose(rng, truth[b][len(done[b]):], parent[b], int(n[b])) for b in range(B)])
        tokens[:, 0] = [x[-1] for x in done]
        tok, par, nn = i32(tokens), i32(parent), i32(n)
        rem = i32([max(0, x) for x in left])
        if form == "chain":
            logits = m.run(tok, lambda i, x, w: sv.spec_append_round(x, kv, i, length, pad, **w),
                           lambda i, q: sv.spec_attend_round(q, kv, i, length, pad))
            out, n_acc, n_emit = sv.spec_verify_greedy(logits.contiguous(), tok[:, 1:].contiguous(), remaining=rem)
        else:
            tree, depth, flags = sv.spec_tree_plan(par, nn)
            assert (flags == 0).all()
            logits = m.run(tok, lambda i, x, w: sv.spec_append_round(x, kv, i, length, pad, depth=depth, n_nodes=nn,
                                                                     idx=idx, staged=staged, **w),
                           lambda i, q: sv.spec_attend_round(q, kv, i, length, pad, tree_mask=tree, n_nodes=nn, idx=idx,
                                                             staged=staged))
            out, path, n_acc, n_emit, flags = sv.spec_verify_tree(logits.contiguous(), tok, par, n_nodes=nn, remaining=rem)
            assert (flags == 0).all()
            flags = sv.spec_commit_tree(staged, kv, length, pad, path, n_emit, idx=idx)
            assert (flags == 0).all()
        for b in range(B):
            done[b] += out[b, :int(n_emit[b])].tolist()
        accepted += int(n_acc.sum())
        if form == "pool":
            assert int(sv.spec_commit_ragged(pool_len, idx, n_emit, S)) == 0
            length = pool_len[idx.long()].contiguous()
        else:
            length, new_pad, _, err = sv.spec_realign_kv(kv, length, pad, n_emit)
            assert int(err) == 0
            sv.spec_rebuild_pos_mask(new_pad, pos, mask, pad_old=pad)
            pad = new_pad
            assert torch.equal(mask.sum(1).cpu(), S - pad.cpu().long())
    for b in range(B):
        assert done[b][:GENERATED] == truth[b], b
    assert accepted > 10  # the rounds did accept proposals


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_tree_round_in_16_bits_gives_the_models_logits(world, dt):
    """One tree round on 16-bit caches: every node's logits near those of its
    path in 64 bits.  The bound is the accumulated rounding of the 16-bit
    projections, attention and residuals: about 3 roundings of unit u in each
    of 2 layers and the output, on vectors whose elements grow to a few units,
    taken 8 times over."""
    m, prompts, truth = world
    m.to(dt)
    B, T, S, rng = len(prompts), 9, 96, np.random.default_rng(4)
    kv = torch.full((LAYERS, 2, B, H, S, D), float("nan"), device="cuda", dtype=dt)
    lens = np.array([len(p) for p in prompts])
    pad, length = i32(lens.max() - lens), i32(lens + 1)
    prefill(m, prompts, kv, pad)
    parent, n = ref.random_trees(rng, B, T, full=True)
    tokens = np.stack([propose(rng, truth[b][1:], parent[b], T) for b in range(B)])
    tokens[:, 0] = [t[0] for t in truth]
    tree, depth, _ = sv.spec_tree_plan(i32(parent))
    staged = torch.full((LAYERS, 2, B, H, T, D), float("nan"), device="cuda", dtype=dt)
    logits = m.run(i32(tokens), lambda i, x, w: sv.spec_append_round(x, kv, i, length, pad, depth=depth, staged=staged, **w),
                   lambda i, q: sv.spec_attend_round(q, kv, i, length, pad, tree_mask=tree, staged=staged))
    bound = 8 * 9 * ref.unit(dt) * 4
    for b in range(B):
        for i in range(T):
            path, a = [], i
            while a >= 0:
                path.append(int(tokens[b, a]))
                a = int(parent[b, a])
            want = m.logits(prompts[b] + path[::-1])
            assert float((logits[b, i].cpu().double() - want).abs().max()) < bound * float(want.abs().max())


def test_a_round_replayed_from_a_graph(world):
    """Appending and attention of a round captured once for every layer and
    replayed on new tokens and lengths."""
    m, prompts, truth = world
    m.to(torch.bfloat16)
    B, T, S = len(prompts), 5, 96
    kv = torch.zeros((LAYERS, 2, B, H, S, D), device="cuda", dtype=torch.bfloat16)
    lens = np.array([len(p) for p in prompts])
    pad, length = i32(lens.max() - lens), i32(lens + 1)
    prefill(m, prompts, kv, pad)
    tok = i32(np.stack([t[:T] for t in truth]))
    fwd = lambda: m.run_quiet(tok, kv, length, pad)  # noqa: E731

    def run_quiet(tokens, kv, length, pad):
        x = m.dev["embed"][tokens.long()]
        for i in range(LAYERS):
            qkv = (x @ m.dev["qkv"][i]).view(*tokens.shape, HQ + 2 * H, D)
            q, _ = sv.spec_append_round(qkv, kv, i, length, pad, m.dev["inv"], q_weight=m.dev["qw"][i],
                                        k_weight=m.dev["kw"][i], eps=EPS)
            o, _ = sv.spec_attend_round(q, kv, i, length, pad)
            x = x + o.reshape(*tokens.shape, DIM) @ m.dev["out"][i]
        return x @ m.dev["embed"].T

    m.run_quiet = run_quiet
    want, keep = fwd().clone(), kv.clone()
    out = torch.zeros_like(want)
    graph = sv.RoundGraph(lambda: out.copy_(fwd()))
    kv.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # other tokens at other lengths: the replay is the eager round
    length.sub_(i32([0, 3, 20]))
    tok.copy_(tok.flip(1))
    kv.copy_(keep)
    want = fwd().clone()
    kv.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
