"""The paged 4-bit cache as a caller runs it, with the operators it stands beside:
prompts in pieces through a 16-bit cache of one layer into pages, sequences forked,
tree rounds (queries and nodes appended, attention, verification, room reserved,
pages copied, the accepted path stored), a sequence freed and the pool compacted.
Attention is held to its formula in 64 bits on what the pages hold, the book to
lists of pages, and what the pages hold to the rows that went in."""
import numpy as np
import pytest
import torch

import forward_ref
import paged_ref as ref
import speculative_decoding_verification_28_gb300 as sv
from test_gpu_forward_e2e import D, EPS, H, HQ, LAYERS, V, Model, i32

pytestmark = pytest.mark.gpu

DIM = HQ * D
PROMPTS = (1, 17, 40)  # tokens
ROWS = [4, 0, 6, 2, 5]  # table rows of the sequences: three prompts, then forks of the second and third
FROM = [1, 2]
N, MP = 7, 8


class Serving:
    def __init__(self, dt, page, T, seed=5):
        self.m = Model(seed).to(dt)
        self.dt, self.page, self.T = dt, page, T
        self.rng = np.random.default_rng(seed)
        self.P = 40 * 16 // page + N
        self.book = ref.Book(N, MP, self.P, page)
        self.t = [x.cuda() for x in self.book.tensors()]
        self.pool = ref.empty_pool(LAYERS, self.P, H, page, D).cuda()
        self.rows = {}  # what table rows were given, [L, 2, H, n, D]

    def forward(self, tokens, append, attend):
        d = self.m.dev
        x = d["embed"][tokens.long()]
        for i in range(LAYERS):
            qkv = (x @ d["qkv"][i]).view(*tokens.shape, HQ + 2 * H, D)
            q = append(i, qkv, dict(inv_freq=d["inv"], q_weight=d["qw"][i], k_weight=d["kw"][i], eps=EPS))
            x = x + attend(i, q).reshape(*tokens.shape, DIM) @ d["out"][i]
        return x @ d["embed"].T / DIM ** 0.5

    def prompts(self):
        rows = ROWS[:len(PROMPTS)]
        row = i32(rows)
        tokens = [self.rng.integers(0, V, n) for n in PROMPTS]
        done = np.zeros(len(PROMPTS), int)
        for r in rows:
            self.rows[r] = torch.zeros((LAYERS, 2, H, 0, D), dtype=self.dt)
        for part in (2, 1):  # the first half of each, and the rest
            n = np.array(PROMPTS) - done if part == 1 else np.array(PROMPTS) // 2
            cu, start, count = i32(np.concatenate([[0], np.cumsum(n)])), i32(done), i32(n)
            self.reserve(done, done + n, rows)
            S = max(PROMPTS) + 3
            one = torch.full((1, 2, len(rows), H, S, D), float("nan"), dtype=self.dt, device="cuda")
            given = []

            def append(i, x, w):
                # what earlier pieces left in the pages, as the values that they stand for
                f = sv.spec_load_pages(self.pool[i:i + 1], one, self.t[0], torch.zeros_like(start), start, row=row)
                assert not f.any()
                for k, r in enumerate(rows):
                    want = ref.get(self.pool.cpu()[i:i + 1], self.page, D, self.t[0].cpu()[r], int(done[k]))
                    assert torch.equal(one[:, :, k, :, :int(done[k])].cpu().double(), want)
                q, f = sv.spec_append_prompt(x, one, 0, cu, None, start=start, **w)
                assert not f.any()
                f = sv.spec_store_pages(one, self.pool, self.t[0], start, count, layer=i, slot=start, row=row)
                assert not f.any()
                given.append(one.cpu())
                return q

            def attend(i, q):
                o, f = sv.spec_attend_prompt(q, one, 0, cu, None, start=start)
                assert not f.any()
                return o

            logits = self.forward(i32(np.concatenate([t[a:a + k] for t, a, k in zip(tokens, done, n)])), append, attend)
            for k, r in enumerate(rows):
                new = torch.cat([g[:, :, k, :, done[k]:done[k] + n[k]] for g in given])
                self.rows[r] = torch.cat([self.rows[r], new], 3)
            done = done + n
        first = logits[(cu[1:] - 1).long()].argmax(-1).int()
        # forks share all pages, the part full ones too
        f = sv.spec_page_fork(*self.t, i32([rows[k] for k in FROM]), self.page, dst=i32(ROWS[len(rows):]))
        assert not f.any()
        self.book.fork([rows[k] for k in FROM], ROWS[len(rows):])
        for k, r in zip(FROM, ROWS[len(rows):]):
            self.rows[r] = self.rows[rows[k]]
        self.check_book()
        self.root = torch.cat([first, first[FROM]])
        self.length = i32([len(tokens[k]) + 1 for k in (0, 1, 2, *FROM)])
        self.idx = i32(ROWS)
        self.staged = torch.full((LAYERS, 2, len(ROWS), H, self.T, D), float("nan"), dtype=self.dt, device="cuda")

    def reserve(self, first, total, rows):
        copies, missing, f = sv.spec_page_reserve(*self.t, i32(first), i32(total), self.page, idx=i32(rows))
        want, short = self.book.reserve(list(first), list(total), list(rows))
        assert not f.any() and int(missing) == short == 0
        assert copies.cpu().tolist() == [list(x) for x in want]
        assert int(sv.spec_page_copy(self.pool, copies)) == 0
        self.check_book()

    def check_book(self):
        for got, want, name in zip(self.t, self.book.tensors(), ("table", "held", "refs")):
            assert torch.equal(got.cpu(), want), name

    def check_rows(self):
        for r, kv in self.rows.items():
            want = ref.unpack(*ref.pack(kv))
            assert torch.equal(ref.get(self.pool.cpu(), self.page, D, self.t[0].cpu()[r], kv.shape[3]), want), r

    def logits(self, tok, par, nn, seen=None):
        """of a round's nodes; seen(layer, q, mask, out): the attention's inputs and outputs"""
        tree, depth, _ = sv.spec_tree_plan(par, nn)
        flags = []

        def append(i, x, w):
            q, f = sv.spec_append_round(x, None, i, self.length, None, depth=depth, n_nodes=nn, idx=self.idx,
                                        staged=self.staged, **w)
            flags.append(f)
            return q

        def attend(i, q):
            out = torch.zeros_like(q)
            o, f = sv.spec_attend_pages(q, self.pool, i, self.t[0], self.length, self.staged, tree_mask=tree, n_nodes=nn,
                                        idx=self.idx, out=out)
            flags.append(f)
            if seen:
                seen(i, q, tree, o)
            return o

        return self.forward(tok, append, attend), flags

    def keep(self, tok, par, nn, logits):
        """The round's end, without a look at the device: what was accepted is in the pages."""
        out, path, n_acc, n_emit, f0 = sv.spec_verify_tree(logits.contiguous(), tok, par, n_nodes=nn)
        before = self.length - 1
        copies, missing, f1 = sv.spec_page_reserve(*self.t, before, before + n_emit, self.page, idx=self.idx)
        err = sv.spec_page_copy(self.pool, copies)
        f2 = sv.spec_store_pages(self.staged, self.pool, self.t[0], before, n_emit, row=self.idx, path=path)
        self.root.copy_(out.gather(1, (n_emit - 1).long()[:, None])[:, 0])
        self.length.add_(n_emit)
        return path, n_emit, (f0, f1, f2, missing, err)


def accepted_somewhere(s, tok, par, nn):
    """tok with the first child of a node the model's own choice there, two levels deep, where there is one"""
    tok, parent, n = tok.clone(), par.cpu().numpy(), nn.cpu().numpy()
    at = np.zeros(len(n), int)
    for _ in range(2):
        best = s.logits(tok, par, nn)[0].argmax(-1).int()
        for b in range(len(n)):
            kids = [c for c in range(at[b] + 1, n[b]) if parent[b, c] == at[b]]
            if kids:
                tok[b, kids[0]] = best[b, at[b]]
                at[b] = kids[0]
    return tok


@pytest.mark.parametrize("dt,page,T", [("bf16", 16, 7), ("f16", 32, 24), ("bf16", 16, 3)])
def test_prompts_rounds_forks_and_compaction(dt, page, T):
    s = Serving({"bf16": torch.bfloat16, "f16": torch.float16}[dt], page, T)
    s.prompts()
    s.check_rows()
    B = len(ROWS)
    for _ in range(4):
        parent, n = forward_ref.random_trees(s.rng, B, T)
        par, nn = i32(parent), i32(n)
        tok = i32(s.rng.integers(0, V, (B, T)))
        tok[:, 0] = s.root
        tok = accepted_somewhere(s, tok, par, nn)

        def seen(i, q, tree, out):
            want, tol = ref.attend(q.cpu(), s.pool.cpu(), i, s.t[0].cpu(), s.length.cpu(), s.staged.cpu(), mask=tree.cpu(),
                                   n=nn.cpu(), idx=s.idx.cpu())
            real = ~torch.isnan(want)
            assert ((out.cpu().double() - want).abs() <= tol)[real].all()

        logits, flags = s.logits(tok, par, nn, seen)
        assert not any(f.any() for f in flags)
        before = s.length.cpu().numpy() - 1
        staged = s.staged.cpu()
        path, n_emit, flags = s.keep(tok, par, nn, logits)
        assert not any(f.any() for f in flags)
        emit = n_emit.cpu().numpy()
        s.book.reserve(list(before), list(before + emit), ROWS)
        s.check_book()
        for b, r in enumerate(ROWS):
            s.rows[r] = torch.cat([s.rows[r], staged[:, :, b][:, :, :, path[b, :emit[b]].cpu().long()]], 3)
        s.check_rows()
    assert (s.length.cpu() - 1).tolist() == [s.rows[r].shape[3] for r in ROWS]

    # the second sequence ends; the pool is made dense, and nobody else sees a difference
    parent, n = forward_ref.random_trees(s.rng, B, T, full=True)
    par, nn, tok = i32(parent), i32(n), i32(s.rng.integers(0, V, (B, T)))
    want = s.logits(tok, par, nn)[0]
    sv.spec_page_fork(*s.t, i32([-1]), page, dst=i32([ROWS[1]]))
    s.book.fork([-1], [ROWS[1]])
    moves, n_moves = sv.spec_page_compact(*s.t)
    assert moves[:int(n_moves)].cpu().tolist() == [list(x) for x in s.book.compact()]
    assert int(sv.spec_page_copy(s.pool, moves, n_moves)) == 0
    s.check_book()
    del s.rows[ROWS[1]]
    s.check_rows()
    live = sum(x > 0 for x in s.book.refs)
    s.pool[:, :, live:] = 0xFF  # free now
    nn[1], s.length[1] = 0, 1
    got = s.logits(tok, par, nn)[0]
    stay = [0, 2, 3, 4]
    assert torch.equal(got[stay], want[stay])


def test_rounds_replayed_from_a_graph():
    """A whole round captured once and replayed on what the replays before it left: the same as eager rounds."""
    T = 6
    s = Serving(torch.bfloat16, 16, T)
    s.prompts()
    B = len(ROWS)
    parent, n = forward_ref.random_trees(s.rng, B, T)
    par, nn, tok = i32(parent), i32(n), i32(s.rng.integers(0, V, (B, T)))
    state = [*s.t, s.pool, s.length, s.root, s.staged]
    keep = [x.clone() for x in state]
    tokens = [i32(s.rng.integers(0, V, (B, T))) for _ in range(3)]

    def one():
        tok[:, 0] = s.root
        s.keep(tok, par, nn, s.logits(tok, par, nn)[0])

    def back():
        for x, y in zip(state, keep):
            x.copy_(y)

    after = []
    for t in tokens:
        tok.copy_(t)
        one()
        after.append([x.clone() for x in state])
    back()
    graph = sv.RoundGraph(one)
    back()
    for t, want in zip(tokens, after):
        tok.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for x, y, name in zip(state, want, ("table", "held", "refs", "pool", "length", "root", "staged")):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), name
    assert int(s.length.sum()) > int(keep[4].sum())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_nodes_are_appended_without_a_cache(dt):
    g = torch.Generator().manual_seed(1)
    B, T, L = 5, 9, 3
    qkv = torch.randn((B, T, HQ + 2 * H, D), generator=g).to(dt).cuda()
    inv = torch.rand(D // 2, generator=g).cuda()
    w = torch.rand(D, generator=g).to(dt).cuda()
    length, idx, nn = i32([1, 5, 70, 9, 33]), i32([9, 3, 4, 0, 7]), i32([9, 1, 0, 7, 9])
    kv = torch.zeros((L, 2, 10, H, 80, D), dtype=dt, device="cuda")
    outs = []
    for cache in (kv, None):
        staged, q = torch.zeros((L, 2, B, H, T, D), dtype=dt, device="cuda"), torch.zeros((B, T, HQ, D), dtype=dt, device="cuda")
        _, flags = sv.spec_append_round(qkv, cache, 1, length, None, inv, q_weight=w, k_weight=w, n_nodes=nn, idx=idx,
                                        staged=staged, q_out=q)
        outs.append((staged, q, flags))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert not kv.any() and not outs[0][2].any() and outs[0][0][1].any()
    # positions and rows that a cache of this size would not have
    staged, q = torch.zeros_like(staged), torch.zeros_like(q)
    _, flags = sv.spec_append_round(qkv, None, 1, i32([1, 5, 70, 9, 0]), None, None, idx=i32([900, -1, 5, 5, 6]),
                                    staged=staged, q_out=q)
    assert (flags != 0).tolist() == [False, True, False, False, True]
    with pytest.raises(ValueError, match="staged"):
        sv.spec_append_round(qkv, None, 1, length, None, inv, staged=staged[:, :1])
