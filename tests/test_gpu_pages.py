"""The book of a page pool (fork, reserve, compact) against lists of pages, and
copies of pages."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Both:
    """The same calls on the device and on lists."""

    def __init__(self, N, MP, P, page):
        self.plain = ref.Book(N, MP, P, page)
        self.t = [x.cuda() for x in self.plain.tensors()]
        self.page = page

    def check(self):
        for got, want, name in zip(self.t, self.plain.tensors(), ("table", "held", "refs")):
            assert torch.equal(got.cpu(), want), name

    def fork(self, src, dst=None, length=None):
        f = sv.spec_page_fork(*self.t, i32(src), self.page, dst=None if dst is None else i32(dst),
                              length=None if length is None else i32(length))
        assert not f.any()
        self.plain.fork(src, dst, length)
        self.check()

    def reserve(self, first, total, idx=None):
        copies, missing, f = sv.spec_page_reserve(*self.t, i32(first), i32(total), self.page,
                                                  idx=None if idx is None else i32(idx))
        want, short = self.plain.reserve(first, total, idx)
        assert not f.any() and int(missing) == short
        assert copies.cpu().tolist() == [list(x) for x in want]
        self.check()
        return copies, missing

    def compact(self):
        moves, n = sv.spec_page_compact(*self.t)
        want = self.plain.compact()
        assert int(n) == len(want) and moves[:len(want)].cpu().tolist() == [list(x) for x in want]
        self.check()
        return moves, n


@pytest.mark.parametrize("N,MP,P,page", [(1, 1, 1, 16), (5, 7, 23, 16), (40, 30, 400, 64), (300, 9, 1500, 32),
                                         (33, 70, 17000, 256), (3, 2100, 40000, 128)])
def test_random_runs_of_calls(N, MP, P, page):
    rng = np.random.default_rng(N + P)
    b = Both(N, MP, P, page)
    most = MP * page
    for step in range(12):
        k = int(rng.integers(1, N + 1))
        idx = rng.permutation(N)[:k].tolist()
        total = rng.integers(0, min(most, 2 * P * page // N + 2) + 1, k)
        first = (rng.random(k) * (total + 2)).astype(int)
        b.reserve(first.tolist(), total.tolist(), idx)
        if step % 3 != 2:
            k = int(rng.integers(1, N + 1))
            dst = rng.permutation(N)[:k]
            src = rng.integers(-1, N, k)
            has = np.array([0 if s < 0 else len(b.plain.rows[s]) for s in src])
            length = (rng.random(k) * (has * page + 1)).astype(int) if step % 2 else None
            b.fork(src.tolist(), dst.tolist(), None if length is None else length.tolist())
        if step % 4 == 3:
            b.compact()


def test_sequences_that_share_a_page_they_write():
    """Of four rows that share their pages three take copies and the last keeps
    them; with a fifth that does not write all four take copies."""
    for extra in (0, 1):
        b = Both(5, 6, 40, 16)
        b.reserve([0], [40], [0])
        b.fork([0] * (3 + extra), [1, 2, 3, 4][:3 + extra])
        copies, _ = b.reserve([40] * 4, [45] * 4)
        assert (copies[:, 0] >= 0).sum() == 3 + extra
        # a second call finds nothing shared
        copies, _ = b.reserve([44] * 4, [50] * 4)
        assert (copies == -1).all()


def test_pages_that_are_full_are_replaced_without_a_copy():
    b = Both(3, 6, 40, 16)
    b.reserve([0], [64], [0])
    b.fork([0, 0], [1, 2])
    copies, _ = b.reserve([32, 33], [64, 60], [1, 2])
    assert copies[0].tolist() == [-1, -1] and copies[1].min() >= 0


def test_too_few_pages():
    b = Both(3, 8, 6, 16)
    b.reserve([0, 0], [48, 32])
    _, missing = b.reserve([16, 0, 0], [16, 64, 64])  # row 0 lets go of two; 3 free for 2 + 4
    assert int(missing) == 3
    b.reserve([16, 32, 0], [16, 32, 48])
    _, missing = b.reserve([0], [16 * 8], [2])
    assert int(missing) == 5


def test_forks_among_one_another():
    b = Both(6, 5, 60, 16)
    b.reserve([0] * 6, [80, 16, 33, 0, 64, 5])
    b.fork([1, 2, 0, 5, 4, -1])
    b.fork([5, 5, 3, 3, 0, 1], [0, 1, 2, 3, 4, 5])
    b.fork([5, 3], [5, 3], [17, 1])  # shortened in place


@pytest.mark.parametrize("P", [1, 16, 17, 16384, 16385, 50000])
def test_compact_of_sparse_and_full_pools(P):
    rng = np.random.default_rng(P)
    for share in (0.0, 0.3, 1.0):
        b = Both(7, P, P, 16)
        live = np.flatnonzero(rng.random(P) < share)
        at = rng.permutation(live)
        cuts = np.sort(rng.integers(0, len(at) + 1, 6))
        b.plain.rows = [x.tolist() for x in np.split(at, cuts)]
        for p in at:
            b.plain.refs[p] = 1
        b.t = [x.cuda() for x in b.plain.tensors()]
        b.compact()
        moves, n = b.compact()
        assert int(n) == 0


@pytest.mark.parametrize("dtype,shape", [(torch.uint8, (2, 2, 9, 3, 544)), (torch.uint8, (1, 2, 40, 1, 16)),
                                         (torch.bfloat16, (3, 2, 11, 2, 16, 64)), (torch.float32, (1, 2, 6, 1, 5000))])
def test_copies(dtype, shape):
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(2)
    pool = torch.randint(0, 200, shape, generator=g).to(dtype)
    P = shape[2]
    perm = rng.permutation(P)
    k = P // 2
    pairs = np.stack([perm[:k], perm[k:2 * k]], 1)
    pairs[k // 2] = -1
    got = pool.cuda()
    err = sv.spec_page_copy(got, i32(pairs))
    want = pool.clone()
    for a, b in pairs:
        if a >= 0:
            want[:, :, b] = pool[:, :, a]
    assert int(err) == 0 and torch.equal(got.cpu(), want)
    # only the first of them, and none
    for n in (1, 0, -3):
        got = pool.cuda()
        sv.spec_page_copy(got, i32(pairs), n_pairs=i32([n]))
        want = pool.clone()
        if n > 0 and pairs[0, 0] >= 0:
            want[:, :, pairs[0, 1]] = pool[:, :, pairs[0, 0]]
        assert torch.equal(got.cpu(), want)
    # a count past the list is the list's; pairs outside the pool are left out
    got = pool.cuda()
    err = sv.spec_page_copy(got, i32([[0, P], [P, 0], [-2, 1], [0, -1], [0, 1], [-1, 3]]), n_pairs=i32([99]))
    want = pool.clone()
    want[:, :, 1] = pool[:, :, 0]
    assert int(err) == 4 and torch.equal(got.cpu(), want)


def test_what_is_flagged_stays_as_it_was():
    b = Both(4, 5, 30, 16)
    b.reserve([0] * 4, [80, 16, 33, 40])
    before = [x.clone() for x in b.t]

    def same(flags, want):
        assert [int(x) for x in flags] == [sv.FLAG_BAD_STATE * w for w in want]
        for x, y in zip(b.t, before):
            assert torch.equal(x, y)

    f = lambda *a, **k: sv.spec_page_fork(*b.t, *a, **k)  # noqa: E731
    same(f(i32([4, -2, 0]), 16, dst=i32([0, 1, 4])), [1, 1, 1])
    same(f(i32([0, 0]), 16, dst=i32([2, 2])), [1, 1])
    same(f(i32([1, 2]), 16, length=i32([17, -1])), [1, 1])
    r = lambda *a, **k: sv.spec_page_reserve(*b.t, *a, **k)  # noqa: E731
    c, m, flags = r(i32([0, -1, 0, 0]), i32([81, 10, -1, 2 ** 31 - 1]), 16)
    same(flags, [1, 1, 1, 1])
    assert int(m) == 0 and (c == -1).all()
    same(r(i32([0, 0, 0]), i32([0, 0, 0]), 16, idx=i32([-1, 4, 9]))[2], [1, 1, 1])
    same(r(i32([0, 0]), i32([0, 0]), 16, idx=i32([3, 3]))[2], [1, 1])
    # entries outside the pool
    b.t[0][0, 1], b.t[0][1, 0] = 30, -5
    before = [x.clone() for x in b.t]
    same(f(i32([0, 1, 3]), 16, dst=i32([2, 3, 0])), [1, 1, 1])
    same(r(i32([0, 0]), i32([32, 3]), 16)[2], [1, 1])
    b.t[1][2] = 6  # held past the row
    before = [x.clone() for x in b.t]
    same(f(i32([2, 3]), 16, dst=i32([3, 2])), [1, 1])
    same(r(i32([0]), i32([3]), 16, idx=i32([2]))[2], [1])


def test_a_captured_round_and_other_streams():
    """Book calls captured once and replayed, and two pools on two streams."""
    b = Both(4, 12, 60, 16)
    b.reserve([0] * 4, [20, 30, 40, 50])
    first, total, src = i32([20, 30, 40, 50]), i32([29, 39, 49, 59]), i32([0, 0, 2, 2])
    pool = torch.randint(0, 255, (2, 2, 60, 1, 544), dtype=torch.uint8).cuda()
    want = pool.clone()

    def step(t, pool, stream=None):
        sv.spec_page_fork(*t, src, 16, length=first, stream=stream)
        copies, missing, _ = sv.spec_page_reserve(*t, first, total, 16, stream=stream)
        sv.spec_page_copy(pool, copies, stream=stream)
        moves, n = sv.spec_page_compact(*t, stream=stream)
        sv.spec_page_copy(pool, moves, n, stream=stream)

    first.copy_(i32([20, 20, 40, 40]))
    start = [x.clone() for x in b.t]
    expect = [x.clone() for x in b.t]
    step(expect, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mine = [x.clone() for x in start]
    got = pool.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pass
    step(mine, got, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(mine, expect)) and torch.equal(got, want)
    held = [x.clone() for x in start]
    got = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held, got)
    for x, y in zip(held, start):
        x.copy_(y)
    got.copy_(pool)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, expect)) and torch.equal(got, want)


@pytest.mark.parametrize("N,MP,P,want", [(3, 40, 9, 25), (40, 300, 33, 300), (2000, 70, 100, 70)])
def test_more_wanted_than_the_pool_has(N, MP, P, want):
    """missing is by how many, also where more are wanted than there are pages; nobody got any."""
    b = Both(N, MP, P, 16)
    b.reserve([0], [5 * 16], [1])
    b.reserve([0] * N, [want * 16] * N)
    b.reserve([3 * 16, 0], [4 * 16, min(P - 4, MP) * 16], [1, 0])  # and what is left can be had


def test_more_wanted_than_31_bits_count():
    """128 sequences want 2^24 pages each, 2^31 in all: sums stop at 2^29, and nothing is handed out."""
    N, MP, P = 128, 1 << 24, 50
    table = torch.full((N, MP), -1, dtype=torch.int32, device="cuda")
    held, refs = i32(np.zeros(N)), i32(np.zeros(P))
    copies, missing, f = sv.spec_page_reserve(table, held, refs, i32(np.zeros(N)), i32(np.full(N, 1 << 28)), 16)
    assert int(missing) == (1 << 29) - P and not f.any() and (copies == -1).all()
    assert (table == -1).all() and not held.any() and not refs.any()


def test_pages_copied_past_32_bits():
    """The ends of slabs of 5 GB."""
    P, page = 150000, 34816
    pool = torch.zeros((2, 1, P, page), dtype=torch.uint8, device="cuda")
    pool[:, :, 3] = torch.arange(page, device="cuda").to(torch.uint8)
    pool[1, 0, 3, 7] = 99
    assert int(sv.spec_page_copy(pool, i32([[3, P - 1], [-1, -1], [P - 2, 0]]))) == 0
    assert torch.equal(pool[:, :, P - 1], pool[:, :, 3]) and int(pool[1, 0, P - 1, 7]) == 99
    assert int(pool[0, 0, 4:P - 1].max()) == 0
