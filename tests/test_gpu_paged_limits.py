"""The paged cache where it runs out: pools with too few pages for a round, calls
without sequences, values at the ends of their ranges."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu
I32 = torch.int32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32).cuda()


class Pool:
    """Rows 0, 1 and 2 of `page`: two forks with a part-full page between them, and one of their own."""

    def __init__(self, page, D, spare, dt=torch.bfloat16):
        self.page, self.D, self.L, self.H = page, D, 2, 2
        self.g = torch.Generator().manual_seed(page + D)
        self.own = 3  # pages of row 2
        self.P = 2 + self.own + spare
        self.book = ref.Book(3, 5, self.P, page)
        self.t = [x.cuda() for x in self.book.tensors()]
        self.pool = torch.zeros((self.L, 2, self.P, self.H, sv.q4_block_bytes(page, D)), dtype=torch.uint8, device="cuda")
        self.first = page + page // 2 + 1  # tokens of rows 0 and 1
        self.last = self.own * page
        rows = i32([0, 2])
        total = i32([self.first, self.last])
        prompt = torch.randn((self.L, 2, 2, self.H, self.last, D), generator=self.g).to(dt).cuda()
        zero = torch.zeros_like(total)
        _, missing, f = sv.spec_page_reserve(*self.t, zero, total, page, idx=rows)
        assert int(missing) == 0 and not f.any()
        assert not sv.spec_store_pages(prompt, self.pool, self.t[0], zero, total, row=rows, missing=missing).any()
        assert not sv.spec_page_fork(*self.t, i32([0]), page, dst=i32([1])).any()
        self.book.reserve([0, 0], [self.first, self.last], [0, 2])
        self.book.fork([0], [1])
        self.length = i32([self.first + 1, self.first + 1, self.last + 1])
        self.T = 3
        self.staged = torch.randn((self.L, 2, 3, self.H, self.T, D), generator=self.g).to(dt).cuda()
        self.path = torch.arange(self.T, dtype=I32, device="cuda").repeat(3, 1)
        self.missing, self.copies = i32([77]), torch.full((3, 2), 7, dtype=I32, device="cuda")
        self.flags = torch.full((3,), 7, dtype=I32, device="cuda")

    def check_book(self):
        for got, want, name in zip(self.t, self.book.tensors(), ("table", "held", "refs")):
            assert torch.equal(got.cpu(), want), name

    def end_of_round(self, n_emit, stream=None):
        """as a program without a look at the device runs it"""
        before = self.length - 1
        sv.spec_page_reserve(*self.t, before, before + n_emit, self.page, copies=self.copies, missing=self.missing)
        sv.spec_page_copy(self.pool, self.copies)
        sv.spec_store_pages(self.staged, self.pool, self.t[0], before, n_emit, path=self.path, flags=self.flags,
                            missing=self.missing)
        self.length += n_emit * (self.missing == 0)

    def row(self, r, n, pos=0):
        return ref.get(self.pool.cpu(), self.page, self.D, self.t[0][r].cpu(), n, pos)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("page,D,spare,short", [(16, 64, 0, 2), (32, 128, 1, 1), (64, 96, 0, 2)])
def test_a_round_with_too_few_pages_stores_nothing(page, D, spare, short, captured):
    """Rows 0 and 1 both write their shared page, row 2 wants one more: 2 pages for them, where there
    are fewer.  Nothing may change but `missing` and the flags; with row 2 freed the same round runs."""
    s = Pool(page, D, spare)
    n_emit = i32([2, 3, 1])
    if captured:
        keep = [x.clone() for x in (*s.t, s.pool, s.length)]
        graph = sv.RoundGraph(lambda: s.end_of_round(n_emit))
        for x, y in zip((*s.t, s.pool, s.length), keep):
            x.copy_(y)
        run = graph.replay
    else:
        run = lambda: s.end_of_round(n_emit)  # noqa: E731
    pool, length = s.pool.clone(), s.length.clone()
    run()
    torch.cuda.synchronize()
    copies, missing = s.book.reserve([s.first, s.first, s.last], [s.first + 2, s.first + 3, s.last + 1])
    assert int(s.missing) == missing == short and (s.copies == -1).all()
    assert (s.flags == sv.FLAG_BAD_STATE).all()
    s.check_book()
    assert int(s.t[2].max()) == 2 and torch.equal(s.pool, pool) and torch.equal(s.length, length)
    # row 2 ends; its part of the round is left out
    sv.spec_page_fork(*s.t, i32([-1]), page, dst=i32([2]))
    s.book.fork([-1], [2])
    n_emit[2] = 0
    s.length[2] = 1
    before = [s.row(r, s.first) for r in (0, 1)]
    run()
    torch.cuda.synchronize()
    copies, missing = s.book.reserve([s.first, s.first, 0], [s.first + 2, s.first + 3, 0])
    assert int(s.missing) == missing == 0 and not s.flags.any()
    assert s.copies.cpu().tolist() == [list(x) for x in copies] and copies[0][0] >= 0
    s.check_book()
    assert s.length.tolist() == [s.first + 3, s.first + 4, 1]
    for r, n in ((0, 2), (1, 3)):
        assert torch.equal(s.row(r, s.first), before[r])
        want = ref.unpack(*ref.pack(s.staged[:, :, r, :, :n].cpu()))
        assert torch.equal(s.row(r, n, s.first), want)


def test_a_store_without_a_reservation_is_as_before():
    s = Pool(16, 64, 3)
    pos, count = i32([5, 1, 0]), i32([0, 0, 2])
    f = sv.spec_store_pages(s.staged, s.pool, s.t[0], pos, count)
    assert not f.any()
    want = ref.unpack(*ref.pack(s.staged[:, :, 2, :, :2].cpu()))
    assert torch.equal(s.row(2, 2), want)
    with pytest.raises(ValueError, match="missing"):
        sv.spec_store_pages(s.staged, s.pool, s.t[0], pos, count, missing=i32([0, 0]))


@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (9, 4)])
@pytest.mark.parametrize("power", [-64, -92, -95, -110, -120])
def test_queries_of_any_size(power, T, G):
    """Rows of queries down to the smallest normal numbers, with a scale to match, in every form: as exact as
    rows of ordinary size.  (All products are normal numbers in fp32: values are 2^-9 .. 2^3 and zeros.)"""
    from test_gpu_attend_q4 import check, make

    c = make(31, "bf16", 4, T, G, 2, 128, 32, [300, 65, 20, 1])
    f = 2.0 ** power
    check(dict(c, q=(c["q"].float() * f).to(torch.bfloat16)), scale=128 ** -0.5 / f)
    # rows of a unit that differ: the smaller ones' weights are nearly even
    g = torch.exp2(-3.0 * (torch.arange(c["q"].shape[2]) % 3))[:, None]
    check(dict(c, q=(c["q"].float() * g * f).to(torch.bfloat16)), scale=128 ** -0.5 / f)


@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (9, 4)])
@pytest.mark.parametrize("scale", [1.0, 1e-4, 1e-30, 1e-37])
def test_queries_of_next_to_nothing(scale, T, G):
    """Subnormal rows and rows of zeros, whose weights are even, in tiles with hidden keys."""
    from test_gpu_attend_q4 import check, make

    c = make(32, "bf16", 4, T, G, 2, 64, 16, [300, 65, 20, 1])
    q = (c["q"].float() * 2.0 ** -130).to(torch.bfloat16)
    q[:, :, ::3] = 0.0
    assert q.any()
    check(dict(c, q=q), scale=scale)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,G", [(1, 4), (3, 4), (9, 4)])
def test_the_largest_scales_and_scores(dt, T, G):
    """Rows of zeros keep even weights under any scale; scores up to 2^23 give finite results, and the
    value of the largest score's key where that leads by 64 and more."""
    from test_gpu_attend_q4 import DT, check, make, run

    c = make(33, dt, 3, T, G, 2, 128, 64, [300, 65, 1])
    check(dict(c, q=torch.zeros_like(c["q"])), scale={"bf16": 2e38, "f16": 1.8e36}[dt])
    eps = torch.finfo(DT[dt]).eps
    for q in (c["q"], c["q"] * 2.0 ** -10, torch.zeros_like(c["q"])):
        if not q.any():
            q[..., 77] = 2.0 ** -24  # scores from a single product
        keys, values = [], []
        for b in range(3):
            pre = ref.get(c["pool"][1:2], 64, 128, c["table"][b], int(c["length"][b]) - 1)[0]
            keys.append([torch.cat([pre[0], c["staged"][1, 0, b, :, :i + 1].double()], 1) for i in range(T)])
            values.append([torch.cat([pre[1], c["staged"][1, 1, b, :, :i + 1].double()], 1) for i in range(T)])
        raw = [[torch.einsum("hgd,hnd->hgn", q[b, i].double().view(2, G, 128), keys[b][i]) for i in range(T)] for b in range(3)]
        top = max(float(x.abs().max()) for r in raw for x in r)
        scale = 2.0 ** 23 / top * (1 - 2.0 ** -10)
        out = run(dict(c, q=q), scale=scale)[0].cpu().double()
        assert torch.isfinite(out).all()
        led = 0
        for b in range(3):
            for i in range(T):
                s, o = raw[b][i] * scale, out[b, i].view(2, G, 128)
                best = s.max(-1, keepdim=True)[0]
                near = s >= best - 64
                # a score's error is 136 * 2^-24 * 2^23 at most, so that what is not within 136 has no weight
                clear = near.sum(-1) == 1
                clear &= (s >= best - 64 - 136).sum(-1) == 1
                want = torch.einsum("hgn,hnd->hgd", near.double(), values[b][i])
                off = ((o - want).abs() - eps * want.abs() - 2.0 ** -25)[clear]
                assert off.numel() == 0 or float(off.max()) <= 0, (b, i, float(off.max()))
                led += int(clear.sum())
        assert led > 0


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,D", [(1, 128), (9, 128), (40, 64), (3, 96)])
def test_the_largest_scores_over_a_16_bit_cache(dt, T, D):
    """The same bound over a contiguous cache."""
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dt]
    g = torch.Generator().manual_seed(34)
    B, H, G, S = 2, 2, 4, 400
    q = torch.randn((B, T, G * H, D), generator=g).to(dtype)
    kv = torch.randn((1, 2, B, H, S, D), generator=g).to(dtype)
    top = torch.einsum("bthgd,bhsd->bthgs", q.double().view(B, T, H, G, D), kv[0, 0].double()).abs().max()
    mask = (2 << torch.arange(T, device="cuda")).sub(1).repeat(B, 1)
    o, flags = sv.spec_attend_round(q.cuda(), kv.cuda(), 0, i32([300, 65]), None, mask, scale=float(2.0 ** 23 / top * 0.999))
    assert not flags.any() and torch.isfinite(o).all()
    assert float(o.abs().max()) <= float(kv.abs().max()) * (1 + torch.finfo(dtype).eps)


def test_a_reservation_for_no_sequences_lacks_nothing():
    """A batch that became empty, with the `missing` word of a call that came short: a store behind it may go on."""
    book = [x.cuda() for x in ref.Book(2, 3, 2, 16).tensors()]
    missing = i32([0])
    sv.spec_page_reserve(*book, i32([0]), i32([48]), 16, missing=missing)
    assert int(missing) == 1
    none = i32([])
    copies, m, flags = sv.spec_page_reserve(*book, none, none, 16, missing=missing)
    assert m is missing and int(missing) == 0 and copies.shape == (0, 2) and flags.shape == (0,)
    assert int(sv.spec_page_reserve(*book, none, none, 16)[1]) == 0
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    missing.fill_(5)
    other.wait_stream(torch.cuda.current_stream())
    sv.spec_page_reserve(*book, none, none, 16, missing=missing, stream=other)
    other.synchronize()
    assert int(missing) == 0
