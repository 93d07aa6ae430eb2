"""The paged 4-bit cache from its definitions, on the CPU: packing in exact
arithmetic (64 bits hold every quotient's comparison exactly enough: values have
11 bits, scales 4), tables of pages as lists, attention by forward_ref.

A bf16 query row is held in fp16 times a power of two that puts its largest
value at 2^8 .. 2^9: elements lose at most 2^-25 of one unit, so 2^-33 of the
row's largest, which adds scale * 2^-33 * max |q| * sum_d |k_d| to a score's
error E of forward_ref.  Weights are fp16 (2^-11) over the prefix and in the
storage type over the nodes (at most its unit).  Codes of 0 are common, so that a
result may consist of one small value alone: below 2^-14 an fp16 result's steps
are 2^-24 whatever its size, so its rounding is off by up to 2^-25, which a unit
relative to the value does not count."""
import numpy as np
import torch

import forward_ref as ref

PAGES = (16, 32, 64, 128, 256)
SCALES = np.array([0.0] + [(b % 8) / 8 * 2.0 ** -14 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 15)
                           for b in range(1, 224)])


def nearest_even(x):
    return np.rint(x)  # ties to even, exact


def pack(x):
    """x [..., D] (16-bit values as a float tensor) -> codes [..., D / 2], scales [..., D / 32] uint8"""
    v = x.double().numpy()
    v = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    odd = ~np.isfinite(v).all(-1)
    v = np.where(odd[..., None], 0.0, v)
    top = np.abs(v).max(-1)
    mid = (SCALES[1:223] + SCALES[2:224]) / 2 * 7  # compared with max |x| itself: exact
    byte = 1 + (top[..., None] > mid).sum(-1)
    at = np.minimum(byte - 1, len(mid) - 1)
    byte = np.where((top == mid[at]) & (byte % 2 == 1), byte + 1, byte)
    code = np.clip(nearest_even(v / SCALES[byte][..., None]), -7, 7) + 8
    code = np.where(odd[..., None], 8, code).astype(np.uint8).reshape(*x.shape)
    byte = np.where(odd, 255, byte).astype(np.uint8)
    return torch.from_numpy(code[..., ::2] | code[..., 1::2] << 4), torch.from_numpy(byte)


def unpack(codes, scales):
    """-> fp64 [..., D]"""
    c, b = codes.numpy(), scales.numpy()
    v = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 2 * c.shape[-1]).astype(np.float64) - 8
    s = np.where(b == 255, np.nan, SCALES[np.minimum(b, 223)])
    return torch.from_numpy(v * np.repeat(s, 32, -1))


def views(pool, page, D):
    """codes [..., page, D / 2] and scales [..., page, D / 32] of pool [..., block], as views"""
    half = page * D // 2
    return pool[..., :half].unflatten(-1, (page, D // 2)), pool[..., half:].unflatten(-1, (page, D // 32))


def empty_pool(L, P, H, page, D, fill=0xFF):
    """bytes of 0xFF: a NaN scale for every group, so that nothing may read what nobody wrote"""
    return torch.full((L, 2, P, H, page * 17 * D // 32), fill, dtype=torch.uint8)


def tables(rng, pages, MP, P):
    """table with pages[r] pages for row r, spread over the pool in no order"""
    table = np.full((len(pages), MP), -1, np.int32)
    free = rng.permutation(P)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = free[at:at + n]
        at += n
    return torch.from_numpy(table)


def put(pool, page, D, table_row, kv, pos=0):
    """writes kv [L, 2, H, n, D] at positions pos .. of a sequence"""
    codes, scales = views(pool, page, D)
    c, s = pack(kv)
    for j in range(kv.shape[3]):
        at, r = int(table_row[(pos + j) // page]), (pos + j) % page
        codes[:, :, at, :, r], scales[:, :, at, :, r] = c[:, :, :, j], s[:, :, :, j]


def get(pool, page, D, table_row, n, pos=0):
    """positions pos .. pos + n - 1 of a sequence -> fp64 [L, 2, H, n, D]"""
    codes, scales = views(pool, page, D)
    i = np.arange(pos, pos + n)
    at = torch.from_numpy(np.asarray(table_row)[i // page].astype(np.int64))
    r = torch.from_numpy(i % page)
    return unpack(codes[:, :, at, :, r], scales[:, :, at, :, r]).permute(1, 2, 3, 0, 4)


def attend(q, pool, layer, table, length, staged, mask=None, n=None, idx=None, scale=None):
    """-> (exact, tolerance) fp64 [B, T, Hq, D]; rows of nodes past n are NaN."""
    B, T, Hq, D = q.shape
    H = staged.shape[3]
    G, page = Hq // H, pool.shape[4] * 32 // (17 * D)
    scale = D ** -0.5 if scale is None else scale
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        nb = T if n is None else int(n[b])
        row = b if idx is None else int(idx[b])
        pre = get(pool[layer:layer + 1], page, D, table[row], int(length[b]) - 1)[0]
        new = staged[layer, :, b].double()
        for h in range(H):
            for i in range(nb):
                bits = (1 << (i + 1)) - 1 if mask is None else int(np.uint64(np.int64(int(mask[b, i]))))
                see = [a for a in range(nb) if bits >> a & 1]
                k, v = (torch.cat([pre[c, h], new[c, h, see]]) for c in (0, 1))
                for g in range(G):
                    x = q[b, i, h * G + g].double()
                    o, t = ref.attend_row(x, k, v, scale, q.dtype)
                    if len(k) and q.dtype == torch.bfloat16:
                        w = torch.softmax((k @ x) * scale, 0)
                        t = t + 2 * scale * 2.0 ** -33 * float(x.abs().max()) * float(k.abs().sum(-1).max()) * (w @ v.abs())
                    if q.dtype == torch.float16:
                        t = t + 2.0 ** -25
                    out[b, i, h * G + g], tol[b, i, h * G + g] = o, t
    return out, tol


class Book:
    """Tables, held and refs as the calls define them, one sequence after another."""

    def __init__(self, N, MP, P, page):
        self.N, self.MP, self.P, self.page = N, MP, P, page
        self.rows = [[] for _ in range(N)]
        self.refs = [0] * P

    def need(self, tokens):
        return -(-tokens // self.page)

    def fork(self, src, dst=None, length=None):
        dst = range(len(src)) if dst is None else dst
        old = [list(r) for r in self.rows]
        for b, d in enumerate(dst):
            for p in old[d]:
                self.refs[p] -= 1
            keep = [] if src[b] < 0 else old[src[b]]
            if length is not None and src[b] >= 0:
                keep = keep[:self.need(length[b])]
            for p in keep:
                self.refs[p] += 1
            self.rows[d] = list(keep)

    def reserve(self, first, total, idx=None):
        """-> (copies, missing)"""
        idx = list(range(len(first))) if idx is None else idx
        want = []  # (sequence, place or None, old page or None)
        for b, r in enumerate(idx):
            n = self.need(total[b])
            for p in self.rows[r][n:]:
                self.refs[p] -= 1
            del self.rows[r][n:]
        left = list(self.refs)  # names of a page that remain while sequences take others
        for b, r in enumerate(idx):
            if first[b] < total[b]:
                for i in range(first[b] // self.page, len(self.rows[r])):
                    p = self.rows[r][i]
                    if left[p] > 1:
                        left[p] -= 1
                        want.append((b, i, p))
            want += [(b, None, None)] * (self.need(total[b]) - len(self.rows[r]))
        copies = [(-1, -1)] * len(idx)
        free = [p for p in range(self.P) if self.refs[p] == 0]
        if len(want) > len(free):
            return copies, len(want) - len(free)
        for (b, i, p), new in zip(want, free):
            r = idx[b]
            self.refs[new] = 1
            if i is None:
                self.rows[r].append(new)
                continue
            self.rows[r][i] = new
            self.refs[p] -= 1
            if i == first[b] // self.page and first[b] % self.page:
                copies[b] = (p, new)
        return copies, 0

    def compact(self):
        """-> moves"""
        n = sum(x > 0 for x in self.refs)
        moves = list(zip([p for p in range(n, self.P) if self.refs[p]], [p for p in range(n) if not self.refs[p]]))
        new = dict(moves)
        self.rows = [[new.get(p, p) for p in r] for r in self.rows]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves

    def tensors(self):
        table = torch.full((self.N, self.MP), -1, dtype=torch.int32)
        for r, row in enumerate(self.rows):
            table[r, :len(row)] = torch.tensor(row, dtype=torch.int32)
        return table, torch.tensor([len(r) for r in self.rows], dtype=torch.int32), torch.tensor(self.refs, dtype=torch.int32)
