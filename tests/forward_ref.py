"""The forward-pass operators from their formulas in 64 bits, on the CPU, and
the error their kernels may have.

Attention, per row: scores s_j with error E <= (D + 8) u32 scale max_j sum_d
|q_d k_jd| + 2^-21 (an fp32 sum of D products in any order, the scaling, the
subtraction of the maximum, the exponential), weights rounded to the storage
type with relative error up to u (tensor-core form) before they meet v, sums of
n terms in fp32, one rounding of the result.  With A = sum_j p_j |v_j|:
    |out - exact| <= u |exact| + A (u + 2 E + 2 (n + 64) u32)
u = eps / 2 of the storage type, u32 = 2^-24.  fp32 caches round no weight.
"""
import numpy as np
import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def attend_row(q, k, v, scale, dtype):
    """q [D], k and v [n, D] seen by the row (n may be 0), fp64.
    -> (exact, tolerance)."""
    D = q.shape[0]
    if k.shape[0] == 0:
        return torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
    s = (k @ q) * scale
    w = torch.exp(s - s.max())
    p = w / w.sum()
    out = p @ v
    a = p @ v.abs()
    e = (D + 8) * U32 * scale * float((k.abs() @ q.abs()).max()) + 2.0 ** -21
    u = unit(dtype)
    rounded = 0.0 if dtype == torch.float32 else u
    return out, u * out.abs() + a * (rounded + 2 * e + 2 * (k.shape[0] + 64) * U32)


def round_keys(kv, layer, b, h, row, length, pad, T, staged):
    """(prefix k, prefix v, node k, node v) of one sequence and key head."""
    pre = kv[layer, :, row, h, pad:pad + length - 1].double()
    new = staged[layer, :, b, h].double() if staged is not None else \
        kv[layer, :, row, h, pad + length - 1:pad + length - 1 + T].double()
    return pre[0], pre[1], new[0], new[1]


def attend_round(q, kv, layer, length, pad, mask=None, n=None, idx=None, staged=None, scale=None):
    """-> (exact, tolerance) fp64 [B, T, Hq, D]; rows of nodes past n are NaN."""
    B, T, Hq, D = q.shape
    H = kv.shape[3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        nb = T if n is None else int(n[b])
        row = b if idx is None else int(idx[b])
        for h in range(H):
            pk, pv, nk, nv = round_keys(kv, layer, b, h, row, int(length[b]), int(pad[b]), T, staged)
            for i in range(nb):
                bits = (1 << (i + 1)) - 1 if mask is None else int(np.uint64(np.int64(int(mask[b, i]))))
                see = [a for a in range(nb) if bits >> a & 1]
                k, v = torch.cat([pk, nk[see]]), torch.cat([pv, nv[see]])
                for g in range(G):
                    out[b, i, h * G + g], tol[b, i, h * G + g] = attend_row(q[b, i, h * G + g].double(), k, v, scale,
                                                                           q.dtype)
    return out, tol


def attend_prompt(q, kv, layer, cu, pad, start=None, idx=None, scale=None):
    M, Hq, D = q.shape
    H = kv.shape[3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(len(cu) - 1):
        row = b if idx is None else int(idx[b])
        past, at = 0 if start is None else int(start[b]), int(pad[b])
        for i in range(int(cu[b + 1]) - int(cu[b])):
            for h in range(H):
                k, v = kv[layer, :, row, h, at:at + past + i + 1].double()
                for g in range(G):
                    m = int(cu[b]) + i
                    out[m, h * G + g], tol[m, h * G + g] = attend_row(q[m, h * G + g].double(), k, v, scale, q.dtype)
    return out, tol


def normed(x, w, eps):
    """x [..., D] fp64 after the RMS norm with weight w (or None)."""
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def turned(x, pos, inv_freq, interleaved):
    """x [n, heads, D] fp64 turned by pos [n]; inv_freq [R / 2] fp32."""
    if inv_freq is None:
        return x
    a = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    half = inv_freq.numel()
    out = x.clone()
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    out[..., i] = x[..., i] * cos - x[..., j] * sin
    out[..., j] = x[..., j] * cos + x[..., i] * sin
    return out


def append_tol(x, dtype):
    """Bound for a normed and turned head x [.., D] (exact values): one rounding
    to the storage type of the element, and fp32 steps -- the sum of D squares
    (up to D u32 of it, halved by the root), five roundings and the angle's
    cosine and sine (2^-22) -- relative to the pair, here to the head's
    largest element."""
    D = x.shape[-1]
    return unit(dtype) * x.abs() + (D / 2 + 24) * U32 * x.abs().amax(-1, keepdim=True)


def walk(logits, tokens, parent, n, eos, rem):
    """One tree: logits [T, V] fp64-exact values.  -> (tokens, path, n_accept)."""
    out, path, accept, at = [], [], 0, 0
    if n <= 0 or rem <= 0:
        return out, path, accept
    while True:
        row = logits[at]
        bad = np.flatnonzero(np.isnan(row))
        t = int(bad[0]) if len(bad) else int(np.argmax(row))
        out.append(t)
        path.append(at)
        kids = [c for c in range(1, n) if parent[c] == at and tokens[c] == t]
        accept += bool(kids)
        if not kids or t == eos or len(out) == rem:
            return out, path, accept
        at = kids[0]


def random_trees(rng, B, T, full=False):
    """parents [B, T] and node counts [B]"""
    parent = np.full((B, T), -1, np.int32)
    for b in range(B):
        for i in range(1, T):
            parent[b, i] = rng.integers(max(0, i - 6), i)
    n = np.full(B, T) if full else rng.integers(1, T + 1, B)
    return parent, n.astype(np.int32)


def plan(parent, n):
    """(mask [B, T] int64, depth [B, T])"""
    B, T = parent.shape
    mask, depth = np.zeros((B, T), np.uint64), np.zeros((B, T), np.int32)
    for b in range(B):
        for i in range(int(n[b])):
            mask[b, i] = np.uint64(1) << np.uint64(i)
            if i:
                mask[b, i] |= mask[b, parent[b, i]]
                depth[b, i] = depth[b, parent[b, i]] + 1
    return mask.view(np.int64), depth
