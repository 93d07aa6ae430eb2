"""The forward-pass operators around a speculative round, as measured cases.

Five operators share one KV cache [L, 2, N, H, S, D] and follow each other in
a user's program:

  append   per-head RMS norm of queries and keys, rotary positions, keys and
           values written to their slots (or to the staged block of a tree);
  attend   attention of the round's T drafted nodes (a chain, a tree or one
           token) over the cached prefix and the nodes they descend from;
  prompt   causal attention of packed prompts of different lengths;
  verify   greedy verification of a drafted tree: the path of accepted nodes;
  commit   the accepted path's staged keys and values copied into the cache.

`own` false: each is computed by elementary torch operations in 32 bits, with
one rounding at the end.  `own` true: the library's calls.  exact() is the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the smallest round: a chain of four proposals on a tiny fp32 model
        dict(name="attend_tiny_f32", op="attend", dtype="f32", B=4, T=5, Hq=4, H=4, D=64, S=256, lo=8, hi=64, tree=0),
        # a single token per sequence: plain decoding between rounds
        dict(name="attend_token_f16", op="attend", dtype="f16", B=32, T=1, Hq=32, H=8, D=128, S=2048, lo=128, hi=1536,
             tree=0),
        # wide trees of up to 64 nodes over long contexts, seven query heads to a key head
        dict(name="attend_tree_g7", op="attend", dtype="bf16", B=32, T=64, Hq=28, H=4, D=128, S=4096, lo=500, hi=4000,
             tree=1),
        # the largest batch: eight proposals each, long ragged contexts
        dict(name="attend_chain_b256", op="attend", dtype="bf16", B=256, T=9, Hq=32, H=8, D=128, S=4096, lo=256,
             hi=4000, tree=0),
        # a few short prompts, one query head to a key head
        dict(name="prompt_short", op="prompt", dtype="f16", B=8, Hq=32, H=32, D=64, S=512, lo=17, hi=300, past=0),
        # packed prompts from a paragraph to a long document
        dict(name="prompt_long", op="prompt", dtype="bf16", B=8, Hq=32, H=8, D=128, S=16384, lo=129, hi=14001, past=0),
        # the projections of a tree round
        dict(name="append_tree", op="append", dtype="bf16", B=64, T=26, Hq=28, H=4, D=128, S=2048, lo=128, hi=1024,
             tree=1, norm=1),
        # the projections of a batch of prompts
        dict(name="append_prompt", op="append", dtype="bf16", B=32, T=0, Hq=32, H=8, D=128, S=2048, lo=128, hi=1536,
             tree=0, norm=1),
        # a few small trees of an fp32 model
        dict(name="verify_tree_f32", op="verify", dtype="f32", B=4, T=13, V=32000, alpha=0.8),
        # a batch of trees over a large vocabulary
        dict(name="verify_tree", op="verify", dtype="bf16", B=64, T=26, V=151936, alpha=0.7),
        # the accepted rows of a small draft model's cache
        dict(name="commit_draft", op="commit", dtype="bf16", L=2, B=8, T=26, H=12, D=64, S=1024, lo=64, hi=512,
             alpha=0.7),
        # the accepted rows of every layer of a target's cache
        dict(name="commit_tree", op="commit", dtype="bf16", L=28, B=64, T=26, H=4, D=128, S=256, lo=64, hi=200,
             alpha=0.7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "prompt", "append", "verify", "commit"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    D = rng.choice([64, 128, 128])
    if op == "attend":
        T = rng.choice([1, _log(rng, 2, 16), _log(rng, 10, 64)])
        top = _log(rng, 64, 4000)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 96 if dtype != "f32" else 24), T=T, Hq=G * H, H=H, D=D,
                    S=top + T + rng.randint(0, 64), lo=max(1, top // 4), hi=top, tree=rng.randint(0, 1))
    if op == "prompt":
        top = _log(rng, 16, 2000)
        past = rng.choice([0, 0, rng.randint(1, 500)])
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 12 if dtype != "f32" else 4), Hq=G * H, H=H, D=D,
                    S=top + past + rng.randint(0, 64), lo=max(1, top // 5), hi=top, past=past)
    if op == "append":
        T = rng.choice([0, rng.randint(1, 64)])
        top = _log(rng, 16, 1000)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 32), T=T, Hq=G * H, H=H, D=D, S=top + T + rng.randint(0, 64),
                    lo=max(1, top // 4), hi=top, tree=int(T > 0 and rng.random() < 0.5), norm=rng.randint(0, 1))
    if op == "verify":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 48), T=rng.randint(2, 48), V=_log(rng, 1000, 151936),
                    alpha=round(rng.uniform(0.2, 0.95), 2))
    top = rng.randint(16, 200)
    return dict(op=op, dtype=dtype, L=rng.randint(1, 16), B=_log(rng, 1, 64), T=rng.randint(2, 64), H=H, D=D,
                S=top + 64 + rng.randint(0, 16), lo=max(1, top // 3), hi=top, alpha=round(rng.uniform(0.2, 0.95), 2))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(r, lo, hi, B):
    """B lengths spread over [lo, hi] whose sum is the range's mean times B, so that packed inputs have one shape."""
    n = r.randint(lo, hi + 1, B)
    off = B * (lo + hi) // 2 - int(n.sum())
    for b in r.permutation(B):
        to = min(hi, max(lo, int(n[b]) + off))
        off -= to - int(n[b])
        n[b] = to
    return n.astype(np.int32)


def _host(case, seed):
    """Everything drawn on the host: lengths, paddings, trees."""
    r = np.random.RandomState(seed % (1 << 31))
    B = case["B"]
    h = {}
    if "lo" in case:
        h["length"] = _lengths(r, case["lo"], case["hi"], B)
    T = case.get("T", 0)
    if T:
        i = np.arange(T)
        if case.get("tree", 1):
            lo, hi = np.maximum(i - 1, 0) // 4, np.maximum(i - 1, 0) // 2
            parent = lo + (r.rand(B, T) * (hi - lo + 1)).astype(np.int64)
            n = r.randint((T + 1) // 2, T + 1, B)
        else:
            parent, n = np.broadcast_to(i - 1, (B, T)).copy(), np.full(B, T)
        parent[:, 0] = -1
        seen = np.zeros((B, T), np.uint64)
        depth = np.zeros((B, T), np.int32)
        for k in range(T):
            up = np.maximum(parent[:, k], 0)
            b = np.arange(B)
            seen[:, k] = np.uint64(1) << np.uint64(k)
            if k:
                seen[:, k] |= seen[b, up]
                depth[:, k] = depth[b, up] + 1
        h.update(parent=parent.astype(np.int32), n=n.astype(np.int32), seen=seen.view(np.int64), depth=depth)
    return h, r


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def prepare(case, seed):
    h, r = _host(case, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, B = case["op"], case["B"]
    s = {"case": case, "host": h}
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for k, v in h.items():
        s[k] = put(v)
    if op in ("attend", "prompt", "append", "commit"):
        H, D, S = case["H"], case["D"], case["S"]
        L = case.get("L", 1)
        s["kv"] = _randn(g, (L, 2, B, H, S, D), dt)
        if op in ("prompt", "append") and not case.get("T", 0):
            n = h["length"]
            cu = np.zeros(B + 1, np.int32)
            cu[1:] = np.cumsum(n)
            past = (r.randint(0, case.get("past", 0) + 1, B)).astype(np.int32)
            room = S - n - past
            M = int(cu[-1])
            s.update(cu=put(cu), start=put(past), M=M)
            s["host"].update(cu=cu, start=past)
            s["pad"] = put(np.minimum(room, (past + n).max() - past - n).astype(np.int32))
        else:
            # left padding to a common width, as the realignment leaves it
            s["pad"] = put((h["length"].max() - h["length"]).astype(np.int32))
    if op == "attend":
        s["q"] = _randn(g, (B, case["T"], case["Hq"], case["D"]), dt)
        if case["tree"]:  # a tree's keys and values are staged until its path is known
            s["staged"] = _randn(g, (1, 2, B, case["H"], case["T"], case["D"]), dt)
    elif op == "prompt":
        s["q"] = _randn(g, (s["M"], case["Hq"], case["D"]), dt)
    elif op == "append":
        heads = case["Hq"] + 2 * case["H"]
        T, D = case["T"], case["D"]
        s["qkv"] = _randn(g, (B, T, heads, D) if T else (s["M"], heads, D), dt)
        s["inv_freq"] = (1.0 / (1e6 ** (torch.arange(0, D, 2, device="cuda").double() / D))).float()
        if case["norm"]:
            s["qw"] = 1 + 0.1 * _randn(g, (D,), dt)
            s["kw"] = 1 + 0.1 * _randn(g, (D,), dt)
        if case["tree"]:
            s["staged"] = _randn(g, (1, 2, B, case["H"], T, D), dt)
    elif op == "verify":
        T, V = case["T"], case["V"]
        s["logits"] = _randn(g, (B, T, V), dt)
        # a node's proposal is its parent's choice with the acceptance rate, on one child of each parent
        best = _first_max(s["logits"])
        tok = put(r.randint(0, V, (B, T)).astype(np.int64))
        up = s["parent"].long().clamp(min=0)
        hit = put(r.rand(B, T) < case["alpha"])
        last = torch.zeros((B, T), dtype=torch.long, device="cuda")
        last.scatter_reduce_(1, up, torch.arange(T, device="cuda").expand(B, T).contiguous(), "amax")
        hit &= last.gather(1, up) == torch.arange(T, device="cuda")
        s["tokens"] = torch.where(hit, best.gather(1, up), tok).int()
    elif op == "commit":
        T = case["T"]
        s["staged"] = _randn(g, (case["L"], 2, B, case["H"], T, case["D"]), dt)
        path = np.full((B, T), -1, np.int32)
        emit = np.zeros(B, np.int32)
        for b in range(B):
            at, steps = 0, 0
            while True:
                path[b, steps] = at
                steps += 1
                kids = np.flatnonzero(h["parent"][b, :h["n"][b]] == at)
                if not len(kids) or r.rand() > case["alpha"]:
                    break
                at = int(r.choice(kids))
            emit[b] = steps
        s.update(path=put(path), emit=put(emit))
        s["host"].update(path=path, emit=emit)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _first_max(x):
    """Lowest index of each row's maximum."""
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _softmax_times(score, sees, v):
    """softmax over the seen places times v; a row that sees nothing gives zeros."""
    score = score.masked_fill(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    return (e @ v) / e.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_attend(s, wide):
    c = s["case"]
    B, T, Hq, H, D, S = (c[k] for k in ("B", "T", "Hq", "H", "D", "S"))
    dev = s["q"].device
    G = Hq // H
    width = int(s["host"]["length"].max()) - 1  # slots of cached prefix, the same for every sequence of the batch
    slot = torch.arange(width, device=dev)
    k, v = s["kv"][0, 0, :, :, :width], s["kv"][0, 1, :, :, :width]
    old = (slot >= s["pad"][:, None])[:, None, None, :]  # [B, 1, 1, width]
    at = (s["pad"] + s["length"] - 1).long()[:, None] + torch.arange(T, device=dev)
    if "staged" in s:
        kn, vn = s["staged"][0, 0], s["staged"][0, 1]
    else:
        at = at[:, None, :, None].expand(B, H, T, D)
        kn, vn = s["kv"][0, 0].gather(2, at), s["kv"][0, 1].gather(2, at)
    k = torch.cat([k.to(wide), kn.to(wide)], 2)
    v = torch.cat([v.to(wide), vn.to(wide)], 2)
    node = torch.arange(T, device=dev)
    new = (s["seen"][:, :, None] >> node & 1).bool() & (node < s["n"][:, None])[:, None, :]  # [B, T, T]
    q = s["q"].to(wide).view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    sees = torch.cat([old.expand(B, 1, T, width), new[:, None]], 3)
    sees = sees.repeat_interleave(G, 2)
    out = _softmax_times((q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D)), sees, v)
    out = out.view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    real = (node < s["n"][:, None])[:, :, None, None]
    return torch.where(real, out, 0.0).to(s["q"].dtype if wide != torch.float64 else wide)


def _plain_prompt(s, wide):
    c = s["case"]
    Hq, H, D = c["Hq"], c["H"], c["D"]
    G = Hq // H
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype if wide != torch.float64 else wide, device=s["q"].device)
    cu, start = s["host"]["cu"], s["host"]["start"]
    pad = s["host"]["pad_h"] if "pad_h" in s["host"] else s["host"].setdefault("pad_h", s["pad"].cpu().numpy())
    for b in range(c["B"]):
        lo, hi, past, at = int(cu[b]), int(cu[b + 1]), int(start[b]), int(pad[b])
        k = s["kv"][0, 0, b, :, at:at + past + hi - lo].to(wide)
        v = s["kv"][0, 1, b, :, at:at + past + hi - lo].to(wide)
        step = max(1, (1 << 28) // (Hq * k.shape[1]))
        for i in range(lo, hi, step):
            j = min(hi, i + step)
            end = past + j - lo
            q = s["q"][i:j].to(wide).view(j - i, H, G, D).permute(1, 0, 2, 3).reshape(H, (j - i) * G, D)
            row = torch.arange(past + i - lo, end, device=q.device).repeat_interleave(G)
            sees = torch.arange(end, device=q.device) <= row[:, None]
            o = _softmax_times((q @ k[:, :end].transpose(1, 2)) * (1.0 / math.sqrt(D)), sees, v[:, :end])
            out[i:j] = o.view(H, j - i, G, D).permute(1, 0, 2, 3).reshape(j - i, Hq, D).to(out.dtype)
    return out


def _turn(x, pos, inv_freq):
    """Rotary positions: pair (i, i + D/2) of each head turns by pos * inv_freq[i]; the angle in 64 bits."""
    a = pos.double()[..., None, None] * inv_freq.double()
    cos, sin = torch.cos(a).to(x.dtype), torch.sin(a).to(x.dtype)
    lo, hi = x.chunk(2, -1)
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)


def _plain_append(s, wide, kv, staged):
    c = s["case"]
    B, T, Hq, H = c["B"], c["T"], c["Hq"], c["H"]
    x = s["qkv"].to(wide)
    dev = x.device
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + H, :], s["qkv"][..., Hq + H:, :].to(kv.dtype)
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["qw"].to(wide)
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["kw"].to(wide)
    if T:
        pos = (s["length"] - 1)[:, None] + (s["depth"] if c["tree"] else torch.arange(T, device=dev))
    else:
        m = torch.arange(s["M"], device=dev)
        b = torch.bucketize(m, s["cu"][1:], right=True)
        pos = s["start"][b] + m - s["cu"][b]
    q, k = _turn(q, pos, s["inv_freq"]).to(kv.dtype), _turn(k, pos, s["inv_freq"]).to(kv.dtype)
    if T:
        real = torch.arange(T, device=dev) < s["n"][:, None]
        q = torch.where(real[..., None, None], q, 0.0)
        if c["tree"]:
            keep = real[:, None, :, None]
            staged[0, 0] = torch.where(keep, k.permute(0, 2, 1, 3), staged[0, 0])
            staged[0, 1] = torch.where(keep, v.permute(0, 2, 1, 3), staged[0, 1])
        else:
            rows = torch.arange(B, device=dev)[:, None]
            slot = (s["pad"] + s["length"] - 1)[:, None] + torch.arange(T, device=dev)
            kv[0, 0][rows, :, slot] = k
            kv[0, 1][rows, :, slot] = v
    else:
        kv[0, 0][b, :, s["pad"][b] + pos] = k
        kv[0, 1][b, :, s["pad"][b] + pos] = v
    return {"q": q, "k_v": staged if c["tree"] else kv}


def _walk(best, s):
    """The accepted path: from the root, the lowest child that carries its parent's choice."""
    T = s["case"]["T"]
    B = best.shape[0]
    dev = best.device
    node = torch.arange(T, device=dev)
    real = node < s["n"][:, None]
    at = torch.zeros((B, 1), dtype=torch.long, device=dev)
    live = torch.ones((B, 1), dtype=torch.bool, device=dev)
    tokens, path = [], []
    for _ in range(T):
        choice = best.gather(1, at)
        tokens.append(torch.where(live, choice, -1))
        path.append(torch.where(live, at, -1))
        fits = (s["parent"] == at) & (s["tokens"] == choice) & real
        nxt = torch.where(fits, node, T).amin(1, keepdim=True)
        live = live & (nxt < T)
        at = torch.where(live, nxt, at)
    tokens, path = torch.cat(tokens, 1).int(), torch.cat(path, 1).int()
    emit = (path >= 0).sum(1).int()
    return {"tokens": tokens, "path": path, "n_accept": emit - 1, "n_emit": emit}


def _plain_commit(s, kv):
    c = s["case"]
    B, T = c["B"], c["T"]
    dev = kv.device
    step = torch.arange(T, device=dev)
    take = step < s["emit"][:, None]
    rows = torch.arange(B, device=dev)[:, None].expand(B, T)
    slot = (s["pad"] + s["length"] - 1)[:, None] + step
    frm = torch.where(take, s["path"], 0)
    slot = torch.where(take, slot, slot[:, :1])  # the places behind the path repeat its root
    kv[:, :, rows, :, slot] = s["staged"][:, :, rows, :, frm]
    return kv


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    op = s["case"]["op"]
    if op == "attend":
        return _plain_attend(s, torch.float32)
    if op == "prompt":
        return _plain_prompt(s, torch.float32)
    if op == "append":
        return _plain_append(s, torch.float32, s["kv"], s.get("staged"))
    if op == "verify":
        return _walk(_first_max(s["logits"]), s)
    return _plain_commit(s, s["kv"])


def _own(s):
    import speculative_decoding_verification_28_gb300 as sv

    c = s["case"]
    op = c["op"]
    if op == "attend":
        if "out" not in s:
            s["out"] = torch.empty_like(s["q"])
        if c["tree"]:  # nodes behind a ragged tree's last are not written
            s["out"].zero_()
        tree = dict(tree_mask=s["seen"], n_nodes=s["n"], staged=s["staged"]) if c["tree"] else {}
        return sv.spec_attend_round(s["q"], s["kv"], 0, s["length"], s["pad"], out=s["out"], **tree)[0]
    if op == "prompt":
        return sv.spec_attend_prompt(s["q"], s["kv"], 0, s["cu"], s["pad"], start=s["start"])[0]
    if op == "append":
        norm = dict(q_weight=s["qw"], k_weight=s["kw"], eps=1e-6) if c["norm"] else {}
        if not c["T"]:
            q = sv.spec_append_prompt(s["qkv"], s["kv"], 0, s["cu"], s["pad"], s["inv_freq"], start=s["start"], **norm)[0]
            return {"q": q, "k_v": s["kv"]}
        if "q" not in s:
            s["q"] = torch.empty((c["B"], c["T"], c["Hq"], c["D"]), dtype=s["qkv"].dtype, device=s["qkv"].device)
        if c["tree"]:
            s["q"].zero_()
        tree = dict(depth=s["depth"], n_nodes=s["n"], staged=s["staged"]) if c["tree"] else {}
        q = sv.spec_append_round(s["qkv"], s["kv"], 0, s["length"], s["pad"], s["inv_freq"], q_out=s["q"], **norm,
                                 **tree)[0]
        return {"q": q, "k_v": s["staged"] if c["tree"] else s["kv"]}
    if op == "verify":
        t, path, na, ne, _ = sv.spec_verify_tree(s["logits"], s["tokens"], s["parent"], n_nodes=s["n"])
        return {"tokens": t, "path": path, "n_accept": na, "n_emit": ne}
    sv.spec_commit_tree(s["staged"], s["kv"], s["length"], s["pad"], s["path"], s["emit"])
    return s["kv"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _tree_rows(case):
    """Mean nodes of a tree that are real, and mean length of an accepted path."""
    T, a = case["T"], case.get("alpha", 0.0)
    n = ((T + 1) // 2 + T) / 2 if case.get("tree", 1) else T
    return n, sum(a ** j for j in range(1 + int(math.log2(max(2, T)))))


def work(case):
    op, e, B = case["op"], SIZE[case["dtype"]], case["B"]
    mean = (case["lo"] + case["hi"]) / 2 if "lo" in case else 0
    if op == "attend":
        n, _ = _tree_rows(case)
        Hq, H, D = case["Hq"], case["H"], case["D"]
        seen = mean - 1 + n / 2
        return {"bytes": e * B * D * (2 * H * (mean - 1 + n) + 2 * Hq * n), "flops": 4.0 * B * n * Hq * D * seen}
    if op == "prompt":
        Hq, H, D, past = case["Hq"], case["H"], case["D"], case["past"] / 2
        square = mean * mean + (case["hi"] - case["lo"]) ** 2 / 12
        return {"bytes": e * B * D * (2 * H * (mean + past) + 2 * Hq * mean),
                "flops": 4.0 * B * Hq * D * (square / 2 + mean * past)}
    if op == "append":
        n = B * (_tree_rows(case)[0] if case["T"] else mean)
        heads = case["Hq"] + 2 * case["H"]
        return {"bytes": 2 * e * n * heads * case["D"], "flops": 10.0 * n * heads * case["D"]}
    if op == "verify":
        return {"bytes": e * B * case["V"] * _tree_rows(case)[1], "flops": B * case["V"] * _tree_rows(case)[1]}
    rows = B * _tree_rows(case)[1] * case["L"] * 2 * case["H"]
    return {"bytes": 2 * e * rows * case["D"], "flops": 0.0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None  # whole numbers
    if op == "commit":
        return None  # copies
    h = s["host"]
    B, H, D, Hq = case["B"], case["H"], case["D"], case["Hq"]
    G = Hq // H
    f = torch.float64
    if op == "attend":
        T = case["T"]
        out = torch.zeros(s["q"].shape, dtype=f, device="cuda")
        seen = h["seen"].view(np.uint64)
        for b in range(B):
            n, ln = int(h["n"][b]), int(h["length"][b])
            lo = int(h["length"].max()) - ln
            bits = (seen[b, :n, None] >> np.arange(n, dtype=np.uint64)) & np.uint64(1)
            see = torch.from_numpy(np.concatenate([np.ones((n, ln - 1)), bits.astype(float)], 1) > 0).cuda()
            side = s["staged"][0, :, b, :, :n] if "staged" in s else s["kv"][0, :, b, :, lo + ln - 1:lo + ln - 1 + n]
            kv = torch.cat([s["kv"][0, :, b, :, lo:lo + ln - 1].to(f), side.to(f)], 2)
            k, v = kv[0].repeat_interleave(G, 0), kv[1].repeat_interleave(G, 0)
            w = torch.einsum("thd,hsd->hts", s["q"][b, :n].to(f), k) / math.sqrt(D)
            w = torch.softmax(w.masked_fill(~see, -math.inf), -1)
            out[b, :n] = torch.einsum("hts,hsd->thd", w, v)
        return out
    if op == "prompt":
        out = torch.empty(s["q"].shape, dtype=f, device="cuda")
        pad = s["pad"].cpu().numpy()
        for b in range(B):
            lo, hi, past, at = int(h["cu"][b]), int(h["cu"][b + 1]), int(h["start"][b]), int(pad[b])
            n = hi - lo
            step = max(1, (1 << 27) // (past + n))
            for head in range(Hq):
                k = s["kv"][0, 0, b, head // G, at:at + past + n].to(f)
                v = s["kv"][0, 1, b, head // G, at:at + past + n].to(f)
                for i in range(0, n, step):
                    j = min(n, i + step)
                    w = s["q"][lo + i:lo + j, head].to(f) @ k[:past + j].T / math.sqrt(D)
                    later = torch.ones(w.shape, dtype=torch.bool, device="cuda").triu(past + i + 1)
                    out[lo + i:lo + j, head] = torch.softmax(w.masked_fill_(later, -math.inf), -1) @ v[:past + j]
        return out
    # append: each head vector as complex numbers, turned by exp(i * position * frequency)
    T, qkv = case["T"], s["qkv"].to(f)
    kv, staged = s["kv"].to(f), s["staged"].to(f) if "staged" in s else None
    q = torch.zeros((*qkv.shape[:-2], Hq, D), dtype=f, device="cuda")
    for b in range(B):
        if T:
            n = int(h["n"][b])
            place = int(h["length"].max()) - 1
            pos = torch.from_numpy((h["depth"][b, :n] if case["tree"] else np.arange(n)) + int(h["length"][b]) - 1).cuda()
            x, to = qkv[b, :n], q[b, :n]
        else:
            lo, hi, past = int(h["cu"][b]), int(h["cu"][b + 1]), int(h["start"][b])
            n = hi - lo
            place = int(s["pad"][b]) + past
            pos = torch.arange(past, past + n, device="cuda")
            x, to = qkv[lo:hi], q[lo:hi]
        turn = torch.polar(torch.ones((), dtype=f, device="cuda"), torch.outer(pos.to(f), s["inv_freq"].to(f)))[:, None]
        parts = []
        for part, w in ((x[:, :Hq], "qw"), (x[:, Hq:Hq + H], "kw")):
            if case["norm"]:
                part = part / torch.sqrt((part * part).mean(-1, keepdim=True) + 1e-6) * s[w].to(f)
            z = torch.complex(part[..., :D // 2].contiguous(), part[..., D // 2:].contiguous()) * turn
            parts.append(torch.cat([z.real, z.imag], -1))
        to.copy_(parts[0])
        new = torch.stack([parts[1], x[:, Hq + H:]]).transpose(1, 2)
        if case["tree"]:
            staged[0, :, b, :, :n] = new
        else:
            kv[0, :, b, :, place:place + n] = new
    return {"q": q, "k_v": staged if case["tree"] else kv}
