"""spec_verify_tree of a chain is spec_verify_greedy: tokens, counts, stops."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_28_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("B,k,V", [(40, 1, 11), (64, 5, 7), (9, 31, 4000), (3, 0, 50)])
@pytest.mark.parametrize("stops", ["none", "eos", "budget", "lengths", "all"])
def test_a_chain_is_the_chain_verification(dt, B, k, V, stops):
    rng = np.random.default_rng(B + k)
    x = torch.randn((B, k + 1, V), generator=torch.Generator().manual_seed(V)).mul(2).round().div(2).to(DT[dt]).cuda()
    best = x.float().argmax(-1).to(torch.int32)
    d = torch.where(torch.from_numpy(rng.random((B, k)) < 0.85).cuda(), best[:, :k],
                    torch.from_numpy(rng.integers(0, V, (B, k)).astype(np.int32)).cuda()).contiguous()
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    kw = {}
    if stops in ("eos", "all"):
        kw["eos_id"] = int(best[0, k // 2])
    if stops in ("budget", "all"):
        kw["remaining"] = i32(rng.integers(-1, k + 3, B))
    n = rng.integers(0, k + 1, B) if stops in ("lengths", "all") else None
    want = sv.spec_verify_greedy(x, d, draft_len=None if n is None else i32(n), **kw)
    tokens = torch.cat([torch.full((B, 1), -7, dtype=torch.int32, device="cuda"), d], 1)
    parent = torch.arange(-1, k, dtype=torch.int32, device="cuda").expand(B, k + 1).contiguous()
    out, path, accept, emit, flags = sv.spec_verify_tree(x, tokens, parent, n_nodes=None if n is None else i32(n + 1), **kw)
    assert (flags == 0).all()
    assert torch.equal(out, want[0]) and torch.equal(accept, want[1]) and torch.equal(emit, want[2])
    at = torch.arange(k + 1, dtype=torch.int32, device="cuda")
    assert torch.equal(path, torch.where(at < emit[:, None], at, -1))
