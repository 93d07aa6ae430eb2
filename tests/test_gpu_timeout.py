"""Attention calls whose waits give up: the library's own test entry makes a
call wait for queries that never come.  Every wait is bounded, so the call
ends, reports it, and the device is as usable as before."""
import pytest
import torch

import speculative_decoding_verification_28_gb300 as sv
from speculative_decoding_verification_28_gb300 import _lib

pytestmark = pytest.mark.gpu
TIMEOUT = 64
CLOCKS = 20_000_000  # about 10 ms


def starve():
    assert _lib.load().spec_attend_starve_next(CLOCKS) == 0


def all_timed_out(flags):
    return flags.tolist() == [TIMEOUT] * flags.numel()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def a_round(T, G, D, dtype, lens):
    """One form of the round kernels by rows a key head: 64, 128 or more."""
    g = torch.Generator(device="cuda").manual_seed(T)
    B, H, S = len(lens), 2, max(lens) + T
    kv = torch.randn((1, 2, B, H, S, D), generator=g, device="cuda").to(dtype)
    q = torch.randn((B, T, G * H, D), generator=g, device="cuda").to(dtype)
    ws = torch.zeros(sv.spec_attend_workspace_bytes(T, G * H, H, D), dtype=torch.uint8, device="cuda")
    return lambda: sv.spec_attend_round(q, kv, 0, i32(lens), None, workspace=ws), ws


ROUNDS = [(1, 4, 64), (9, 4, 128), (20, 5, 64), (20, 5, 128), (64, 4, 64), (64, 4, 128)]


@pytest.mark.parametrize("T,G,D", ROUNDS)
def test_a_round_that_gives_up_ends_and_says_so(T, G, D):
    call, ws = a_round(T, G, D, torch.bfloat16, [300, 40, 700])
    want, flags = call()
    assert (flags == 0).all()
    starve()
    _, flags = call()
    torch.cuda.synchronize()
    assert (flags & TIMEOUT).any()
    # cleared, the workspace is as good as new; so are the tensor cores' memory and the SMs
    ws[:sv.ATTEND_ZERO].zero_()
    for _ in range(3):
        out, flags = call()
        assert (flags == 0).all() and torch.equal(out, want)


@pytest.mark.parametrize("lens", [[40, 3, 100], [700, 600]])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_that_give_up_end_and_say_so(lens, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    B, H, G = len(lens), 1, 2
    cu = i32([sum(lens[:b]) for b in range(B + 1)])
    kv = torch.randn((1, 2, B, H, max(lens), D), generator=g, device="cuda").half()
    q = torch.randn((sum(lens), G * H, D), generator=g, device="cuda").half()
    want, flags = sv.spec_attend_prompt(q, kv, 0, cu, None)
    assert (flags == 0).all()
    starve()
    _, flags = sv.spec_attend_prompt(q, kv, 0, cu, None)
    torch.cuda.synchronize()
    assert (flags & TIMEOUT).any()
    for _ in range(3):
        out, flags = sv.spec_attend_prompt(q, kv, 0, cu, None)
        assert (flags == 0).all() and torch.equal(out, want)


def test_calls_off_the_tensor_cores_do_not_wait():
    kv = torch.randn((1, 2, 2, 1, 40, 64), device="cuda")
    q = torch.randn((2, 3, 2, 64), device="cuda")
    want, _ = sv.spec_attend_round(q, kv, 0, i32([30, 5]), None)
    starve()
    out, flags = sv.spec_attend_round(q, kv, 0, i32([30, 5]), None)
    assert (flags == 0).all() and torch.equal(out, want)


@pytest.mark.parametrize("T,G,D", ROUNDS)
def test_a_round_that_gives_up_flags_every_sequence(T, G, D):
    """More units than CTAs: each CTA stands on the first of its run when it gives up."""
    lens = [130 + 17 * (b % 23) for b in range(200)]
    call, ws = a_round(T, G, D, torch.float16, lens)
    want, flags = call()
    assert (flags == 0).all()
    starve()
    _, flags = call()
    assert all_timed_out(flags)
    # and so does every later call on the workspace, until it is cleared
    _, flags = call()
    assert all_timed_out(flags)
    ws[:sv.ATTEND_ZERO].zero_()
    out, flags = call()
    assert (flags == 0).all() and torch.equal(out, want)


def test_prompts_that_give_up_flag_every_sequence():
    lens = [40, 0, 100, 7]
    cu = i32([sum(lens[:b]) for b in range(5)])
    kv = torch.randn((1, 2, 4, 2, 128, 64), device="cuda").bfloat16()
    q = torch.randn((147, 4, 64), device="cuda").bfloat16()
    starve()
    _, flags = sv.spec_attend_prompt(q, kv, 0, cu, None)
    assert all_timed_out(flags)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,G", [(1, 1), (9, 4), (20, 5), (64, 4)])
def test_rounds_on_a_workspace_of_a_call_that_gave_up(dt, T, G):
    """Whatever kernel comes next: its counters may be off, and it says so."""
    call, ws = a_round(T, G, 64, dt, [300, 40, 700])
    want, _ = call()
    ws[:sv.ATTEND_ZERO].view(torch.int32)[-1] = 1
    for _ in range(2):
        _, flags = call()
        assert all_timed_out(flags)
    assert not ws[:sv.ATTEND_ZERO - 4].any()
    ws[:sv.ATTEND_ZERO].zero_()
    out, flags = call()
    assert (flags == 0).all() and torch.equal(out, want)


@pytest.mark.parametrize("own_stream", [False, True])
def test_reset_of_the_scratch_kept_for_a_stream(own_stream):
    """Calls without a workspace of their own, after one that gave up."""
    kv = torch.randn((1, 2, 3, 2, 900, 128), device="cuda").bfloat16()
    q = torch.randn((3, 5, 8, 128), device="cuda").bfloat16()
    length = i32([800, 30, 500])
    kw = {"stream": torch.cuda.Stream()} if own_stream else {}
    torch.cuda.synchronize()

    def call():
        out, flags = sv.spec_attend_round(q, kv, 0, length, None, **kw)
        torch.cuda.synchronize()
        return out, flags

    want, flags = call()
    assert (flags == 0).all()
    starve()
    assert all_timed_out(call()[1]) and all_timed_out(call()[1])
    # a captured call has scratch of its own
    graph, o = torch.cuda.CUDAGraph(), torch.empty_like(q)
    f = torch.empty_like(length)
    with torch.cuda.graph(graph):
        sv.spec_attend_round(q, kv, 0, length, None, out=o, flags=f)
    graph.replay()
    torch.cuda.synchronize()
    assert (f == 0).all() and torch.equal(o, want)
    sv.spec_attend_reset(**kw)
    out, flags = call()
    assert (flags == 0).all() and torch.equal(out, want)
