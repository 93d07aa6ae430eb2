"""What surrounds an attention call whose waits gave up, on the CPU."""
from speculative_decoding_verification_28_gb300 import _lib
from speculative_decoding_verification_28_gb300 import build as libbuild


def test_starve_next_refusals():
    libbuild.build()
    lib = _lib.load()
    assert lib.spec_attend_starve_next(0) == -1 and lib.spec_attend_starve_next(-5) == -1


def test_reset_clears_the_head_of_the_current_streams_scratch(monkeypatch):
    import torch

    import speculative_decoding_verification_28_gb300 as sv
    from speculative_decoding_verification_28_gb300 import forward

    mine, other = ("attend", 0, 50), ("attend", 0, 60)
    kept = {k: torch.full((sv.ATTEND_ZERO + 64,), 5, dtype=torch.uint8) for k in (mine, other)}
    monkeypatch.setattr(forward, "_scratch", kept)
    monkeypatch.setattr(forward, "_device_now", lambda: 0)
    monkeypatch.setattr(forward, "_raw_stream", lambda i: {0: 50, 1: 50}[i])
    sv.spec_attend_reset("cuda:1")  # nothing is kept for that device
    assert all((b == 5).all() for b in kept.values())
    sv.spec_attend_reset()
    assert not kept[mine][:sv.ATTEND_ZERO].any() and (kept[mine][sv.ATTEND_ZERO:] == 5).all()
    assert (kept[other] == 5).all() and sv.FLAG_TIMEOUT == 64
