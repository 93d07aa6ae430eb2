"""What surrounds an attention call whose waits gave up, on the CPU."""
from speculative_decoding_verification_28_gb300 import _lib
from speculative_decoding_verification_28_gb300 import build as libbuild


def test_starve_next_refusals():
    libbuild.build()
    lib = _lib.load()
    assert lib.spec_attend_starve_next(0) == -1 and lib.spec_attend_starve_next(-5) == -1
