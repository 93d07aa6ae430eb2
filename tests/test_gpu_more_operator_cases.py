"""The measured cases of the paged cache (perf/more_operators.py), in small: a pass
gives what the plain form gives, whole, whatever the buffers held before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

CASES = [
    dict(op="attend", dtype="bf16", B=5, T=9, Hq=8, H=2, D=64, page=16, lo=3, hi=90, tree=1),
    dict(op="attend", dtype="f16", B=3, T=1, Hq=4, H=4, D=128, page=32, lo=1, hi=200, tree=0),
    dict(op="attend", dtype="bf16", B=4, T=5, Hq=2, H=1, D=128, page=64, lo=20, hi=300, tree=0),
    dict(op="keep", dtype="f16", L=3, B=5, T=9, H=2, D=64, page=16, lo=3, hi=50, path=1),
    dict(op="keep", dtype="bf16", L=1, B=3, T=130, H=2, D=128, page=32, lo=1, hi=100, path=0),
    dict(op="branch", L=2, B=3, K=4, H=2, D=64, page=16, lo=5, hi=70, room=9, spare=7),
    dict(op="turn", L=2, B=9, H=2, D=64, page=16, lo=5, hi=90, spare=11),
]


def outputs(m, s):
    o = m.run(s)
    return o if isinstance(o, dict) else {"out": o}


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['op']}-{c.get('dtype', '')}-{c.get('T', '')}-{c['page']}")
def test_a_pass_gives_the_plain_forms_outputs(case, monkeypatch):
    from perf import more_operators as m

    plain = {k: v.clone() for k, v in outputs(m, m.prepare(case, 11)).items()}
    monkeypatch.setattr(m, "own", True)
    s = m.prepare(case, 11)
    if case["op"] in ("attend", "keep"):
        for v in outputs(m, s).values():
            v.fill_(77)
        if case["op"] == "keep":
            s["back"].zero_()  # rows behind a sequence's last are left as they are
    got = outputs(m, s)
    assert got.keys() == plain.keys()
    for k, v in got.items():
        if case["op"] == "attend":
            # two weighted sums of values below 8 (the 4-bit ones of normal numbers), rounded once to 16 bits,
            # with weights in 16 bits and in 32
            assert float((v.double() - plain[k].double()).abs().max()) <= 8 * (3 * torch.finfo(v.dtype).eps / 2 + 2.0 ** -11)
        else:
            assert torch.equal(v, plain[k]), k
