"""The measured operator cases (perf/operators.py), in small: a pass gives
whole outputs, whatever the buffers held before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

CASES = [
    dict(op="attend", dtype="bf16", B=5, T=7, Hq=4, H=2, D=64, S=80, lo=3, hi=50, tree=1),
    dict(op="attend", dtype="f32", B=3, T=4, Hq=2, H=2, D=64, S=80, lo=3, hi=50, tree=0),
    dict(op="prompt", dtype="f16", B=3, Hq=4, H=2, D=64, S=90, lo=5, hi=60, past=20),
    dict(op="append", dtype="bf16", B=5, T=7, Hq=4, H=2, D=64, S=80, lo=3, hi=50, tree=1, norm=1),
    dict(op="append", dtype="bf16", B=4, T=5, Hq=4, H=2, D=64, S=80, lo=3, hi=50, tree=0, norm=0),
    dict(op="append", dtype="f32", B=3, T=0, Hq=4, H=2, D=64, S=80, lo=3, hi=50, tree=0, norm=1),
    dict(op="verify", dtype="f32", B=4, T=9, V=300, alpha=0.8),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['op']}-{c['dtype']}-{c.get('T', '')}-{c.get('tree', '')}")
def test_a_pass_writes_all_of_its_outputs(case, monkeypatch):
    from perf import operators

    monkeypatch.setattr(operators, "own", True)
    s = operators.prepare(case, 11)

    def outputs():
        o = operators.run(s)
        o = o if isinstance(o, dict) else {"out": o}
        return {k: v for k, v in o.items() if k != "k_v"}  # the cache itself is updated, not written whole

    first = {k: v.clone() for k, v in outputs().items()}
    for v in outputs().values():
        v.fill_(77)
    second = outputs()
    assert first.keys() == second.keys()
    for k, v in second.items():
        assert torch.equal(v, first[k]), k
        assert not (v == 77).all(), k
