"""Attention passes of the paged cache's measured cases (perf/more_operators.py), in
small, element by element against the formula in 64 bits: a key left out, a node
too many or the wrong tail of a page is more than an element may be off by."""
import pytest
import torch

import paged_ref as ref
from test_gpu_more_operator_cases import CASES

pytestmark = pytest.mark.gpu

ATTEND = [c for c in CASES if c["op"] == "attend"] + [
    dict(op="attend", dtype="bf16", B=4, T=3, Hq=8, H=2, D=128, page=32, lo=3, hi=150, tree=1),  # 12 rows a key head
    dict(op="attend", dtype="f16", B=3, T=30, Hq=14, H=2, D=64, page=16, lo=2, hi=140, tree=1),
    dict(op="attend", dtype="bf16", B=6, T=1, Hq=8, H=1, D=64, page=256, lo=1, hi=500, tree=0),
]


def inputs(s):
    tree = dict(mask=s["seen"].cpu(), n=s["n"].cpu()) if s["case"]["tree"] else {}
    return [s["q"].cpu(), s["pool"].cpu(), 0, s["table"].cpu(), s["length"].cpu(), s["staged"].cpu()], tree


def beyond(got, want, tol):
    """[B] whether some element of a sequence is off by more than it may be"""
    off = (got.cpu().double() - want).abs() > tol
    return (off & ~torch.isnan(want)).flatten(1).any(1)


@pytest.mark.parametrize("own", [False, True], ids=["plain", "own"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c['dtype']}-{c['T']}-{c['Hq']}-{c['page']}")
def test_a_pass_is_the_formula_element_by_element(case, own, monkeypatch):
    from perf import more_operators as m

    monkeypatch.setattr(m, "own", own)
    s = m.prepare(case, 23)
    got = m.run(s)
    args, tree = inputs(s)
    want, tol = ref.attend(*args, **tree)
    assert not beyond(got, want, tol).any()
    assert not got.cpu()[torch.isnan(want)].any()  # nodes behind a tree's last
    # mistakes, planted in the formula's inputs, are seen: a prefix without its last token ...
    less = list(args)
    less[4] = torch.where(args[4] > 1, args[4] - 1, args[4])
    there = args[4] > 1
    assert bool(beyond(got, *ref.attend(*less, **tree))[there].all())
    # ... and nodes that do not see themselves, or see the one before who should not
    T = case["T"]
    seen = tree.get("mask", (2 << torch.arange(T)).sub(1).repeat(case["B"], 1))
    own_bit = 1 << torch.arange(T)
    for mask in (seen & ~own_bit, seen ^ (own_bit >> 1) if T > 1 else seen & ~own_bit):
        assert bool(beyond(got, *ref.attend(*args, mask=mask, n=tree.get("n")))[(tree["n"] > 1) if tree else there].all())
