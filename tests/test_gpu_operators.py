"""The workloads of perf/operators.py: the library's calls there give the plain forms' outputs, bit for bit."""
import pytest
import torch

from perf import operators

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", operators.listed(), ids=lambda c: c["name"])
def test_listed_case_equals_its_plain_form(case, monkeypatch):
    state = operators.prepare(case, 11)
    want = {k: v.clone() for k, v in operators.run(state).items()}
    monkeypatch.setattr(operators, "own", True)
    got = operators.run(state)
    assert got.keys() == want.keys()
    for name, w in want.items():
        assert got[name].dtype == w.dtype and torch.equal(got[name], w), name
