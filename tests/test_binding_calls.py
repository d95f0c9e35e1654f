"""The binding's wrappers hand their arguments to the library and return, on the CPU: the
library is a stand-in whose entries note what they are given and return MGEMM_OK."""

import ast
import inspect
import types

import pytest
import torch

from mixture_experts_grouped_gmm_gb300 import binding as B
from mixture_experts_grouped_gmm_gb300 import moe


class Library:
    """Every entry returns 0 and is noted with its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*a):
            assert len(a) == len(B._SIGS[name][1]), name
            self.calls.append((name, a))
            return 0

        return entry


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(B, "lib", lambda: lib)
    monkeypatch.setattr(B, "_cuda", lambda *ts: None)
    monkeypatch.setattr(B, "_stream", lambda t=None: 0)
    monkeypatch.setattr(B, "calls", lambda: types.SimpleNamespace(balance_bwd=lambda *a: None, balance=lambda *a: None))
    monkeypatch.setattr(torch.cuda, "device", lambda d: torch.no_grad())
    return lib


def test_every_check_has_a_code_and_a_name():
    for node in ast.walk(ast.parse(inspect.getsource(B))):
        if isinstance(node, ast.Call) and getattr(node.func, "id", "") == "_check":
            assert len(node.args) == 2 and not node.keywords, f"line {node.lineno}"


def test_balance_gradient(library):
    logits, slopes = torch.zeros(6, 8), torch.zeros(9)
    g = torch.ones((), dtype=torch.float64)
    for l, o, m in ((logits, None, None), (logits.t().contiguous().t(), None, torch.ones(12, dtype=torch.bool)[::2]),
                    (logits, torch.tensor([0, 9, 6, 9])[::2], None)):
        out = moe.balance_loss_backward(g, l, slopes, offsets=o, mask=m)
        name, a = library.calls[-1]
        assert name == "mgemm_balance_bwd" and out.shape == l.shape and a[-3] == out.data_ptr() and a[8:10] == (6, 8)
        assert (a[5] is None) == (o is None) and (a[7] is None) == (m is None)
    assert len(library.calls) == 3
