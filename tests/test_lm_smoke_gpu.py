"""GPU: the smoke run calls every token-model operator."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_smoke_runs_the_token_model_operators(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import __graft_entry__ as entry
    from sparse_gradient_backward_amd import lm
    called = set()
    for cls, name in ((lm.BlockNorm, "forward"), (lm.BlockNorm, "backward"),
                      (lm.TopkDistill, "loss_grad"), (lm.LogitsPenalty, "apply")):
        real = getattr(cls, name)

        def seen(self, *a, _real=real, _name=(cls.__name__, name), **kw):
            called.add(_name)
            return _real(self, *a, **kw)
        monkeypatch.setattr(cls, name, seen)
    entry.smoke()
    assert called == {("BlockNorm", "forward"), ("BlockNorm", "backward"),
                      ("TopkDistill", "loss_grad"), ("LogitsPenalty", "apply")}
