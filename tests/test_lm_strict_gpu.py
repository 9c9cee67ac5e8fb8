"""GPU: the penalties' tests again with infinities held to their places: a
barred token is -inf and nothing else, an allowed one a number."""
import pytest
import torch

import lm_strict as strict
import test_lm_penalty_gpu as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


@pytest.fixture(autouse=True)
def strictly(monkeypatch):
    monkeypatch.setattr(base.ref, "check", strict.check)


@pytest.mark.parametrize("V", [1, 7, 8, 31, 33, 1000, 1023, 1024, 1025, 4097, 20011])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_vocabularies(lm, V, dt):
    base.test_vocabularies(lm, V, dt)


@pytest.mark.parametrize("rows,V", [(600, 900), (130, 9000), (40, 40000)])
def test_slices(lm, rows, V):
    base.test_slices(lm, rows, V)


@pytest.mark.parametrize("V", [8193, 8199, 16385, 24571])
def test_last_slices(lm, V):
    base.test_last_slices(lm, V)


def test_masks_and_infinite_logits(lm):
    base.test_a_mask_for_every_row(lm)
    base.test_infinite_and_nan_logits(lm)
    base.test_repeated_biases_add_up(lm)
    base.test_bad_contents_are_reported_and_left_out(lm)
