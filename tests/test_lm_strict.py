"""CPU: the comparison of the token-model outputs tells infinities from numbers."""
import pytest
import torch

import lm_reference as ref
import lm_strict as strict

INF = torch.inf


def want_of(*values):
    v = torch.tensor(values, dtype=torch.float64)
    return {"out": (v, ref.half_step(v, torch.float32))}


@pytest.mark.parametrize("got", [0.5, INF, 3e38, -3.4028234663852886e38])
def test_a_barred_token_has_to_be_minus_infinity(got):
    with pytest.raises(AssertionError):
        strict.check({"out": torch.tensor([1.0, got])}, want_of(1.0, -INF))


@pytest.mark.parametrize("got,want", [(INF, 1.0), (-INF, 2.0), (INF, -INF), (1.0, INF),
                                      (torch.nan, INF), (INF, torch.nan), (1.5, 1.25)])
def test_what_else_is_off(got, want):
    with pytest.raises(AssertionError):
        strict.check({"out": torch.tensor([got])}, want_of(want))


def test_what_is_not():
    v = [1.0, -INF, INF, torch.nan, 0.0, 1.0 + 2.0 ** -25]
    strict.check({"out": torch.tensor(v)}, want_of(*v))
    top = torch.finfo(torch.float32).max
    # rounding decides between the largest number and infinity
    strict.check({"out": torch.tensor([top, INF])}, want_of(top, top * (1 + 2.0 ** -25)))
