"""The checks of linattn_precision.py tell right from wrong: on a model of the tensor-core route's arithmetic they pass,
and with a mistake planted in the model they fail."""
import pytest
import torch

from linattn_precision import model, one_product_values, row_excess, state_excess
from linattn_util import inputs

BF16 = torch.bfloat16


@pytest.mark.parametrize("L", [9, 33, 128, 129, 300])
@pytest.mark.parametrize("decay", [1 - 2.0 ** -9, 0.9, 0.7])
def test_state_check_counts_the_terms_of_a_weighted_key(L, decay):
    q, k, _, _ = inputs(2, L, 2, 2, 64, 64, BF16, L)
    v = one_product_values(2, L, 2, 64, L)
    dec = torch.full((2,), decay)
    off = {m: state_excess(model(q, k, v, dec, 1.0, terms=m)[1], k, v, dec) for m in (2, 3, 4)}
    assert off[4] <= 1 < off[3] < off[2], off


@pytest.mark.parametrize("L,lost", [(128, (100, 3)), (300, (100, 3)), (300, (127, 0)), (300, (9, 9))])
@pytest.mark.parametrize("decay", [1.0, 1 - 2.0 ** -12, 1 - 2.0 ** -6])
@pytest.mark.parametrize("carry", [False, True])
def test_row_check_sees_one_lost_token(L, lost, decay, carry):
    q, k, v, S = inputs(3, L, 4, 4, 64, 64, BF16, L + 1, carry=carry)
    S = None if S is None else S / 3
    dec = torch.full((4,), decay)
    assert row_excess(model(q, k, v, dec, 0.125, S)[0], q, k, v, dec, 0.125, None, S) <= 1
    assert row_excess(model(q, k, v, dec, 0.125, S, lost=lost)[0], q, k, v, dec, 0.125, None, S) > 1


@pytest.mark.parametrize("decay", [0.0, 1e-3, 0.5, 0.875, 1.0])
@pytest.mark.parametrize("dk,dv", [(128, 128), (24, 72)])
def test_row_check_passes_the_models_roundings(decay, dk, dv):
    q, k, v, S = inputs(2, 200, 2, 2, dk, dv, BF16, dk, carry=True)
    dec = torch.full((2,), decay)
    assert row_excess(model(q, k, v, dec, 0.125, S)[0], q, k, v, dec, 0.125, None, S) <= 1
