"""The steps of orthogonalise: each one a triple, whatever the count of all coefficients."""
import pytest
import torch

import mhc_hyper_connection_gb300 as mp
from mhc_hyper_connection_gb300 import _update_ops


@pytest.mark.parametrize("steps", [((1, 2), (3, 4, 5, 6)), ((1, 2, 3, 4), (5, 6)), ((), (1, 2, 3, 4, 5, 6)), ((1, 2, 3), (4, 5)), ((1,),),
                                   [[1, 2, 3, 4, 5, 6]], ([1.5, -0.5], [0.0, 1.5, -0.5, 0.0])])
def test_steps_that_are_no_triples(steps):
    with pytest.raises(ValueError, match="triples"):
        mp.orthogonalise(torch.zeros((4, 8)), steps=steps)


def test_steps_in_order():
    assert list(_update_ops._coefficients(((1, 2, 3), (4.5, -5, 6)))) == [1, 2, 3, 4.5, -5, 6]
    assert len(_update_ops._coefficients(mp.NEWTON_SCHULZ)) == 15
