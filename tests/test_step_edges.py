"""References and refusals of the page, position, sampling and adapter calls, without a GPU."""

import math

import numpy as np
import pytest
import torch

import oracle.step as ref
import weight_streaming_linear_amd as wsl


def test_min_p_above_every_weight():
    """By hand: no weight is 7 or more, and the first entry is kept always."""
    z = np.array([1.0, 3.0, 3.0, 0.0])
    assert (ref.sample_ref(z, min_p=7.0)[1] == [0, 1, 0, 0]).all() and ref.sample_ref(z, 0.99, min_p=7.0)[0] == 1
    assert (ref.sample_ref(z, min_p=1.0)[1] == [0, 0.5, 0.5, 0]).all()
    assert (ref.sample_ref(z, min_p=float("inf"))[1] == [0, 1, 0, 0]).all()


def test_positions_are_in_the_order_of_their_tokens():
    """[n_seq][q_len] tokens take positions of that shape, or all in one row; as many in another order are refused.
    Dimensions of one change no order."""
    size = torch.Size
    for shape, tokens in (((6,), (2, 3)), ((6,), (6,)), ((2, 3), (6,)), ((0,), (0, 3)), ((0, 4), (0,)), ((1, 6), (2, 3)), ((2, 3, 1), (2, 3)),
                          ((), (1,)), ((6, 1), (1, 6)), ((1, 2, 3), (6,)), ((3, 0), (0, 3))):
        wsl._one_each(size(shape), size(tokens), math.prod(tokens))
    for shape, tokens in (((3, 2), (2, 3)), ((3, 1, 2), (2, 3)), ((6, 2), (3, 4)), ((5,), (2, 3)), ((7,), (6,)), ((2, 4), (6,)), ((), (6,)),
                          ((2, 2), (2, 3)), ((2, 3), (1, 5))):
        with pytest.raises(ValueError, match="positions: shape"):
            wsl._one_each(size(shape), size(tokens), math.prod(tokens))
