"""What the binding and the examples check on the host before a call of the cache, the attention and the
verification, without a GPU."""

import pytest
import torch

import weight_streaming_linear_amd as wsl

CPU = torch.device("cpu")


@pytest.mark.parametrize("shape", [(2, 3, 7), (1, 3, 7), (4, 1, 7), (2, 2, 1)])
@pytest.mark.parametrize("step", [0, 1])
def test_rows_that_lie_over_each_other_are_no_rows(shape, step):
    """Broadcast rows (a drafter with one distribution for every position), and rows that overlap: a step
    below vocab from row to row must not be handed on, least of all 0, which could stand for no rows."""
    n, rows, vocab = shape
    wide = torch.zeros(n * rows + vocab)
    t = wide.as_strided(shape, (rows * step, step, 1))
    if step >= vocab:
        assert wsl._prob_rows(t, "q", CPU, shape) == vocab
        return
    with pytest.raises(ValueError, match="q: rows"):
        wsl._prob_rows(t, "q", CPU, shape)


def test_rows_of_their_own_keep_their_step():
    wide = torch.zeros(2, 3, 11)
    assert wsl._prob_rows(wide, "p", CPU, (2, 3, 11)) == 11
    assert wsl._prob_rows(wide[..., 2:9], "p", CPU, (2, 3, 7)) == 11
    assert wsl._prob_rows(wide[:, :1, :7], "p", CPU, (2, 1, 7)) == 33
    assert wsl._prob_rows(wide[:1, 1:2, :7], "p", CPU, (1, 1, 7)) == 7
    assert wsl._prob_rows(wide[:0], "p", CPU, (0, 3, 11)) == 11
