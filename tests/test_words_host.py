"""AdamW's random words: a change of any one bit of a value's number, of the step or of the
seed changes each bit of the word half of the time."""
import pytest
import torch

from tests import _block_reference as R

N = 1 << 16


def _bits(w):
    return (w[:, None] >> torch.arange(32)) & 1


@pytest.mark.parametrize("bit", range(40))
def test_a_bit_of_the_number_changes_half_of_the_word(bit):
    """Within five standard deviations for each of the word's bits; a number's bits from 32 on change the key.  Among N
    numbers the pairs that differ in a bit below N are N / 2, each counted twice."""
    base, step = R.words(0, N, 3, 11, "cpu"), 1 << bit
    if step < N:
        other = base[torch.arange(N) ^ step]
    else:
        other = R.words(step, N, 3, 11, "cpu")
    share = _bits(base ^ other).double().mean(0)
    assert float((share - 0.5).abs().max()) <= 5 * 0.5 / (N / 2 if step < N else N) ** 0.5


@pytest.mark.parametrize("bit", range(0, 31, 3))
def test_a_bit_of_the_step_or_seed_changes_half_of_the_word(bit):
    base = R.words(0, N, 1 << 31, 0, "cpu")
    for other in (R.words(0, N, (1 << 31) ^ (1 << bit), 0, "cpu"), R.words(0, N, 1 << 31, 1 << bit, "cpu")):
        share = _bits(base ^ other).double().mean(0)
        assert float((share - 0.5).abs().max()) <= 5 * 0.5 / N ** 0.5
