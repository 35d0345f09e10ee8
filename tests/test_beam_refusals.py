"""beam_reorder with more tensors than one call of the library takes (no GPU
needed): what a later call would refuse is refused before the first."""
import pytest

from gated_delta_rule_25_amd.beam import BEAM_REORDER_MAX, _refuse_reorder

PARENTS = (1 << 40, 64)


def states(n=11, size=4096, row=64):
    return [((i + 1) << 20, size, row) for i in range(n)]


def test_states_apart_are_taken():
    _refuse_reorder(states(), PARENTS)
    s = states()
    s[10] = (s[9][0] + 4096, 4096, 64)      # next to one another
    s[3] = (0, 0, 0)                        # nothing in it
    _refuse_reorder(s, (s[0][0] - 64, 64))


@pytest.mark.parametrize("i,j", [(0, 10), (2, 3), (8, 9), (7, 8)])
@pytest.mark.parametrize("shift", [-4095, -16, 1, 4095])
def test_states_that_overlap(i, j, shift):
    s = states()
    s[j] = (s[i][0] + shift, 4096, 64)
    with pytest.raises(ValueError, match="overlap"):
        _refuse_reorder(s, PARENTS)


@pytest.mark.parametrize("i", [0, 7, 8, 10])
def test_states_over_parents(i):
    s = states()
    with pytest.raises(ValueError, match="overlap"):
        _refuse_reorder(s, (s[i][0] + 4000, 64))
    with pytest.raises(ValueError, match="overlap"):
        _refuse_reorder(s, (s[i][0] - 60, 64))


@pytest.mark.parametrize("i", [0, 8, 10])
@pytest.mark.parametrize("at,row", [(1, 2 ** 32), (4, 2 ** 34), (16, 2 ** 36)])
def test_rows_too_long_for_a_launch(i, at, row):
    """A launch has fewer than 2^32 threads, one for each unit of a row (16,
    4 or 1 bytes by its alignment) of its up to eight tensors together."""
    s = states()
    s[i] = ((1 << 41) + at, 2 * row, row)
    with pytest.raises(ValueError, match="too long"):
        _refuse_reorder(s, PARENTS)
    s[i] = ((1 << 41) + at, row, row // 2)
    _refuse_reorder(s, PARENTS)
    # two halves of it in one call of the library, and in two
    j = (i + 1) % len(s)
    s[j] = ((1 << 43) + at, row, row // 2)
    if i // BEAM_REORDER_MAX == j // BEAM_REORDER_MAX:
        with pytest.raises(ValueError, match="too long"):
            _refuse_reorder(s, PARENTS)
    else:
        _refuse_reorder(s, PARENTS)
