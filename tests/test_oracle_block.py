"""The oracle's generator against the published vectors of Philox 4x32-10 (those of its authors' library: counter and key of
all zeros, of all ones, and of the digits of pi), and the masks' order of halves."""

import numpy as np
import pytest

from oracle import block as oblk

ONES = (1 << 64) - 1


@pytest.mark.parametrize("counter,call,seed,words", [
    (0, 0, 0, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    (ONES, ONES, ONES, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    (0x85a308d3243f6a88, 0x0370734413198a2e, 0x299f31d0a4093822, (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_published_vectors(counter, call, seed, words):
    assert tuple(oblk.philox(counter, call, seed)) == words


def test_masks_take_the_halves_low_first():
    """Group 0 of row 0 with seed and call 0: the halves of the first published vector, in order."""
    halves = [0xe8d5, 0x6627, 0xc58d, 0xe169, 0xac4c, 0xbc57, 0xdbd8, 0x9b00]
    for p in (0.25, 0.5, 0.75, 0.875):
        kept = oblk.dropout_mask(1, 8, p, 0, 0)[0] > 0
        assert (kept == (np.array(halves) >= round(65536 * p))).all()
