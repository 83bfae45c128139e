"""Numbers of pairs that rope_frequencies takes: whole ones, as they are."""
import numpy as np
import pytest

import w4a4_rank_corrected_quantize_amd as svdq


@pytest.mark.parametrize("sections", [[21.5, 21.5, 21.0], np.array([32.0]), [8, 8.0], ["8"], [None]])
def test_sections_that_are_no_whole_numbers_are_refused(sections):
    with pytest.raises(TypeError):
        svdq.rope_frequencies(sections)


@pytest.mark.parametrize("sections", [np.array([2 ** 32 + 8]), [2 ** 32 + 8], [2 ** 63 + 8], np.array([2 ** 63 + 8], np.uint64),
                                      np.array([8, -2 ** 32 + 8]), [-2 ** 63 + 8]])
def test_sections_past_32_bits_are_refused(sections):
    with pytest.raises(svdq.SvdqError):
        svdq.rope_frequencies(sections)


@pytest.mark.parametrize("kind", [list, tuple, lambda s: np.array(s, np.uint8), lambda s: np.array(s, np.int64)])
def test_sections_of_any_whole_type(kind):
    want = svdq.rope_frequencies([16, 24, 24])
    for a, b in zip(want, svdq.rope_frequencies(kind([16, 24, 24]))):
        assert np.array_equal(a, b)


def test_sections_of_two_dimensions_are_refused():
    with pytest.raises(ValueError):
        svdq.rope_frequencies([[8], [8]])
