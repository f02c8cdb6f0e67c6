"""Numbers that the binding hands to the library in 32 bits: what does not fit is refused, not cut off."""
import ctypes

import pytest

from paged_kv_cache_127_gb300 import build as pa_build


@pytest.fixture(scope="module")
def pa():
    pa_build.build()
    from paged_kv_cache_127_gb300 import binding
    return binding


BEYOND = (2 ** 31, 2 ** 32, 2 ** 32 + 40, -2 ** 31 - 1, 10 ** 12)


def test_numbers_beyond_32_bits_are_refused(pa):
    for x in (0, 1, 2 ** 31 - 1, -1, -2 ** 31):
        assert pa._i32(x, "x") == x == ctypes.c_int32(x).value
    for x in BEYOND:
        with pytest.raises(ValueError):
            pa._i32(x, "x")


def test_windows_of_scores_beyond_32_bits_are_refused(pa):
    for x in BEYOND:
        with pytest.raises(ValueError):
            pa._marshal_score(pa.make_score(window=x), 8, 3, None)
    _, keep = pa._marshal_score(pa.make_score(window=2 ** 31 - 1), 8, 3, None)
    assert keep[0].window == 2 ** 31 - 1
