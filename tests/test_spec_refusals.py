"""Further refusals of the drafted tokens' calls, on the host before any launch."""
import ctypes

import pytest

from paged_kv_cache_188_gb300 import api
from paged_kv_cache_188_gb300 import build as B

FAKE = 0x10000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.lib()


@pytest.mark.parametrize("move", [False, True])
def test_lengths_that_overlap_in_part(lib, move):
    """Requests' new lengths among others' old ones: one request's would be written before another's is read."""
    kv = (P(FAKE), P(FAKE), api.KvShape(1, 64, 2, 64), 2) if move else (None, None, api.KvShape(0, 0, 0, 0), 0)

    def call(seq, new, r, table=FAKE):
        return lib.pa_kv_accept(P(table), 2, 32, P(FAKE), P(seq), P(FAKE), 4, r, P(FAKE), 4, P(FAKE), P(new), P(FAKE), *kv,
                                None, None)
    for shift in (4, -4, 8, -8):
        assert call(FAKE, FAKE + shift, 3) == 2
    # beside one another, or (in the table form) the same: looked at no further than the next argument
    for shift in (12, -12) + (() if move else (0,)):
        assert call(FAKE, FAKE + shift, 3, table=0) == 1
