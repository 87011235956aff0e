"""Attention over the 4-bit cache at the borders of what a call may ask for,
against 64 bits (tolerances: tests/_kv4.py)."""
import numpy as np
import pytest

import ternary_absmax_int8_b200 as tq
from tests._kv4 import Cache, assert_attention, attention, queries, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 5, 1 << 30, 129, 128, 127])
def test_windows_beyond_the_table(cuda_device, decode, window):
    """A window that hides no key, up to the largest whole number, beside rows
    before position 0; and the border itself (a table of 128 tokens)."""
    rng = np.random.default_rng(30)
    lens, n = [3, 128, 0], ([1] * 3 if decode else [10, 128, 4])
    cache = Cache(rng, lens, 2, 64, 16, max_pages=8)
    c, keep = cache.on_gpu()
    q = queries(rng, sum(n), 4, 64)
    got = run_attention(c, keep, q, lens, n, 0.125, window, decode=decode)
    assert_attention(got, attention(cache, q, n, 0.125, window))
    assert tq.tq_device_error() == 0


def test_queries_before_position_0_see_nothing_whatever_they_hold(cuda_device):
    """Rows before position 0 are 0 and -infinity, whether the rows beside them see
    keys or not and though they hold a NaN or an infinity; such a row that sees a
    key is NaN, and no other. (One unit of 256 rows, parts of keys, 64 and 128.)"""
    rng = np.random.default_rng(31)
    for D, lens, n, max_pages in ((64, [3, 0, 40], [10, 4, 40], None), (128, [3, 2], [70, 2], 40),
                                  (128, [200, 0, 5], [210, 3, 5], None)):
        cache = Cache(rng, lens, 2, D, 64, max_pages=max_pages)
        c, keep = cache.on_gpu()
        q = queries(rng, sum(n), 8, D)
        clean = q.copy()
        first = n[0] - lens[0]  # tokens before position 0 of sequence 0
        q[0, 0, 0] = np.nan
        q[first - 1, 5, D - 1] = -np.inf
        q[1, :, 3] = np.inf
        seen = q.copy()
        seen[:first] = clean[:first]
        seen[first, 2, 7] = q[first, 2, 7] = np.nan
        got = run_attention(c, keep, q, lens, n, 0.1, decode=False)
        assert (got[0][:first] == 0).all() and np.isneginf(got[1][:first]).all()
        ref = attention(cache, seen, n, 0.1)
        assert np.isnan(ref[0]).any(-1).sum() == 1
        nan = np.isnan(ref[1])
        assert np.array_equal(np.isnan(got[1]), nan)
        # (the logarithms of the others: a row that is NaN has no tolerance)
        lse, rlse, ltol = (np.where(nan, 0, x) for x in (got[1], ref[1], ref[3]))
        assert_attention((got[0], lse), (ref[0], rlse, ref[2], ltol))
        assert tq.tq_device_error() == 0
