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
