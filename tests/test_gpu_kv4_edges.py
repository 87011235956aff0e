"""Attention over the 4-bit cache at the borders of what a call may ask for,
against 64 bits (tolerances: tests/_kv4.py)."""
import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("window", [0, 5, 100, 2 ** 31 - 1])
def test_rows_far_before_position_0(cuda_device, window):
    """tok_start that names 2^31 - 1 tokens of which the call has five."""
    rng = np.random.default_rng(33)
    cache = Cache(rng, [100], 2, 64, 16)
    c, keep = cache.on_gpu()
    f = dict(device="cuda", dtype=torch.int32)
    q = torch.from_numpy(queries(rng, 5, 4, 64)).cuda().bfloat16()
    out, lse = torch.full_like(q, 7.0), torch.full((5, 4), 7.0, device="cuda")
    size = tq.tq_kv4_prefill_workspace(c, 4, 5)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    tq.tq_kv4_prefill(c, q, torch.tensor([0, 2 ** 31 - 1], **f), torch.tensor([100], **f), out, lse,
                      5, 4, 0.1, window, ws, size)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all() and tq.tq_device_error() == 0


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


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("D,rep", [(128, 4), (64, 7), (64, 16)])
def test_scores_beyond_fp32(cuda_device, decode, D, rep):
    """Keys whose scores are 0, 2^134 or -2^134 times a little: a row that sees one
    of the large ones is NaN, those far below count as not seen, and the others
    weigh the same. The weights are equal and exact, so the tolerance is that of
    tests/_kv4.py without the part of the scores."""
    rng = np.random.default_rng(32)
    lens = [200, 200, 150, 300, 1, 1]
    n = [1] * 6 if decode else [170, 30, 2, 5, 1, 1]
    hk = 2
    cache = Cache(rng, lens, hk, D, 32)
    kind = [rng.integers(-1, 1, L) for L in lens]  # 0, or far below
    kind[1][40] = 1                                # one far above
    kind[2][:] = -1                                # nothing else
    kind[3][:] = np.where(np.arange(300) < 131, -1, 0)
    kind[4][:], kind[5][:] = 1, -1
    for b, ks in enumerate(kind):
        for j, x in enumerate(ks):
            at = cache.table[b, j // 32], 0, slice(None), j % 32
            cache.codes[at], cache.scales[at] = 7 * x, np.float32(2.0 ** 60)
    c, keep = cache.on_gpu()
    q = np.full((sum(n), hk * rep, D), 2.0 ** 66, np.float32)
    out, lse = run_attention(c, keep, q, lens, n, 1.0, decode=decode)
    t = 0
    for b, nb in enumerate(n):
        v = cache.rows(b, 1)
        for p in range(lens[b] - nb, lens[b]):
            seen = kind[b][:p + 1]
            if (seen > 0).any():
                assert np.isnan(out[t]).all() and np.isnan(lse[t]).all()
            elif (seen < 0).all():
                assert (out[t] == 0).all() and np.isneginf(lse[t]).all()
            else:
                vv = np.repeat(v[:, :p + 1][:, seen == 0], rep, 0)  # [heads, keys, D]
                ref, A = vv.mean(1), np.abs(vv).mean(1)
                tol = (2.0 ** -8 * np.abs(ref) + A * (2.0 ** -8 + 2.0 ** -12)
                       + 2.0 ** -39 * vv.shape[1] * np.abs(vv).max())
                assert (np.abs(out[t] - ref) <= tol).all()
                want = np.log(vv.shape[1])
                assert (np.abs(lse[t] - want) <= 2.0 ** -18 + 2.0 ** -22 * want).all()
            t += 1
    assert tq.tq_device_error() == 0


def without(cache, q, n, scale, window, gone):
    """tests/_kv4.py's attention, of sequences whose keys gone[b] are not there."""
    class Rest:
        hk, lens = cache.hk, cache.lens

        @staticmethod
        def rows(b, which):
            x = cache.rows(b, which).copy()
            x[:, gone[b][:x.shape[1]]] = 0
            return x

    out, lse, tol, ltol = attention(Rest, q, n, scale, window)
    rep, t = q.shape[1] // cache.hk, 0
    for b, nb in enumerate(n):
        k, v = (cache.rows(b, w) for w in (0, 1))
        for p in range(cache.lens[b] - nb, cache.lens[b]):
            seen = np.arange(k.shape[1])
            seen = seen[(seen <= p) & (seen > p - (window or p + 1)) & ~gone[b][:len(seen)]]
            for h in range(q.shape[1]):
                out[t, h], lse[t, h] = 0, -np.inf
                if len(seen):
                    z = scale * (k[h // rep, seen] @ q[t, h].astype(np.float64))
                    lse[t, h] = z.max() + np.log(np.exp(z - z.max()).sum())
                    w, vv = np.exp(z - lse[t, h]), v[h // rep, seen]
                    out[t, h] = w @ vv
                    # (attention's bound with this A; its dz is of all keys that are left)
                    A = w @ np.abs(vv)
                    tol[t, h] = (2.0 ** -8 * np.abs(out[t, h]) + 2.0 ** -39 * len(vv) * np.abs(vv).max()
                                 + A * (2.0 ** -8 + 2 * (ltol[t, h] - 2.0 ** -18) + 2.0 ** -12) + 1e-30)
            t += 1
    return out, lse, tol, ltol


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("D,ps,window", [(64, 32, 0), (128, 16, 0), (128, 128, 0), (64, 64, 90)])
def test_keys_of_pages_outside_the_cache_are_left_out(cuda_device, decode, D, ps, window):
    """The sequences that name such pages: their other keys count, a row without any
    is 0 and -infinity; and lengths beyond the table are cut to it."""
    rng = np.random.default_rng(34)
    lens, n = [300, 130, 2, 256], ([1] * 4 if decode else [120, 30, 2, 3])
    cache = Cache(rng, lens, 2, D, ps, max_pages=384 // ps)
    gone = [np.zeros(384, bool) for _ in lens]
    good = cache.table.copy()
    for b, page, name in ((0, 0, -1), (0, 200 // ps, cache.num_pages), (0, 299 // ps, 2 ** 31 - 1),
                          (1, 0, -2 ** 31), (2, 0, cache.num_pages + 7)):
        cache.table[b, page] = name
        gone[b][page * ps:(page + 1) * ps] = True
    c, keep = cache.on_gpu()
    q = queries(rng, sum(n), 8, D)
    got = run_attention(c, keep, q, lens, n, 0.1, window, decode=decode)
    assert tq.tq_device_error(reset=True) == 2
    cache.table = good
    assert_attention(got, without(cache, q, n, 0.1, window, gone))

    cut = [384, 40]
    cache = Cache(rng, cut, 2, D, ps, max_pages=384 // ps)
    c, keep = cache.on_gpu()
    n = [1, 1] if decode else [150, 40]
    q = queries(rng, sum(n), 8, D)
    for beyond in (385, 2 ** 31 - 1):
        got = run_attention(c, keep, q, [beyond, 40], n, 0.1, window, decode=decode)
        assert tq.tq_device_error(reset=True) == 2
        assert_attention(got, attention(cache, q, n, 0.1, window))
