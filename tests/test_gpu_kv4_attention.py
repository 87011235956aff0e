"""tq_kv4_decode and tq_kv4_prefill against attention in 64 bits over the
values that the cache's codes and scales stand for."""
import numpy as np
import pytest
import torch

import ternary_absmax_int8_b200 as tq
from tests._kv4 import Cache, assert_attention, attention, queries, run_attention

pytestmark = pytest.mark.gpu


def check(rng, lens, n, hk, rep, D, ps, window=0, scale=None, spread=1.0, **kw):
    cache = Cache(rng, lens, hk, D, ps, max_pages=kw.pop("max_pages", None))
    c, keep = cache.on_gpu(pad_bytes=kw.pop("pad_bytes", 0))
    q = queries(rng, sum(n), hk * rep, D, spread)
    scale = D ** -0.5 if scale is None else scale
    got = run_attention(c, keep, q, lens, n, scale, window, **kw)
    ref = attention(cache, q, n, scale, window)
    if not kw.get("want_lse", True):
        got = (got[0], ref[1])
    assert_attention(got, ref)
    assert tq.tq_device_error() == 0


@pytest.mark.parametrize("D,ps,hk,rep,lens,window", [
    (128, 64, 5, 4, [1], 0),
    (128, 64, 5, 4, [777], 0),
    (128, 64, 5, 4, [0, 1, 2, 63, 64, 65, 127, 128, 129, 300], 0),
    (128, 16, 2, 8, [5, 16, 17, 1000], 0),
    (128, 32, 1, 7, [31, 32, 33, 500], 100),
    (128, 128, 3, 1, [127, 128, 129, 700], 1),
    (64, 16, 4, 5, [15, 16, 400, 0], 33),
    (64, 32, 1, 16, [640, 90], 0),
    (64, 64, 2, 12, [200, 0, 0, 1], 64),
    (64, 128, 8, 3, [129, 511], 200),
    (128, 64, 1, 64, [321, 64], 0),
    (64, 64, 2, 33, [130], 70),
])
def test_decode(cuda_device, D, ps, hk, rep, lens, window):
    rng = np.random.default_rng(D + ps + hk * rep + len(lens))
    check(rng, lens, [1] * len(lens), hk, rep, D, ps, window)


@pytest.mark.parametrize("D,ps,hk,rep,lens,n,window", [
    (128, 64, 5, 4, [77], [77], 0),
    (128, 64, 1, 1, [1], [1], 0),
    (128, 64, 2, 4, [130, 5, 64, 0], [130, 1, 0, 0], 0),
    (128, 16, 1, 3, [300], [150], 0),
    (128, 32, 2, 2, [200, 65], [3, 65], 50),
    (128, 128, 1, 5, [257], [257], 128),
    (64, 16, 2, 1, [129, 40, 1], [129, 7, 1], 0),
    (64, 64, 1, 8, [190], [190], 1),
    (64, 32, 3, 12, [50, 333], [20, 20], 0),
    (64, 128, 1, 64, [150], [9], 31),
    (128, 64, 1, 4, [3, 2], [10, 2], 0),       # rows before position 0 see nothing
    (64, 64, 1, 2, [0, 5, -3], [4, 5, 2], 0),
])
def test_prefill(cuda_device, D, ps, hk, rep, lens, n, window):
    rng = np.random.default_rng(D + ps + hk * rep + sum(n))
    check(rng, lens, n, hk, rep, D, ps, window, decode=False)


@pytest.mark.parametrize("decode", [True, False])
def test_strides_no_lse_and_padded_pages(cuda_device, decode):
    rng = np.random.default_rng(3)
    n = [1, 1, 1] if decode else [40, 1, 3]
    check(rng, [90, 64, 3], n, 2, 4, 128, 64, decode=decode, q_row=8 * 128 + 64,
          out_row=8 * 128 + 8, want_lse=False, pad_bytes=16, max_pages=9)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("spread,scale", [(30.0, 0.5), (1e-6, 1.0), (1e18, 1e-18), (2e35, 1e-35)])
def test_sharp_flat_and_huge_queries(cuda_device, decode, spread, scale):
    """One key takes all, all keys weigh the same, query values beyond fp16.
    (2e35: a sum of 128 products with codes up to 7 is still below FLT_MAX, for
    kernels that take queries as they are.)"""
    rng = np.random.default_rng(4)
    n = [1, 1] if decode else [70, 2]
    cache = Cache(rng, [200, 131], 2, 128, 64)
    c, keep = cache.on_gpu()
    q = np.clip(queries(rng, sum(n), 8, 128), -1, 1) * np.float32(spread)
    q = (q.view(np.uint32) & 0xFFFF0000).view(np.float32)
    got = run_attention(c, keep, q, cache.lens, n, scale, decode=decode)
    assert_attention(got, attention(cache, q, n, scale))


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("scale", [0.1, 2.0 ** -30, 2.0 ** -90])
def test_zero_queries_weigh_all_keys_the_same(cuda_device, decode, scale):
    """Padding rows of zeros, whose scores are 0 whatever the scale, beside keys
    that a row does not see."""
    rng = np.random.default_rng(14)
    lens, n = [70, 200, 3], ([1] * 3 if decode else [70, 20, 1])
    cache = Cache(rng, lens, 2, 128, 64)
    c, keep = cache.on_gpu()
    q = np.zeros((sum(n), 8, 128), np.float32)
    q[0, 0] = 1.0
    got = run_attention(c, keep, q, lens, n, scale, 30, decode=decode)
    assert_attention(got, attention(cache, q, n, scale, 30))


@pytest.mark.parametrize("decode", [True, False])
def test_scales_of_any_size(cuda_device, decode):
    """Key and value rows from 2^-40 to 2^40, neighbours in one tile."""
    rng = np.random.default_rng(5)
    n = [1, 1] if decode else [66, 5]
    for which, span in ((0, 3), (1, 40)):
        cache = Cache(rng, [200, 131], 2, 64, 32)
        e = rng.integers(-span, span + 1, cache.scales[:, which].shape)
        cache.scales[:, which] *= (2.0 ** e).astype(np.float32)
        c, keep = cache.on_gpu()
        q = queries(rng, sum(n), 4, 64)
        got = run_attention(c, keep, q, cache.lens, n, 0.125, decode=decode)
        assert_attention(got, attention(cache, q, n, 0.125))


@pytest.mark.parametrize("decode", [True, False])
def test_nan_rows_reach_only_who_sees_them(cuda_device, decode):
    rng = np.random.default_rng(6)
    lens, n, window = [150, 70, 64], ([1] * 3 if decode else [150, 20, 2]), 40
    cache = Cache(rng, lens, 2, 128, 64)
    # a key and a value that some windows hold and others do not
    cache.scales[cache.table[0, 30 // 64], 0, 1, 30] = np.nan
    cache.scales[cache.table[1, 0], 1, 0, 60] = np.nan
    cache.scales[cache.table[1, 0], 1, 1, 5] = np.nan
    c, keep = cache.on_gpu()
    q = queries(rng, sum(n), 8, 128)
    q[-1, 3, 7] = np.nan
    got = run_attention(c, keep, q, lens, n, 0.1, window, decode=decode)
    ref = attention(cache, q, n, 0.1, window)
    assert np.array_equal(np.isnan(got[0]), np.isnan(ref[0]))
    fine = ~np.isnan(ref[0])
    assert (np.abs(got[0] - ref[0])[fine] <= ref[2][fine]).all()
    assert np.array_equal(np.isnan(got[1]), np.isnan(ref[1]))


@pytest.mark.parametrize("decode", [True, False])
def test_same_bits_every_run_and_two_streams(cuda_device, decode):
    rng = np.random.default_rng(7)
    lens = [2500, 1, 700, 0, 64]
    n = [1] * 5 if decode else [130, 1, 64, 0, 64]
    cache = Cache(rng, lens, 2, 128, 64)
    c, keep = cache.on_gpu()
    q = queries(rng, sum(n), 8, 128)
    first = run_attention(c, keep, q, lens, n, 0.09, decode=decode)
    assert_attention(first, attention(cache, q, n, 0.09))
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in range(2)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for s in streams:
            with torch.cuda.stream(s):
                again = run_attention(c, keep, q, lens, n, 0.09, decode=decode, stream=s)
            assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("decode", [True, False])
def test_replay_with_other_lengths(cuda_device, decode):
    """A captured call, replayed as the sequences change length on the device."""
    rng = np.random.default_rng(8)
    full = [600, 257, 64]
    cache = Cache(rng, full, 2, 128, 64)
    c, keep = cache.on_gpu()
    hq, T = 8, 3 if decode else 90
    f = dict(device="cuda", dtype=torch.int32)
    lens_g, start_g = torch.tensor(full, **f), torch.tensor([0, 30, 60, 90], **f)
    q = queries(rng, T, hq, 128)
    qg = torch.from_numpy(q).cuda().bfloat16()
    out = torch.empty((T, hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, hq), device="cuda")
    size = (tq.tq_kv4_decode_workspace(c, hq) if decode
            else tq.tq_kv4_prefill_workspace(c, hq, T))
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if decode:
            tq.tq_kv4_decode(c, qg, lens_g, out, lse, hq, 0.1, 0, ws, size)
        else:
            tq.tq_kv4_prefill(c, qg, start_g, lens_g, out, lse, T, hq, 0.1, 0, ws, size)
    for lens, start in (([600, 257, 64], [0, 30, 60, 90]), ([1, 0, 64], [0, 1, 1, 65]),
                        ([599, 3, 0], [0, 88, 90, 90]), ([600, 257, 63], [0, 2, 32, 90])):
        n = [1] * 3 if decode else list(np.diff(start))
        lens_g.copy_(torch.tensor(lens, dtype=torch.int32))
        start_g.copy_(torch.tensor(start, dtype=torch.int32))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        cache.lens = lens
        used = T if decode else start[-1]
        assert (out[used:] == 7).all() and (lse[used:] == 7).all()
        got = (out[:used].double().cpu().numpy(), lse[:used].double().cpu().numpy())
        assert_attention(got, attention(cache, q[:used], n, 0.1))


@pytest.mark.parametrize("decode", [True, False])
def test_bad_pages_are_reported_and_skipped(cuda_device, decode):
    """A page index outside the cache: reported, never followed, and the other
    sequences are right."""
    rng = np.random.default_rng(9)
    lens, n = [300, 130], ([1, 1] if decode else [20, 30])
    for bad in (-1, 10 ** 6):
        cache = Cache(rng, lens, 2, 64, 32)
        q = queries(rng, sum(n), 4, 64)
        ref = attention(cache, q, n, 0.125)
        cache.table[0, 3] = bad
        c, keep = cache.on_gpu()
        got = run_attention(c, keep, q, lens, n, 0.125, decode=decode)
        assert tq.tq_device_error(reset=True) == 2
        at = n[0]
        assert_attention(tuple(x[at:] for x in got), tuple(x[at:] for x in ref))
    # a length beyond the table is cut to it
    cache = Cache(rng, [64, 32], 1, 64, 32)
    c, keep = cache.on_gpu()
    n = [1, 1]
    q = queries(rng, 2, 2, 64)
    run_attention(c, keep, q, [2 ** 30, 32], n, 0.125, decode=decode)
    assert tq.tq_device_error(reset=True) == 2


@pytest.mark.parametrize("decode", [True, False])
def test_far_pages(cuda_device, decode):
    rng = np.random.default_rng(10)
    lens, n = [400, 3], ([1, 1] if decode else [140, 3])
    cache = Cache(rng, lens, 5, 128, 64)
    lead = (1 << 32) // tq.tq_kv4_page_bytes(64, 5, 128) + 7
    c, keep = cache.on_gpu(lead_pages=lead)
    q = queries(rng, sum(n), 20, 128)
    got = run_attention(c, keep, q, lens, n, 0.1, decode=decode)
    assert_attention(got, attention(cache, q, n, 0.1))


@pytest.mark.parametrize("D,rep,batch", [(128, 4, 33), (128, 1, 450), (64, 9, 300), (64, 2, 1100)])
def test_decode_of_many_sequences(cuda_device, D, rep, batch):
    """More sequences than a warp has lanes, or a CTA threads: empty ones first,
    last and in long runs, one far longer than the others."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 100, batch)
    lens[rng.integers(0, 2, batch) == 0] = 0
    lens[:3] = lens[-2:] = 0
    lens[batch // 3:batch // 3 + 20] = 0
    lens[batch - 5] = 900
    check(rng, lens.tolist(), [1] * batch, 1, rep, D, 32)


def test_prefill_of_many_sequences(cuda_device):
    rng = np.random.default_rng(15)
    lens = rng.integers(-1, 40, 1100)
    n = np.minimum(np.maximum(lens, 0), rng.integers(0, 4, 1100))
    n[::7] = 0
    n[600], lens[600] = 300, 310
    check(rng, lens.tolist(), n.tolist(), 1, 2, 64, 16, decode=False)


@pytest.mark.parametrize("D,n,window", [(128, [7, 0, 1], 0), (64, [5, 9, 0], 0),
                                        (64, [33, 2, 2], 70), (128, [3, 3, 3], 1)])
def test_few_rows_over_a_long_cache(cuda_device, D, n, window):
    """Key tiles in parts that are joined; parts that no row of a sequence sees."""
    rng = np.random.default_rng(16)
    check(rng, [2000, 130, 4], n, 2, 4, D, 64, window, decode=False)


@pytest.mark.parametrize("decode", [True, False])
def test_caches_without_pages(cuda_device, decode):
    """No page, or tables of no entry: all sequences empty, or reported."""
    n = [1, 1] if decode else [3, 2]
    q = queries(np.random.default_rng(17), sum(n), 4, 64)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    for kw in (dict(max_pages=0), dict(max_pages=2, page_table=table)):
        c = tq.make_kv4_cache(num_pages=0, page_size=16, kv_heads=2, head_dim=64, batch=2, **kw)
        for lens, error in (([0, 0], 0), ([0, 20], 2)):
            out, lse = run_attention(c, None, q, lens, n, 0.1, decode=decode)
            assert (out == 0).all() and np.isneginf(lse).all()
            assert tq.tq_device_error(reset=True) == error


def test_prefill_of_fewer_rows_than_tok_start_names(cuda_device):
    """tok_start beyond T: rows up to T only, at the positions they have in all."""
    rng = np.random.default_rng(18)
    cache = Cache(rng, [90], 1, 128, 64)
    c, keep = cache.on_gpu()
    q = queries(rng, 40, 4, 128)
    ref = attention(cache, q, [40], 0.1)
    f = dict(device="cuda", dtype=torch.int32)
    out = torch.full((40, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((40, 4), 7.0, device="cuda")
    size = tq.tq_kv4_prefill_workspace(c, 4, 25)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    tq.tq_kv4_prefill(c, torch.from_numpy(q).cuda().bfloat16(), torch.tensor([0, 40], **f),
                      torch.tensor([90], **f), out, lse, 25, 4, 0.1, 0, ws, size)
    torch.cuda.synchronize()
    assert (out[25:] == 7).all() and (lse[25:] == 7).all()
    got = (out[:25].double().cpu().numpy(), lse[:25].double().cpu().numpy())
    assert_attention(got, tuple(x[:25] for x in ref))


@pytest.mark.parametrize("decode", [True, False])
def test_shared_pages(cuda_device, decode):
    """Sequences with a common beginning, whose tables name the same pages."""
    rng = np.random.default_rng(19)
    lens, n = [130, 129, 128], ([1] * 3 if decode else [60, 1, 3])
    cache = Cache(rng, lens, 3, 128, 32)
    cache.table[1, :4] = cache.table[2, :4] = cache.table[0, :4]
    c, keep = cache.on_gpu()
    q = queries(rng, sum(n), 3, 128)
    got = run_attention(c, keep, q, lens, n, 0.1, decode=decode)
    assert_attention(got, attention(cache, q, n, 0.1))


@pytest.mark.parametrize("decode", [True, False])
def test_two_graphs_at_once(cuda_device, decode):
    """Two captured calls with a workspace each, replayed on two streams: the
    bits of calls that run alone."""
    rng = np.random.default_rng(20)
    lens, hq = [3000, 500], 8
    T = 2 if decode else 40
    cache = Cache(rng, lens, 2, 64, 64)
    c, keep = cache.on_gpu()
    f = dict(device="cuda", dtype=torch.int32)
    lens_g, start_g = torch.tensor(lens, **f), torch.tensor([0, T - 1, T], **f)
    size = max(16, tq.tq_kv4_decode_workspace(c, hq) if decode
               else tq.tq_kv4_prefill_workspace(c, hq, T))
    runs = []
    for _ in range(2):
        q = torch.from_numpy(queries(rng, T, hq, 64)).cuda().bfloat16()
        out = torch.empty((T, hq, 64), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((T, hq), device="cuda")
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")

        def call(q=q, out=out, lse=lse, ws=ws):
            if decode:
                tq.tq_kv4_decode(c, q, lens_g, out, lse, hq, 0.1, 0, ws, size)
            else:
                tq.tq_kv4_prefill(c, q, start_g, lens_g, out, lse, T, hq, 0.1, 0, ws, size)

        call()
        torch.cuda.synchronize()
        alone = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                call()
        runs.append((graph, torch.cuda.Stream(), out, lse, alone, (q, ws)))
    for _ in range(5):
        for graph, stream, out, lse, alone, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, out, lse, alone, _ in runs:
            assert torch.equal(out, alone[0]) and torch.equal(lse, alone[1])
