"""tq_kv4_append against the definition: bytes of the whole cache, bit for bit."""
import numpy as np
import pytest
import torch

import ternary_absmax_int8_b200 as tq
from tests._kv4 import Cache, bf16_round, quantise, to_gpu

pytestmark = pytest.mark.gpu


def rows(rng, T, hk, D, f32):
    x = rng.standard_normal((T, hk, D)) * np.exp(rng.standard_normal((T, hk, 1)))
    x = x.astype(np.float32)
    return x if f32 else bf16_round(x).reshape(x.shape)


def append(c, keep, k, v, f32, n, lens, tail=0, row=0, tok_start=True):
    T, hk, D = k.shape
    kg, vg = to_gpu(k, f32, row), to_gpu(v, f32, row)
    start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    lens_g = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
    a = (None, None, kg, vg) if f32 else (kg, vg, None, None)
    tq.tq_kv4_append(c, *a, start if tok_start else None, lens_g, T, k_stride=row, v_stride=row)
    torch.cuda.synchronize()


def put(cache, k, v, n, lens):
    t = 0
    for b, nb in enumerate(n):
        for i in range(nb):
            j = lens[b] - nb + i
            if j >= 0:
                pg, slot = cache.table[b, j // cache.ps], j % cache.ps
                for w, x in enumerate((k, v)):
                    cache.codes[pg, w, :, slot], cache.scales[pg, w, :, slot] = quantise(x[t])
            t += 1


@pytest.mark.parametrize("D,ps,hk,f32,n,lens,row", [
    (128, 64, 5, True, [1] * 7, [1, 64, 65, 128, 200, 33, 2], 0),
    (128, 64, 5, False, [3, 0, 130, 1], [3, 5, 131, 64], 0),
    (64, 16, 8, False, [17, 1, 31], [17, 16, 48], 8 * 64 + 8),
    (64, 32, 1, True, [1, 40], [300, 40], 68),
    (128, 128, 2, True, [2, 129, 1], [1, 129, 0], 0),   # tokens before position 0 are dropped
    (128, 16, 3, False, [0, 0], [4, 0], 0),
])
def test_append(cuda_device, D, ps, hk, f32, n, lens, row):
    rng = np.random.default_rng(D + ps + hk)
    cache = Cache(rng, lens, hk, D, ps)
    c, keep = cache.on_gpu()
    tail = 2  # padding rows behind the last sequence
    T = sum(n) + tail
    k, v = rows(rng, T, hk, D, f32), rows(rng, T, hk, D, f32)
    append(c, keep, k, v, f32, n, lens, row=row)
    put(cache, k, v, n, lens)
    assert np.array_equal(keep[0].cpu().numpy(), cache.bytes())
    assert tq.tq_device_error() == 0


def test_append_one_token_without_tok_start(cuda_device):
    rng = np.random.default_rng(5)
    lens = [1, 17, 0, 64]
    cache = Cache(rng, lens, 5, 128, 64)
    c, keep = cache.on_gpu(pad_bytes=48)
    k, v = rows(rng, 4, 5, 128, True), rows(rng, 4, 5, 128, True)
    append(c, keep, k, v, True, [1] * 4, lens, tok_start=False)
    put(cache, k, v, [1] * 4, lens)
    size = cache.bytes().shape[1]
    got = keep[0].cpu().numpy()
    assert np.array_equal(got[:, :size], cache.bytes())
    assert (got[:, size:] == 255).all()


@pytest.mark.parametrize("f32", [True, False])
def test_append_borders(cuda_device, f32):
    """Ties, values a step from a tie, zeros, tiny and huge rows, NaN, infinities."""
    rng = np.random.default_rng(9)
    D, hk, T = 64, 2, 40
    k = rows(rng, T, hk, D, True)
    scales = bf16_round(np.exp(rng.uniform(-80, 80, T)).astype(np.float32))
    for t in range(24):  # x = s (m + 1/2) and its neighbours; 7 s on top fixes the scale
        s = scales[t]
        h = (rng.integers(-7, 7, (hk, D)) + 0.5).astype(np.float32) * s
        step = rng.integers(-1, 2, (hk, D))
        k[t] = np.where(step > 0, np.nextafter(h, np.float32(np.inf)),
                        np.where(step < 0, np.nextafter(h, np.float32(-np.inf)), h))
        k[t, :, 0] = 7 * s
    k[24] = 0
    k[25] = -0.0
    k[26] *= np.float32(1e-38)
    k[27] = rng.integers(-3, 4, (hk, D)) * np.float32(1e-45)
    k[28] = np.float32(3e38) * np.sign(k[28])
    k[29, 0, 5] = np.nan
    k[30, 1, 63] = np.inf
    k[31, 0, 0] = -np.inf
    k[32] = rng.integers(-40, 40, (hk, D)) * np.float32(2.0 ** -133)
    if not f32:
        k = bf16_round(np.nan_to_num(k, nan=1.0, posinf=1.0, neginf=1.0)).reshape(k.shape)
        k[29, 0, 5], k[30, 1, 63], k[31, 0, 0] = np.nan, np.inf, -np.inf
    v = k[::-1].copy()
    cache = Cache(rng, [T], hk, D, 16)
    c, keep = cache.on_gpu()
    append(c, keep, k, v, f32, [T], [T])
    put(cache, k, v, [T], [T])
    got, want = keep[0].cpu().numpy(), cache.bytes()
    # NaN scales: the definition names no payload
    g, w = (x.reshape(cache.num_pages, hk, -1) for x in (got, want))
    sc = cache.ps * D
    assert np.array_equal(g[..., :sc], w[..., :sc])
    gs, ws = (np.ascontiguousarray(x[..., sc:]).view(np.uint16).astype(np.uint32) << 16
              for x in (g, w))
    gs, ws = gs.view(np.float32), ws.view(np.float32)
    assert np.array_equal(np.isnan(gs), np.isnan(ws))
    assert np.array_equal(gs[~np.isnan(gs)], ws[~np.isnan(ws)])


@pytest.mark.parametrize("f32", [True, False])
def test_append_subnormal_scales(cuda_device, f32):
    """Rows of a few of bf16's last steps, 2^-133: s rounds to 1 of them for all
    up to 10, and codes end at 7."""
    D, hk, T = 64, 1, 64
    rng = np.random.default_rng(13)
    k = np.empty((T, hk, D), np.float32)
    for t in range(T):
        k[t] = rng.integers(-t, t + 1, (hk, D)) * np.float32(2.0 ** -133)
        k[t, :, 3] = t * np.float32(2.0 ** -133)
    v = -k[::-1].copy()
    assert k.max() == np.float32(63 * 2.0 ** -133)  # the host does not flush them
    cache = Cache(rng, [T], hk, D, 64)
    c, keep = cache.on_gpu()
    append(c, keep, k, v, f32, [T], [T])
    put(cache, k, v, [T], [T])
    assert np.array_equal(keep[0].cpu().numpy(), cache.bytes())


def test_append_bad_pages_are_reported_and_skipped(cuda_device):
    rng = np.random.default_rng(11)
    lens = [70, 5]
    cache = Cache(rng, lens, 2, 64, 16)
    good = cache.table.copy()
    cache.table[0, 4] = cache.num_pages  # positions 64..69 of sequence 0
    c, keep = cache.on_gpu()
    before = keep[0].clone()
    k, v = rows(rng, 2, 2, 64, True), rows(rng, 2, 2, 64, True)
    append(c, keep, k, v, True, [1, 1], lens)
    assert tq.tq_device_error(reset=True) == 2
    pg, slot = good[1, 0], 4
    (cache.codes[pg, 0, :, slot], cache.scales[pg, 0, :, slot]) = quantise(k[1])
    (cache.codes[pg, 1, :, slot], cache.scales[pg, 1, :, slot]) = quantise(v[1])
    assert np.array_equal(keep[0].cpu().numpy(), cache.bytes())
    # a length beyond the table
    keep[0].copy_(before)
    append(c, keep, k, v, True, [1, 1], [cache.max_pages * 16 + 1, 0])
    assert tq.tq_device_error(reset=True) == 2
    assert torch.equal(keep[0], before)


def test_append_far_pages(cuda_device):
    """Pages more than 4 GiB into the cache."""
    rng = np.random.default_rng(12)
    cache = Cache(rng, [200, 3], 5, 128, 64)
    lead = (1 << 32) // tq.tq_kv4_page_bytes(64, 5, 128) + 7
    c, keep = cache.on_gpu(lead_pages=lead)
    k, v = rows(rng, 12, 5, 128, False), rows(rng, 12, 5, 128, False)
    append(c, keep, k, v, False, [10, 2], [200, 3])
    put(cache, k, v, [10, 2], [200, 3])
    assert np.array_equal(keep[0][lead:].cpu().numpy(), cache.bytes())


@pytest.mark.parametrize("D,hk,f32,batch", [(64, 9, False, 700), (128, 45, True, 100),
                                            (64, 80, True, 100)])
def test_append_of_many_sequences(cuda_device, D, hk, f32, batch):
    """More (token, head) pairs than the GPU takes at once, sequences of 0 to 3
    tokens and one long one, tokens beyond tok_start's end ignored."""
    rng = np.random.default_rng(21)
    n = rng.integers(0, 4, batch)
    n[::5] = 0
    n[60] = 900
    lens = n + rng.integers(0, 20, batch)
    cache = Cache(rng, lens.tolist(), hk, D, 16)
    c, keep = cache.on_gpu()
    T = int(n.sum()) + 5
    k, v = rows(rng, T, hk, D, f32), rows(rng, T, hk, D, f32)
    append(c, keep, k, v, f32, n.tolist(), lens.tolist())
    put(cache, k, v, n, lens)
    assert np.array_equal(keep[0].cpu().numpy(), cache.bytes())
    assert tq.tq_device_error() == 0


def test_append_to_no_pages(cuda_device):
    """Tables of no entry: tokens of empty sequences are dropped, others reported."""
    rng = np.random.default_rng(22)
    k, v = rows(rng, 2, 1, 64, False), rows(rng, 2, 1, 64, False)
    c = tq.make_kv4_cache(page_size=16, kv_heads=1, head_dim=64, batch=2)
    for lens, error in (([0, 0], 0), ([0, 3], 2)):
        append(c, None, k, v, False, [1, 1], lens)
        assert tq.tq_device_error(reset=True) == error
