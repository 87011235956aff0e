"""Argument checks of the rotary and key/value cache calls, through the C ABI.
No GPU: a refused call touches nothing, a no-op returns before the device."""
import ctypes

import pytest
import torch

import ternary_absmax_int8_b200 as tq

P = 4096  # an aligned address that is never followed


def cache(**kw):
    a = dict(pages=P, page_table=P, num_pages=4, page_size=64, kv_heads=5, head_dim=128, batch=2,
             max_pages=3)
    a.update(kw)
    return tq.make_kv4_cache(**a)


def rope(rows=None, pos=P, inv=P, sections=(64,), T=3, D=128, rot=128, flags=0, pos_stride=0):
    rows = [dict(x_f32=P, y_bf16=2 * P, heads=4)] if rows is None else rows
    tq.tq_rope(tq.make_rope_rows(rows, D), pos, inv, list(sections), T, D, rot, flags,
               pos_stride, stream=0)


def append(c=None, k_bf16=None, v_bf16=None, k_f32=P, v_f32=P, start=P, lens=P, T=2, **kw):
    tq.tq_kv4_append(c or cache(), k_bf16, v_bf16, k_f32, v_f32, start, lens, T, stream=0, **kw)


def decode(c=None, q=P, lens=P, out=P, lse=P, hq=20, scale=0.1, window=0, ws=P,
           size=1 << 40, **kw):
    tq.tq_kv4_decode(c or cache(), q, lens, out, lse, hq, scale, window, ws, size,
                     stream=0, **kw)


def prefill(c=None, q=P, start=P, lens=P, out=P, lse=P, T=7, hq=20, scale=0.1, window=0,
            ws=P, size=1 << 40, **kw):
    tq.tq_kv4_prefill(c or cache(), q, start, lens, out, lse, T, hq, scale, window,
                      ws, size, stream=0, **kw)


def refused(name, fn, *a, **kw):
    with pytest.raises(tq.TQError) as e:
        fn(*a, **kw)
    assert e.value.name == name, str(e.value)


@pytest.mark.parametrize("name,kw", [
    ("TQ_ERR_SHAPE", dict(T=-1)),
    ("TQ_ERR_SHAPE", dict(D=12, rot=0, sections=[0])),
    ("TQ_ERR_SHAPE", dict(D=2048, rot=128)),
    ("TQ_ERR_SHAPE", dict(rot=8, sections=[4])),
    ("TQ_ERR_SHAPE", dict(D=64)),
    ("TQ_ERR_SHAPE", dict(sections=[])),
    ("TQ_ERR_SHAPE", dict(sections=[60])),
    ("TQ_ERR_SHAPE", dict(sections=[65, -1])),
    ("TQ_ERR_SHAPE", dict(sections=[20, 20, 8, 8, 8])),
    ("TQ_ERR_SHAPE", dict(sections=[32, 32], pos_stride=2)),
    ("TQ_ERR_VALUE", dict(flags=2)),
    ("TQ_ERR_NULL", dict(pos=None)),
    ("TQ_ERR_NULL", dict(inv=None)),
    ("TQ_ERR_ALIGN", dict(pos=P + 2)),
    ("TQ_ERR_VALUE", dict(rows=[dict(x_f32=P, heads=4)])),
    ("TQ_ERR_VALUE", dict(rows=[dict(x_f32=P, x_bf16=P, y_bf16=P, heads=4)])),
    ("TQ_ERR_ALIGN", dict(rows=[dict(x_f32=P + 4, y_bf16=P, heads=4)])),
    ("TQ_ERR_ALIGN", dict(rows=[dict(x_f32=P, y_bf16=2 * P, heads=4, y_stride=516)])),
    ("TQ_ERR_SHAPE", dict(rows=[dict(x_f32=P, y_bf16=2 * P, heads=4, x_stride=256)])),
    ("TQ_ERR_SHAPE", dict(rows=[dict(x_f32=P, y_bf16=2 * P, heads=-1)])),
    ("TQ_ERR_VALUE", dict(rows=[dict(x_f32=P, y_bf16=P, heads=4)])),           # in place, two types
    ("TQ_ERR_VALUE", dict(rows=[dict(x_f32=P, y_f32=P, heads=4, x_stride=1024)])),
    ("TQ_ERR_SHAPE", dict(rows=[dict(x_f32=P, y_bf16=2 * P, heads=1)] * 5)),
])
def test_rope_refuses(name, kw):
    refused(name, rope, **kw)


def test_rope_no_ops():
    rope(T=0)
    rope(rows=[])
    rope(rows=[dict(heads=0)])


BAD_CACHE = [
    ("TQ_ERR_SHAPE", dict(page_size=48)),
    ("TQ_ERR_SHAPE", dict(page_size=256)),
    ("TQ_ERR_UNSUPPORTED", dict(head_dim=96)),
    ("TQ_ERR_SHAPE", dict(kv_heads=0)),
    ("TQ_ERR_SHAPE", dict(batch=-1)),
    ("TQ_ERR_SHAPE", dict(num_pages=-1)),
    ("TQ_ERR_SHAPE", dict(max_pages=-1)),
    ("TQ_ERR_UNSUPPORTED", dict(max_pages=1 << 24)),
    ("TQ_ERR_UNSUPPORTED", dict(batch=70000)),
    ("TQ_ERR_SHAPE", dict(page_stride=16)),
    ("TQ_ERR_ALIGN", dict(page_stride=64 * 132 * 5 + 8)),
    ("TQ_ERR_NULL", dict(pages=None)),
    ("TQ_ERR_NULL", dict(page_table=None)),
    ("TQ_ERR_ALIGN", dict(pages=P + 8)),
    ("TQ_ERR_ALIGN", dict(page_table=P + 2)),
]


@pytest.mark.parametrize("name,kw", BAD_CACHE)
def test_bad_caches_are_refused(name, kw):
    c = cache(**kw)
    refused(name, append, c)
    refused(name, decode, c, hq=c.kv_heads or 1)
    refused(name, prefill, c, hq=c.kv_heads or 1)


@pytest.mark.parametrize("name,kw", [
    ("TQ_ERR_SHAPE", dict(T=-1)),
    ("TQ_ERR_SHAPE", dict(start=None, T=3)),
    ("TQ_ERR_VALUE", dict(v_f32=None)),
    ("TQ_ERR_VALUE", dict(k_bf16=P)),
    ("TQ_ERR_VALUE", dict(k_f32=None, v_f32=None)),
    ("TQ_ERR_VALUE", dict(k_f32=None, v_f32=None, k_bf16=P)),
    ("TQ_ERR_NULL", dict(lens=None)),
    ("TQ_ERR_ALIGN", dict(lens=P + 1)),
    ("TQ_ERR_ALIGN", dict(start=P + 2)),
    ("TQ_ERR_ALIGN", dict(k_f32=P + 8)),
    ("TQ_ERR_ALIGN", dict(v_stride=641)),
    ("TQ_ERR_SHAPE", dict(k_stride=320)),
])
def test_append_refuses(name, kw):
    refused(name, append, **kw)


BAD_QUERY = [
    ("TQ_ERR_SHAPE", dict(hq=18)),
    ("TQ_ERR_SHAPE", dict(hq=0)),
    ("TQ_ERR_UNSUPPORTED", dict(hq=5 * 65)),
    ("TQ_ERR_VALUE", dict(scale=0.0)),
    ("TQ_ERR_VALUE", dict(scale=-1.0)),
    ("TQ_ERR_VALUE", dict(scale=float("inf"))),
    ("TQ_ERR_VALUE", dict(scale=float("nan"))),
    ("TQ_ERR_VALUE", dict(window=-1)),
    ("TQ_ERR_NULL", dict(q=None)),
    ("TQ_ERR_NULL", dict(out=None)),
    ("TQ_ERR_NULL", dict(lens=None)),
    ("TQ_ERR_ALIGN", dict(q=P + 2)),
    ("TQ_ERR_ALIGN", dict(out=P + 2)),
    ("TQ_ERR_ALIGN", dict(lse=P + 2)),
    ("TQ_ERR_ALIGN", dict(lens=P + 2)),
    ("TQ_ERR_ALIGN", dict(q_stride=20 * 128 + 4)),
    ("TQ_ERR_SHAPE", dict(out_stride=1280)),
]


@pytest.mark.parametrize("name,kw", BAD_QUERY)
def test_attention_refuses(name, kw):
    refused(name, decode, **kw)
    refused(name, prefill, **kw)


def test_prefill_refuses():
    refused("TQ_ERR_SHAPE", prefill, T=-1)
    refused("TQ_ERR_NULL", prefill, start=None)
    refused("TQ_ERR_ALIGN", prefill, start=P + 2)


def test_empty_calls_return_before_the_device():
    append(T=0)
    append(cache(batch=0), T=5)
    decode(cache(batch=0))
    prefill(cache(batch=0))
    prefill(T=0)


def test_page_bytes():
    assert tq.tq_kv4_page_bytes(64, 5, 128) == 64 * 5 * 132
    assert tq.tq_kv4_page_bytes(16, 1, 64) == 16 * 68
    assert tq.tq_kv4_page_bytes(48, 1, 64) == 0
    assert tq.tq_kv4_page_bytes(64, 0, 64) == 0
    assert tq.tq_kv4_page_bytes(64, 1, 96) == 0


def test_binding_refuses_wrong_tensors():
    """Element sizes and places that a kernel would misread."""
    refused("TQ_ERR_VALUE", tq.make_kv4_cache, pages=torch.zeros(16, dtype=torch.int32))
    refused("TQ_ERR_VALUE", append, lens=torch.zeros(2, dtype=torch.int64))
    refused("TQ_ERR_VALUE", append, lens=torch.zeros(2, dtype=torch.int32))  # not on the GPU
    refused("TQ_ERR_VALUE", decode, q=torch.zeros(8, dtype=torch.float32))


def test_structs_match_the_header():
    assert ctypes.sizeof(tq.TqRopeRows) == 56
    assert ctypes.sizeof(tq.TqKv4Cache) == 48
    assert ctypes.sizeof(tq.TqKv4Query) == 56


@pytest.mark.parametrize("fn,kw", [
    (append, dict(T=(1 << 30) // 5 + 1)),
    (append, dict(k_stride=1 << 32)),
    (append, dict(v_stride=1 << 32)),
    (append, dict(c=cache(page_stride=1 << 32))),
    (decode, dict(c=cache(batch=65536, max_pages=1 << 16))),
    (decode, dict(c=cache(batch=4096, kv_heads=1, max_pages=1 << 18), hq=17)),
    (prefill, dict(T=(1 << 28) + 1)),
    (prefill, dict(T=1 << 29, c=cache(kv_heads=1024), hq=1024)),
])
def test_counts_beyond_32_bits_are_refused(fn, kw):
    refused("TQ_ERR_UNSUPPORTED", fn, **kw)
