"""What the Python bindings of the rotary and cache calls take for a tensor. No
GPU: tensors in host memory stand for the current device's, and every call has
nothing to do (no sequence, no token), so that its pointers are not followed."""
import pytest
import torch

import ternary_absmax_int8_b200 as tq


@pytest.fixture(autouse=True)
def host_tensors_are_here(monkeypatch):
    monkeypatch.setattr(tq, "_device", lambda: -1)
    monkeypatch.setattr(tq, "_here", lambda stream: (-1, 0))


def t(dtype, *shape):
    return torch.zeros(shape or (16,), dtype=dtype)


GOOD = dict(x_bf16=torch.bfloat16, x_f32=torch.float32, y_bf16=torch.bfloat16, y_f32=torch.float32,
            pos=torch.int32, inv_freq=torch.float32, pages=torch.uint8, page_table=torch.int32,
            k_bf16=torch.bfloat16, v_bf16=torch.bfloat16, k_f32=torch.float32, v_f32=torch.float32,
            tok_start=torch.int32, lens=torch.int32, q=torch.bfloat16, out=torch.bfloat16,
            lse=torch.float32, workspace=torch.uint8)


def cache(**a):
    return tq.make_kv4_cache(pages=a.get("pages"), page_table=a.get("page_table"), kv_heads=1,
                             page_size=16, head_dim=64)


def calls(a):
    """Every call of the bindings with the tensors of `a`."""
    g = {n: a.get(n) for n in GOOD}
    rows = [{n: g[n] for n in ("x_bf16", "x_f32", "y_bf16", "y_f32")} | dict(heads=0)]
    tq.tq_rope(tq.make_rope_rows(rows, 64), g["pos"], g["inv_freq"], [32], 0, 64, 64)
    c = cache(**a)
    tq.tq_kv4_append(c, g["k_bf16"], g["v_bf16"], g["k_f32"], g["v_f32"], g["tok_start"], g["lens"],
                     0)
    tq.tq_kv4_decode(c, g["q"], g["lens"], g["out"], g["lse"], 1, 0.1, workspace=g["workspace"])
    tq.tq_kv4_prefill(c, g["q"], g["tok_start"], g["lens"], g["out"], g["lse"], 0, 1, 0.1,
                      workspace=g["workspace"])


def test_the_types_that_the_calls_name():
    calls({n: t(d) for n, d in GOOD.items()})
    calls({n: 4096 for n in GOOD})
    calls({})
    # the bits of bf16 as whole numbers
    calls(dict(x_bf16=t(torch.int16), q=t(torch.int16), out=t(torch.uint16)))


@pytest.mark.parametrize("name,dtype", [
    (n, d) for n, g in GOOD.items()
    for d in (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float64,
              torch.uint8, torch.bool)
    if d != g])
def test_other_types_are_refused(name, dtype):
    """Of the same size too: fp16 for bf16, fp32 for int32, bool for bytes."""
    with pytest.raises(tq.TQError) as e:
        calls({name: t(dtype)})
    assert e.value.name == "TQ_ERR_VALUE" and str(dtype) in str(e.value)


def wide(dtype, T, columns, rows=()):
    """[T, columns] of rows of 1000 elements, or in the dimensions `rows` + columns."""
    x = torch.zeros((T, 1000), dtype=dtype)[:, 8:8 + columns]
    return x.unflatten(1, rows) if rows else x


def test_rows_of_a_wider_tensor():
    """Views whose rows lie as far apart as the call is told."""
    for x in (wide(torch.bfloat16, 3, 128), wide(torch.bfloat16, 3, 128, (2, 64)),
              torch.zeros((2, 3, 1000), dtype=torch.bfloat16)[..., :64],
              wide(torch.bfloat16, 1, 128), torch.zeros((3, 1000), dtype=torch.bfloat16)):
        c = cache()
        tq.tq_kv4_append(c, x, x, None, None, None, None, 0, k_stride=1000, v_stride=1000)
        tq.tq_kv4_decode(c, x, None, x, None, 1, 0.1, q_stride=1000, out_stride=1000)
        tq.tq_kv4_prefill(c, x, None, None, x, None, 0, 1, 0.1, q_stride=1000, out_stride=1000)
        tq.make_rope_rows([dict(x_bf16=x, y_bf16=x, heads=1, x_stride=1000, y_stride=1000)], 64)
    pos = torch.zeros((3, 50), dtype=torch.int32)
    for p, T, stride in ((pos[:, :7], 7, 50), (pos[:, 4:5], 1, 50), (pos[:1, 3:9], 6, 0),
                         (pos[0], 50, 0), (pos, 50, 0), (pos[::2, :2], 2, 100)):
        tq.tq_rope(tq.make_rope_rows([], 64), p, None, [32], T, 64, 64, pos_stride=stride)
    tq.make_kv4_cache(page_table=torch.zeros((4, 20), dtype=torch.int32)[:, :7], max_pages=20)
    tq.make_kv4_cache(pages=torch.zeros((4, 2000), dtype=torch.uint8)[:, :1088], page_stride=2000)


@pytest.mark.parametrize("stride", [0, 64, 128, 999])
def test_views_that_would_be_misread_are_refused(stride):
    """Rows at another distance than the call is told, and elements that do not
    follow one another."""
    def refused(fn, *a, **kw):
        with pytest.raises(tq.TQError) as e:
            fn(*a, **kw)
        assert e.value.name == "TQ_ERR_VALUE" and "view" in str(e.value)

    c, none = cache(), [None] * 4
    for x in (wide(torch.bfloat16, 3, 128), wide(torch.bfloat16, 3, 128, (2, 64)),
              torch.zeros((8, 4, 64), dtype=torch.bfloat16).transpose(0, 1),
              torch.zeros((3, 128), dtype=torch.bfloat16)[:, ::2],
              torch.zeros((1, 64), dtype=torch.bfloat16).expand(3, 64)):
        refused(tq.tq_kv4_append, c, x, None, *none, 0, k_stride=stride)
        refused(tq.tq_kv4_append, c, None, x, *none, 0, v_stride=stride)
        refused(tq.tq_kv4_decode, c, x, *none[:3], 1, 0.1, q_stride=stride)
        refused(tq.tq_kv4_decode, c, None, None, x, None, 1, 0.1, out_stride=stride)
        refused(tq.tq_kv4_prefill, c, x, *none, 0, 1, 0.1, q_stride=stride)
        for n in ("x", "y"):
            refused(tq.make_rope_rows, [{n + "_bf16": x, "heads": 1, n + "_stride": stride}], 64)
    i = torch.zeros((4, 20), dtype=torch.int32)
    refused(tq.make_kv4_cache, page_table=i[:, :7], max_pages=7)
    refused(tq.make_kv4_cache, page_table=i.t(), max_pages=20)
    refused(tq.make_kv4_cache, pages=torch.zeros((4, 2000), dtype=torch.uint8)[:, :1088])
    for p, T in ((i[0, ::2], 10), (i[:, :7], 7), (i[0, :4:2], 2), (i[:1, :4:2], 2)):
        refused(tq.tq_rope, tq.make_rope_rows([], 64), p, None, [32], T, 64, 64)
    for lens in (i[:, 0], i[0, ::3]):
        refused(tq.tq_kv4_append, c, *none, None, lens, 0)
        refused(tq.tq_kv4_append, c, *none, lens, None, 0)
        refused(tq.tq_kv4_decode, c, None, lens, None, None, 1, 0.1)
    refused(tq.tq_kv4_decode, c, None, None, None, torch.zeros(4, 8)[:, :4], 1, 0.1)
    refused(tq.tq_rope, tq.make_rope_rows([], 64), None, torch.zeros(64)[::2], [32], 0, 64, 64)


def test_descriptions_of_another_device_are_refused(monkeypatch):
    """A cache or rows described while another device was the current one."""
    c = cache(pages=t(torch.uint8), page_table=4096)
    rows = tq.make_rope_rows([dict(heads=0, y_f32=t(torch.float32))], 64)
    none = [None] * 6

    def call(c, rows):
        return [lambda: tq.tq_rope(rows, None, None, [32], 0, 64, 64),
                lambda: tq.tq_kv4_append(c, *none, 0),
                lambda: tq.tq_kv4_decode(c, *none[:4], 1, 0.1),
                lambda: tq.tq_kv4_prefill(c, *none[:5], 0, 1, 0.1)]

    for f in call(c, rows):
        f()
    monkeypatch.setattr(tq, "_here", lambda stream: (1, 0))
    for f in call(c, rows):
        with pytest.raises(tq.TQError) as e:
            f()
        assert e.value.name == "TQ_ERR_VALUE" and "device" in str(e.value)
    # addresses as whole numbers, structs filled in by hand: the caller's business
    monkeypatch.setattr(tq, "_device", lambda: 0)
    for f in call(cache(pages=4096, page_table=4096), tq.make_rope_rows([dict(heads=0, x_f32=64)], 64)):
        f()
    for f in call(tq.TqKv4Cache(page_size=16, kv_heads=1, head_dim=64), (tq.TqRopeRows * 1)()):
        f()
