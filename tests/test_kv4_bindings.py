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
