"""tq_rope against the formula in 64 bits.

Tolerance per value: the angle's reduced part of a turn, |r| <= 1/2, is
rounded to fp32 (2^-25 turns at most, 2 pi 2^-25 < 2^-22 rad), cosine and sine
are off by 2^-23 at most, and the two products and their sum round three
times (2^-24 each): with u, v the pair, |u| + |v| times 2^-21 in all. Storing
bf16 adds half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import ternary_absmax_int8_b200 as tq
from tests._kv4 import bf16_round

pytestmark = pytest.mark.gpu


def reference(x, pos, inv, sections, rot, inter):
    x = x.astype(np.float64)
    axis = np.repeat(np.arange(len(sections)), sections)
    turns = pos[axis].T.astype(np.float64) * inv.astype(np.float64)  # [T, rot/2]
    c, s = np.cos(turns)[:, None], np.sin(turns)[:, None]
    y, size = x.copy(), np.zeros(x.shape)
    i = slice(0, rot, 2) if inter else slice(0, rot // 2)
    j = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, size * 2.0 ** -21


def freq(rot):
    return (1.0 / 500000.0 ** (np.arange(0, rot, 2) / max(1, rot))).astype(np.float32)


@pytest.mark.parametrize("T,hq,hk,D,rot,sections,inter,src,dst,far", [
    (1, 20, 5, 128, 128, [64], False, "f32", "bf16", 0),
    (7, 20, 5, 128, 128, [64], False, "f32", "bf16", 131072),
    (700, 4, 1, 128, 128, [16, 24, 24], False, "bf16", "bf16", 9000),
    (593, 3, 2, 64, 32, [8, 8], True, "f32", "f32", 1000000),
    (33, 1, 1, 80, 48, [10, 0, 14], True, "bf16", "f32", 2 ** 31 - 50),
    (5, 2, 0, 24, 0, [0], False, "f32", "bf16", 10),
    (9, 2, 2, 256, 256, [1, 2, 3, 122], False, "bf16", "f32", 77777),
    (3, 1, 70, 104, 80, [40], False, "f32", "f32", 5),
])
def test_rope(cuda_device, T, hq, hk, D, rot, sections, inter, src, dst, far):
    rng = np.random.default_rng(T)
    inv = freq(rot)
    pos = (far - rng.integers(0, far + 1, (len(sections), T)) // 3).astype(np.int32)
    rows, refs, outs = [], [], []
    for heads in (hq, hk):
        x = rng.standard_normal((T, heads, D)).astype(np.float32)
        if src == "bf16":
            x = bf16_round(x).reshape(x.shape)
        g = torch.from_numpy(x).cuda()
        g = g if src == "f32" else g.bfloat16()
        y = torch.full((T, heads, D), 9.0, device="cuda",
                       dtype=torch.float32 if dst == "f32" else torch.bfloat16)
        rows.append({"x_" + src: g, "y_" + dst: y, "heads": heads})
        refs.append(reference(x, pos, inv, sections, rot, inter))
        outs.append(y)
    tq.tq_rope(tq.make_rope_rows(rows, D), torch.from_numpy(pos).cuda(),
               torch.from_numpy(inv).cuda(), sections, T, D, rot,
               flags=tq.TQ_ROPE_INTERLEAVED if inter else 0)
    torch.cuda.synchronize()
    for y, (ref, tol) in zip(outs, refs):
        off = np.abs(y.double().cpu().numpy() - ref)
        assert (off <= tol + (2.0 ** -8 * (np.abs(ref) + tol) if dst == "bf16" else 0)).all()


def test_rope_in_place_strided_and_captured(cuda_device):
    """q and k as columns of one fused projection's rows, turned in place, the
    launch replayed at new positions."""
    T, hq, hk, D = 6, 4, 2, 128
    rng = np.random.default_rng(1)
    width = (hq + 2 * hk) * D
    x = rng.standard_normal((T, width)).astype(np.float32)
    g = torch.from_numpy(x).cuda()
    inv, pos = freq(D), np.arange(50, 50 + T, dtype=np.int32)[None]
    pos_g, inv_g = torch.from_numpy(pos).cuda(), torch.from_numpy(inv).cuda()
    rows = tq.make_rope_rows(
        [dict(x_f32=g.data_ptr() + 4 * o, y_f32=g.data_ptr() + 4 * o, heads=h, x_stride=width,
              y_stride=width) for o, h in ((0, hq), (hq * D, hk))], D)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tq.tq_rope(rows, pos_g, inv_g, [D // 2], T, D, D)
    for shift in (0, 1000):
        g.copy_(torch.from_numpy(x))
        pos_g.copy_(torch.from_numpy(pos + shift))
        graph.replay()
        torch.cuda.synchronize()
        got = g.cpu().numpy()
        ref, tol = reference(x[:, :(hq + hk) * D].reshape(T, hq + hk, D), pos + shift, inv,
                             [D // 2], D, False)
        assert (np.abs(got[:, :(hq + hk) * D].reshape(ref.shape) - ref) <= tol).all()
        assert np.array_equal(got[:, (hq + hk) * D:], x[:, (hq + hk) * D:])


def test_rope_infinite_and_nan_values_stay_in_their_pair(cuda_device):
    T, D = 2, 64
    x = np.ones((T, 1, D), np.float32)
    x[0, 0, 3], x[1, 0, 40] = np.nan, np.inf
    g = torch.from_numpy(x).cuda()
    y = torch.empty_like(g)
    tq.tq_rope(tq.make_rope_rows([dict(x_f32=g, y_f32=y, heads=1)], D),
               torch.full((1, T), 12, dtype=torch.int32, device="cuda"),
               torch.from_numpy(freq(D)).cuda(), [D // 2], T, D, D)
    bad = ~np.isfinite(y.cpu().numpy())
    want = np.zeros_like(bad)
    want[0, 0, [3, 35]] = want[1, 0, [8, 40]] = True
    assert np.array_equal(bad, want)
