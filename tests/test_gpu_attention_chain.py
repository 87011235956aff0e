"""A decoder layer's attention half as it is used: projections, rotary
positions, cache, attention, sub-layer norm and the output projection, for a
prompt and then for single tokens, against the same steps in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
import ternary_absmax_int8_b200 as tq
from tests._gpu import dev, host_pack
from tests._kv4 import bf16_bits, bf16_round, quantise

pytestmark = pytest.mark.gpu

HQ, HK, D, HID, PS = 8, 2, 64, 512, 16
EPS = 1e-5
SCALE = D ** -0.5


def layer(rng):
    shapes = dict(q=(HQ * D, HID), k=(HK * D, HID), v=(HK * D, HID), o=(HID, HQ * D))
    w = {n: rng.integers(-1, 2, s).astype(np.int8) for n, s in shapes.items()}
    return w, {n: np.float32(rng.uniform(0.02, 0.05)) for n in shapes}


class Gpu:
    """The library's side, with a cache that grows over the calls."""

    def __init__(self, w, ws, gain, inv, batch, max_pages):
        self.w = {n: dev(host_pack(x)) for n, x in w.items()}
        self.ws, self.gain, self.inv = ws, dev(gain), dev(inv)
        self.table = torch.randperm(batch * max_pages, dtype=torch.int32).view(batch, max_pages).cuda()
        self.pages = torch.zeros(batch * max_pages, tq.tq_kv4_page_bytes(PS, HK, D),
                                 dtype=torch.uint8, device="cuda")
        self.cache = tq.make_kv4_cache(pages=self.pages, page_table=self.table,
                                       num_pages=batch * max_pages, page_size=PS, kv_heads=HK,
                                       head_dim=D, batch=batch, max_pages=max_pages)

    def linear(self, n, xq, xs, xsum, M):
        N, K = self.w[n].shape[0] * 4, self.w[n].shape[1]
        y = torch.empty((M, N), device="cuda")
        call = tq.tq_gemv if M <= 24 else tq.tq_gemm_prefill
        call(self.w[n], float(self.ws[n]), xq, xs, xsum, y, None, M, N, K)
        return y

    def codes(self, M, K):
        return (torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                torch.empty(M, dtype=torch.int32, device="cuda"))

    def __call__(self, x, start, lens, pos):
        M = x.shape[0]
        c = self.codes(M, HID)
        tq.tq_quantize_act(dev(bf16_bits(x).reshape(x.shape).view(np.int16)), *c, M, 0, HID)
        q, k, v = (self.linear(n, *c, M) for n in "qkv")
        qr = torch.empty((M, HQ * D), dtype=torch.bfloat16, device="cuda")
        tq.tq_rope(tq.make_rope_rows([dict(x_f32=q, y_bf16=qr, heads=HQ),
                                      dict(x_f32=k, y_f32=k, heads=HK)], D),
                   dev(pos.astype(np.int32)), self.inv, [D // 2], M, D, D)
        start_g, lens_g = dev(np.int32(start)), dev(np.int32(lens))
        tq.tq_kv4_append(self.cache, None, None, k, v, start_g, lens_g, M)
        out = torch.empty_like(qr)
        if M == len(lens):
            size = tq.tq_kv4_decode_workspace(self.cache, HQ)
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            tq.tq_kv4_decode(self.cache, qr, lens_g, out, None, HQ, SCALE, 0, ws, size)
        else:
            size = tq.tq_kv4_prefill_workspace(self.cache, HQ, M)
            ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
            tq.tq_kv4_prefill(self.cache, qr, start_g, lens_g, out, None, M, HQ, SCALE, 0, ws, size)
        c = self.codes(M, HQ * D)
        tq.tq_rmsnorm_quantize(out, None, self.gain, EPS, *c, M, HQ * D)
        y = self.linear("o", *c, M)
        torch.cuda.synchronize()
        return (q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), qr.float().cpu().numpy(),
                out.float().cpu().numpy(), c, y.cpu().numpy())


def turn(x, pos, inv):
    a = pos.reshape(-1, 1).astype(np.float64) * inv.astype(np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    u, v = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([u * c - v * s, v * c + u * s], -1)


def test_prompt_then_single_tokens(cuda_device):
    """Each step is held to the library's own inputs to it (the projections are
    exact, a code of a 64-bit recomputation could fall on the other side of a
    half): rotary values to 2^-21 of their pair, attention to the tolerance that
    tests/_kv4.py derives, the norm's codes to one step."""
    rng = np.random.default_rng(3)
    B, max_pages = 3, 8
    w, ws = layer(rng)
    inv = (1.0 / 10000.0 ** (np.arange(0, D, 2) / D)).astype(np.float32)
    gain = rng.uniform(0.5, 1.5, HQ * D).astype(np.float32)
    gpu = Gpu(w, ws, gain, inv, B, max_pages)
    keys, values = [np.zeros((0, HK, D)) for _ in range(B)], [np.zeros((0, HK, D)) for _ in range(B)]
    lens = np.zeros(B, np.int64)
    for n in ([37, 5, 64], [1, 1, 1], [1, 1, 1], [17, 16, 1], [1, 1, 1]):
        lens = lens + n
        start = np.concatenate([[0], np.cumsum(n)])
        pos = np.concatenate([np.arange(l - m, l) for l, m in zip(lens, n)])
        x = bf16_round(rng.standard_normal((sum(n), HID)).astype(np.float32)).reshape(-1, HID)
        q, k, v, qr, out, (xq, xs, _), y = gpu(x, start, lens, pos)
        M = len(x)
        q0 = oracle.forward(oracle.pack(w["q"]), HQ * D, ws["q"], bf16_bits(x).reshape(x.shape))[4]
        assert np.allclose(q, q0, rtol=1e-5, atol=0)
        t = turn(q.reshape(M, HQ, D).astype(np.float64), pos, inv)
        assert (np.abs(qr.reshape(t.shape) - t) <= 2.0 ** -8 * np.abs(t)
                + 2.0 ** -20 * np.abs(q).max()).all()
        qr = qr.reshape(M, HQ, D).astype(np.float64)
        for b in range(B):
            rows = slice(start[b], start[b + 1])
            for kept, new in ((keys, k), (values, v)):
                c, s = quantise(new.reshape(M, HK, D)[rows])
                kept[b] = np.concatenate([kept[b], c * s.astype(np.float64)[..., None]])
            for i in range(start[b], start[b + 1]):
                L = pos[i] + 1
                for h in range(HQ):
                    kk, vv = keys[b][:L, h // (HQ // HK)], values[b][:L, h // (HQ // HK)]
                    z = SCALE * (kk @ qr[i, h])
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    ref, A = p @ vv, p @ np.abs(vv)
                    off = np.abs(out[i, h * D:(h + 1) * D] - ref)
                    assert (off <= 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -8 + 2.0 ** -11)
                            + 2.0 ** -39 * L * np.abs(vv).max()).all()
        o = out.astype(np.float64)
        g = o / np.sqrt((o * o).mean(-1, keepdims=True) + EPS) * gain
        assert (np.abs(g / np.abs(g).max(-1, keepdims=True) * 127 - xq.cpu().numpy()) <= 0.501).all()
        acc = xq.cpu().numpy().astype(np.int64) @ w["o"].T.astype(np.int64)
        assert np.allclose(y, acc * (np.float64(ws["o"]) * xs.double().cpu().numpy()[:, None]),
                           rtol=1e-5, atol=0)
    assert tq.tq_device_error() == 0


def test_decode_step_replayed_from_a_graph(cuda_device):
    """Rotary, append and attention of single tokens in one captured graph; the
    sequences grow by device-side lengths and positions between replays."""
    rng = np.random.default_rng(4)
    B, max_pages, steps = 4, 4, 40
    table = torch.randperm(B * max_pages, dtype=torch.int32).view(B, max_pages).cuda()
    pages = torch.zeros(B * max_pages, tq.tq_kv4_page_bytes(PS, HK, D), dtype=torch.uint8,
                        device="cuda")
    cache = tq.make_kv4_cache(pages=pages, page_table=table, num_pages=B * max_pages, page_size=PS,
                              kv_heads=HK, head_dim=D, batch=B, max_pages=max_pages)
    inv_np = (1.0 / 10000.0 ** (np.arange(0, D, 2) / D)).astype(np.float32)
    inv = dev(inv_np)
    q, k, v = (torch.empty((B, h * D), device="cuda") for h in (HQ, HK, HK))
    qr, out = (torch.empty((B, HQ * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = torch.zeros((1, B), dtype=torch.int32, device="cuda")
    rows = tq.make_rope_rows([dict(x_f32=q, y_bf16=qr, heads=HQ), dict(x_f32=k, y_f32=k, heads=HK)],
                             D)
    size = tq.tq_kv4_decode_workspace(cache, HQ)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos.copy_(lens.view(1, B))
        lens.add_(1)
        tq.tq_rope(rows, pos, inv, [D // 2], B, D, D)
        tq.tq_kv4_append(cache, None, None, k, v, None, lens, B)
        tq.tq_kv4_decode(cache, qr, lens, out, None, HQ, SCALE, 0, ws, size)
    lens.zero_()
    keys, values = [], []
    for step in range(steps):
        x = [rng.standard_normal((B, h * D)).astype(np.float32) for h in (HQ, HK, HK)]
        for t, a in zip((q, k, v), x):
            t.copy_(torch.from_numpy(a))
        graph.replay()
        torch.cuda.synchronize()
        for kept, new in ((keys, k), (values, v)):  # k holds the turned keys now
            c, s = quantise(new.cpu().numpy().reshape(B, HK, D))
            kept.append(c * s.astype(np.float64)[..., None])
        assert (lens == step + 1).all()
        K, V = np.stack(keys, 1), np.stack(values, 1)  # [B, step + 1, HK, D]
        Q = qr.double().cpu().numpy().reshape(B, HQ, D)
        t = turn(x[0].reshape(B, HQ, D).astype(np.float64), np.full(B, step), inv_np)
        assert (np.abs(Q - t) <= 2.0 ** -8 * np.abs(t) + 2.0 ** -20 * np.abs(x[0]).max()).all()
        kk, vv = (np.repeat(a, HQ // HK, 2) for a in (K, V))
        z = SCALE * np.einsum("bhd,bjhd->bhj", Q, kk)
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        ref, A = np.einsum("bhj,bjhd->bhd", p, vv), np.einsum("bhj,bjhd->bhd", p, np.abs(vv))
        off = np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref)
        assert (off <= 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -8 + 2.0 ** -11)
                + 2.0 ** -39 * (step + 1) * np.abs(vv).max()).all()
