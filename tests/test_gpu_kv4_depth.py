"""Attention over the 4-bit cache where the kernels' loops run deep: several
tiles, items and page batches to a warp in single-token calls, more key tiles to
a CTA than it has stages, scale slots and barrier phases in prompts. Against 64
bits, computed on the GPU by plain products.

Tolerances as tests/_kv4.py derives them, with the sums counted for these lengths.
Single tokens: a value passes through at most 16 tiles of a warp, 64 products
each in the matrix unit (2^-23 an addition), 16 warps and 148 SMs one after
another, fewer than 300 additions: 2^-14 of A, within the 2^-12 that stand there for
sums and exponentials. Prompts: at most 16,400 keys, 16 to an addition, in up to 32
parts: 1060 additions of 2^-23 in the matrix unit, 2^-12.9 of A, and what the sum of
weights loses (1 / 8 of that many additions, 2^-24 each, 2^-17): within 2^-12 as well.
The logarithm of a sum of weights moves by its relative error: fewer than 250
additions of 2^-24 one after another (8 a tile and lane, then lanes, warps, SMs),
2^-16, for the 2^-18 of short sequences."""
import math

import numpy as np
import pytest
import torch

import ternary_absmax_int8_b200 as tq

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Deep:
    """A cache on the GPU: random codes, scales that grow along a sequence (so do
    the running maxima), stay or shrink, NaN scales in slots without a token, pages
    in any order."""

    def __init__(self, seed, lens, hk, D, ps):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.hk, self.D, self.ps = lens, hk, D, ps
        need = [-(-n // ps) for n in lens]
        total = sum(need) + 2
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(lens), max(need)), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
        scale = torch.full((total, hk, 2, ps), math.nan, device=DEV)
        at = 0
        for b, (n, m) in enumerate(zip(lens, need)):
            mine = order[at:at + m]
            self.table[b, :m] = mine
            j = torch.arange(m * ps, device=DEV).view(m, 1, 1, ps)
            s = torch.exp(0.4 * torch.randn((m, hk, 2, ps), generator=g, device=DEV))
            s *= 0.2 + (0.1, 0, -0.1)[b % 3] * (2 * j / max(n, 1) - 1)
            scale[mine.long()] = torch.where(j < n, s, math.nan)
            at += m
        codes = torch.randint(1, 16, (total, hk, 2, ps, D), generator=g, device=DEV,
                              dtype=torch.uint8)
        packed = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(total, hk, -1)
        self.codes, self.scale = codes, scale.bfloat16()
        raw = self.scale.view(torch.uint8).reshape(total, hk, -1)
        self.pages = torch.cat([packed, raw], -1).reshape(total, -1).contiguous()
        assert self.pages.shape[1] == tq.tq_kv4_page_bytes(ps, hk, D)
        self.cache = tq.make_kv4_cache(pages=self.pages, page_table=self.table, num_pages=total,
                                       page_size=ps, kv_heads=hk, head_dim=D, batch=len(lens),
                                       max_pages=max(need))

    def rows(self, b, h, which):
        n = self.lens[b]
        mine = self.table[b, :-(-n // self.ps)].long()
        c = self.codes[mine, h, which].reshape(-1, self.D)[:n].double() - 8
        return c * self.scale[mine, h, which].reshape(-1)[:n].double().unsqueeze(1)


def check(deep, q, out, lse, start, n, window):
    """Every row of every sequence against softmax in 64 bits."""
    T, hq, D = q.shape
    rep, scale = hq // deep.hk, D ** -0.5
    x = q.double()
    for b, L in enumerate(deep.lens):
        if n[b] == 0:
            continue
        rows = slice(start[b], start[b] + n[b])
        p = torch.arange(L - n[b], L, device=DEV).repeat_interleave(rep).unsqueeze(1)
        for h in range(deep.hk):
            heads = slice(h * rep, (h + 1) * rep)
            xx = x[rows, heads].reshape(-1, D)
            k, v = deep.rows(b, h, 0), deep.rows(b, h, 1)
            z = xx @ k.t() * scale
            if n[b] > 1 or window:
                j = torch.arange(L, device=DEV)
                z.masked_fill_((j > p) | (j <= p - (window or L + 1)), -math.inf)
            rlse = torch.logsumexp(z, -1)
            w = z.sub_(rlse.unsqueeze(1)).exp_()
            ref, A = w @ v, w @ v.abs()
            del z, w
            size = scale * xx.abs().amax(-1) * k.abs().sum(-1).max()  # (above any score's)
            dz = 2.0 ** -25 * size + 2.0 ** -20 * scale * (xx.abs() @ k.abs().t()).amax(-1)
            tol = (2.0 ** -8 * ref.abs() + A * (2.0 ** -8 + 2.0 ** -12 + 2 * dz.unsqueeze(1))
                   + 2.0 ** -39 * L * v.abs().max() + 1e-30)
            got = out[rows, heads].double().reshape(-1, D)
            off = (got - ref).abs() / tol
            assert (off <= 1).all(), f"sequence {b}, head {h}: {off.max().item():.2f} tolerances"
            ltol = dz + 2.0 ** -16 + 2.0 ** -22 * rlse.abs()
            off = (lse[rows, heads].double().reshape(-1) - rlse).abs() / ltol
            assert (off <= 1).all(), f"sequence {b}, head {h}: lse {off.max().item():.2f} tolerances"
    assert tq.tq_device_error() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def buffers(seed, T, hq, D, spread):
    """Queries of which all keys count (spread 2: the logarithm of the sum tells
    what is missing), or a few (12: the values tell which), and what is written."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    q = (spread * torch.randn((T, hq, D), generator=g, device=DEV)).bfloat16()
    return q, torch.full_like(q, 7.0), torch.full((T, hq), 7.0, device=DEV)


def lengths(kind, rng):
    if kind == "ragged":  # page batches, ring and maxima within a warp; joins over several SMs
        lens = rng.integers(1000, 8192, 25).tolist()
        lens[11] = 131099
        return lens, 2
    if kind == "many":    # shares of several items, more sequences than threads
        lens = rng.integers(60, 400, 420).tolist()
        lens[7:300:40] = [0] * len(lens[7:300:40])
        return lens, 5
    return [300007], 1    # one sequence over all SMs


@pytest.mark.parametrize("kind", ["ragged", "many", "one"])
@pytest.mark.parametrize("D,rep,ps,window", [(128, 4, 64, 0), (128, 8, 16, 0), (128, 16, 128, 0),
                                             (64, 3, 128, 0), (64, 7, 16, 3001), (64, 16, 32, 0),
                                             (128, 1, 32, 200)])
def test_deep_decode(cuda_device, kind, D, rep, ps, window):
    rng = np.random.default_rng(40)
    lens, hk = lengths(kind, rng)
    if not window:
        # 64 keys a tile, at most 16 warps on each SM: two tiles a warp and more
        warps = 16 * torch.cuda.get_device_properties(0).multi_processor_count
        assert hk * sum(-(-n // 64) for n in lens) > (1.9 if kind == "one" else 2) * warps
    deep = Deep(D + rep, lens, hk, D, ps)
    size = tq.tq_kv4_decode_workspace(deep.cache, hk * rep)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    empty = i32(lens) == 0
    for seed, spread in enumerate((2, 12) if kind == "many" else (2, 12, 12, 12)):
        q, out, lse = buffers(seed, len(lens), hk * rep, D, spread)
        tq.tq_kv4_decode(deep.cache, q, i32(lens), out, lse, hk * rep, D ** -0.5, window, ws, size)
        torch.cuda.synchronize()
        assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
        check(deep, q, out, lse, list(range(len(lens))), [int(n > 0) for n in lens], window)


@pytest.mark.parametrize("D,rep,hk,ps,lens,n,window,parts", [
    (128, 4, 2, 64, [2500], [2500], 0, False),            # 20 key tiles a CTA
    (64, 4, 2, 16, [2500], [2500], 0, False),
    (128, 3, 2, 128, [2000, 40, 2100], [2000, 40, 2100], 700, False),
    (64, 8, 1, 32, [2111, 900], [2111, 900], 0, False),
    (128, 4, 2, 64, [16300, 9001], [300, 257], 0, True),  # 18 tiles a part
    (64, 4, 2, 128, [16300, 9001], [300, 257], 0, True),
    (128, 2, 1, 16, [16390], [77], 9000, True),
    (64, 16, 1, 32, [12345, 0, 16390], [33, 0, 1], 0, True),
])
def test_deep_prefill(cuda_device, D, rep, hk, ps, lens, n, window, parts):
    deep = Deep(D + rep, lens, hk, D, ps)
    T, hq = sum(n), hk * rep
    size = tq.tq_kv4_prefill_workspace(deep.cache, hq, T)
    assert (size > 0) == parts
    ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device=DEV)
    start = [0] + np.cumsum(n).tolist()
    for spread in (2, 12):
        q, out, lse = buffers(D + rep, T, hq, D, spread)
        tq.tq_kv4_prefill(deep.cache, q, i32(start), i32(lens), out, lse, T, hq, D ** -0.5, window,
                          ws, size)
        torch.cuda.synchronize()
        check(deep, q, out, lse, start, n, window)
