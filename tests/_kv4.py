"""Plain 64-bit implementations of the rotary positions, the 4-bit key/value
cache and the attention over it, and helpers that run the library on the same
inputs. Nothing here shares code with the library.

Tolerance of attention outputs, per value. With p the softmax weights,
A = sum_j p_j |v_j| and out = sum_j p_j v_j:
  - storing bf16 moves out by at most 2^-8 |out| (half a step);
  - a weight times its value's scale is rounded once to bf16 on its way into
    the matrix units: 2^-8 of itself, in sum 2^-8 A. Single tokens round to
    fp16 in units of 2^-14 of the largest value scale S near it: 2^-11 of
    itself, or where that is smaller than fp16's last step of 2^-24, half of
    it: 2^-25 2^-14 S = 2^-39 S. With codes up to 7, n keys move out by
    7 n 2^-39 S = n 2^-39 max |v| (seen where one key takes all and its code is 0);
  - a query value may be held in fp16 against its row's largest: bf16's 8 bits
    fit, what falls below fp16's range moves by 2^-25 of the row's largest. The
    scores move by at most dz, so every weight by a factor within exp(+-2 dz)
    and out by 2 dz A;
  - fp32 sums over at most a few thousand keys and the exponential's
    approximation: 2^-12 A together.
"""
import numpy as np
import torch

import ternary_absmax_int8_b200 as tq


def bf16_round(x):
    """fp32 array -> the nearest bf16 values (ties to even), as fp32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16
    return (b.astype(np.uint32) << 16).view(np.float32)


def bf16_bits(x):
    return (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def quantise(x):
    """Rows [..., D] -> codes int (-7..7), scales fp32 (bf16 values)."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    amax = np.where(bad, np.float32(0), amax)
    s = bf16_round((amax / np.float32(7)).astype(np.float32)).reshape(amax.shape)
    d = np.where(s > 0, s, 1).astype(np.float64)[..., None]
    c = np.rint(np.where(bad[..., None], 0, x).astype(np.float64) / d) * (s > 0)[..., None]
    c = np.clip(c, -7, 7)  # (a subnormal s may be far below absmax / 7)
    return c.astype(np.int64), np.where(bad, np.float32(np.nan), s)


class Cache:
    """A cache on the host, as numbers: codes [pages, 2, heads, ps, D] and
    scales [pages, 2, heads, ps] (0 keys, 1 values), and its page table."""

    def __init__(self, rng, lens, hk, D, ps, spare=3, max_pages=None, junk=True):
        self.hk, self.D, self.ps, self.lens = hk, D, ps, list(lens)
        need = [-(-max(0, n) // ps) for n in lens]
        self.max_pages = max_pages or max(1, max(need, default=1))
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        # entries behind a sequence's pages are never to be followed
        self.table = np.full((len(lens), self.max_pages), 2 ** 31 - 1 if junk else 0, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, 2, hk, ps)
        # unwritten slots: any nibble, scales NaN (a leak shows)
        self.codes = rng.integers(-8, 8, shape + (D,))
        self.scales = np.full(shape, np.nan if junk else 0, np.float32)
        for b, n in enumerate(lens):
            for j in range(max(0, n)):
                pg, slot = self.table[b, j // ps], j % ps
                x = rng.standard_normal((2, hk, D)) * np.exp(0.5 * rng.standard_normal((2, hk, 1)))
                self.codes[pg, :, :, slot], self.scales[pg, :, :, slot] = quantise(x)

    def bytes(self):
        n = (self.codes + 8).astype(np.uint8)
        n = n[..., 0::2] | (n[..., 1::2] << 4)  # [pages, 2, hk, ps, D/2]
        c = n.transpose(0, 2, 1, 3, 4).reshape(self.num_pages, self.hk, -1)
        s = bf16_bits(self.scales).reshape(self.scales.shape).transpose(0, 2, 1, 3)
        s = np.ascontiguousarray(s).reshape(self.num_pages, self.hk, -1).view(np.uint8)
        return np.concatenate([c, s], -1).reshape(self.num_pages, -1)

    def rows(self, b, which):
        """Keys (0) or values (1) of sequence b, [heads, len, D], fp64."""
        n = min(max(0, self.lens[b]), self.max_pages * self.ps)
        j = np.arange(n)
        pg, slot = self.table[b, j // self.ps], j % self.ps
        v = self.codes[pg, which, :, slot].astype(np.float64)
        return (v * self.scales[pg, which, :, slot].astype(np.float64)[..., None]).transpose(1, 0, 2)

    def on_gpu(self, lead_pages=0, pad_bytes=0):
        """(tq cache, tensors to keep): pages behind `lead_pages` others, each
        padded by `pad_bytes`."""
        raw = self.bytes()
        size = raw.shape[1]
        pages = torch.empty((lead_pages + self.num_pages, size + pad_bytes), dtype=torch.uint8,
                            device="cuda")
        pages[lead_pages:] = 255
        pages[lead_pages:, :size] = torch.from_numpy(raw).cuda()
        t = self.table.astype(np.int64)
        t = np.where((t >= 0) & (t < self.num_pages), t + lead_pages, t).astype(np.int32)
        table = torch.from_numpy(t).cuda()
        cache = tq.make_kv4_cache(pages=pages, page_table=table,
                                  num_pages=lead_pages + self.num_pages, page_size=self.ps,
                                  kv_heads=self.hk, head_dim=self.D, batch=len(self.lens),
                                  max_pages=self.max_pages,
                                  page_stride=size + pad_bytes if pad_bytes else 0)
        return cache, (pages, table)


def attention(cache, q, n, scale, window=0):
    """(out, lse, tolerance of out, tolerance of lse) for the queries q
    [tokens, heads, D] of sequences with n[b] new tokens each."""
    T, hq, D = q.shape
    rep = hq // cache.hk
    q = q.astype(np.float64)
    out, lse = np.zeros((T, hq, D)), np.full((T, hq), -np.inf)
    tol, ltol = np.zeros((T, hq, D)), np.zeros((T, hq))
    t = 0
    for b, nb in enumerate(n):
        k, v = cache.rows(b, 0), cache.rows(b, 1)
        L = k.shape[1]
        for i in range(nb):
            p = cache.lens[b] - nb + i
            lo, hi = (max(0, p - window + 1) if window else 0), min(p + 1, L)
            if hi > lo:
                for h in range(hq):
                    kk, vv, x = k[h // rep, lo:hi], v[h // rep, lo:hi], q[t, h]
                    z = scale * (kk @ x)
                    with np.errstate(invalid="ignore"):
                        m = np.max(z)
                        w = np.exp(z - m)
                        s = w.sum()
                        w = w / s
                        A = w @ np.abs(vv)
                        out[t, h] = w @ vv
                        lse[t, h] = m + np.log(s)
                        size = scale * (np.abs(kk) @ np.abs(x)).max()
                        dq = 2.0 ** -25 * np.abs(x).max()
                        dz = scale * dq * np.abs(kk).sum(-1).max() + 2.0 ** -20 * size
                        tol[t, h] = (2.0 ** -8 * np.abs(out[t, h])
                                     + A * (2.0 ** -8 + 2 * dz + 2.0 ** -12)
                                     + 2.0 ** -39 * len(vv) * np.abs(vv).max() + 1e-30)
                        ltol[t, h] = dz + 2.0 ** -18 + 2.0 ** -22 * abs(lse[t, h])
            t += 1
    return out, lse, tol, ltol


def queries(rng, T, hq, D, spread=1.0):
    x = (spread * rng.standard_normal((T, hq, D))).astype(np.float32)
    return bf16_round(x).reshape(x.shape)


def to_gpu(x, f32, row=0):
    """Rows [T, ...] on the GPU, in rows of `row` values where that is more."""
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    t = t if f32 else t.bfloat16()
    flat = t.reshape(t.shape[0], -1)
    if row > flat.shape[1]:
        wide = torch.full((flat.shape[0], row), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :flat.shape[1]] = flat
        return wide
    return flat


def run_attention(cache, keep, q, lens, n, scale, window=0, decode=None, tail=2, q_row=0,
                  out_row=0, want_lse=True, stream=None):
    """The library's (out fp64, lse) [tokens, heads(, D)]; checks that `tail`
    rows behind the last sequence keep what they held."""
    T, hq, D = q.shape
    decode = all(x == 1 for x in n) if decode is None else decode
    tail = 0 if decode else tail
    qg = to_gpu(np.concatenate([q, np.full((tail, hq, D), np.nan, np.float32)]), False,
                q_row)
    width = max(hq * D, out_row)
    out = torch.full((T + tail, width), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + tail, hq), 7.0, device="cuda")
    lens_g = torch.tensor(list(lens), dtype=torch.int32, device="cuda")
    start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    kw = dict(q_stride=q_row if q_row > hq * D else 0, out_stride=out_row if out_row > hq * D else 0)
    if decode:
        size = tq.tq_kv4_decode_workspace(cache, hq)
        ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device="cuda")
        tq.tq_kv4_decode(cache, qg, lens_g, out, lse if want_lse else None, hq, scale, window, ws,
                         size, stream=stream, **kw)
    else:
        size = tq.tq_kv4_prefill_workspace(cache, hq, T + tail)
        ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device="cuda")
        tq.tq_kv4_prefill(cache, qg, start, lens_g, out, lse if want_lse else None, T + tail, hq,
                          scale, window, ws, size, stream=stream, **kw)
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (lse[T:] == 7).all(), "rows behind the last sequence changed"
    assert (out[:, hq * D:] == 7).all(), "values behind a row changed"
    if not want_lse:
        assert (lse == 7).all()
    return (out[:T, :hq * D].double().cpu().numpy().reshape(T, hq, D), lse[:T].double().cpu().numpy())


def assert_attention(got, ref):
    (out, lse), (rout, rlse, tol, ltol) = got, ref
    nan = np.isnan(rout)
    assert np.array_equal(np.isnan(out), nan), "NaN in other places"
    off = np.abs(out - rout)[~nan]
    assert (off <= tol[~nan]).all(), f"off by {np.max(off / tol[~nan]):.2f} tolerances"
    fin = np.isfinite(rlse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rlse)) and np.isfinite(lse[fin]).all()
    off = np.abs(lse[fin] - rlse[fin])
    assert (off <= ltol[fin]).all(), f"lse off by {np.max(off / ltol[fin]):.2f} tolerances"
