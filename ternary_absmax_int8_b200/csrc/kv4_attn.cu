// kv4_attn.cu -- attention over the 4-bit cache, the plain kernel: one warp
// per (token, query head), 32 keys at a time, running maximum and sum.
#include "kv4_common.cuh"
#include "quant_core.cuh"

namespace tq {

namespace {

template <int D>
__global__ void __launch_bounds__(128) kv4_attn_kernel(const __grid_constant__ Kv4View c,
                                                       const __grid_constant__ Kv4Query q,
                                                       const int32_t *tok_start,
                                                       const int32_t *lens, int T)
{
    __shared__ float sq[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 4 + warp;
    if (item >= (long long)T * q.q_heads)
        return;
    const int t = int(item / q.q_heads), h = int(item - (long long)t * q.q_heads);
    int b = t, behind = 1;
    if (tok_start) {
        int lo = 0, hi = c.batch;
        if (t < tok_start[0] || t >= tok_start[hi])
            return;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            (tok_start[mid] <= t ? lo : hi) = mid;
        }
        b = lo;
        behind = tok_start[lo + 1] - t;
    }
    for (int d = lane; d < D; d += 32) {
        const long long at = t * q.q_stride + h * D + d;
        sq[warp][d] = __uint_as_float(uint32_t(q.q[at]) << 16);
    }
    __syncwarp();
    const int end = kv4_len(c, lens, b) - behind + 1;  // keys 0 .. end - 1 are seen
    const int begin = q.window > 0 ? max(0, end - q.window) : 0;
    const int kvh = h / (q.q_heads / c.kv_heads);
    const int ps = c.page_size();
    float m = -INFINITY, l = 0.0f, o[D / 32] = {};
    for (int j0 = begin; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY, vs = 0.0f;
        const uint8_t *vrow = nullptr;
        if (j < end) {
            const uint8_t *page = kv4_page(c, b, j >> c.lg_ps);
            if (page) {
                const uint8_t *blk = page + kvh * c.head_bytes<D>();
                const int slot = j & (ps - 1);
                const uint16_t *sc = reinterpret_cast<const uint16_t *>(blk + (long long)ps * D);
                const uint8_t *kr = blk + slot * (D / 2);
                float dot = 0.0f;
                for (int i = 0; i < D / 2; ++i)
                    dot += sq[warp][2 * i] * float(int(kr[i] & 15) - 8) +
                           sq[warp][2 * i + 1] * float(int(kr[i] >> 4) - 8);
                s = dot * __uint_as_float(uint32_t(sc[slot]) << 16) * q.scale;
                vs = __uint_as_float(uint32_t(sc[ps + slot]) << 16);
                vrow = kr + ps * (D / 2);
            }
        }
        float mx = s;
        for (int x = 16; x > 0; x >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m, mx);
        const float mr = mn == -INFINITY ? 0.0f : mn;
        const float alpha = __expf(m - mr);
        const float pr = vrow ? __expf(s - mr) : 0.0f;
        m = mn;
        l = l * alpha + pr;
        for (int i = 0; i < D / 32; ++i)
            o[i] *= alpha;
        for (int x = 0; x < 32; ++x) {
            const float w = __shfl_sync(0xffffffffu, pr * vs, x);
            const uint8_t *vr = reinterpret_cast<const uint8_t *>(
                __shfl_sync(0xffffffffu, (unsigned long long)vrow, x));
            if (vr)
                for (int i = 0; i < D / 32; ++i) {
                    const int d = lane * (D / 32) + i;
                    const int byte = vr[d >> 1];
                    o[i] += w * float(((d & 1) ? byte >> 4 : byte & 15) - 8);
                }
        }
    }
    for (int x = 16; x > 0; x >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, x);
    const bool none = m == -INFINITY && l == 0.0f;
    for (int i = 0; i < D / 32; ++i)
        q.out[t * q.out_stride + h * D + lane * (D / 32) + i] =
            bf16_bits(none ? 0.0f : o[i] / l);
    if (q.lse && lane == 0)
        q.lse[item] = none ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4View &c, int D, const Kv4Query &q, const int32_t *tok_start,
                            const int32_t *lens, int T, cudaStream_t stream)
{
    const unsigned grid = unsigned(((long long)T * q.q_heads + 3) / 4);
    if (D == 128)
        kv4_attn_kernel<128><<<grid, 128, 0, stream>>>(c, q, tok_start, lens, T);
    else
        kv4_attn_kernel<64><<<grid, 128, 0, stream>>>(c, q, tok_start, lens, T);
    return cudaGetLastError();
}

}  // namespace tq
