// rope.cu -- rotary positions of query and key rows (include/tq.h, tq_rope).
//
// Pair i of a head's rot_dim / 2 pairs turns by angle = pos[a(i)][t] *
// inv_freq[i], where a(i) is the axis whose section holds i. The product and
// its reduction to a part of a turn are taken in fp64, because in fp32 a
// position of 100,000 has no bits left for the angle (its step is 2^-7
// radian); what is left, |r| <= 1/2 turn, is rounded to fp32 once and turned
// into a cosine and a sine there.
//
// Bound by HBM at a prompt's length: every row is read and written once, with
// 16-byte accesses, and a token's angles are computed once for all its heads
// (they live in shared memory). 8192 tokens of 25 heads of 128, fp32 to bf16:
// 27.5 us, 5.71 TB/s (87% of a plain copy). A CTA takes one token while tokens
// are few (a decode step of 16 is 2.1 us, with two tokens a CTA 2.9), two from 4
// tokens per SM, where one leaves threads idle in the angles (30.0 us at 8192,
// when two took 27.8) and four too few CTAs (29.4).
#include <algorithm>

#include "divisor.cuh"
#include "quant_core.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
    RopeRows r[kRopeMaxRows];
    int head0[kRopeMaxRows + 1];  // first head of each entry among all entries' heads
    const int32_t *pos;
    long long pos_stride;
    const float *inv_freq;
    int section_end[kRopeMaxAxes];
    int n, n_axes, T, D, rot, interleaved, tokens_per_cta;
    Divisor by_half, by_units, by_heads;
};

__device__ __forceinline__ void load8(const RopeRows &r, long long at, float (&v)[8])
{
    if (r.x_f32) {
        const float4 a = *reinterpret_cast<const float4 *>(r.x_f32 + at);
        const float4 b = *reinterpret_cast<const float4 *>(r.x_f32 + at + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(r.x_bf16 + at);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
}

__device__ __forceinline__ void store8(const RopeRows &r, long long at, const float (&v)[8])
{
    if (r.y_f32) {
        *reinterpret_cast<float4 *>(r.y_f32 + at) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(r.y_f32 + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 u;
        u.x = pack_bf16(v[0], v[1]);
        u.y = pack_bf16(v[2], v[3]);
        u.z = pack_bf16(v[4], v[5]);
        u.w = pack_bf16(v[6], v[7]);
        *reinterpret_cast<uint4 *>(r.y_bf16 + at) = u;
    }
}

// A unit is what one thread turns at a time: two vectors of 8 values, i.e.
// 8 pairs (i, i + rot/2) or, interleaved, 16 consecutive values; the values
// behind rot are copied in the same units.
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    extern __shared__ float2 cs[];  // [tokens_per_cta][rot / 2] cosine, sine
    const int half = p.rot >> 1;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int tokens = min(p.tokens_per_cta, p.T - t0);
    const int turn_units = p.rot >> 4;
    const int units = turn_units + ((p.D - p.rot + 15) >> 4);  // per head
    const int heads = p.head0[p.n];

    pdl_wait();
    pdl_launch_dependents();
    for (int j = threadIdx.x; j < tokens * half; j += kRopeThreads) {
        const int t = p.by_half.of(j), i = j - t * half;
        int a = 0;
        while (a + 1 < p.n_axes && i >= p.section_end[a])
            ++a;
        const double turns = double(p.pos[a * p.pos_stride + t0 + t]) * double(p.inv_freq[i]) *
                             0.15915494309189533577;  // 1 / (2 pi)
        const float r = float(turns - rint(turns));
        float s, c;
        sincospif(2.0f * r, &s, &c);
        cs[j] = make_float2(c, s);
    }
    __syncthreads();
    for (int j = threadIdx.x; j < tokens * heads * units; j += kRopeThreads) {
        const int th = p.by_units.of(j), u = j - th * units;
        const int t = p.by_heads.of(th), h = th - t * heads;
        int e = 0;
        while (e + 1 < p.n && h >= p.head0[e + 1])
            ++e;
        const RopeRows &r = p.r[e];
        const long long x0 = (long long)(t0 + t) * r.x_stride + (long long)(h - p.head0[e]) * p.D;
        const long long y0 = (long long)(t0 + t) * r.y_stride + (long long)(h - p.head0[e]) * p.D;
        float a[8], b[8];
        if (u >= turn_units) {
            const int d = p.rot + (u - turn_units) * 16;
            load8(r, x0 + d, a);
            const bool two = d + 8 < p.D;
            if (two)
                load8(r, x0 + d + 8, b);
            store8(r, y0 + d, a);
            if (two)
                store8(r, y0 + d + 8, b);
            continue;
        }
        const float2 *w = cs + t * half + u * 8;
        const int d0 = p.interleaved ? u * 16 : u * 8;
        const int d1 = p.interleaved ? d0 + 8 : half + d0;
        load8(r, x0 + d0, a);
        load8(r, x0 + d1, b);
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 f = w[i >> 1], g = w[4 + (i >> 1)];
                const float a0 = a[i], b0 = b[i];
                a[i] = a0 * f.x - a[i + 1] * f.y;
                a[i + 1] = a[i + 1] * f.x + a0 * f.y;
                b[i] = b0 * g.x - b[i + 1] * g.y;
                b[i + 1] = b[i + 1] * g.x + b0 * g.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = w[i];
                const float a0 = a[i];
                a[i] = a0 * f.x - b[i] * f.y;
                b[i] = b[i] * f.x + a0 * f.y;
            }
        }
        store8(r, y0 + d0, a);
        store8(r, y0 + d1, b);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeRows *rows, int n, const int32_t *pos, long long pos_stride,
                        const float *inv_freq, const int *sections, int n_axes, int T, int D,
                        int rot, bool interleaved, cudaStream_t stream)
{
    RopeParams p = {};
    p.n = n;
    for (int i = 0; i < n; ++i) {
        p.r[i] = rows[i];
        p.head0[i + 1] = p.head0[i] + rows[i].heads;
    }
    p.pos = pos;
    p.pos_stride = pos_stride;
    p.inv_freq = inv_freq;
    for (int i = 0, end = 0; i < n_axes; ++i)
        p.section_end[i] = end += sections[i];
    p.n_axes = n_axes;
    p.T = T;
    p.D = D;
    p.rot = rot;
    p.interleaved = interleaved;
    p.tokens_per_cta = T >= 4 * device_sm_count() ? 2 : 1;
    p.by_half = Divisor(std::max(1, rot / 2));
    p.by_units = Divisor((rot >> 4) + ((D - rot + 15) >> 4));
    p.by_heads = Divisor(p.head0[n]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((T + p.tokens_per_cta - 1) / p.tokens_per_cta));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = size_t(p.tokens_per_cta) * size_t(rot / 2) * sizeof(float2);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel, p);
}

}  // namespace tq
