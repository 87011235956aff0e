// kv4_append.cu -- new tokens' keys and values into the 4-bit cache
// (include/tq.h, tq_kv4_append).
//
// Per token and head: s = bf16(fl32(absmax / 7)), code = the whole number
// nearest to x / s (ties to even, decided exactly), stored as code + 8. The
// scale is bf16, the range of fp32 at 2 bytes: fp16 would overflow or lose
// small rows, fp32 would add 3% to every later read of the cache. Codes are
// taken against the rounded scale, so its rounding (2^-9) costs no accuracy
// beyond the code's own half step; |x / s| stays below 7.04.
//
// Bound by HBM (K and V read once, D + 4 bytes a token and head written): a
// group of D/8 lanes holds one (token, head) pair of rows, 8 values of each
// per lane with 16-byte loads, and the largest magnitude is a shuffle
// reduction inside the group.
#include "kv4_common.cuh"
#include "quant_core.cuh"

namespace tq {

namespace {

constexpr int kAppendThreads = 256;

struct AppendParams {
    Kv4View c;
    const void *k, *v;  // rows [T, kv_heads, D], bf16 or fp32
    long long k_stride, v_stride;
    const int32_t *tok_start, *lens;
    int T;
};

// Eight codes + 8, four bits each, first value lowest: the whole numbers
// nearest to x / s, ties to even. x times the rounded 1 / s is off by less than
// 2^-20, so its nearest whole number q is the right one or its neighbour, and
// the exact remainder x - q s (24 bits hold it: q s has 11, and it is smaller
// than x or than s) tells: beyond s / 2, or at it with q odd, the code is the
// neighbour on x's side. Adding 1.5 2^23 rounds to a whole number and leaves it
// in the low bits, where the sum of 16^i times those bits packs the codes. (A
// correctly rounded quotient and its checks took 40 instructions a value and
// bound prompts by arithmetic at 29 us; this takes 8.)
__device__ __forceinline__ uint32_t pack_codes(const float (&x)[8], float s)
{
    constexpr float kMagic = 12582912.0f;
    constexpr uint32_t kOnes = 0x11111111u;
    // a scale below 2^-100 is lifted: its reciprocal could overflow
    const float lift = s < 7.9e-31f ? 1.2676506e30f : 1.0f;  // 2^100
    const float sl = s * lift, inv = __frcp_rn(sl);
    float t[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float xl = x[i] * lift;
        t[i] = __fmaf_rn(xl, inv, kMagic);
        far = fmaxf(far, fabsf(__fmaf_rn(kMagic - t[i], sl, xl)));
    }
    if (2.0f * far >= sl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __fmaf_rn(kMagic - t[i], sl, x[i] * lift), h = 2.0f * fabsf(e);
            if (h > sl || (h == sl && (__float_as_uint(t[i]) & 1u)))
                t[i] += e > 0.0f ? 1.0f : -1.0f;
        }
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w += __float_as_uint(t[i]) << (4 * i);
    // less the magic number's own bits, plus 8 in each place
    return w - 0x4B400000u * kOnes + 8u * kOnes;
}

template <bool F32>
__device__ __forceinline__ void load_row8(const void *base, long long at, float (&v)[8])
{
    if constexpr (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
}

// Quantise the group's row and store its codes (4 bytes a lane) and scale.
template <int D>
__device__ __forceinline__ void put_row(const float (&x)[8], int lane, uint8_t *codes,
                                        uint16_t *scale, bool store)
{
    // The largest magnitude; as unsigned whole numbers the bit patterns of
    // magnitudes order with infinity and NaN on top, so neither is dropped.
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint32_t packed = 0x88888888u;  // eight codes 0
    uint16_t sbits = 0x7FC0;        // NaN: the row holds a NaN or an infinity
    if (m < 0x7F800000u) {
        sbits = bf16_bits(__fdiv_rn(__uint_as_float(m), 7.0f));
        if (sbits != 0)
            packed = pack_codes(x, __uint_as_float(uint32_t(sbits) << 16));
    }
    if (store) {
        *reinterpret_cast<uint32_t *>(codes + 4 * lane) = packed;
        if (lane == 0)
            *scale = sbits;
    }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kAppendThreads)
    kv4_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const long long item =
        (long long)blockIdx.x * (kAppendThreads / kLanes) + threadIdx.x / kLanes;
    pdl_wait();
    pdl_launch_dependents();
    // Lanes without a row stay for the shuffles and store nothing.
    const bool real = item < (long long)p.T * p.c.kv_heads;
    const int t = real ? int(item / p.c.kv_heads) : 0;
    const int h = real ? int(item - (long long)t * p.c.kv_heads) : 0;
    float k[8], v[8];
    load_row8<F32>(p.k, t * p.k_stride + h * D + lane * 8, k);
    load_row8<F32>(p.v, t * p.v_stride + h * D + lane * 8, v);

    // The token's sequence: the last b with tok_start[b] <= t.
    bool store = real;
    int b = t, behind = 1;  // tokens from t to its sequence's end
    if (p.tok_start) {
        int lo = 0, hi = p.c.batch;  // tok_start[lo] <= t < tok_start[hi]
        store = store && p.tok_start[0] <= t && t < p.tok_start[hi];
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            (p.tok_start[mid] <= t ? lo : hi) = mid;
        }
        b = lo;
        behind = p.tok_start[lo + 1] - t;
    }
    uint8_t *codes = nullptr;
    uint16_t *scale = nullptr;
    const int ps = p.c.page_size();
    if (store) {
        const long long at = (long long)p.lens[b] - behind;
        if (at < 0) {
            store = false;
        } else if (at >= p.c.max_len()) {
            store = false;
            atomicOr(p.c.err, kErrBadPage);
        } else {
            uint8_t *page = kv4_page(p.c, b, int(at) >> p.c.lg_ps);
            store = page != nullptr;
            if (store) {
                const int slot = int(at) & (ps - 1);
                uint8_t *block = page + h * p.c.head_bytes<D>();
                codes = block + slot * (D / 2);
                scale = reinterpret_cast<uint16_t *>(block + (long long)ps * D) + slot;
            }
        }
    }
    put_row<D>(k, lane, codes, scale, store);
    put_row<D>(v, lane, codes + ps * (D / 2), scale + ps, store);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4View &c, int D, const void *k, const void *v, bool f32,
                              long long k_stride, long long v_stride, const int32_t *tok_start,
                              const int32_t *lens, int T, cudaStream_t stream)
{
    const AppendParams p{c, k, v, k_stride, v_stride, tok_start, lens, T};
    const long long groups = (long long)T * c.kv_heads;
    const int per_cta = kAppendThreads / (D / 8);
    const long long grid = (groups + per_cta - 1) / per_cta;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (D == 128)
        return f32 ? cudaLaunchKernelEx(&cfg, kv4_append_kernel<128, true>, p)
                   : cudaLaunchKernelEx(&cfg, kv4_append_kernel<128, false>, p);
    return f32 ? cudaLaunchKernelEx(&cfg, kv4_append_kernel<64, true>, p)
               : cudaLaunchKernelEx(&cfg, kv4_append_kernel<64, false>, p);
}

}  // namespace tq
