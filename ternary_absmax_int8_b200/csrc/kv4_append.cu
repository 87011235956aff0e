// kv4_append.cu -- new tokens' keys and values into the 4-bit cache
// (include/tq.h, tq_kv4_append).
//
// Per token and head: s = bf16(fl32(absmax / 7)), code = the whole number
// nearest to x / s (ties to even, decided exactly), stored as code + 8. The
// scale is bf16, the range of fp32 at 2 bytes: fp16 would overflow or lose
// small rows, fp32 would add 3% to every later read of the cache. Codes are
// taken against the rounded scale, so its rounding (2^-9) costs no accuracy
// beyond the code's own half step; |x / s| stays below 7.04 (but for subnormal s).
//
// Bound by HBM (K and V read once, D + 4 bytes a token and head written): a
// group of D/8 lanes holds one (token, head) pair of rows, 8 values of each
// per lane with 16-byte loads, and the largest magnitude is a shuffle
// reduction inside the group. Prompts of 13,400 tokens in all, 5 heads of
// 128 in fp32 (77 MB), take 16.2 us from memory, 4.7 TB/s, and 14.9 where the
// inputs of the call before are still in L2, with 65% of the issue slots busy: no
// unit is full. bf16 rows of as many tokens, 43 MB, take 18.9 and 16.7: as many
// instructions a value, 73% of the slots, with all of a CTA's start for each item.
#include <algorithm>

#include "kv4_common.cuh"
#include "quant_core.cuh"

namespace tq {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kLoopCtas = 3, kOnceCtas = 4;  // of an SM

struct AppendParams {
    Kv4View c;
    const void *k, *v;  // rows [T, kv_heads, D], bf16 or fp32
    // strides and counts fit 32 bits, so that an address is one multiply-add
    unsigned k_stride, v_stride, page_stride;
    const int32_t *tok_start, *lens;
    int T, items;  // items: (token, head) pairs
    Divisor by_heads;
    int each, more;  // rounds (an item of each group) of a CTA: the first `more` have each + 1
};

// Eight codes + 8, four bits each, first value lowest: the whole numbers
// nearest to x / s, ties to even; inv is 1 / s to 2^-22. x times inv is off by
// less than 2^-18, so its nearest whole number q is the right one or its
// neighbour, and the exact remainder x - q s (24 bits hold it: q s has 11, and
// it is smaller than x or than s) tells: beyond s / 2, or at it with q odd, the
// code is the neighbour on x's side. Adding 1.5 2^23 rounds to a whole number
// and leaves it in the low bits, where the sum of 16^i times those bits packs
// the codes. (A correctly rounded quotient and its checks took 40 instructions
// a value and bound prompts by arithmetic.)
__device__ __forceinline__ uint32_t pack_codes(const float (&x)[8], float s, float inv)
{
    constexpr float kMagic = 12582912.0f;
    constexpr uint32_t kOnes = 0x11111111u;
    float t[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = __fmaf_rn(x[i], inv, kMagic);
        far = fmaxf(far, fabsf(__fmaf_rn(kMagic - t[i], s, x[i])));
    }
    if (2.0f * far >= s) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __fmaf_rn(kMagic - t[i], s, x[i]), h = 2.0f * fabsf(e);
            if (h > s || (h == s && (__float_as_uint(t[i]) & 1u)))
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

__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The larger, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Bits of the row's largest magnitude; as unsigned whole numbers they order with
// infinity and NaN on top, so neither is dropped.
template <int D>
__device__ __forceinline__ uint32_t row_top(const float (&x)[8])
{
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        m = max_nan(m, fabsf(x[i]));
    uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
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

// Store the group's row as codes (4 bytes a lane) and its scale's bits; inv is
// the scale's reciprocal.
template <int D>
__device__ __forceinline__ void put_row(const float (&x)[8], uint32_t sbits, float inv, int lane,
                                        uint8_t *codes, uint16_t *scale, bool store)
{
    uint32_t packed = 0x88888888u;  // eight codes 0: a row of zeros, or one that holds a NaN
    if (inv != 0.0f) {
        float s = __uint_as_float(sbits << 16);
        if (s < 7.9e-31f) {
            // below 2^-100 all is lifted by 2^100, as 1 / s might be infinite;
            // a subnormal s may be so far below absmax / 7 that codes end at 7
            constexpr float kLift = 1.2676506002282294e30f;
            const float top = 7.0f * (s * kLift);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = fminf(fmaxf(x[i] * kLift, -top), top);
            packed = pack_codes(y, s * kLift, inv);
        } else {
            packed = pack_codes(x, s, inv);
        }
    }
    if (store) {
        *reinterpret_cast<uint32_t *>(codes + 4 * lane) = packed;
        if (lane == 0)
            *scale = uint16_t(sbits);
    }
}

// kLoop: a CTA's items go round; else each group has one.
template <int D, bool F32, bool kLoop>
__global__ void __launch_bounds__(kAppendThreads, kLoop ? kLoopCtas : kOnceCtas)
    kv4_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 8, kGroups = kAppendThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    pdl_wait();
    pdl_launch_dependents();
    // A CTA's items are consecutive (token, head) pairs, kGroups at a time; where
    // it goes round, the next ones' rows are on their way while the present ones
    // are quantised.
    const int cta = blockIdx.x, round0 = cta * p.each + min(cta, p.more);
    const int first = round0 * kGroups + threadIdx.x / kLanes;
    const int stop = min(p.items, (round0 + p.each + (cta < p.more)) * kGroups);
    float k[8], v[8], next_k[8], next_v[8];
    int t = p.by_heads.of(first), h = first - t * p.c.kv_heads;
    auto load = [&](bool real, int at, int head, float (&kk)[8], float (&vv)[8]) {
        if (real) {
            const unsigned in = head * D + lane * 8;
            load_row8<F32>(p.k, (long long)((unsigned long long)unsigned(at) * p.k_stride + in), kk);
            load_row8<F32>(p.v, (long long)((unsigned long long)unsigned(at) * p.v_stride + in), vv);
        }
    };
    load(first < stop, t, h, k, v);

    // The token's sequence: the last b with tok_start[b] <= t.
    int b = t, seq_end = t + 1, begin = 0, end = p.T;
    if (p.tok_start) {
        begin = p.tok_start[0];
        end = p.tok_start[p.c.batch];
        int lo = 0, hi = p.c.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            (p.tok_start[mid] <= t ? lo : hi) = mid;
        }
        b = lo;
        seq_end = p.tok_start[lo + 1];
    }
    const int ps = p.c.page_size();
    // Position of token t, -1 where it has none, and the number of its page; the
    // sequence moves on with t.
    auto locate = [&](bool real, int at_t, int *page) {
        if (!real || at_t < begin || at_t >= end)
            return -1;
        if (p.tok_start) {
            while (at_t >= seq_end && b + 1 < p.c.batch)
                seq_end = p.tok_start[++b + 1];
        } else {
            b = at_t;
            seq_end = at_t + 1;
        }
        const long long at = (long long)p.lens[b] - (seq_end - at_t);
        if (at >= p.c.max_len()) {
            atomicOr(p.c.err, kErrBadPage);
            return -1;
        }
        if (at >= 0)
            *page = p.c.table[(long long)b * p.c.max_pages + (int(at) >> p.c.lg_ps)];
        return int(max(at, -1ll));
    };
    int page = 0, at = locate(first < stop, t, &page);
    // (a warp's groups go round together: lanes without a row stay for the
    // shuffles and store nothing)
#pragma unroll 2
    for (int item = first; item - int(threadIdx.x / kLanes) < stop; item += kGroups) {
        int next_t = t, next_h = h + kGroups, next_page = 0;
        while (next_h >= p.c.kv_heads) {
            next_h -= p.c.kv_heads;
            ++next_t;
        }
        const bool more = kLoop && stop - item > kGroups;
        load(more, next_t, next_h, next_k, next_v);
        const int next_at = locate(more, next_t, &next_page);

        uint8_t *codes = nullptr;
        uint16_t *scale = nullptr;
        bool store = at >= 0;
        if (store && unsigned(page) >= unsigned(p.c.num_pages)) {
            atomicOr(p.c.err, kErrBadPage);
            store = false;
        }
        if (store) {
            const int slot = at & (ps - 1);
            uint8_t *block = p.c.pages + (unsigned long long)unsigned(page) * p.page_stride +
                             unsigned(h * (D + 4)) * (unsigned long long)ps;
            codes = block + slot * (D / 2);
            scale = reinterpret_cast<uint16_t *>(block + ps * D) + slot;
        }
        // Even lanes work out the key row's scale, odd ones the value row's.
        const uint32_t top_k = row_top<D>(k), top_v = row_top<D>(v);
        const uint32_t top = (lane & 1) ? top_v : top_k;
        uint32_t sbits = 0x7FC0;  // NaN: the row holds a NaN or an infinity
        float inv = 0.0f;
        if (top < 0x7F800000u) {
            sbits = bf16_bits(__fdiv_rn(__uint_as_float(top), 7.0f));
            const float s = __uint_as_float(sbits << 16);
            if (sbits != 0)
                inv = reciprocal(s < 7.9e-31f ? s * 1.2676506002282294e30f : s);
        }
        const int even = threadIdx.x & 30;
        put_row<D>(k, __shfl_sync(0xffffffffu, sbits, even), __shfl_sync(0xffffffffu, inv, even),
                   lane, codes, scale, store);
        put_row<D>(v, __shfl_sync(0xffffffffu, sbits, even + 1),
                   __shfl_sync(0xffffffffu, inv, even + 1), lane, codes + ps * (D / 2), scale + ps,
                   store);
        if (!kLoop)
            break;
        t = next_t;
        h = next_h;
        at = next_at;
        page = next_page;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] = next_k[i];
            v[i] = next_v[i];
        }
    }
}

template <int D>
cudaError_t launch(const cudaLaunchConfig_t *cfg, bool f32, bool loop, const AppendParams &p)
{
    if (!f32)
        return cudaLaunchKernelEx(cfg, kv4_append_kernel<D, false, false>, p);
    return loop ? cudaLaunchKernelEx(cfg, kv4_append_kernel<D, true, true>, p)
                : cudaLaunchKernelEx(cfg, kv4_append_kernel<D, true, false>, p);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4View &c, int D, const void *k, const void *v, bool f32,
                              long long k_stride, long long v_stride, const int32_t *tok_start,
                              const int32_t *lens, int T, cudaStream_t stream)
{
    const long long items = (long long)T * c.kv_heads;
    const int groups = kAppendThreads / (D / 8);
    // A round is an item for each group of a CTA. Each CTA has one, so that small
    // calls spread over all SMs; fp32 rows beyond 16 rounds an SM go round in 3
    // CTAs per SM, the next ones' loads in flight, as there bytes count more than
    // instructions. fp32, heads of 128, in us, one round : going round, at 7, 12,
    // 16, 20, 24 and 40 rounds an SM: 5.1:5.5, 7.2:7.5, 9.7:9.9, 13.2:12.6,
    // 16.0:14.5, 24.4:21.7; bf16 at 7, 16, 40: 5.5:6.5, 10.2:11.2, 24.8:29.1.
    const int rounds = int((items + groups - 1) / groups);  // of one CTA
    const bool loop = f32 && rounds > 16 * device_sm_count();
    const int grid = loop ? std::min(rounds, kLoopCtas * device_sm_count()) : rounds;
    const AppendParams p{c, k, v, unsigned(k_stride), unsigned(v_stride), unsigned(c.page_stride),
                         tok_start, lens, T, int(items), Divisor(c.kv_heads), rounds / grid,
                         rounds % grid};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 128 ? launch<128>(&cfg, f32, loop, p) : launch<64>(&cfg, f32, loop, p);
}

}  // namespace tq
