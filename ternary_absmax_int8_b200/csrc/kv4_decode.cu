// kv4_decode.cu -- attention of one new token per sequence over the 4-bit
// cache (include/tq.h, tq_kv4_decode).
//
// Every cached code is read once, so HBM sets the floor: (D + 4) bytes a
// token and head. At 6.5 TB/s that is 13e12 codes a second against 36e12
// instruction lanes, so a code may cost no more than about two lanes of work
// from load to result, and scalar products cannot do it (4 query heads x 2
// products). Hence the warp-level MMA (m16n8k16, fp16 x fp16 + fp32), with
//  - keys on the 16-row side and the query heads that share them on the
//    8-column side, S^T = K q^T and O^T = V^T P^T: 4 heads waste half of a
//    product of 8 columns, not three quarters of one of 16 rows. (The
//    tensor-memory MMA wants 64 or 128 rows and its operands in shared
//    memory: codes would be written back there, 4 bytes for each one read.)
//  - operands from the packed nibbles in nine instructions for eight codes: a
//    nibble n masked in place under the exponent of 1024 (of 64, one nibble
//    higher) is the fp16 number 1024 + n (64 + n), and one subtraction leaves
//    the code, exactly. (Leaving out the subtraction, with masked nibbles as
//    subnormals n 2^-24 and the +8 taken off the sums, costs five; but the
//    matrix unit aligns a subnormal's products as if it were 2^-14, and the
//    sums lost up to 2^-13 of the weights' sum.) Which 16 codes form an MMA's
//    k range is free as long as both operands agree, so a lane takes
//    contiguous bytes of a row and no data moves between lanes.
//  - P^T from S^T's registers by one transposing move per 8 x 8 block.
// Scores, running maxima and sums are fp32. A weight times its value's scale
// is rounded to fp16 (2^-11) against the largest value scale of its tile, and
// a tile's 64 products are added up by the MMA, the tiles in fp32 registers.
//
// Work split: the tiles (64 tokens of one sequence and head) of all sequences
// form one list, cut into equal shares per SM and per warp, whatever the
// sequences' lengths. Each warp walks its share alone: a private ring of
// shared-memory stages filled by bulk copies (a tile of one page is one copy
// of 64 (D + 4) bytes) and no barrier with other warps until its share is
// done. Then the warps of an SM that ended in one sequence are merged in
// shared memory, and kv4_combine_kernel joins what several SMs hold of one
// sequence, in a fixed order.
#include <algorithm>

#include "kv4_common.cuh"
#include "quant_core.cuh"
#include "tc_common.cuh"

#include <cuda_fp16.h>

namespace tq {

namespace {

constexpr int kTile = 64;  // tokens of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Warps of a CTA (one CTA per SM) and ring stages per warp: as many bytes in
// flight as shared memory holds, with registers for the heads' results (NT
// groups of 8 heads x D values x fp32 over 32 lanes).
template <int D, int NT>
struct DecodeShape {
    static constexpr int kWarps = D == 128 ? (NT == 1 ? 12 : 8) : (NT == 1 ? 16 : 12);
    static constexpr int kStages = D == 128 ? (NT == 1 ? 2 : 3) : (NT == 1 ? 3 : 4);
    static constexpr int kStageBytes = kTile * (D + 4);
    static constexpr int kHeads = 8 * NT;          // heads of an item
    static constexpr int kPartFloats = D + 2;      // one head's part: values, maximum, sum
};

struct DecodeParams {
    Kv4View c;
    Kv4Query q;
    const int32_t *lens;
    int rep;     // query heads per key/value head
    int groups;  // of up to 8 NT query heads each
    // workspace
    long long *total;  // tiles of the call
    long long *start;  // [items] first tile of each item that has any
    float *parts;      // [workers][2][rows][D + 2]
    int rows;          // heads of a part: min(rep, 8 NT)
};

// A sequence's keys that its query sees: [begin, end), tiles of 64 from the
// one that holds begin.
struct Span {
    int begin, end, tile0, tiles;
};

__device__ __forceinline__ Span span_of(const DecodeParams &p, int b)
{
    Span s;
    s.end = kv4_len(p.c, p.lens, b);
    s.begin = p.q.window > 0 ? max(0, s.end - p.q.window) : 0;
    s.tile0 = s.begin / kTile;
    s.tiles = (s.end + kTile - 1) / kTile - s.tile0;
    return s;
}

// Shares: CTA c of n takes tiles [c total / n, (c + 1) total / n), its warp w
// of them [w per, (w + 1) per) with per = ceil(count / warps).
struct Share {
    long long first;
    int count, per;
};

__device__ __forceinline__ Share share_of(long long total, int cta, int ctas, int warps)
{
    Share s;
    s.first = total * cta / ctas;
    s.count = int(total * (cta + 1) / ctas - s.first);
    s.per = (s.count + warps - 1) / warps;
    return s;
}

__device__ __forceinline__ int cta_of(long long tile, long long total, int ctas)
{
    return int(((tile + 1) * ctas - 1) / total);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The codes at bits 0-3 and 16-19 (low4) or 4-7 and 20-23 (high4) of a word of
// nibbles code + 8, as two fp16 numbers.
__device__ __forceinline__ uint32_t sub_half2(uint32_t v, uint32_t c)
{
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t low4(uint32_t w)
{
    return sub_half2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);  // 1024 + n - 1032
}
__device__ __forceinline__ uint32_t high4(uint32_t w)
{
    return sub_half2((w & 0x00F000F0u) | 0x54005400u, 0x54805480u);  // 64 + n - 72
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The token of a 16-token group that stands at MMA row i. Rows 2t, 2t + 1
// (and + 8) are lane t's value tokens: neighbouring t and the two of a lane
// alternate in parity, so that rows of 64 bytes spread over all banks in the
// key loads and over half in the value loads.
__device__ __forceinline__ int token_at(int i)
{
    const int j = i & 7;
    return (i & 8) + ((j & 1) ? 4 + ((j >> 1) ^ 1) : j >> 1);
}

// One head group's running result over part of a sequence.
template <int D, int NT>
struct Running {
    float o[NT][D / 16][4];  // [d-tile]: elements d (0, 1) and d + 1 (2, 3) of heads 2t, 2t + 1
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[n][i][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[n][j] = 0.0f;
                m[n][j] = -INFINITY;
            }
        }
    }
};

// A head group's queries as MMA operands, with what their scaling needs.
template <int D, int NT>
struct Queries {
    uint32_t b[NT][D / 16][2];
    float mul[NT][2];  // accumulator x key scale -> log2 of the weight; heads 2t, 2t + 1
};

template <int D, int NT>
__device__ __forceinline__ void load_queries(const DecodeParams &p, long long row, int head0,
                                             int heads, Queries<D, NT> &q)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // lane's D/4 consecutive values of head 8n + g
        float v[D / 4];
        const bool real = n * 8 + g < heads;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q.q + row + (long long)(head0 + (real ? n * 8 + g : 0)) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 u = real ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
            v[8 * i] = bf16_lo(u.x), v[8 * i + 1] = bf16_hi(u.x);
            v[8 * i + 2] = bf16_lo(u.y), v[8 * i + 3] = bf16_hi(u.y);
            v[8 * i + 4] = bf16_lo(u.z), v[8 * i + 5] = bf16_hi(u.z);
            v[8 * i + 6] = bf16_lo(u.w), v[8 * i + 7] = bf16_hi(u.w);
        }
        // Scaled by a power of two so that the largest magnitude of the head
        // lies in [2^14, 2^15): bf16's 8 bits fit fp16's 11.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
            top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int k = min(max(int(top >> 23) - 127, -100), 117);
        const float up = __uint_as_float(uint32_t(14 - k + 127) << 23);
#pragma unroll
        for (int u = 0; u < D / 32; ++u)  // one 32-bit word of a key row: 8 codes
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q.b[n][2 * u + (i >> 1)][i & 1] = pack_half(v[8 * u + i] * up, v[8 * u + 4 + i] * up);
        // 1 / up, scale and the change to base 2
        const float mul = __uint_as_float(uint32_t(k - 14 + 127) << 23) * (p.q.scale * kLog2e);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            q.mul[n][j] = __shfl_sync(0xffffffffu, mul, 8 * t + 4 * j);
    }
}

// One tile: scores, softmax step, weighted values. `sps` tokens of the tile
// come from one page: in shared memory its key codes, value codes, key scales
// and value scales follow one another, blocks of sps (D + 4) bytes. With
// kEdge, tokens outside [begin, end) and pages whose bit of `good` is clear
// take no part.
template <int D, int NT, bool kEdge>
__device__ __forceinline__ void tile_step(const uint8_t *stage, int lg_sps, int j0, int begin,
                                          int end, uint32_t good, const Queries<D, NT> &q,
                                          Running<D, NT> &r)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int sps = 1 << lg_sps;
    const int row0 = token_at(g);
    float x[NT][4][4];
    uint32_t sv[4][2];  // value scales (fp32 bits) of rows g and g + 8
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
        const int blk = (mt * 16) >> lg_sps;
        const uint8_t *base = stage + (blk << lg_sps) * (D + 4);
        const int in0 = ((mt * 16) & (sps - 1)) + row0;  // row within the block
        const uint16_t *sc = reinterpret_cast<const uint16_t *>(base + (sps * D));
        float ks[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ks[h] = __uint_as_float(uint32_t(sc[in0 + 8 * h]) << 16);
            sv[mt][h] = uint32_t(sc[sps + in0 + 8 * h]) << 16;
        }
        uint32_t w0[D / 32], w1[D / 32];  // rows g and g + 8, lane's D/4 codes
        const uint8_t *kr = base + in0 * (D / 2) + t * (D / 8);
        if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4 *>(kr);
            const uint4 b = *reinterpret_cast<const uint4 *>(kr + 8 * (D / 2));
            w0[0] = a.x, w0[1] = a.y, w0[2] = a.z, w0[3] = a.w;
            w1[0] = b.x, w1[1] = b.y, w1[2] = b.z, w1[3] = b.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(kr);
            const uint2 b = *reinterpret_cast<const uint2 *>(kr + 8 * (D / 2));
            w0[0] = a.x, w0[1] = a.y;
            w1[0] = b.x, w1[1] = b.y;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[n][mt][i] = 0.0f;
#pragma unroll
        for (int u = 0; u < 2 * (D / 32); ++u) {
            const uint32_t a = (u & 1) ? w0[u >> 1] >> 8 : w0[u >> 1];
            const uint32_t b = (u & 1) ? w1[u >> 1] >> 8 : w1[u >> 1];
            const uint32_t a0 = low4(a), a1 = low4(b), a2 = high4(a), a3 = high4(b);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mma_f16(x[n][mt], a0, a1, a2, a3, q.b[n][u][0], q.b[n][u][1]);
        }
        bool in[2] = {true, true};
        if constexpr (kEdge) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = j0 + mt * 16 + row0 + 8 * h;
                in[h] = j >= begin && j < end && ((good >> blk) & 1u);
                if (!in[h])
                    sv[mt][h] = 0;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = x[n][mt][i] * ks[i >> 1];
                x[n][mt][i] = kEdge && !in[i >> 1] ? -INFINITY : s;
            }
    }

    // The largest value scale of the tile, as a power of two (NaN stays NaN):
    // weights x value scales go to fp16 as multiples of sref, below 2^15, so
    // that all above 2^-28 of the largest possible keep 11 bits.
    uint32_t top = 0;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
        top = max(top, max(sv[mt][0], sv[mt][1]));
    top = max(__reduce_max_sync(0xffffffffu, top) & 0x7F800000u, 15u << 23);
    const float sref = top == 0x7F800000u ? NAN : __uint_as_float(top - (14u << 23));
    const float rs = top == 0x7F800000u ? NAN : __uint_as_float((268u << 23) - top);

    // Running maximum per head, in units of accumulator x key scale.
    float mn[NT][2];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = fmaxf(x[n][0][j], x[n][0][2 + j]);
#pragma unroll
            for (int mt = 1; mt < 4; ++mt)
                v = fmaxf(v, fmaxf(x[n][mt][j], x[n][mt][2 + j]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            mn[n][j] = fmaxf(r.m[n][j], v);
            grew = grew || mn[n][j] != r.m[n][j];
        }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float a[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // nothing seen yet: nothing to scale (and no infinity minus itself)
                a[j] = r.m[n][j] == mn[n][j] ? 1.0f : ex2((r.m[n][j] - mn[n][j]) * q.mul[n][j]);
                r.l[n][j] *= a[j];
                r.m[n][j] = mn[n][j];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r.o[n][i][j] *= a[j & 1];
        }
    }

    // Weights, and the operands P^T of the second product.
    uint32_t pb[NT][4][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            c[j] = r.m[n][j] == -INFINITY ? 0.0f : -r.m[n][j] * q.mul[n][j];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = ex2(fmaf(x[n][mt][i], q.mul[n][i & 1], c[i & 1]));
                r.l[n][i & 1] += w[i];
                w[i] *= __uint_as_float(sv[mt][i >> 1]) * rs;
            }
            pb[n][mt][0] = transpose8x8(pack_half(w[0], w[1]));
            pb[n][mt][1] = transpose8x8(pack_half(w[2], w[3]));
        }
    }
    // Values: lane g's D/8 consecutive elements, 8 (one word) at a time.
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        float acc[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[n][i][j] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const int blk = (mt * 16) >> lg_sps;
            const uint8_t *vr = stage + (blk << lg_sps) * (D + 4) + sps * (D / 2) +
                                ((mt * 16) & (sps - 1)) * (D / 2) + g * (D / 16) + u * 4;
            uint32_t w[4];  // tokens at rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = *reinterpret_cast<const uint32_t *>(
                    vr + (t + ((i & 1) ? 4 + (t ^ 1) - t : 0) + ((i & 2) ? 8 : 0)) * (D / 2));
            uint32_t lo[2], hi[2];  // the two tokens' elements 0..3 and 4..7
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                lo[h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x5410);
                hi[h] = __byte_perm(w[2 * h], w[2 * h + 1], 0x7632);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = (i & 2) ? hi[0] : lo[0], b = (i & 2) ? hi[1] : lo[1];
                const uint32_t as = (i & 1) ? a >> 8 : a, bs = (i & 1) ? b >> 8 : b;
                const uint32_t a0 = low4(as), a1 = high4(as), a2 = low4(bs), a3 = high4(bs);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma_f16(acc[n][i], a0, a1, a2, a3, pb[n][mt][0], pb[n][mt][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r.o[n][4 * u + i][j] = fmaf(acc[n][i][j], sref, r.o[n][4 * u + i][j]);
    }
}

// The lane's result for head 8n + 2t + j, element pair i: even, odd element.
template <int D, int NT>
__device__ __forceinline__ float2 value_pair(const Running<D, NT> &r, int n, int i, int j)
{
    return make_float2(r.o[n][i][j], r.o[n][i][2 + j]);
}

// The sums of weights lie spread over the lanes of a column: add them up.
template <int D, int NT>
__device__ __forceinline__ void close_sums(Running<D, NT> &r)
{
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1)
                r.l[n][j] += __shfl_xor_sync(0xffffffffu, r.l[n][j], o);
}

// A part [heads][D + 2]: values, then the maximum (base 2) and the sum. For
// heads beyond `rows` nothing is stored.
template <int D, int NT>
__device__ __forceinline__ void store_part(const Running<D, NT> &r, const Queries<D, NT> &q,
                                           float *part, int rows)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 8 * n + 2 * t + j;
            if (h >= rows)
                continue;
            float *row = part + h * (D + 2);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2 *>(row + g * (D / 8) + 2 * i) = value_pair(r, n, i, j);
            if (g == 0)
                *reinterpret_cast<float2 *>(row + D) = make_float2(
                    r.m[n][j] == -INFINITY ? -INFINITY : r.m[n][j] * q.mul[n][j], r.l[n][j]);
        }
}

template <int D>
__device__ __forceinline__ void store_out(const DecodeParams &p, int b, int head, int d, float2 v,
                                          float inv)
{
    *reinterpret_cast<uint32_t *>(p.q.out + b * p.q.out_stride + (long long)head * D + d) =
        pack_bf16(v.x * inv, v.y * inv);
}

// Final values of one head from its sum: what saw nothing is 0.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

template <int D, int NT>
__device__ __forceinline__ void store_final(const DecodeParams &p, const Running<D, NT> &r,
                                            const Queries<D, NT> &q, int b, int head0, int heads)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 8 * n + 2 * t + j;
            if (h >= heads)
                continue;
            const float inv = inverse_sum(r.l[n][j]);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                store_out<D>(p, b, head0 + h, g * (D / 8) + 2 * i, value_pair(r, n, i, j), inv);
            if (p.q.lse && g == 0)
                p.q.lse[(long long)b * p.q.q_heads + head0 + h] =
                    log_sum(r.m[n][j] * q.mul[n][j], r.l[n][j]);
        }
}

// The weighted sum of one head's element pair d over n parts `stride` floats
// apart, and that head's maximum and sum.
template <int D, class PartAt>
__device__ __forceinline__ void join(int n, PartAt part_at, int d, float2 *v, float *m, float *l)
{
    float top = -INFINITY;
    for (int i = 0; i < n; ++i)
        top = fmaxf(top, part_at(i)[D]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float2 s = make_float2(0.0f, 0.0f);
    float sum = 0.0f;
    for (int i = 0; i < n; ++i) {
        const float *part = part_at(i);
        const float2 ml = *reinterpret_cast<const float2 *>(part + D);
        const float2 x = *reinterpret_cast<const float2 *>(part + d);
        const float w = ex2(ml.x - ref);
        s.x = fmaf(w, x.x, s.x);
        s.y = fmaf(w, x.y, s.y);
        sum = fmaf(w, ml.y, sum);
    }
    *v = s;
    *m = top;
    *l = sum;
}

struct Segment {  // a warp's last stretch, for the merge within the CTA
    long long item;    // -1: none
    long long first, last;  // the item's tiles [first, last) among all
};

template <int D, int NT>
__global__ void __launch_bounds__(DecodeShape<D, NT>::kWarps * 32, 1)
    kv4_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using S = DecodeShape<D, NT>;
    constexpr int kThreads = S::kWarps * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[S::kWarps][S::kStages];
    __shared__ long long scan[S::kWarps], s_total;
    __shared__ long long warp_base[S::kWarps];  // tiles before the warp's first sequence
    __shared__ int warp_b[S::kWarps];           // that sequence
    __shared__ Segment seg[S::kWarps];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        for (int s = 0; s < S::kStages; ++s)
            mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
    const uint64_t policy = policy_evict_first();
    pdl_wait();
    pdl_launch_dependents();

    // Tiles of all sequences.
    const int hg = p.c.kv_heads * p.groups;
    long long mine = 0;
    for (int b = threadIdx.x; b < p.c.batch; b += kThreads)
        mine += span_of(p, b).tiles;
    for (int o = 16; o > 0; o >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0)
        scan[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        long long sum = 0;
        for (int w = 0; w < S::kWarps; ++w)
            sum += scan[w];
        s_total = sum * hg;
        if (blockIdx.x == 0)
            *p.total = sum * hg;
    }
    __syncthreads();
    const long long total = s_total;
    const Share share = share_of(total, blockIdx.x, gridDim.x, S::kWarps);
    long long at = share.first + min(share.count, warp * share.per);
    const long long stop = share.first + min(share.count, (warp + 1) * share.per);

    // The sequence that holds each warp's first tile: a running sum over the
    // lengths, a block of them at a time.
    if (share.count > 0) {
        long long before = 0;  // tiles (x hg) of the sequences before this block
        for (int b0 = 0; b0 < p.c.batch && before <= share.first + share.count - 1; b0 += kThreads) {
            const int b = b0 + threadIdx.x;
            const long long n = b < p.c.batch ? (long long)span_of(p, b).tiles * hg : 0;
            long long incl = n;
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            __syncthreads();
            if (lane == 31)
                scan[warp] = incl;
            __syncthreads();
            long long base = before, all = 0;
            for (int w = 0; w < S::kWarps; ++w) {
                if (w < warp)
                    base += scan[w];
                all += scan[w];
            }
            const long long lo = base + incl - n;  // this sequence's tiles: [lo, lo + n)
            for (int w = 0; w < S::kWarps; ++w) {
                const long long t = share.first + (long long)w * share.per;
                if (w * share.per < share.count && t >= lo && t < lo + n) {
                    warp_b[w] = b;
                    warp_base[w] = lo;
                }
            }
            before += all;
        }
    }
    __syncthreads();

    uint8_t *ring = smem + warp * (S::kStages * S::kStageBytes);
    const int worker = blockIdx.x * S::kWarps + warp;
    const int lg_sps = min(p.c.lg_ps, 6), sps = 1 << lg_sps;
    const int per_tile = kTile >> lg_sps;  // page stretches of a tile
    uint32_t phase = 0;                    // one bit per stage
    Running<D, NT> run;
    Queries<D, NT> qs;
    bool fine = true;
    Segment last{-1, 0, 0};
    int b = 0;
    long long seq0 = 0;
    if (at < stop) {
        b = warp_b[warp];
        seq0 = warp_base[warp];
    }
    while (at < stop && fine) {
        Span sp = span_of(p, b);
        while ((long long)sp.tiles * hg <= at - seq0 && b + 1 < p.c.batch) {
            seq0 += (long long)sp.tiles * hg;  // on to the sequence with tile `at`
            sp = span_of(p, ++b);
        }
        if ((long long)sp.tiles * hg <= at - seq0)
            break;  // only if lengths change while the kernel runs
        const int ig = int((at - seq0) / sp.tiles);  // head group of the sequence
        const long long item0 = seq0 + (long long)ig * sp.tiles;
        const int n0 = int(at - item0);
        const int n1 = int(min((long long)sp.tiles, stop - item0));
        const int kvh = ig / p.groups, grp = ig - kvh * p.groups;
        const int head0 = kvh * p.rep + grp * S::kHeads;
        const int heads = min(S::kHeads, p.rep - grp * S::kHeads);
        if (n0 == 0 && lane == 0)
            p.start[(long long)b * hg + ig] = item0;

        // Page numbers of the next tiles, one lane each (a page of 128 tokens
        // serves two tiles); -1 for one outside the cache.
        const int lg_batch = 5 - (6 - lg_sps);  // log2 of the tiles 32 lanes cover
        int batch0 = -1, page = -1;
        const long long head_at = kvh * p.c.head_bytes<D>();
        auto fetch = [&](int n, int s) {  // tile n of the sequence into stage s
            const int tile = sp.tile0 + n;
            if ((n >> lg_batch) != batch0) {
                batch0 = n >> lg_batch;
                const int j = ((sp.tile0 + (batch0 << lg_batch)) << 6) + (lane << lg_sps);
                page = -1;
                // (pages in front of a window may have gone to other sequences)
                if (j < sp.end && j + sps > sp.begin) {
                    const int pg = p.c.table[(long long)b * p.c.max_pages + (j >> p.c.lg_ps)];
                    if (unsigned(pg) < unsigned(p.c.num_pages))
                        page = pg;
                    else
                        atomicOr(p.c.err, kErrBadPage);
                }
            }
            const int i0 = (n & ((1 << lg_batch) - 1)) * per_tile;
            uint8_t *dst = ring + s * S::kStageBytes;
            uint64_t *bar = &bars[warp][s];
            const int pg = __shfl_sync(0xffffffffu, page, i0 + (per_tile > 1 ? lane % per_tile : 0));
            const uint32_t good = __ballot_sync(0xffffffffu, pg >= 0) & ((1u << per_tile) - 1u);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, __popc(good) * uint32_t(sps) * (D + 4));
            __syncwarp();
            const uint8_t *src = p.c.pages + (long long)max(pg, 0) * p.c.page_stride + head_at;
            if (p.c.lg_ps <= 6) {
                if (lane < per_tile && pg >= 0)
                    bulk_g2s(dst + lane * sps * (D + 4), src, sps * (D + 4), bar, policy);
            } else if (lane < 4 && pg >= 0) {
                // half of a page of 128: its keys, its values, their scales
                const int half = tile & 1;
                const int ps = 128;
                const int part = lane;
                const int off = part < 2 ? part * ps * (D / 2) + half * kTile * (D / 2)
                                         : ps * D + (part - 2) * ps * 2 + half * kTile * 2;
                const int to = part < 2 ? part * kTile * (D / 2) : kTile * D + (part - 2) * kTile * 2;
                bulk_g2s(dst + to, src + off, part < 2 ? kTile * (D / 2) : kTile * 2, bar, policy);
            }
            return good;
        };

        uint32_t good = 0;  // four bits per stage: which stretches arrive
        for (int s = 0; s < S::kStages && n0 + s < n1; ++s)
            good |= fetch(n0 + s, s) << (4 * s);
        load_queries<D, NT>(p, b * p.q.q_stride, head0, heads, qs);
        run.clear();
#pragma unroll 1
        for (int n = n0, s = 0; n < n1; ++n, s = s + 1 == S::kStages ? 0 : s + 1) {
            fine = mbar_wait_warp(&bars[warp][s], (phase >> s) & 1u, p.c.err);
            phase ^= 1u << s;
            if (!fine)
                break;
            const uint8_t *stage = ring + s * S::kStageBytes;
            const int j0 = (sp.tile0 + n) * kTile;
            const uint32_t here = (good >> (4 * s)) & 15u;
            if (j0 < sp.begin || j0 + kTile > sp.end || here != (1u << per_tile) - 1u)
                tile_step<D, NT, true>(stage, lg_sps, j0, sp.begin, sp.end, here, qs, run);
            else
                tile_step<D, NT, false>(stage, lg_sps, j0, 0, 0, 0, qs, run);
            __syncwarp();
            if (n + S::kStages < n1)
                good = (good & ~(15u << (4 * s))) | fetch(n + S::kStages, s) << (4 * s);
        }
        if (!fine)
            break;
        close_sums<D, NT>(run);
        at = item0 + n1;
        if (n0 == 0 && n1 == sp.tiles) {
            store_final<D, NT>(p, run, qs, b, head0, heads);
        } else if (n1 == sp.tiles && at < stop) {
            // the end of a sequence that other warps began
            store_part<D, NT>(run, qs, p.parts + (long long)(2 * worker) * p.rows * (D + 2),
                              min(p.rows, heads));
        } else {
            last = Segment{(long long)b * hg + ig, item0, item0 + sp.tiles};
        }
    }

    // Merge the warps whose shares ended in one sequence.
    if (lane == 0)
        seg[warp] = last;
    __syncthreads();  // also: every ring is idle
    if (last.item >= 0 && fine)
        store_part<D, NT>(run, qs,
                          reinterpret_cast<float *>(smem) + warp * (S::kHeads * S::kPartFloats),
                          S::kHeads);
    __syncthreads();
    for (int w = 0; w < S::kWarps;) {
        const Segment s = seg[w];
        int n = 1;
        while (w + n < S::kWarps && s.item >= 0 && seg[w + n].item == s.item)
            ++n;
        if (s.item >= 0) {
            const int sb = int(s.item / hg), ig = int(s.item - (long long)sb * hg);
            const int kvh = ig / p.groups, grp = ig - kvh * p.groups;
            const int head0 = kvh * p.rep + grp * S::kHeads;
            const int heads = min(S::kHeads, p.rep - grp * S::kHeads);
            // complete if these warps hold all of it (a share that goes on
            // past it would have been the end of a sequence, above)
            const long long from = share.first + (long long)w * share.per;
            const long long to = share.first + min(share.count, (w + n) * share.per);
            const bool whole = from <= s.first && to >= s.last;
            const float *first = reinterpret_cast<const float *>(smem) +
                                 w * (S::kHeads * S::kPartFloats);
            float *dst = p.parts +
                         (long long)(2 * (blockIdx.x * S::kWarps + w) + 1) * p.rows * (D + 2);
            for (int i = threadIdx.x; i < heads * (D / 2); i += kThreads) {
                const int h = i / (D / 2), d = 2 * (i - h * (D / 2));
                float2 v;
                float m, l;
                join<D>(n, [&](int k) { return first + (k * S::kHeads + h) * S::kPartFloats; }, d,
                        &v, &m, &l);
                if (whole) {
                    store_out<D>(p, sb, head0 + h, d, v, inverse_sum(l));
                    if (p.q.lse && d == 0)
                        p.q.lse[(long long)sb * p.q.q_heads + head0 + h] = log_sum(m, l);
                } else {
                    *reinterpret_cast<float2 *>(dst + h * (D + 2) + d) = v;
                    if (d == 0)
                        *reinterpret_cast<float2 *>(dst + h * (D + 2) + D) = make_float2(m, l);
                }
            }
        }
        w += n;
    }
}

// Joins the parts of each item that several CTAs (or a CTA's merged warps and
// the warp behind them) hold, in the order of the tiles, and writes the rows
// of sequences without a visible token. One CTA per item.
template <int D, int NT>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const __grid_constant__ DecodeParams p,
                                                          int ctas)
{
    using S = DecodeShape<D, NT>;
    pdl_wait();
    pdl_launch_dependents();
    const int hg = p.c.kv_heads * p.groups;
    const int b = blockIdx.x / hg, ig = blockIdx.x - b * hg;
    const int kvh = ig / p.groups, grp = ig - kvh * p.groups;
    const int head0 = kvh * p.rep + grp * S::kHeads;
    const int heads = min(S::kHeads, p.rep - grp * S::kHeads);
    const Span sp = span_of(p, b);
    long long first = 0, end = 0, total = 1;
    int cta0 = 0, cta1 = -1;
    if (sp.tiles > 0) {
        total = *p.total;
        first = p.start[blockIdx.x];
        end = first + sp.tiles;
        cta0 = cta_of(first, total, ctas);
        cta1 = cta_of(end - 1, total, ctas);
        if (cta0 == cta1) {
            // one CTA: whole there unless the warp behind the merged ones ended it
            const Share s = share_of(total, cta0, ctas, S::kWarps);
            const int w0 = int(first - s.first) / s.per, w1 = int(end - 1 - s.first) / s.per;
            const long long stop1 = s.first + min(s.count, (w1 + 1) * s.per);
            if (w0 == w1 || stop1 == end)
                return;
        }
    }
    // Part k of the item: per CTA the merged warps' part, then, in the last
    // CTA, that of a warp that ended the item and went on.
    __shared__ int slot[2 * 160];
    __shared__ int slots;
    if (threadIdx.x == 0) {
        int n = 0;
        for (int c = cta0; c <= cta1; ++c) {
            const Share s = share_of(total, c, ctas, S::kWarps);
            if (s.count == 0)
                continue;
            const int w0 = max(0, int(max(first, s.first) - s.first) / s.per);
            const long long lim = min(end, s.first + s.count);
            const int w1 = int(lim - 1 - s.first) / s.per;
            const long long stop1 = s.first + min(s.count, (w1 + 1) * s.per);
            const bool ended = lim == end && stop1 > end;  // w1 went on to the next item
            if (w0 < w1 || !ended)
                slot[n++] = 2 * (c * S::kWarps + w0) + 1;
            if (ended)
                slot[n++] = 2 * (c * S::kWarps + w1);
        }
        slots = n;
    }
    __syncthreads();
    const int n = slots;
    for (int i = threadIdx.x; i < heads * (D / 2); i += blockDim.x) {
        const int h = i / (D / 2), d = 2 * (i - h * (D / 2));
        float2 v;
        float m, l;
        join<D>(n, [&](int k) {
            return p.parts + ((long long)slot[k] * p.rows + h) * (D + 2);
        }, d, &v, &m, &l);
        store_out<D>(p, b, head0 + h, d, v, inverse_sum(l));
        if (p.q.lse && d == 0)
            p.q.lse[(long long)b * p.q.q_heads + head0 + h] = log_sum(m, l);
    }
}

struct DecodePlan {
    int rep, nt, groups, rows, ctas, warps;
    long long items;
    size_t start_at, parts_at, bytes;
};

DecodePlan plan_decode(const Kv4View &c, int D, int q_heads)
{
    DecodePlan d;
    d.rep = q_heads / c.kv_heads;
    d.nt = d.rep <= 8 ? 1 : 2;
    d.groups = (d.rep + 8 * d.nt - 1) / (8 * d.nt);
    d.rows = std::min(d.rep, 8 * d.nt);
    d.ctas = std::min(device_sm_count(), 160);
    d.warps = D == 128 ? (d.nt == 1 ? DecodeShape<128, 1>::kWarps : DecodeShape<128, 2>::kWarps)
                       : (d.nt == 1 ? DecodeShape<64, 1>::kWarps : DecodeShape<64, 2>::kWarps);
    d.items = (long long)c.batch * c.kv_heads * d.groups;
    d.start_at = 16;
    d.parts_at = (d.start_at + size_t(d.items) * sizeof(long long) + 15) & ~size_t(15);
    d.bytes = d.parts_at +
              size_t(d.ctas) * d.warps * 2 * d.rows * size_t(D + 2) * sizeof(float);
    return d;
}

template <int D, int NT>
cudaError_t launch(const DecodeParams &p, const DecodePlan &plan, cudaStream_t stream)
{
    using S = DecodeShape<D, NT>;
    constexpr size_t kSmem = size_t(S::kWarps) * S::kStages * S::kStageBytes;
    static_assert(size_t(S::kWarps) * S::kHeads * S::kPartFloats * 4 <= kSmem, "merge space");
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_dev != dev) {
        e = cudaFuncSetAttribute(kv4_decode_kernel<D, NT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
        if (e == cudaSuccess)
            configured_dev = dev;
    }
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(unsigned(plan.ctas));
    cfg.blockDim = dim3(S::kWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    e = cudaLaunchKernelEx(&cfg, kv4_decode_kernel<D, NT>, p);
    if (e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(unsigned(plan.items));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, NT>, p, plan.ctas);
}

}  // namespace

size_t kv4_decode_workspace(const Kv4View &c, int D, int q_heads)
{
    return c.batch > 0 ? plan_decode(c, D, q_heads).bytes : 0;
}

cudaError_t launch_kv4_decode(const Kv4View &c, int D, const Kv4Query &q, const int32_t *lens,
                              void *workspace, cudaStream_t stream)
{
    const DecodePlan plan = plan_decode(c, D, q.q_heads);
    if (plan.items > INT32_MAX)
        return cudaErrorInvalidValue;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    DecodeParams p;
    p.c = c;
    p.q = q;
    p.lens = lens;
    p.rep = plan.rep;
    p.groups = plan.groups;
    p.total = reinterpret_cast<long long *>(ws);
    p.start = reinterpret_cast<long long *>(ws + plan.start_at);
    p.parts = reinterpret_cast<float *>(ws + plan.parts_at);
    p.rows = plan.rows;
    if (D == 128)
        return plan.nt == 1 ? launch<128, 1>(p, plan, stream) : launch<128, 2>(p, plan, stream);
    return plan.nt == 1 ? launch<64, 1>(p, plan, stream) : launch<64, 2>(p, plan, stream);
}

}  // namespace tq
