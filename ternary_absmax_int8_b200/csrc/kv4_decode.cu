// kv4_decode.cu -- attention of one new token per sequence over the 4-bit
// cache (include/tq.h, tq_kv4_decode).
//
// Every cached code is read once, so HBM sets the floor: (D + 4) bytes a
// token and head. At 6.5 TB/s that is 13e12 codes a second against 36e12
// instruction lanes, so a code may cost no more than about two lanes of work
// from load to result, and scalar products cannot do it (4 query heads x 2
// products). Hence the warp-level MMA, with keys on its 16-row side and the
// query heads that share them on its 8-column side, S^T = K q^T and
// O^T = V^T P^T. (The tensor-memory MMA wants 64 or 128 rows and its operands
// in shared memory: codes would be written back there, 4 bytes for each one
// read.) Which codes form an MMA's k range is free as long as both operands
// agree, so a lane takes contiguous bytes of a row and nothing moves between
// lanes but P, by one transposing move per 8 x 8 block.
//  - Scores: m16n8k32, u8 x s8 -> s32. A word of 8 codes masked with 0F0F0F0F
//    and F0F0F0F0 is two operand registers as it stands (the upper one 16
//    times too large): two instructions for eight codes. The query is a whole
//    number of 23 bits in three signed bytes, against the power of two above
//    its head's largest value; they fill the columns that 4 heads would leave
//    empty: upper and middle byte of head t in columns 2t and 2t + 1, the lower
//    byte in a second product. The sums are exact; -8 sum(q), for the stored
//    code + 8, is their starting value.
//  - Values: m16n8k16 fp16. A nibble n masked in place under the exponent of
//    1024 (of 64, one nibble higher) is the fp16 number 1024 + n (64 + n), and
//    one subtraction leaves the code, exactly. (Leaving it out, with masked
//    nibbles as subnormals n 2^-24 and the +8 taken off the sums, is cheaper
//    by 4 in 10, but the matrix unit aligns a subnormal's products as if it
//    were 2^-14: the results lost up to 2^-13 of the weights' sum.) Weights
//    cannot be bytes: a long context holds many that are tiny and count.
// Running maxima and sums are fp32. A weight times its value's scale is
// rounded to fp16 (2^-11) against the largest value scale of its tile; a
// tile's 64 products are added up by the MMA, the tiles in fp32 registers.
//
// Work split: the tiles (64 tokens of one sequence and head) of all sequences
// form one list, cut into equal shares per SM and per warp, whatever the
// sequences' lengths. Each warp walks its share alone: a private ring of
// shared-memory stages filled by bulk copies (a tile of one page is one copy
// of 64 (D + 4) bytes) and no barrier with other warps until its share is
// done. Then the warps of an SM that ended in one sequence are merged in
// shared memory, and kv4_combine_kernel joins what several SMs hold of one
// sequence, in a fixed order.
//
// Measured (20 heads on 5 of 128, pages of 64): one sequence of 777 tokens
// 6.4 us; 24 of up to 8191 (65 MB) 22.1 us from memory, 2.9 TB/s, 20.4 with the
// cache in L2; one of 262143 (173 MB) 38.1 us, 4.5 TB/s. Of the long call the
// start (lengths, page numbers, first copies) takes 2.7 us, merge and join 4;
// between them it runs at 6 TB/s with the issue slots 57%, ALUs 54% and matrix
// pipes 28% busy. The batch's tiles are a third of that, and its start and end,
// with more joins, the same.
#include <algorithm>

#include "kv4_common.cuh"
#include "quant_core.cuh"
#include "tc_common.cuh"

#include <cuda_fp16.h>

namespace tq {

namespace {

constexpr int kTile = 64;      // tokens of a tile
constexpr int kMaxCtas = 160;  // of a launch: one per SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Warps of a CTA (one CTA per SM) and ring stages per warp: as many as shared
// memory and the registers for the heads' results allow (a tile is 2000 cycles
// of latency to a warp; with 10 warps instead of 12 of D = 128 a long context
// took 43 us, not 39). HG groups of four heads share a pass over the codes.
template <int D, int HG>
struct DecodeShape {
    static constexpr int kWarps = HG == 4 ? 8 : D == 128 ? 12 : 16;
    static constexpr int kStages = D == 128 ? (HG == 4 ? 3 : 2) : (HG == 4 ? 6 : 3);
    static constexpr int kStageBytes = kTile * (D + 4);
    static constexpr int kHeads = 4 * HG;      // heads of an item
    static constexpr int kPartFloats = D + 2;  // one head's part: values, maximum, sum
};

struct Crossing;

struct DecodeParams {
    Kv4View c;
    Kv4Query q;
    const int32_t *lens;
    int rep;     // query heads per key/value head
    int groups;  // items per key/value head: of up to 4 HG query heads each
    int rows;    // heads of a part: min(rep, 4 HG)
    Divisor by_groups, by_ctas;
    // workspace
    Crossing *crossing;  // [CTAs]
    float *parts;               // [warps of all CTAs][2][rows][D + 2]
};

// A sequence's keys that its query sees: [begin, end), tiles of 64 from the
// one that holds begin.
struct Span {
    int begin, end, tile0, tiles;
};

__device__ __forceinline__ Span span_of_length(const DecodeParams &p, int len)
{
    Span s;
    s.end = len;
    s.begin = p.q.window > 0 ? max(0, s.end - p.q.window) : 0;
    s.tile0 = s.begin / kTile;
    s.tiles = (s.end + kTile - 1) / kTile - s.tile0;
    return s;
}

__device__ __forceinline__ Span span_of(const DecodeParams &p, int b)
{
    return span_of_length(p, kv4_len(p.c, p.lens, b));
}

// `count` tiles in `n` shares: the first `more` have each + 1, the others each.
struct Shares {
    int each, more;

    __device__ __forceinline__ Shares(int count, int n) : each(count / n), more(count - each * n) {}
    __device__ __forceinline__ Shares(int count, int n, const Divisor &by_n)
        : each(by_n.of(count)), more(count - each * n)
    {
    }
    __device__ __forceinline__ int first(int i) const { return i * each + min(i, more); }
    __device__ __forceinline__ int of(int tile) const  // the share that holds tile
    {
        const int split = more * (each + 1);
        return tile < split ? tile / (each + 1) : more + (tile - split) / each;
    }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
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
// (w & mask) | c in one instruction: left to itself the compiler takes two,
// as only one of the constants fits the instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t low4(uint32_t w)
{
    return sub_half2(and_or(w, 0x000F000Fu, 0x64006400u), 0x64086408u);  // 1024 + n - 1032
}
__device__ __forceinline__ uint32_t high4(uint32_t w)
{
    return sub_half2(and_or(w, 0x00F000F0u, 0x54005400u), 0x54805480u);  // 64 + n - 72
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

// The heads' running results over part of a sequence. Lane (g, t) holds head
// 4j + t of group j: elements d and d + 1 of d-tile i at o[j / 2][i][j % 2] and
// [2 + j % 2], d = g D/8 + 2 i.
template <int D, int HG>
struct Running {
    static constexpr int kV = (HG + 1) / 2;  // value products' column tiles
    float o[kV][D / 16][4];
    float m[HG], l[HG];  // maximum (accumulator x key scale), sum over the lane's tokens

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[v][i][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < HG; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.0f;
        }
    }
};

// The heads' queries as MMA operands: [column tile][high, low nibbles][k step].
template <int D, int HG>
struct Queries {
    static constexpr int kT = HG + (HG + 1) / 2;  // upper + middle bytes, then lower bytes
    uint32_t b[kT][2][D / 64][2];
    int init[kT][2];  // -128 sum of the column's bytes; columns 2t, 2t + 1
    float mul[HG];    // accumulator x key scale -> log2 of the weight; head 4j + t
};

// Lane (g, t) takes part t of head 4j + g/2 of each group j: bf16 as stored.
template <int D, int HG>
__device__ __forceinline__ void fetch_queries(const DecodeParams &p, long long row, int head0,
                                              int heads, uint4 (&raw)[HG][D / 32])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        const int h = 4 * j + (g >> 1);
        const bool real = h < heads;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q.q + row + (long long)(head0 + (real ? h : 0)) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            raw[j][i] = real ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    }
}

// Its values go into both columns of a pair: upper byte in the even one,
// middle in the odd.
template <int D, int HG>
__device__ __forceinline__ void convert_queries(const DecodeParams &p,
                                                const uint4 (&raw)[HG][D / 32],
                                                Queries<D, HG> &q)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t y[HG][D / 4];  // the values' three bytes
    float mul[HG];
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        float v[D / 4];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 u = raw[j][i];
            v[8 * i] = bf16_lo(u.x), v[8 * i + 1] = bf16_hi(u.x);
            v[8 * i + 2] = bf16_lo(u.y), v[8 * i + 3] = bf16_hi(u.y);
            v[8 * i + 4] = bf16_lo(u.z), v[8 * i + 5] = bf16_hi(u.z);
            v[8 * i + 6] = bf16_lo(u.w), v[8 * i + 7] = bf16_hi(u.w);
        }
        // As multiples of 2^(k - 21), 2^k <= the head's largest magnitude
        // < 2^(k + 1): bf16 values down to 2^-14 of it are exact.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
            top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int k = max(int(top >> 23) - 127, -100);
        const float up = __uint_as_float(uint32_t(21 - k + 127) << 23);
        // Adding 1.5 2^23 leaves the whole number in the low bits; with 128
        // added in each byte, a byte less 128 is the signed digit.
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
            y[j][i] = __float_as_uint(fmaf(v[i], up, 12582912.0f)) - 0x4B400000u + 0x00808080u;
        // the unit, scale and the change to base 2; an infinite or NaN query
        // makes all of its head's scores NaN
        mul[j] = __uint_as_float(uint32_t(k - 21 + 127) << 23) * (p.q.scale * kLog2e);
        mul[j] = fmaxf(mul[j], 1.40129846e-45f);  // no zero, which masks would meet
        if (top >= 0x7F800000u)
            mul[j] = NAN;
        q.mul[j] = __shfl_sync(0xffffffffu, mul[j], 8 * t);
    }
#pragma unroll
    for (int c = 0; c < Queries<D, HG>::kT; ++c) {
        // Lower bytes: of group 2 (c - HG) in the even column, of the next in
        // the odd one.
        const bool lower = c >= HG;
        const int j0 = lower ? 2 * (c - HG) : c;
        const bool odd = g & 1;
        const uint32_t pick = lower ? 0u : odd ? 1u : 2u;  // byte of y
        const uint32_t sel = pick | (pick + 4) << 4;       // of two values
        int sum = 0;
#pragma unroll
        for (int u = 0; u < D / 32; ++u)  // a word of a key row: 8 codes
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // its high nibbles: odd elements; its low
                uint32_t z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 8 * u + 2 * i + (half == 0);
                    z[i] = y[j0][e];
                    if (lower)  // a group beyond the last: digits 0
                        z[i] = odd ? (j0 + 1 < HG ? y[j0 + 1 < HG ? j0 + 1 : j0][e] : 0x80u) : z[i];
                }
                const uint32_t w = __byte_perm(__byte_perm(z[0], z[1], sel),
                                               __byte_perm(z[2], z[3], sel), 0x5410) ^
                                   0x80808080u;
                sum = __dp4a(int(w), 0x01010101, sum);
                q.b[c][half][u >> 1][u & 1] = w;
            }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        q.init[c][0] = -128 * __shfl_sync(0xffffffffu, sum, 8 * t);
        q.init[c][1] = -128 * __shfl_sync(0xffffffffu, sum, 8 * t + 4);
    }
}

// One tile: scores, softmax step, weighted values. `sps` tokens of the tile
// come from one page: in shared memory its key codes, value codes, key scales
// and value scales follow one another, blocks of sps (D + 4) bytes. Tokens
// outside [begin, end) and pages whose bit of `good` is clear take no part
// (tested in every tile: a second copy of this code without the tests costs a
// short call more in instruction fetches than a long one gains).
template <int D, int HG>
__device__ __forceinline__ void tile_step(const uint8_t *stage, int lg_sps, int j0, int begin,
                                          int end, uint32_t good, const Queries<D, HG> &q,
                                          Running<D, HG> &r)
{
    constexpr int kV = Running<D, HG>::kV, kT = Queries<D, HG>::kT;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int sps = 1 << lg_sps;
    const int row0 = token_at(g);
    float x[HG][4][2];
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
        int s[kT][4];
#pragma unroll
        for (int c = 0; c < kT; ++c) {
            s[c][0] = s[c][2] = q.init[c][0];
            s[c][1] = s[c][3] = q.init[c][1];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t mask = half ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const uint32_t a0 = w0[2 * u] & mask, a1 = w1[2 * u] & mask;
                const uint32_t a2 = w0[2 * u + 1] & mask, a3 = w1[2 * u + 1] & mask;
#pragma unroll
                for (int c = 0; c < kT; ++c)
                    mma_u8s8(s[c], a0, a1, a2, a3, q.b[c][half][u][0], q.b[c][half][u][1]);
            }
            if (half == 0) {  // the high nibbles stood for 16 times their codes
#pragma unroll
                for (int c = 0; c < kT; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[c][i] >>= 4;
            }
        }
        bool in[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[h] = unsigned(j0 + mt * 16 + row0 + 8 * h - begin) < unsigned(end - begin) &&
                    ((good >> blk) & 1u);
            if (!in[h])
                sv[mt][h] = 0;
        }
#pragma unroll
        for (int j = 0; j < HG; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float upper = float(s[j][2 * h] * 256 + s[j][2 * h + 1]);
                const float lower = float(s[HG + j / 2][2 * h + (j & 1)]);
                const float z = fmaf(upper, 256.0f, lower) * ks[h];
                x[j][mt][h] = in[h] ? z : -INFINITY;
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

    // Running maximum per head.
    float mn[HG];
    bool grew = false;
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        float v = fmaxf(x[j][0][0], x[j][0][1]);
#pragma unroll
        for (int mt = 1; mt < 4; ++mt)
            v = fmaxf(v, fmaxf(x[j][mt][0], x[j][mt][1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        mn[j] = fmaxf(r.m[j], v);
        grew = grew || mn[j] != r.m[j];
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int j = 0; j < HG; ++j) {
            // nothing seen yet: nothing to scale (and no infinity minus itself)
            const float a = r.m[j] == mn[j] ? 1.0f : ex2((r.m[j] - mn[j]) * q.mul[j]);
            r.l[j] *= a;
            r.m[j] = mn[j];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                r.o[j / 2][i][j & 1] *= a;
                r.o[j / 2][i][2 + (j & 1)] *= a;
            }
        }
    }

    // Weights, and the operands P^T of the second product.
    uint32_t pb[kV][4][2];
    float c[HG];
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        const float top = r.m[j] * q.mul[j];
        c[j] = top == -INFINITY ? 0.0f : -top;  // nothing seen, or nothing above -FLT_MAX
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float by = __uint_as_float(sv[mt][h]) * rs;
            float w[HG];
#pragma unroll
            for (int j = 0; j < HG; ++j) {
                w[j] = ex2(fmaf(x[j][mt][h], q.mul[j], c[j]));
                r.l[j] += w[j];
                w[j] *= by;
            }
#pragma unroll
            for (int v = 0; v < kV; ++v)
                pb[v][mt][h] = transpose8x8(pack_half(w[2 * v], 2 * v + 1 < HG ? w[2 * v + 1] : 0.0f));
        }
    // Values: lane g's D/8 consecutive elements, 8 (one word) at a time.
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
        float acc[kV][4][4];
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[v][i][j] = 0.0f;
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
                for (int v = 0; v < kV; ++v)
                    mma_f16(acc[v][i], a0, a1, a2, a3, pb[v][mt][0], pb[v][mt][1]);
            }
        }
#pragma unroll
        for (int j = 0; j < HG; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float &o = r.o[j / 2][4 * u + i][2 * h + (j & 1)];
                    o = fmaf(acc[j / 2][i][2 * h + (j & 1)], sref, o);
                }
    }
}

// The lane's result for head 4j + t, element pair i.
template <int D, int HG>
__device__ __forceinline__ float2 value_pair(const Running<D, HG> &r, int j, int i)
{
    return make_float2(r.o[j / 2][i][j & 1], r.o[j / 2][i][2 + (j & 1)]);
}

// The sums of weights lie spread over the lanes of a column: add them up. Where
// the largest score is above fp32's numbers no weight is known.
template <int D, int HG>
__device__ __forceinline__ void close_sums(Running<D, HG> &r, const Queries<D, HG> &q)
{
#pragma unroll
    for (int j = 0; j < HG; ++j) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1)
            r.l[j] += __shfl_xor_sync(0xffffffffu, r.l[j], o);
        if (r.m[j] * q.mul[j] == INFINITY)
            r.l[j] = NAN;
    }
}

// A part [heads][D + 2]: values, then the maximum (base 2) and the sum. For
// heads beyond `rows` nothing is stored.
template <int D, int HG>
__device__ __forceinline__ void store_part(const Running<D, HG> &r, const Queries<D, HG> &q,
                                           float *part, int rows)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        const int h = 4 * j + t;
        if (h >= rows)
            continue;
        float *row = part + h * (D + 2);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2 *>(row + g * (D / 8) + 2 * i) = value_pair(r, j, i);
        if (g == 0)
            *reinterpret_cast<float2 *>(row + D) =
                make_float2(r.m[j] == -INFINITY ? -INFINITY : r.m[j] * q.mul[j], r.l[j]);
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

template <int D, int HG>
__device__ __forceinline__ void store_final(const DecodeParams &p, const Running<D, HG> &r,
                                            const Queries<D, HG> &q, int b, int head0, int heads)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < HG; ++j) {
        const int h = 4 * j + t;
        if (h >= heads)
            continue;
        const float inv = inverse_sum(r.l[j]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            store_out<D>(p, b, head0 + h, g * (D / 8) + 2 * i, value_pair(r, j, i), inv);
        if (p.q.lse && g == 0)
            p.q.lse[(long long)b * p.q.q_heads + head0 + h] = log_sum(r.m[j] * q.mul[j], r.l[j]);
    }
}

// Parts of one head joined one after another: v = sum_k 2^(m_k - m) v_k, and l
// alike, m the largest m_k.
struct Joined {
    float2 v = make_float2(0.0f, 0.0f);
    float m = -INFINITY, l = 0.0f;

    __device__ __forceinline__ void rescale(float top)  // top >= m
    {
        const float a = m == top ? 1.0f : ex2(m - top);
        v.x *= a;
        v.y *= a;
        l *= a;
        m = top;
    }
    __device__ __forceinline__ void add_below(float2 x, float2 ml)  // ml.x <= m
    {
        const float b = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
        v.x = fmaf(x.x, b, v.x);
        v.y = fmaf(x.y, b, v.y);
        l = fmaf(ml.y, b, l);
    }
    __device__ __forceinline__ void add(float2 x, float2 ml)
    {
        rescale(fmaxf(m, ml.x));
        add_below(x, ml);
    }
};

template <int D>
__device__ __forceinline__ void store_joined(const DecodeParams &p, const Joined &r, int b,
                                             int head, int d)
{
    store_out<D>(p, b, head, d, r.v, inverse_sum(r.l));
    if (p.q.lse && d == 0)
        p.q.lse[(long long)b * p.q.q_heads + head] = log_sum(r.m, r.l);
}

// The item that a CTA's share begins in, where it began in an earlier CTA: the
// combine kernel's work list.
struct alignas(8) Crossing {
    int b;       // its sequence; -1: none, or one that began further back than the CTA before
    int head0, heads;  // its query heads
    int parts;   // CTAs that hold a part of it, from the one before on
    int warp0;   // the warp that it begins in there
    int ended;   // its last part is in that CTA's first warp's slot 0
};

struct Segment {  // a warp's last stretch, for the merge within the CTA
    int item;         // -1: none
    int first, last;  // the item's tiles [first, last) among all
    int b, head0, heads;  // its sequence and query heads
};

template <int D, int HG>
__global__ void __launch_bounds__(DecodeShape<D, HG>::kWarps * 32, 1)
    kv4_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using S = DecodeShape<D, HG>;
    constexpr int kThreads = S::kWarps * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[S::kWarps][S::kStages];
    __shared__ int scan[S::kWarps], scan2[S::kWarps];
    __shared__ int warp_base[S::kWarps];  // tiles before the warp's first sequence
    __shared__ int warp_b[S::kWarps];     // that sequence
    __shared__ Segment seg[S::kWarps];
    __shared__ int ended[S::kWarps];  // item whose end is in the warp's slot 0, or -1

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        for (int s = 0; s < S::kStages; ++s)
            mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
    const uint64_t policy = policy_evict_first();
    pdl_wait();
    pdl_launch_dependents();

    // Tiles of all sequences; rows of a sequence without a visible token are
    // written here, its CTA taken in turn. Up to 32 sequences each warp sums up
    // for itself; beyond, the CTA does, a block of lengths at a time.
    const int hg = p.c.kv_heads * p.groups;
    auto tiles_of = [&](int b) {
        if (b >= p.c.batch)
            return 0;
        return span_of(p, b).tiles * hg;
    };
    auto empty_rows = [&](int b, int n) {
        if (n != 0 || b >= p.c.batch || b % int(gridDim.x) != int(blockIdx.x))
            return;
#pragma unroll 1
        for (int h = 0; h < p.q.q_heads; ++h) {
#pragma unroll 1
            for (int d = 0; d < D; d += 2)
                store_out<D>(p, b, h, d, make_float2(0.0f, 0.0f), 0.0f);
            if (p.q.lse)
                p.q.lse[(long long)b * p.q.q_heads + h] = -INFINITY;
        }
    };
    auto running_sum = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += u;
        }
        return v;
    };
    int b = 0, seq0 = 0, total = 0;  // the warp's first sequence, tiles before it
    int len = 0;                     // its length
    int cta_first, cta_stop;
    if (p.c.batch <= 32) {
        const Span mine = lane < p.c.batch ? span_of(p, lane) : Span{0, 0, 0, 0};
        const int own = mine.tiles * hg;
        if (warp == S::kWarps - 1)
            empty_rows(lane, own);
        const int incl = running_sum(own);
        total = __shfl_sync(0xffffffffu, incl, 31);
        const Shares ctas(total, gridDim.x, p.by_ctas);
        cta_first = ctas.first(blockIdx.x);
        cta_stop = ctas.first(blockIdx.x + 1);
        const int at = cta_first + Shares(cta_stop - cta_first, S::kWarps).first(warp);
        b = min(31, __popc(__ballot_sync(0xffffffffu, incl <= at)));
        seq0 = __shfl_sync(0xffffffffu, incl - own, b);
        len = __shfl_sync(0xffffffffu, mine.end, b);
    } else {
        int mine = 0, own = 0;  // own: of the thread's sequence in the first block
        for (int i = threadIdx.x; i < p.c.batch; i += kThreads) {
            const int n = tiles_of(i);
            mine += n;
            if (i < kThreads)
                own = n;
            empty_rows(i, n);
        }
        int incl = running_sum(own);
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 31) {
            scan[warp] = incl;
            scan2[warp] = mine;
        }
        __syncthreads();
        int base = 0, before = 0;  // before: tiles of the sequences before this block
        for (int w = 0; w < S::kWarps; ++w) {
            total += scan2[w];
            base += w < warp ? scan[w] : 0;
            before += scan[w];
        }
        const Shares ctas(total, gridDim.x, p.by_ctas);
        cta_first = ctas.first(blockIdx.x);
        cta_stop = ctas.first(blockIdx.x + 1);
        const Shares warps(cta_stop - cta_first, S::kWarps);
        auto place = [&](int i, int lo, int n) {  // sequence i has tiles [lo, lo + n)
            for (int w = 0; w < S::kWarps; ++w) {
                const int t = cta_first + warps.first(w);
                if (t < cta_stop && t >= lo && t < lo + n) {
                    warp_b[w] = i;
                    warp_base[w] = lo;
                }
            }
        };
        place(threadIdx.x, base + incl - own, own);
        for (int b0 = kThreads; b0 < p.c.batch && before < cta_stop;
             b0 += kThreads) {
            own = tiles_of(b0 + threadIdx.x);
            incl = running_sum(own);
            __syncthreads();
            if (lane == 31)
                scan[warp] = incl;
            __syncthreads();
            base = before;
            for (int w = 0; w < S::kWarps; ++w) {
                base += w < warp ? scan[w] : 0;
                before += scan[w];
            }
            place(b0 + threadIdx.x, base + incl - own, own);
        }
        __syncthreads();
        if (cta_first + warps.first(warp) < cta_stop) {
            b = warp_b[warp];
            seq0 = warp_base[warp];
            len = kv4_len(p.c, p.lens, b);
        }
    }
    const Shares warps(cta_stop - cta_first, S::kWarps);
    const int warp_first = cta_first + warps.first(warp), stop = cta_first + warps.first(warp + 1);
    int at = warp_first;

    uint8_t *ring = smem + warp * (S::kStages * S::kStageBytes);
    const int worker = blockIdx.x * S::kWarps + warp;
    const int lg_sps = min(p.c.lg_ps, 6), sps = 1 << lg_sps;
    const int per_tile = kTile >> lg_sps;  // page stretches of a tile
    uint32_t phase = 0;                    // one bit per stage
    Running<D, HG> run;
    Queries<D, HG> qs;
    bool fine = true;
    Segment last{-1, 0, 0, 0, 0, 0};
    Crossing cross{-1, 0, 0, 0, 0, 0};
    int end_item = -1;
    while (at < stop && fine) {
        Span sp = span_of_length(p, len);
        while (sp.tiles * hg <= at - seq0 && b + 1 < p.c.batch) {
            seq0 += sp.tiles * hg;  // on to the sequence with tile `at`
            len = kv4_len(p.c, p.lens, ++b);
            sp = span_of_length(p, len);
        }
        if (sp.tiles * hg <= at - seq0)
            break;  // only if lengths change while the kernel runs
        const int ig = (at - seq0) / sp.tiles;  // head group of the sequence
        const int item0 = seq0 + ig * sp.tiles;
        const int n0 = at - item0;
        const int n1 = min(sp.tiles, stop - item0);
        const int kvh = p.by_groups.of(ig), grp = ig - kvh * p.groups;
        const int head0 = kvh * p.rep + grp * S::kHeads;
        const int heads = min(S::kHeads, p.rep - grp * S::kHeads);
        // Page numbers of the next tiles, one lane each (a page of 128 tokens
        // serves two tiles); -1 for one outside the cache.
        const int lg_batch = lg_sps - 1;  // log2 of the tiles that 32 lanes cover
        int batch0 = n0 >> lg_batch, page = 0;
        bool checked = false;
        auto key_of = [&] { return ((sp.tile0 + (batch0 << lg_batch)) << 6) + (lane << lg_sps); };
        auto wanted = [&](int j) {
            // (pages in front of a window may have gone to other sequences)
            return j < sp.end && j + sps > sp.begin;
        };
        auto look_up = [&] {
            if (wanted(key_of()))
                page = p.c.table[(long long)b * p.c.max_pages + (key_of() >> p.c.lg_ps)];
            checked = false;
        };
        look_up();
        uint4 raw[HG][D / 32];  // (both are on their way together)
        fetch_queries<D, HG>(p, b * p.q.q_stride, head0, heads, raw);
        const long long head_at = kvh * p.c.head_bytes<D>();
        auto fetch = [&](int n, int s) {  // tile n of the sequence into stage s
            const int tile = sp.tile0 + n;
            if ((n >> lg_batch) != batch0) {
                batch0 = n >> lg_batch;
                look_up();
            }
            if (!checked) {
                if (!wanted(key_of())) {
                    page = -1;
                } else if (unsigned(page) >= unsigned(p.c.num_pages)) {
                    page = -1;
                    atomicOr(p.c.err, kErrBadPage);
                }
                checked = true;
            }
            const int i0 = (n & ((1 << lg_batch) - 1)) * per_tile;
            uint8_t *dst = ring + s * S::kStageBytes;
            uint64_t *bar = &bars[warp][s];
            const int pg = __shfl_sync(0xffffffffu, page, i0 + (lane & (per_tile - 1)));
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
        if (n0 > 0 && at == cta_first) {
            // (while the first tile is on its way)
            const Shares ctas(total, gridDim.x, p.by_ctas);
            const int first0 = ctas.first(blockIdx.x - 1);
            if (item0 >= first0) {
                const int end = item0 + sp.tiles, cta1 = ctas.of(end - 1);
                const int first1 = ctas.first(cta1);
                cross.b = b;
                cross.head0 = head0;
                cross.heads = heads;
                cross.parts = cta1 - int(blockIdx.x) + 2;
                cross.warp0 = Shares(cta_first - first0, S::kWarps).of(item0 - first0);
                cross.ended = end < first1 + Shares(ctas.first(cta1 + 1) - first1, S::kWarps).first(1);
            }
        }
        convert_queries<D, HG>(p, raw, qs);
        run.clear();
#pragma unroll 1
        for (int n = n0, s = 0; n < n1; ++n, s = s + 1 == S::kStages ? 0 : s + 1) {
            fine = mbar_wait_warp(&bars[warp][s], (phase >> s) & 1u, p.c.err);
            if (!fine) {
                // The merge writes where the rings are, and the CTA may retire: not
                // while copies of this and the next tiles are on their way.
                for (int i = n; i < n1 && i < n + S::kStages; ++i) {
                    mbar_wait_warp(&bars[warp][s], (phase >> s) & 1u, p.c.err);
                    s = s + 1 == S::kStages ? 0 : s + 1;
                }
                break;
            }
            phase ^= 1u << s;
            const uint8_t *stage = ring + s * S::kStageBytes;
            const int j0 = (sp.tile0 + n) * kTile;
            const uint32_t here = (good >> (4 * s)) & 15u;
            tile_step<D, HG>(stage, lg_sps, j0, sp.begin, sp.end, here, qs, run);
            __syncwarp();
            if (n + S::kStages < n1)
                good = (good & ~(15u << (4 * s))) | fetch(n + S::kStages, s) << (4 * s);
        }
        if (!fine)
            break;
        close_sums<D, HG>(run, qs);
        at = item0 + n1;
        if (n0 == 0 && n1 == sp.tiles) {
            store_final<D, HG>(p, run, qs, b, head0, heads);
        } else if (n1 == sp.tiles && at < stop) {
            // the end of a sequence that other warps began
            store_part<D, HG>(run, qs, p.parts + (long long)(2 * worker) * p.rows * (D + 2),
                              min(p.rows, heads));
            end_item = b * hg + ig;
        } else {
            last = Segment{b * hg + ig, item0, item0 + sp.tiles, b, head0, heads};
        }
    }

    if (threadIdx.x == 0)
        p.crossing[blockIdx.x] = cross;
    // A part that no other warp of this CTA adds to needs no merge.
    const bool alone = last.item >= 0 && fine &&
                       (warp == 0 || last.first >= warp_first) &&
                       (stop == cta_stop || last.last <= stop);
    if (alone) {
        store_part<D, HG>(run, qs, p.parts + (long long)(2 * worker + 1) * p.rows * (D + 2), p.rows);
        last.item = -1;
    }
    // Merge what the CTA's warps hold of one sequence: the shares that ended in
    // it (shared memory) and the one behind them that ended it and went on.
    if (lane == 0) {
        seg[warp] = last;
        ended[warp] = end_item;
    }
    if (!__syncthreads_or(last.item >= 0))  // also: every ring is idle
        return;
    float *mine_at = reinterpret_cast<float *>(smem) + warp * (S::kHeads * S::kPartFloats);
    if (last.item >= 0 && fine)
        store_part<D, HG>(run, qs, mine_at, S::kHeads);
    __syncthreads();
    // Runs of warps whose shares ended in one item; a task is one head's 64
    // values (32 element pairs) of a run, a warp's at a time.
    const int item_w = lane < S::kWarps ? seg[lane].item : -1;
    const int item_before = __shfl_up_sync(0xffffffffu, item_w, 1);
    uint32_t starts = __ballot_sync(0xffffffffu, item_w >= 0 && (lane == 0 || item_w != item_before));
    constexpr int kTasks = S::kHeads * (D / 64);  // of a run
    int task = warp;
    while (starts) {
        if (task >= kTasks) {
            task -= kTasks;
            starts &= starts - 1;
            continue;
        }
        const int w = __ffs(starts) - 1;
        const Segment sg = seg[w];
        const int n = __popc(__ballot_sync(0xffffffffu, item_w == sg.item));
        const int h = task / (D / 64), d = (task % (D / 64)) * 64 + 2 * lane;
        task += S::kWarps;
        if (h >= sg.heads)
            continue;
        const bool more = w + n < S::kWarps && ended[w + n] == sg.item;
        const int from = cta_first + warps.first(w), to = cta_first + warps.first(w + n);
        const bool whole = from <= sg.first && (more || to >= sg.last);
        const float *first =
            reinterpret_cast<const float *>(smem) + (w * S::kHeads + h) * S::kPartFloats;
        const float *tail =
            p.parts + ((long long)(2 * (blockIdx.x * S::kWarps + w + n)) * p.rows + h) * (D + 2);
        float2 ml_tail = make_float2(-INFINITY, 0.0f), x_tail = make_float2(0.0f, 0.0f);
        if (more) {  // from L2, while the others are added up
            ml_tail = *reinterpret_cast<const float2 *>(tail + D);
            x_tail = *reinterpret_cast<const float2 *>(tail + d);
        }
        Joined r;
        float2 ml[S::kWarps];
#pragma unroll
        for (int k = 0; k < S::kWarps; ++k) {
            ml[k] = make_float2(-INFINITY, 0.0f);
            if (k < n)
                ml[k] = *reinterpret_cast<const float2 *>(
                    first + k * (S::kHeads * S::kPartFloats) + D);
            r.m = fmaxf(r.m, ml[k].x);
        }
#pragma unroll
        for (int k = 0; k < S::kWarps; ++k)
            if (k < n)
                r.add_below(*reinterpret_cast<const float2 *>(
                                first + k * (S::kHeads * S::kPartFloats) + d),
                            ml[k]);
        if (more)
            r.add(x_tail, ml_tail);
        if (whole) {
            store_joined<D>(p, r, sg.b, sg.head0 + h, d);
        } else {
            float *dst =
                p.parts + ((long long)(2 * (blockIdx.x * S::kWarps + w) + 1) * p.rows + h) * (D + 2);
            *reinterpret_cast<float2 *>(dst + d) = r.v;
            if (d == 0)
                *reinterpret_cast<float2 *>(dst + D) = make_float2(r.m, r.l);
        }
    }
}

// Joins the parts of each item that several CTAs hold, in the order of the
// tiles. Block (c - 1, h): head h of the item that CTA c's share begins in, if
// it began in CTA c - 1. Groups of D/2 threads take every kGroups-th part each,
// eight loads in flight at once.
constexpr int kCombineThreads = 128;

template <int D, int HG>
__global__ void __launch_bounds__(kCombineThreads)
    kv4_combine_kernel(const __grid_constant__ DecodeParams p)
{
    using S = DecodeShape<D, HG>;
    constexpr int kGroups = kCombineThreads / (D / 2), kBatch = 8;
    __shared__ float2 vs[kGroups][D / 2], mls[kGroups];
    pdl_wait();
    pdl_launch_dependents();
    const int c0 = blockIdx.x, h = blockIdx.y;
    const Crossing x = p.crossing[c0 + 1];
    if (x.b < 0 || h >= x.heads)
        return;
    // A CTA holds its part in the slot 1 of the first of its warps that worked
    // on it, or, where its first warp ended the item and went on, in slot 0.
    const int n = x.parts;
    const int group = threadIdx.x / (D / 2), d = 2 * (threadIdx.x % (D / 2));
    Joined r;
#pragma unroll 1
    for (int k0 = group; k0 < n; k0 += kGroups * kBatch) {
        float2 v[kBatch], ml[kBatch];
        float top = r.m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + i * kGroups;
            v[i] = make_float2(0.0f, 0.0f);
            ml[i] = make_float2(-INFINITY, 0.0f);
            if (k < n) {
                const int slot = 2 * ((c0 + k) * S::kWarps + (k == 0 ? x.warp0 : 0)) + 1 -
                                 (k == n - 1 && x.ended);
                const float *part = p.parts + ((long long)slot * p.rows + h) * (D + 2);
                v[i] = *reinterpret_cast<const float2 *>(part + d);
                ml[i] = *reinterpret_cast<const float2 *>(part + D);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            top = fmaxf(top, ml[i].x);
        r.rescale(top);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            r.add_below(v[i], ml[i]);
    }
    vs[group][d / 2] = r.v;
    if (d == 0)
        mls[group] = make_float2(r.m, r.l);
    __syncthreads();
    if (group == 0) {
        for (int i = 1; i < kGroups; ++i)
            r.add(vs[i][d / 2], mls[i]);
        store_joined<D>(p, r, x.b, x.head0 + h, d);
    }
}

struct DecodePlan {
    int rep, hg, groups, rows, ctas, warps;
    long long items, tiles;  // tiles: at most so many
    size_t parts_at, bytes;
};

DecodePlan plan_decode(const Kv4View &c, int D, int q_heads)
{
    DecodePlan d;
    d.rep = q_heads / c.kv_heads;
    d.hg = d.rep <= 4 ? 1 : d.rep <= 8 ? 2 : 4;
    d.groups = (d.rep + 4 * d.hg - 1) / (4 * d.hg);
    d.rows = std::min(d.rep, 4 * d.hg);
    d.ctas = std::min(device_sm_count(), kMaxCtas);
    d.warps = d.hg == 4 ? DecodeShape<128, 4>::kWarps
                        : D == 128 ? DecodeShape<128, 1>::kWarps : DecodeShape<64, 1>::kWarps;
    d.items = (long long)c.batch * c.kv_heads * d.groups;
    d.tiles = d.items * ((c.max_len() + kTile - 1) / kTile);
    d.parts_at = size_t(d.ctas) * sizeof(Crossing);
    d.bytes = d.parts_at +
              size_t(d.ctas) * d.warps * 2 * d.rows * size_t(D + 2) * sizeof(float);
    return d;
}

template <int D, int HG>
cudaError_t launch(const DecodeParams &p, const DecodePlan &plan, cudaStream_t stream)
{
    using S = DecodeShape<D, HG>;
    constexpr size_t kSmem = size_t(S::kWarps) * S::kStages * S::kStageBytes;
    static_assert(size_t(S::kWarps) * S::kHeads * S::kPartFloats * 4 <= kSmem, "merge space");
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_dev != dev) {
        e = cudaFuncSetAttribute(kv4_decode_kernel<D, HG>,
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
    e = cudaLaunchKernelEx(&cfg, kv4_decode_kernel<D, HG>, p);
    if (e != cudaSuccess || plan.tiles == plan.items || plan.ctas == 1)
        return e;  // at most one tile per item, or one CTA: nothing is shared
    cfg.gridDim = dim3(unsigned(plan.ctas - 1), unsigned(plan.rows));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, HG>, p);
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
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    DecodeParams p;
    p.c = c;
    p.q = q;
    p.lens = lens;
    p.rep = plan.rep;
    p.groups = plan.groups;
    p.crossing = reinterpret_cast<Crossing *>(ws);
    p.parts = reinterpret_cast<float *>(ws + plan.parts_at);
    p.rows = plan.rows;
    p.by_groups = Divisor(plan.groups);
    p.by_ctas = Divisor(plan.ctas);
    if (D == 128)
        return plan.hg == 1   ? launch<128, 1>(p, plan, stream)
               : plan.hg == 2 ? launch<128, 2>(p, plan, stream)
                              : launch<128, 4>(p, plan, stream);
    return plan.hg == 1   ? launch<64, 1>(p, plan, stream)
           : plan.hg == 2 ? launch<64, 2>(p, plan, stream)
                          : launch<64, 4>(p, plan, stream);
}

}  // namespace tq
