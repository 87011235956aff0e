// kv4_prefill.cu -- attention of any number of new tokens per sequence over
// the 4-bit cache (include/tq.h, tq_kv4_prefill), on the tensor cores.
//
// A CTA takes 256 query rows of one sequence and key/value head, a row being
// (token, query head of the group), tokens first: the heads that share keys
// share their expansion. Two tiles of 128 rows take turns on the tensor core
// and in the softmax, over tiles of 128 keys:
//   S = Q K^T (fp16; fp32 in tensor memory) -> softmax weights in registers,
//   one thread a row -> P (bf16) back into S's tensor memory -> O += P V.
// Roundings: a query row is bf16 values against the power of two above its
// largest (fp16 has 11 bits for their 8), a key code x scale of at most 3 + 8
// bits against the largest scale of its tile: both exact down to 2^-25 of that,
// so the scores and the logarithm of the sum are as exact as fp32 sums. Values
// are their codes (exact in bf16); a weight times its value's scale is rounded
// to bf16 once (2^-8: fp16's range would not do, as rows that do not see a key
// share its tile). Folding the value scales into the values instead is cheaper
// in the softmax, but a second bf16 rounding of every product.
//
// Each runs in warps of its own:
//   warps 0-3, 4-7  softmax of row tile 0, 1 (also the final division)
//   warps 8-11      codes -> 16-bit operands, swizzled for the MMA
//   warps 12, 14    issue the MMAs of row tile 0, 1
//   warp 13         looks up pages and issues bulk copies of packed codes, two
//                   tiles ahead
// The running maximum may lag by a factor 2^8 (weights up to 256 in fp32 and
// bf16 lose nothing): results in tensor memory are scaled anew only beyond.
//
// What bounds it: the softmax. Per pair of row tiles and key tile (D = 128) the
// tensor core needs 4 x 512 cycles, the 2 x 16384 exponentials 2048 at 16 a
// cycle, shared memory about 2300 (operands 1536, expanded codes 512, scales
// 256), all instructions about 2600 issue slots of each scheduler; but a pair of
// tiles takes 4200, as the two softmax warps of a scheduler do not cover the
// latencies of their own chain (scores from tensor memory, maximum, exponentials,
// weights back). A CTA's start takes 9000 cycles (lengths, keys and queries from
// memory, their expansion), its end 4500, the next CTA's arrival 1900. A prompt of
// 8192 tokens (20 heads on 5, D = 128; 344 GFLOP) takes 365 us, 942 TFLOP/s, 57%
// of a plain library product's rate (tensor pipe 39% busy, issue slots 51%,
// exponentials 41% over 4096 tokens). What was tried, in us for that prompt:
// scores of whole tiles, not ahead 519, of half tiles two ahead 422 (380 with all
// heads' long units first, 367 with the shorter start); four softmax warpgroups
// 490 where two took 449; the next scores fetched before the exponentials 534
// then (spills). Where 380 was the measure: registers dealt anew between the
// roles 386; the row tiles' softmax taking turns 394; a part of the exponentials
// as polynomials 387 and more; waits that sleep longer 395. Where 367 was: the
// next scores asked for before the weights' arrival is awaited, with the weights
// handed on then 375, in time 412 (spills).
//
// Few rows over a long cache are split along the keys, into parts that
// kv4_prefill_join_kernel adds up in order.
#include <algorithm>

#include "kv4_common.cuh"
#include "quant_core.cuh"
#include "tc_common.cuh"

#include <cuda_fp16.h>

namespace tq {

namespace {

constexpr int kRows = 256, kKeys = 128, kHalf = 64;
constexpr int kPrefillThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kScaleSlots = 3;

template <int D>
struct PrefillShape {
    // 128 rows or keys, bf16, in blocks of 64 values (rows of 128 bytes)
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kPacked = 128 * D / 2;  // a tile's key or value codes
};

struct PrefillParams {
    Kv4View c;
    Kv4Query q;
    const int32_t *tok_start, *lens;
    int T, rep, splits;
    Divisor by_rep, by_heads, by_splits;  // of rep, kv_heads, splits
    float *parts;   // [units][kv_heads][splits][256][D] where splits > 1
    float2 *sums;   // [units][kv_heads][splits][256]: maximum (base 2), sum
};

// Unit (256 rows) `unit` of the call: its sequence, and where its rows begin.
struct Unit {
    int b;       // -1: none
    int row0;    // of the sequence's n x rep rows
    int start;   // the sequence's first token
    int n;       // its tokens
    int pos0;    // position of its first token
};

// The sequence that unit `u` counted from the call's last one belongs to: late
// units of a prompt see most keys, so they start first.
__device__ Unit find_unit(const PrefillParams &p, int u, int *scratch)
{
    const int threads = blockDim.x, warps = threads >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Unit *found = reinterpret_cast<Unit *>(scratch + 32);
    int before = 0;  // units of the sequences behind the present block (from the back)
    for (int b0 = 0; b0 < p.c.batch; b0 += threads) {
        const int b = p.c.batch - 1 - b0 - int(threadIdx.x);
        Unit mine{b, 0, 0, 0, 0};
        int own = 0, end = 0, len = 0;
        if (b >= 0) {
            len = p.lens[b];
            end = p.tok_start[b + 1];
            mine.start = max(p.tok_start[b], 0);
            mine.n = max(min(end, p.T) - mine.start, 0);
            own = (mine.n * p.rep + kRows - 1) / kRows;
        }
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            scratch[warp] = incl;
        __syncthreads();
        int base = before;
        for (int w = 0; w < warps; ++w) {
            base += w < warp ? scratch[w] : 0;
            before += scratch[w];
        }
        const int lo = base + incl - own;
        if (u >= lo && u < lo + own) {
            mine.row0 = (own - 1 - (u - lo)) * kRows;
            mine.pos0 = kv4_cut(p.c, len) - (end - mine.start);
            *found = mine;
        }
        __syncthreads();
        if (u < before)
            return *found;
    }
    return Unit{-1, 0, 0, 0, 0};
}

// Key tiles [first, last) of 128 that a unit's split works through.
struct Tiles {
    int first, last;
    int begin, end;  // keys that any row sees: [begin, end)
};

__device__ __forceinline__ Tiles tiles_of(const PrefillParams &p, const Unit &u, int split)
{
    const int last_row = min(u.row0 + kRows, u.n * p.rep) - 1;
    const int p0 = u.pos0 + p.by_rep.of(u.row0), p1 = u.pos0 + p.by_rep.of(last_row);
    Tiles t;
    // (p0 may be 2^30 or more below 0 where tok_start names far more tokens than
    // the call has: then p1 < 0, and there are no tiles whatever begin is)
    t.end = min(max(p1 + 1, 0), p.c.max_len());
    t.begin = p.q.window > 0 ? max(0, p0 - p.q.window + 1) : 0;
    const int a = t.begin / kKeys, n = max(0, (t.end + kKeys - 1) / kKeys - a);
    t.first = a + p.by_splits.of(n * split);  // (at most 2^23 tiles, 32 parts)
    t.last = a + p.by_splits.of(n * (split + 1));
    return t;
}

// ------------------------------------------------------------- PTX wrappers
// Bulk copy with L2's own policy: other CTAs of the sequence read the same codes.
__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16, bool b_mn_major)
{
    return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(b_mn_major) << 16) |
           (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// Operand whose rows of 64 values run along the MMA's N (values: N = elements,
// K = keys): 8 keys are 1024 bytes apart, blocks of 64 values block_bytes.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t block_bytes)
{
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t(block_bytes >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

// 32 columns of the thread's lane; the values are there after tmem_arrived().
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Ties the registers of an asynchronous load to the wait before this line: no
// use of them can be moved above it.
__device__ __forceinline__ void tmem_arrived(uint32_t *v)
{
    asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
    asm volatile("" : "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]),
                 "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]),
                 "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]));
}

// One arrival for the warp, after all of its lanes' work (32 arrivals on one
// barrier go through shared memory one by one).
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
}

// Pairs of fp32 values in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Of a query row whose largest magnitude has these fp32 bits: the power of two
// that its fp16 values are taken against.
__device__ __forceinline__ int row_exponent(uint32_t top)
{
    return min(max(int(top >> 23) - 127, -100), 126);
}

template <class T2>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b)
{
    const T2 r = __hsub2(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(c));
    return r;
}

// A word of 8 nibbles n = code + 8 as 16-bit numbers, in the order 0 4 1 5 2 6
// 3 7 in which the masks deliver them; the queries are stored in the same
// order, and so come out the values' elements. Keys: under the exponent of
// 1024 (64, one nibble higher) n is the fp16 number 1024 + n (64 + n), and the
// code is multiplied by its scale. Values: under the exponent of 128 it is the
// bf16 number 128 + n.
__device__ __forceinline__ uint4 expand_keys(uint32_t w, uint32_t scale)
{
    const __half2 f = *reinterpret_cast<const __half2 *>(&scale);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = i < 2 ? w : w >> 8;
        r[i] = (i & 1) ? sub2<__half2>(and_or(x, 0x00F000F0u, 0x54005400u), 0x54805480u)
                       : sub2<__half2>(and_or(x, 0x000F000Fu, 0x64006400u), 0x64086408u);
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&r[i]), f);
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint4 expand_values(uint32_t w)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = sub2<__nv_bfloat162>(and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u), 0x43084308u);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// ------------------------------------------------------------------ kernel
struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t scales[kScaleSlots];
    uint64_t q_raw[8], q_full[2];  // q_raw: of each softmax warp
    uint64_t s_full[2][2], p_full[2][2], o_done[2], o_final[2];  // [row tile][half tile]
    uint64_t packed_full[2][2], packed_empty[2][2];  // [keys, values][stage]
};

// Shared memory. Operand tiles stand on 1024 bytes (the swizzle's period):
// the struct is all of the kernel's shared memory, which begins there.
template <int D>
struct Shared {
    uint8_t q[2][PrefillShape<D>::kTileBytes];
    uint8_t k[2][PrefillShape<D>::kTileBytes];
    uint8_t v[2][PrefillShape<D>::kTileBytes];
    uint8_t packed[2][2][PrefillShape<D>::kPacked];  // [keys, values][stage] codes
    uint16_t scales[2][2][kKeys];                    // [stage][keys, values] as stored
    float vs[kScaleSlots][kKeys];                    // value scales
    uint4 skip[kScaleSlots];    // keys of pages outside the cache, a bit each
    uint4 poison[kScaleSlots];  // keys whose value scale is NaN
    float unit[kScaleSlots];    // what 1 in the tile's key operand stands for
    uint32_t pages[2];          // [stage] pages that are there, and << 16 bad ones
    uint32_t tmem;
    Bars bar;
    __device__ __forceinline__ int *scratch()  // only until the roles part
    {
        return reinterpret_cast<int *>(vs[0]);
    }
};

template <int D>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    kv4_prefill_kernel(const __grid_constant__ PrefillParams p)
{
    using S = PrefillShape<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Shared<D> &sh = *reinterpret_cast<Shared<D> *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Units are counted from the call's last row, and their heads and parts stand
    // next to each other: the CTAs that see most keys start first. (With one
    // head's units after the other's, the last head's long ones start when SMs
    // run dry: 422 us for 8192 tokens where this order took 380.)
    const int item = p.by_heads.of(blockIdx.x), kvh = int(blockIdx.x) - item * p.c.kv_heads;
    const int unit = p.by_splits.of(item), split = item - unit * p.splits;

    pdl_wait();
    pdl_launch_dependents();
    if (warp == 12) {  // (while the others look up lengths)
        tmem_alloc(&sh.tmem, 512);
        tc_fence_before();
    }
    const Unit u = find_unit(p, unit, sh.scratch());
    if (u.b < 0) {
        if (warp == 12)
            tmem_dealloc(sh.tmem, 512);
        return;
    }
    const Tiles tl = tiles_of(p, u, split);
    const int n = tl.last - tl.first;
    const int rows = min(kRows, u.n * p.rep - u.row0);
    const int nq = rows > 128 ? 2 : 1;  // row tiles at work
    // The softmax warps' rows, one a thread. A warp's query rows come by bulk
    // copies, one for each token's heads, into the value tiles, which wait for
    // them (plain loads took 5000 cycles, longer than the first keys).
    const int row = threadIdx.x;
    const int tok = p.by_rep.of(u.row0 + row), h = (u.row0 + row) - tok * p.rep;
    const bool real = row < rows;
    const long long row_at = (long long)(kvh * p.rep + h) * D;  // within its token's row
    const uint8_t *raw = sh.v[0] + row * (2 * D);
    if (warp < 8 && n > 0 && (warp >> 2) < nq) {
        uint64_t *bar = &sh.bar.q_raw[warp];
        if (lane == 0) {
            mbar_init(bar, 1);
            fence_mbar_init();
            mbar_arrive_expect_tx(bar, max(0, min(32, rows - warp * 32)) * uint32_t(2 * D));
        }
        __syncwarp();
        if (real && (h == 0 || lane == 0))
            bulk_copy(const_cast<uint8_t *>(raw), p.q.q + (u.start + tok) * p.q.q_stride + row_at,
                      2 * D * min(p.rep - h, min(32 - lane, rows - row)), bar);
    }

    // Copies of packed codes, by warp 13. Lane 4 g + w: page g of a tile; w: its
    // key codes, value codes, key scales, value scales.
    const int copy_g = lane >> 2, copy_w = lane & 3;
    auto wanted = [&](int tile) {
        const int index = tile * (kKeys >> p.c.lg_ps) + copy_g;
        // (a page in front of a window may have gone to another sequence)
        return copy_g < kKeys >> p.c.lg_ps && index << p.c.lg_ps < tl.end &&
               (index + 1) << p.c.lg_ps > tl.begin;
    };
    auto page_of = [&](int tile) {
        return wanted(tile) ? p.c.table[(long long)u.b * p.c.max_pages +
                                        tile * (kKeys >> p.c.lg_ps) + copy_g]
                            : 0;
    };
    int next_page = 0;
    auto copy_tile = [&](int j) {
        const int ps = p.c.page_size(), g = copy_g, w = copy_w;
        const int st = j & 1, parity = ((j >> 1) & 1) ^ 1, page = next_page;
        if (j + 1 < n)
            next_page = page_of(tl.first + j + 1);
        const bool want = wanted(tl.first + j);
        const bool bad = want && unsigned(page) >= unsigned(p.c.num_pages);
        const uint32_t there = __ballot_sync(0xffffffffu, want && !bad && w == 0);
        const uint32_t wrong = __ballot_sync(0xffffffffu, bad && w == 0);
        const uint8_t *src = p.c.pages + kvh * p.c.template head_bytes<D>() +
                             (long long)page * p.c.page_stride +
                             (w < 2 ? (long long)w * ps * (D / 2)
                                    : (long long)ps * D + (w - 2) * 2 * ps);
        if (j >= 2 && !mbar_wait_warp(&sh.bar.packed_empty[0][st], parity, p.c.err))
            return false;
        if (lane == 0) {
            uint32_t a = 0, b = 0;  // a bit a page
            for (int k = 0; k < 8; ++k) {
                a |= (there >> (4 * k) & 1) << k;
                b |= (wrong >> (4 * k) & 1) << k;
            }
            if (b)
                atomicOr(p.c.err, kErrBadPage);
            sh.pages[st] = a | b << 16;
            mbar_arrive_expect_tx(&sh.bar.packed_full[0][st],
                                  __popc(there) * uint32_t(ps) * (D / 2 + 4));
        }
        __syncwarp();
        if (want && !bad && w != 1)
            bulk_copy(w == 0 ? sh.packed[0][st] + g * ps * (D / 2)
                             : reinterpret_cast<uint8_t *>(&sh.scales[st][w - 2][g * ps]),
                      src, w == 0 ? ps * (D / 2) : ps * 2, &sh.bar.packed_full[0][st]);
        if (j >= 2 && !mbar_wait_warp(&sh.bar.packed_empty[1][st], parity, p.c.err))
            return false;
        if (lane == 0)
            mbar_arrive_expect_tx(&sh.bar.packed_full[1][st],
                                  __popc(there) * uint32_t(ps) * (D / 2));
        __syncwarp();
        if (want && !bad && w == 1)
            bulk_copy(sh.packed[1][st] + g * ps * (D / 2), src, ps * (D / 2),
                      &sh.bar.packed_full[1][st]);
        return true;
    };

    if (n > 0) {
        if (warp == 13) {  // the first keys come while all else is set up
            next_page = page_of(tl.first);
            if (lane < 4) {
                mbar_init(&sh.bar.packed_full[lane & 1][lane >> 1], 1);
                mbar_init(&sh.bar.packed_empty[lane & 1][lane >> 1], 4);
                fence_mbar_init();
            }
            __syncwarp();
            copy_tile(0);
        }
        if (warp == 15) {
            if (lane < 2) {
                const int i = lane;
                mbar_init(&sh.bar.k_full[i], 4);
                mbar_init(&sh.bar.k_empty[i], nq);
                mbar_init(&sh.bar.v_full[i], 4);
                mbar_init(&sh.bar.v_empty[i], nq);
                for (int h = 0; h < 2; ++h) {
                    mbar_init(&sh.bar.s_full[i][h], 1);
                    mbar_init(&sh.bar.p_full[i][h], 4);
                }
                mbar_init(&sh.bar.o_done[i], 1);
                mbar_init(&sh.bar.o_final[i], 1);
                mbar_init(&sh.bar.q_full[i], 4);
            }
            if (lane < kScaleSlots)
                mbar_init(&sh.bar.scales[lane], 4);
            fence_mbar_init();
        }
        __syncthreads();
        tc_fence_after();
    }
    const uint32_t tmem = n > 0 ? sh.tmem : 0;

    if (warp < 8) {
        // ---------------------------------------------------------- softmax
        const int s = warp >> 2;
        const int pos = real ? u.pos0 + tok : -1;  // below 0: sees nothing
        const int low = p.q.window > 0 ? pos - p.q.window + 1 : 0;  // first key seen
        // what all rows of the tile see: keys [low_max, pos_min]
        const int pos_min = u.pos0 + p.by_rep.of(u.row0 + s * 128);
        const int last = min(s * 128 + 127, rows - 1);
        const int low_max =
            p.q.window > 0 ? u.pos0 + p.by_rep.of(u.row0 + last) - p.q.window + 1 : 0;
        const uint32_t lane_at = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_at + s * 128, to = tmem + lane_at + 256 + s * D;
        // The thread's query row as fp16 against its largest magnitude: 16 bytes at
        // a time in an order (c = k ^ twist) in which neither the reads nor the
        // swizzled writes of eight lanes meet in a bank: twist, and twist ^ lane,
        // take all values of three bits.
        float row_mul = 0.0f;  // what 1 in the row stands for x scale, base 2
        bool fine = s < nq;
        if (n > 0 && s < nq) {
            const int twist = ((lane << 1) & 7) ^ ((lane & 4) ? 3 : 0);
            fine = mbar_wait_warp(&sh.bar.q_raw[warp], 0, p.c.err);
            if (!fine)  // (the CTA does not retire under the warp's copies)
                mbar_wait_warp(&sh.bar.q_raw[warp], 0, p.c.err);
            // (a row before position 0 sees nothing: were it NaN, its masked scores
            // would be, so it counts as zeros)
            auto chunk = [&](int c) {
                return pos >= 0 ? lds128(raw + (c << 4)) : make_uint4(0, 0, 0, 0);
            };
            uint4 v[D / 8];
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
                v[k] = chunk(k ^ twist);
            uint32_t tops = 0;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const uint4 x = v[k];
                tops = __vmaxu2(tops, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                               __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
            }
            const uint32_t top = max(tops & 0xFFFFu, tops >> 16) << 16;  // fp32 bits
            const float down = __uint_as_float(uint32_t(127 - row_exponent(top)) << 23);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const int c = k ^ twist;
                const uint4 x = v[k];
                const float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                                    bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 y = __floats2half2_rn(f[e] * down, f[4 + e] * down);
                    w[e] = *reinterpret_cast<const uint32_t *>(&y);
                }
                *reinterpret_cast<uint4 *>(sh.q[s] + (c >> 3) * 16384 +
                                           sw128_off(row & 127, c & 7)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            row_mul = top >= 0x7F800000u ? NAN
                                         : __uint_as_float(uint32_t(127 + row_exponent(top)) << 23) *
                                               (p.q.scale * kLog2e);
            fence_proxy_async_smem();
            warp_arrive(&sh.bar.q_full[s]);
        }
        float m = -INFINITY, lsum = 0.0f;  // m: base 2, of scale x scores
        bool poisoned = false;
#pragma unroll 1
        for (int i = 0; i < 2 * n && fine; ++i) {  // half tiles
            const int slot = (i >> 1) % kScaleSlots, half = i & 1;
            const int j0 = (tl.first + (i >> 1)) * kKeys + half * kHalf;
            if (half == 0)
                fine = mbar_wait_warp(&sh.bar.scales[slot], ((i >> 1) / kScaleSlots) & 1, p.c.err);
            fine = fine && mbar_wait_warp(&sh.bar.s_full[s][half], (i >> 1) & 1, p.c.err);
            if (!fine)
                break;
            tc_fence_after();
            uint32_t t[kHalf];
            tmem_ld32_async(ts + half * kHalf, t);
            tmem_ld32_async(ts + half * kHalf + 32, t + 32);
            float mul = row_mul * sh.unit[slot];
            if (mul < 1.17549435e-38f)  // (NaN stays) no zero, which masks would meet
                mul = 1.17549435e-38f;
            const uint2 skip = reinterpret_cast<const uint2 *>(&sh.skip[slot])[half];
            const uint2 poison = reinterpret_cast<const uint2 *>(&sh.poison[slot])[half];
            tmem_ld_wait();
            tmem_arrived(t);
            tmem_arrived(t + 32);
            const bool special = (skip.x | skip.y | poison.x | poison.y) != 0;
            if (special || j0 + kHalf - 1 > pos_min || j0 < low_max) {
                const int hi = pos - j0, lo = low - j0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    // keys of these 32 that the row sees, a bit each
                    uint32_t see = hi >= 32 * w + 31 ? 0xFFFFFFFFu
                                   : hi < 32 * w     ? 0u
                                                     : 0xFFFFFFFFu >> (31 - (hi - 32 * w));
                    see &= lo <= 32 * w          ? 0xFFFFFFFFu
                           : lo > 32 * w + 31 ? 0u
                                              : 0xFFFFFFFFu << (lo - 32 * w);
                    see &= ~(w ? skip.y : skip.x);
                    poisoned = poisoned || (see & (w ? poison.y : poison.x));
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        t[32 * w + k] = (see >> k) & 1 ? t[32 * w + k] : 0xFF800000u;
                }
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                top[c] = fmaxf(__uint_as_float(t[16 * c]), __uint_as_float(t[16 * c + 1]));
#pragma unroll
                for (int k = 2; k < 16; k += 2)
                    top[c] = fmaxf(top[c], fmaxf(__uint_as_float(t[16 * c + k]),
                                                 __uint_as_float(t[16 * c + k + 1])));
            }
            const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mul;
            if (m == -INFINITY)
                m = mt;  // nothing summed up yet
            const bool grew = mt - m > 8.0f;
            if (__any_sync(0xffffffffu, grew)) {
                const float a = grew ? ex2(m - mt) : 1.0f;
                if (grew)
                    m = mt;
                lsum *= a;
                if (i > 0) {
                    // (the scores of i came after product i - 2: at most one
                    // phase is out, and its parity is enough)
                    fine = mbar_wait_warp(&sh.bar.o_done[s], (i - 1) & 1, p.c.err);
                    if (!fine)
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_async(to + 32 * c, o);
                        tmem_ld_wait();
                        tmem_arrived(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                        tmem_st32_async(to + 32 * c, o);
                    }
                    tmem_st_wait();
                }
            }
            const float neg = m == -INFINITY ? 0.0f : -m;
            const float4 *vs = reinterpret_cast<const float4 *>(sh.vs[slot] + half * kHalf);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float4 v = vs[k];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float2 x = fma2(make_float2(__uint_as_float(t[4 * k + 2 * c]),
                                                __uint_as_float(t[4 * k + 2 * c + 1])),
                                    make_float2(mul, mul), make_float2(neg, neg));
                    x.x = ex2(x.x);
                    x.y = ex2(x.y);
                    sum[c] = add2(sum[c], x);
                    x = mul2(x, c ? make_float2(v.z, v.w) : make_float2(v.x, v.y));
                    pk[2 * k + c] = pack_bf16(x.x, x.y);
                }
            }
            tmem_st32_async(ts + half * kHalf, pk);
            lsum += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sh.bar.p_full[s][half]);
        }
        // A largest score above fp32's numbers: no weight is known.
        if (m == INFINITY)
            lsum = NAN;
        // Output rows (a row tile without keys, or without rows, has none).
        const float inv = lsum == 0.0f ? 0.0f : poisoned ? NAN : 1.0f / lsum;
        const long long token = u.start + tok;
        const long long part = ((((long long)unit * p.c.kv_heads + kvh) * p.splits + split) *
                                kRows + row);
        if (s < nq) {
            // Rows change lanes in shared memory (the row tile's queries are done
            // with), so that D/8 lanes store the 2 D bytes of one row: results in
            // bf16, or fp32 parts D/2 values at a time.
            constexpr int kChunks = D / 8;  // of 16 bytes
            uint8_t *stage = sh.q[s] + (warp & 3) * 32 * (2 * D);
            const bool parts = p.splits > 1;
            const float by = !parts || lsum == 0.0f ? inv : poisoned ? NAN : 1.0f;
            char *dst = parts ? reinterpret_cast<char *>(p.parts + part * D)
                              : reinterpret_cast<char *>(p.q.out + token * p.q.out_stride + row_at);
            if (!real)
                dst = nullptr;
            if (n > 0) {
                fine = fine && mbar_wait_warp(&sh.bar.o_final[s], 0, p.c.err);
                tc_fence_after();
            }
            auto put = [&](int chunk, uint4 v) {
                *reinterpret_cast<uint4 *>(stage + lane * 2 * D + ((chunk ^ (lane & 7)) << 4)) = v;
            };
            auto flush = [&](int offset) {
                __syncwarp();
#pragma unroll 4
                for (int r0 = 0; r0 < 32; r0 += 32 / kChunks) {
                    const int r = r0 + lane / kChunks, c = lane % kChunks;
                    const uint4 v = lds128(stage + r * 2 * D + ((c ^ (r & 7)) << 4));
                    char *to_row = reinterpret_cast<char *>(__shfl_sync(
                        0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
                    if (to_row)
                        *reinterpret_cast<uint4 *>(to_row + offset + c * 16) = v;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32_async(to + 32 * i, o);
                    tmem_ld_wait();
                    tmem_arrived(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = 0;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float e[8];  // back from the order 0 4 1 5 2 6 3 7
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e[k] = __uint_as_float(o[8 * c + 2 * k]);
                        e[4 + k] = __uint_as_float(o[8 * c + 2 * k + 1]);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        e[k] *= by;
                    if (parts) {
                        const int at = (32 * i) % (D / 2) / 4 + 2 * c;
                        put(at, make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]),
                                           __float_as_uint(e[2]), __float_as_uint(e[3])));
                        put(at + 1, make_uint4(__float_as_uint(e[4]), __float_as_uint(e[5]),
                                               __float_as_uint(e[6]), __float_as_uint(e[7])));
                    } else {
                        put(4 * i + c, make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]),
                                                  pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])));
                    }
                }
                if (parts && 32 * (i + 1) % (D / 2) == 0)
                    flush(32 * i / (D / 2) * 2 * D);
            }
            if (!parts)
                flush(0);
            if (real && parts)
                p.sums[part] = make_float2(m, lsum);
            else if (real && p.q.lse)
                p.q.lse[token * p.q.q_heads + kvh * p.rep + h] =
                    lsum == 0.0f ? -INFINITY : (m + __log2f(lsum)) * kLn2;
        }
        tc_fence_before();
    } else if (warp < 12) {
        // ------------------------------------------------- codes to operands
        // Thread i takes 16 bytes of codes of every kRowsAtOnce-th key. Lane l
        // of each warp looks after the scales of keys l, l + 32, ...
        constexpr int kPerRow = D / 32, kRowsAtOnce = 128 / kPerRow, kSteps = 128 / kRowsAtOnce;
        const int i = threadIdx.x - 256, w4 = warp - 8;
        const int part = i % kPerRow, row0 = i / kPerRow;
        // Word w goes to chunk (part % 2) 4 + w of block part / 2; the two
        // blocks of a row of 128 values take their words in another order, so
        // that eight lanes' stores meet eight bank groups.
        const int turn = D == 128 ? (part >> 1) * 2 : 0;
        auto expand = [&](uint8_t *tile, const uint8_t *packed, bool keys, const uint32_t *scale) {
#pragma unroll
            for (int r = 0; r < kSteps; ++r) {
                const int key = r * kRowsAtOnce + row0;
                uint32_t f = 0;
                if (keys) {
                    const int from = D == 128 ? r : 2 * r + (w4 >> 1);  // key / 32, the warp's
                    f = __shfl_sync(0xffffffffu, from == 0 ? scale[0] : from == 1 ? scale[1]
                                                 : from == 2 ? scale[2] : scale[3], key & 31);
                }
                uint4 x = lds128(packed + (r * 128 + i) * 16);
                if (turn)
                    x = make_uint4(x.z, x.w, x.x, x.y);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint8_t *row = tile + (part >> 1) * 16384 + (key >> 3) * 1024 + (key & 7) * 128;
                const int c0 = ((part & 1) * 4 + turn) ^ (key & 7);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(row + ((c0 ^ q) << 4)) =
                        keys ? expand_keys(w[q], f) : expand_values(w[q]);
            }
        };
        bool fine = true;
        int j = 0;
#pragma unroll 1
        for (; j < n; ++j) {
            const int st = j & 1, slot = j % kScaleSlots, parity = (j >> 1) & 1;
            fine = (j < 2 || mbar_wait_warp(&sh.bar.k_empty[st], parity ^ 1, p.c.err)) &&
                   mbar_wait_warp(&sh.bar.packed_full[0][st], parity, p.c.err);
            if (!fine)
                break;
            // Key scales against the tile's largest (NaN and infinity aside),
            // which becomes 2^11 .. 2^12: times 7 that is in fp16's range. Keys
            // that no row sees, or that are not there, have scale 0.
            const uint32_t pages = sh.pages[st];
            uint32_t ks[4], top = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int key = w * 32 + lane, at = (tl.first + j) * kKeys + key;
                const bool in = at >= tl.begin && at < tl.end && (pages >> (key >> p.c.lg_ps) & 1);
                ks[w] = in ? sh.scales[st][0][key] : 0u;
                top = max(top, (ks[w] & 0x7F80) == 0x7F80 ? 0u : ks[w] >> 7);
            }
            top = max(__reduce_max_sync(0xffffffffu, top), 13u);
            uint32_t scale[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const __half h = __float2half_rn(__uint_as_float(ks[w] << 16) *
                                                 __uint_as_float((265u - top) << 23));
                const uint32_t b = __half_as_ushort(h);
                scale[w] = b | b << 16;
            }
            // A NaN value scale would reach, as 0 x NaN, rows that do not see
            // the key: it is noted, and the rows that do see it find it there.
            const int own = (tl.first + j) * kKeys + i;
            const bool in = own >= tl.begin && own < tl.end && (pages >> (i >> p.c.lg_ps) & 1);
            const uint32_t vs = in ? sh.scales[st][1][i] : 0u;
            const uint32_t skip =
                __ballot_sync(0xffffffffu, (pages >> (16 + (i >> p.c.lg_ps))) & 1);
            const bool nan = (vs & 0x7F80) == 0x7F80;
            const uint32_t poison = __ballot_sync(0xffffffffu, nan);
            sh.vs[slot][i] = nan ? 0.0f : __uint_as_float(vs << 16);
            if (lane == 0) {
                reinterpret_cast<uint32_t *>(&sh.skip[slot])[w4] = skip;
                reinterpret_cast<uint32_t *>(&sh.poison[slot])[w4] = poison;
            }
            if (i == 0)
                sh.unit[slot] = __uint_as_float((top - 11u) << 23);
            warp_arrive(&sh.bar.scales[slot]);
            expand(sh.k[st], sh.packed[0][st], true, scale);
            fence_proxy_async_smem();
            warp_arrive(&sh.bar.k_full[st]);
            if (lane == 0)
                mbar_arrive(&sh.bar.packed_empty[0][st]);
            fine = (j < 2 || mbar_wait_warp(&sh.bar.v_empty[st], parity ^ 1, p.c.err)) &&
                   mbar_wait_warp(&sh.bar.packed_full[1][st], parity, p.c.err);
            if (!fine)
                break;
            if (j == 0)  // the query rows lie there until they are converted
                for (int s = 0; s < nq; ++s)
                    fine = fine && mbar_wait_warp(&sh.bar.q_full[s], 0, p.c.err);
            if (!fine)
                break;
            expand(sh.v[st], sh.packed[1][st], false, scale);
            fence_proxy_async_smem();
            warp_arrive(&sh.bar.v_full[st]);
            if (lane == 0)
                mbar_arrive(&sh.bar.packed_empty[1][st]);
        }
        // Where a wait gave up, the CTA does not retire under the copies that may
        // be on their way: this tile's and the next one's.
        if (!fine)
            for (int h = 2 * j; h < min(2 * j + 4, 2 * n); ++h)
                mbar_wait_warp(&sh.bar.packed_full[h & 1][(h >> 1) & 1], (h >> 2) & 1, p.c.err);
    } else {
        // -------------------------------------------------------------- MMAs
        // One warp per row tile: a product is queued only a few deep, so what
        // one warp spends on waits and commits the other's products cover. The
        // whole warp walks the loop, so that addresses and descriptors stay in
        // uniform registers; one elected lane issues (issue by a lone lane of a
        // divergent branch took 100 cycles a product, twice its execution).
        const int s = (warp - 12) >> 1;
        if ((warp & 1) == 0 && s < nq && n > 0) {
            constexpr uint32_t kQk = idesc_f16(128, kHalf, false, false);
            constexpr uint32_t kPv = idesc_f16(128, D, true, true);
            const uint64_t q0 = umma_desc_sw128(smem_u32(sh.q[s]));
            const uint64_t k0 = umma_desc_sw128(smem_u32(sh.k));
            const uint64_t v0 = umma_desc_mn_sw128(smem_u32(sh.v), 16384);
            const uint32_t s_at = tmem + s * 128, o_at = tmem + 256 + s * D;
            const bool lead = elect_one();
            // Scores of a half tile of 64 keys of the stage, and the products
            // with its values. Scores run two half tiles ahead: the softmax
            // finds them ready. A half tile's weights lie in its scores'
            // columns, which the scores after next may overwrite as one
            // thread's products execute in order.
            auto scores = [&](int stage, int half) {
                const uint64_t b = umma_desc_advance(k0, stage * S::kTileBytes + half * kHalf * 128);
                if (lead) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                        umma_f16(s_at + half * kHalf, umma_desc_advance(q0, at),
                                 umma_desc_advance(b, at), kQk, k > 0);
                    }
                    umma_commit(&sh.bar.s_full[s][half]);
                }
            };
            auto values = [&](int stage, int half, bool first, bool final) {
                const uint64_t b = umma_desc_advance(v0, stage * S::kTileBytes + half * kHalf * 128);
                if (lead) {
#pragma unroll
                    for (int k = 0; k < kHalf / 16; ++k)
                        umma_f16_ts(o_at, s_at + half * kHalf + k * 8, umma_desc_advance(b, k * 2048),
                                    kPv, !first || k > 0);
                    umma_commit(final ? &sh.bar.o_final[s] : &sh.bar.o_done[s]);
                }
            };
            bool fine = mbar_wait_warp(&sh.bar.q_full[s], 0, p.c.err) &&
                        mbar_wait_warp(&sh.bar.k_full[0], 0, p.c.err);
            if (fine) {
                tc_fence_after();
                scores(0, 0);
                scores(0, 1);
                if (n > 2 && lead)  // (no arrival that nobody waits for)
                    umma_commit(&sh.bar.k_empty[0]);
            }
#pragma unroll 1
            for (int j = 0; j < n && fine; ++j) {
                const int st = j & 1;
                fine = mbar_wait_warp(&sh.bar.v_full[st], (j >> 1) & 1, p.c.err) &&
                       mbar_wait_warp(&sh.bar.p_full[s][0], j & 1, p.c.err);
                if (!fine)
                    break;
                tc_fence_after();
                values(st, 0, j == 0, false);
                if (j + 1 < n) {
                    fine = mbar_wait_warp(&sh.bar.k_full[st ^ 1], ((j + 1) >> 1) & 1, p.c.err);
                    if (!fine)
                        break;
                    tc_fence_after();
                    scores(st ^ 1, 0);
                }
                fine = mbar_wait_warp(&sh.bar.p_full[s][1], j & 1, p.c.err);
                if (!fine)
                    break;
                tc_fence_after();
                values(st, 1, false, j == n - 1);
                if (j + 2 < n && lead)
                    umma_commit(&sh.bar.v_empty[st]);
                if (j + 1 < n) {
                    scores(st ^ 1, 1);
                    if (j + 3 < n && lead)
                        umma_commit(&sh.bar.k_empty[st ^ 1]);
                }
            }
            // Where a wait gave up, the tensor memory is not freed, nor does the CTA
            // retire, under the products that were issued.
            if (!fine) {
                if (lead)
                    umma_commit(&sh.bar.o_final[s]);
                mbar_wait_warp(&sh.bar.o_final[s], 0, p.c.err);
            }
        }
        // ------------------------------------------------------------ copies
        if (warp == 13) {
#pragma unroll 1
            for (int j = 1; j < n && copy_tile(j); ++j)
                ;
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

// Adds up the parts of a unit's rows, one warp a row at a time.
constexpr int kJoinThreads = 256, kJoinRows = 32;

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    kv4_prefill_join_kernel(const __grid_constant__ PrefillParams p)
{
    __shared__ int scratch[40];
    pdl_wait();
    pdl_launch_dependents();
    const Unit u = find_unit(p, blockIdx.x, scratch);
    if (u.b < 0)
        return;
    const int kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(kRows, u.n * p.rep - u.row0);
    const long long unit = ((long long)blockIdx.x * p.c.kv_heads + kvh) * p.splits * kRows;
    for (int r = blockIdx.z * kJoinRows + warp; r < min(rows, int(blockIdx.z + 1) * kJoinRows);
         r += kJoinThreads / 32) {
        auto part = [&](int k) { return unit + (long long)k * kRows + r; };
        // lane k: part k's maximum and sum
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < p.splits)
            ml = p.sums[part(lane)];
        float m = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float w = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
        float l = w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, o);
        float2 v[D / 64] = {};
        for (int k = 0; k < p.splits; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const float2 x = *reinterpret_cast<const float2 *>(p.parts + part(k) * D + i * 64 + 2 * lane);
                v[i].x = fmaf(wk, x.x, v[i].x);
                v[i].y = fmaf(wk, x.y, v[i].y);
            }
        }
        const int tok = p.by_rep.of(u.row0 + r), h = (u.row0 + r) - tok * p.rep;
        const long long token = u.start + tok;
        const int head = kvh * p.rep + h;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            *reinterpret_cast<uint32_t *>(p.q.out + token * p.q.out_stride + (long long)head * D +
                                          i * 64 + 2 * lane) = pack_bf16(v[i].x * inv, v[i].y * inv);
        if (p.q.lse && lane == 0)
            p.q.lse[token * p.q.q_heads + head] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }
}

struct PrefillPlan {
    int rep, units, splits;
    size_t bytes;
};

// Units at most (rows fill them but for one per sequence), and parts per unit.
// CTAs run one to an SM, so s parts of c units' tiles take ceil(c s / SMs)
// turns of tiles / s each, and about four tiles' time for every turn's start,
// end and joining; from two turns on, parts gain less than they cost. (Two
// sequences of 512 tokens behind up to 16000, 5 heads of 4: 238, 177, 156, 156,
// 152, 167, 166, 174, 179, 195, 216 us with 1 to 9, 11 and 14 parts; 5 are taken.)
// The host knows the table's width alone, not the lengths: in a table of 131072
// tokens those two sequences get 17 parts and take 234 us, a prompt of 2048
// tokens 12 parts and 192 us where its own width gives one part and 46.
PrefillPlan plan_prefill(const Kv4View &c, int D, int q_heads, int T)
{
    PrefillPlan d;
    d.rep = q_heads / c.kv_heads;
    const long long rows = (long long)T * d.rep;
    const long long units = rows / kRows + std::min(c.batch, T);
    d.units = int(std::min<long long>(units, INT32_MAX));
    const int sms = device_sm_count();
    const long long ctas =
        std::max<long long>((rows + kRows - 1) / kRows, std::min(c.batch, T)) * c.kv_heads;
    const int tiles = (c.max_len() + kKeys - 1) / kKeys;
    d.splits = 1;
    double best = 1e30;
    for (int s = 1; s <= 32 && s <= std::max(1, tiles); ++s) {
        if (s > 1 && ctas >= 2ll * sms)
            break;
        const double turns = double((ctas * s + sms - 1) / sms);
        const double cost = turns * (double(tiles) / s + 4.0) + (s > 1 ? 4.0 : 0.0);
        if (cost < best) {
            best = cost;
            d.splits = s;
        }
    }
    d.bytes = d.splits == 1 ? 0
                            : size_t(d.units) * c.kv_heads * d.splits * kRows *
                                  (size_t(D) * sizeof(float) + sizeof(float2));
    return d;
}

template <int D>
cudaError_t launch(const PrefillParams &p, const PrefillPlan &plan, cudaStream_t stream)
{
    using S = PrefillShape<D>;
    static thread_local int configured_dev = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured_dev != dev) {
        e = cudaFuncSetAttribute(kv4_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(sizeof(Shared<D>)));
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
    cfg.gridDim = dim3(unsigned(plan.units) * unsigned(p.c.kv_heads) * unsigned(plan.splits));
    cfg.blockDim = dim3(kPrefillThreads);
    cfg.dynamicSmemBytes = int(sizeof(Shared<D>));
    e = cudaLaunchKernelEx(&cfg, kv4_prefill_kernel<D>, p);
    if (e != cudaSuccess || plan.splits == 1)
        return e;
    cfg.gridDim = dim3(unsigned(plan.units), unsigned(p.c.kv_heads), kRows / kJoinRows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv4_prefill_join_kernel<D>, p);
}

}  // namespace

size_t kv4_prefill_workspace(const Kv4View &c, int D, int q_heads, int T)
{
    return c.batch > 0 && T > 0 ? plan_prefill(c, D, q_heads, T).bytes : 0;
}

cudaError_t launch_kv4_prefill(const Kv4View &c, int D, const Kv4Query &q,
                               const int32_t *tok_start, const int32_t *lens, int T,
                               void *workspace, cudaStream_t stream)
{
    const PrefillPlan plan = plan_prefill(c, D, q.q_heads, T);
    PrefillParams p;
    p.c = c;
    p.q = q;
    p.tok_start = tok_start;
    p.lens = lens;
    p.T = T;
    p.rep = plan.rep;
    p.splits = plan.splits;
    p.by_rep = Divisor(plan.rep);
    p.by_heads = Divisor(c.kv_heads);
    p.by_splits = Divisor(plan.splits);
    p.parts = static_cast<float *>(workspace);
    p.sums = reinterpret_cast<float2 *>(p.parts + size_t(plan.units) * c.kv_heads * plan.splits *
                                                      kRows * size_t(D));
    return D == 128 ? launch<128>(p, plan, stream) : launch<64>(p, plan, stream);
}

}  // namespace tq
