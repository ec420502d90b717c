// Attention of single tokens over a paged cache in 8 bits, with a scale for each
// 16 tokens of a head: 2 D bytes for 4 D operations a key and query head, so the
// bound is HBM, at half the FP16 cache's bytes.
//
// Arithmetic.  Codes are whole numbers up to 127, exact in FP16, so the products
// are those of the FP16 decode kernel over the codes, a block's scale applied
// once to what its 16 keys gave:
//   s = (S_hi + 2^-10 S_lo) (scale kscale)     q split into hi and lo;
//   o = o 2^(m_old - m_new) + vscale (O'_hi + O'_lo)   2^14 p split into hi and lo.
// A product over a block's 16 keys starts afresh and is added up in FP32 registers.
//
// Products.  With half the bytes of the FP16 cache, time is as short for the
// arithmetic, so the keys are the 16 rows of an m16n8k16 product and the eight
// columns are query heads (the FP16 kernel has eight heads in the rows, hi and lo):
//   S^T = K q^T      a lane has two keys of a head (or of two);
//   O^T = V^T p^T    a lane has DP/8 dimensions of it.
// The weights go from one layout to the other by a transposition of 8 x 8 FP16
// values (movmatrix).  Where up to four heads share a key head, hi and lo of each
// stand side by side (Four): half the products, weights and sums of rows of eight
// heads, 48 sequences of 129 to 6001 tokens take 41 us instead of 45.  Otherwise the
// columns are eight heads, hi in one product and lo in another, and a lane has two
// heads side by side for packed arithmetic (Eight): 16 sequences of 20001 to 65536
// tokens with 16 heads a key head take 173 us, as two Fours for each eight 203.
//
// Large values.  The sums hold 2^14 p times the values, and leave binary32 with one
// value of 2^114, or 2^16 of 2^98, where their mean is an ordinary number.  A warp whose
// results are not all numbers goes through its keys once more with values of kDown
// times their size, and replaces those that were not.  The second pass is a copy of the
// first in the code, so that the first is what it would be alone: a flag in one copy, or a
// look at each tile's scales before its products, took 1 to 3 % of every call.  The 48
// sequences take 78 us where all of them go through it.
//
// Layout.  The sum over the head dimension may go in any order, and so may the
// rows of the output and the keys of a block: a lane's operands are 16 codes that
// stand side by side in a row, one 16-byte load from shared memory, and which keys
// it has is chosen so that no load has bank conflicts (see key_of).  Codes become
// FP16 two at a time, 1024 + 128 + code by a bitwise operation and one subtraction.
// A warp loads its own tiles (TMA, keys and values apart).  An earlier form, in which each lane
// copied just its own words with cp.async, needed no barrier and no swizzle, but
// moved 3.9 TB/s at most: eight rows of 64 bytes an instruction.
//
// Work is cut and joined as in the FP16 kernel (attn_line.cuh).
#include <cuda_fp16.h>

#include <cmath>

#include "attn.h"

namespace compfp32 {
namespace {
constexpr int kTileShift = 0;       // a tile's size goes by the heads: see Cfg
constexpr int kLeastKeys = 32;      // a sequence of 777 alone takes 12.3 us, with 64 12.8, with 128 13.2
// A row's beginning (its queries, rotated and split, and its end) takes the time of
// some tiles: 96 sequences of 33 to 2500 tokens of 16 heads of 64 take 30 us, 43 if
// rows count by their keys alone (31 with 3, 33 with 4); 16 of 20001 to 65536 with 16
// heads a key head 173, 181 and (170, 173).
constexpr int kRowCost = 2;
// With the next call's kernel on the SMs before the join has begun, its CTAs are
// spread unevenly: 16 sequences of 20001 to 65536 tokens, four heads a key head, take
// 149 us a call in a row of calls where they take 111 (eight heads 125 and 120; the 48
// ragged sequences 40.8 and 41.2).
constexpr bool kJoinEarly = false;
constexpr float kJoinWeight = 0x1p-12f;  // a row has fewer than 2^12 parts
}
}  // namespace compfp32

#include "attn_line.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

// Keys that are added up before they are added to the sums so far, as in the FP16 kernel.
constexpr int kRunKeys = 1024;
constexpr uint32_t kFaultDecode8 = 0xB01;

// The sums over all keys that a table can name, fewer than 2^30, stay below 2^124 with
// this for any values that are binary32 numbers.
constexpr float kDown = 0x1p-48f;

// DP: head dimension padded to 64 or 128; NT: query heads of a warp, in fours.
// A tile is some blocks of 16 keys.  What a tile costs whatever its size (waits, loads,
// the maximum) is some 190 instructions, a block's products and conversions are 300 to
// 400, so larger tiles are faster until the SM waits for their loads: with four heads of
// 128 tiles of 32 keys take 41 us where 64 take 45 (48 ragged sequences), with eight 31
// and 34; with two heads of 64, 129 where 64 take 111, with 16 of 128, 181 where 64
// take 173 (16 long ones).
// One stage each for keys and values is enough, each filled again as soon as it has been
// read, as the other is: an earlier form took 42 us with two stages where it took 41 with
// one (ragged), and 133 where 124 (eight heads, long).
template <int DP, int NT>
struct Cfg {
    static constexpr int kWords = DP / 64;                  // 16-byte words of a key that a lane has
    static constexpr int kTileShift = DP == 128 && NT < 4 ? 5 : 6;
    static constexpr int kTile = 1 << kTileShift, kBlocks = kTile / COMP_KV8_BLOCK;
    static constexpr uint32_t kPlane = kTile * DP;          // the keys or the values of a tile
    static constexpr int kCtas = NT == 4 ? 2 : 3;           // an SM
    static constexpr size_t kSmem = 1024 + kWarps * 2 * kPlane;
};

struct Cache8 {
    const float* k_scale;
    const float* v_scale;
    comp_rope_t rope;
    int wide;               // its angles stand on 16 bytes
};

// Rows of DP codes in shared memory, swizzled by the TMA: the 16-byte chunk
// `chunk` of a row (128-byte rows), or the same of 64-byte rows.
template <int DP>
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk)
{
    return DP == 128 ? sw128(row, chunk) : row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}

// The key that stands at place `at` of eight.  A quarter of a warp loads four chunks
// of the keys at two places, 2 a and 2 a + 1: with 128-byte rows their numbers
// differ in bit 2, with 64-byte rows in bit 0.  For the values it (with 64-byte rows
// half a warp, 8 bytes a lane) loads two (four) columns of dimensions of the keys at
// the four even or the four odd places: with 128-byte rows these differ above bit 0,
// with 64-byte rows in bit 0 or in bit 2.  So all 32 banks are read once.
template <int DP>
__device__ __forceinline__ int key_of(int at)
{
    return ((DP == 128 ? 0x36147250u : 0x65217430u) >> (4 * at)) & 7u;
}

// The largest magnitude of three; NaN if one of them is.
__device__ __forceinline__ float largest(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ bool is_number(float x) { return fabsf(x) < INFINITY; }

// A 4-byte copy that the barrier waits for: it counts one arrival of this thread
// when the copy has landed.
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src, bool there, uint64_t* bar)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Loads from shared memory, in order after the wait for the stage.
__device__ __forceinline__ void lds(uint32_t at, uint32_t (&v)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void lds(uint32_t at, uint32_t (&v)[2])
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at) : "memory");
}

__device__ __forceinline__ uint32_t lds(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// c += a b: a 16 x 16, b 16 x 8, FP16 in, FP32 sums.  Not volatile: the compiler
// may mix the products of one block with the conversions of the next.
__device__ __forceinline__ void mma16816_free(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes 0 and 2 of w, two codes, as FP16: 0x6400 + u is 1024 + u, u = code + 128.
// One bitwise operation by hand: the compiler makes two of it.
__device__ __forceinline__ uint32_t even_codes(uint32_t w)
{
    const uint32_t mask = 0x00ff00ffu, bias = 0x64806480u;  // 1152 twice
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x) : "r"(w), "r"(mask), "r"(bias));  // (w & mask) ^ bias
    return pack_h2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias)));
}

__device__ __forceinline__ uint32_t odd_codes(uint32_t w)
{
    return even_codes(w >> 8);
}

// An 8 x 8 matrix of FP16 values, two a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t t;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
    return t;
}

// The bytes of w that are -128, a code that is not a number: 0x80 each.
__device__ __forceinline__ uint32_t odd_bytes(uint32_t w)
{
    return __vcmpeq4(w, 0x80808080u) & 0x80808080u;
}

__device__ __forceinline__ void prefetch_l1(const void* p)
{
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

__device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Whether a block has such codes: the sign of its scale.
__device__ __forceinline__ bool has_odd(float scale)
{
    return __float_as_int(scale) < 0;
}

// A query head's values in a lane: step 4 j + w of the head dimension takes word w of the
// lane's codes, whose four stand in the order 0, 2, 1, 3.
__device__ __forceinline__ void split_step(const float4& x, uint32_t (&hi)[2], uint32_t (&lo)[2])
{
    split2(x.x, x.z, hi[0], lo[0]);
    split2(x.y, x.w, hi[1], lo[1]);
}

__device__ __forceinline__ float warp_max_of_places(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

__device__ __forceinline__ float warp_sum_of_places(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Up to four query heads: hi and lo of each side by side in a product's eight columns.
// A lane has head quad's scores of its two keys, its part of the sum, DP/8 dimensions.
template <int DP, int BLOCKS>
struct Four {
    static constexpr int kHeads = 1;                    // of a lane
    uint32_t q[DP / 16][2], pb[BLOCKS][2];
    float s[2][4], x[BLOCKS][2], m, l;
    uint64_t o[DP / 16];

    static __device__ __forceinline__ int q_head(int lane) { return lane >> 3; }
    static __device__ __forceinline__ int out_head(int quad, int) { return quad; }
    __device__ __forceinline__ void put(int k, const float4& v, int g)
    {
        uint32_t hi[2], lo[2];
        split_step(v, hi, lo);
        q[k][0] = g & 1 ? lo[0] : hi[0];
        q[k][1] = g & 1 ? lo[1] : hi[1];
    }
    __device__ __forceinline__ void reset()
    {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            o[d] = 0;
    }
    __device__ __forceinline__ void begin_scores()
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[0][e] = s[1][e] = 0.0f;
    }
    // two chains, the even and the odd steps
    __device__ __forceinline__ void score(int k, const uint32_t (&a)[4])
    {
        mma16816_free(s[k & 1], a, q[k][0], q[k][1]);
    }
    __device__ __forceinline__ void end_scores(int b, float kc)
    {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint64_t both = add2(f2_bits(s[0][2 * e], s[0][2 * e + 1]), f2_bits(s[1][2 * e], s[1][2 * e + 1]));
            x[b][e] = __fmul_rn(fmaf(hi_f(both), 0x1p-10f, lo_f(both)), kc);
        }
    }
    __device__ __forceinline__ void set_score(int b, int e, float v) { x[b][e] = v; }
    // 2^14 p as the values' products take them; the sums so far follow the maximum
    __device__ __forceinline__ void weights()
    {
        float top = fmaxf(x[0][0], x[0][1]);
#pragma unroll
        for (int b = 1; b < BLOCKS; ++b)
            top = fmaxf(top, fmaxf(x[b][0], x[b][1]));
        const float m_new = fmaxf(m, warp_max_of_places(top)), shift = m_new == -INFINITY ? 0.0f : m_new;
        if (__any_sync(0xffffffffu, m_new > m)) {  // rare after some tiles
            const float alpha = ex2(m - shift);
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
                o[d] = mul2(o[d], f2_bits(alpha, alpha));
        }
        m = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            // each step rounded as the maximum was, or large scores would not end at 0
            const uint64_t e = add2(add2(f2_bits(x[b][0], x[b][1]), f2_bits(-shift, -shift)), f2_bits(14.0f, 14.0f));
            const float w0 = ex2(lo_f(e)), w1 = ex2(hi_f(e));
            uint32_t hi, lo;
            split_p(w0, w1, hi, lo);
            pb[b][0] = transposed(__byte_perm(hi, lo, 0x5410));
            pb[b][1] = transposed(__byte_perm(hi, lo, 0x7632));
            sum += w0 + w1;
        }
        l += sum;
    }
    // dimensions 2 d and 2 d + 1 of a block
    __device__ __forceinline__ void value(int b, int d, const uint32_t (&a)[4], float vs)
    {
        float y[4] = {};
        mma16816_free(y, a, pb[b][0], pb[b][1]);
        o[d] = fma2(f2_bits(y[0] + y[1], y[2] + y[3]), f2_bits(vs, vs), o[d]);
    }
    // dimensions 4 j .. 4 j + 3 of the lane's head
    __device__ __forceinline__ float4 four(int j, int) const
    {
        return make_float4(lo_f(o[2 * j]), hi_f(o[2 * j]), lo_f(o[2 * j + 1]), hi_f(o[2 * j + 1]));
    }
    __device__ __forceinline__ void set_four(int j, int, const float4& v)
    {
        o[2 * j] = f2_bits(v.x, v.y);
        o[2 * j + 1] = f2_bits(v.z, v.w);
    }
    __device__ __forceinline__ float2 sums(int) const { return make_float2(m, l); }
    __device__ __forceinline__ void set_sum(int, float v) { l = v; }
};

// Up to eight query heads: a product's eight columns are hi of all, another's lo.  A lane
// has the heads 2 quad and 2 quad + 1 side by side, so that most operations do two.
template <int DP, int BLOCKS>
struct Eight {
    static constexpr int kHeads = 2;
    uint32_t q[DP / 16][2][2], pb[BLOCKS][2][2];        // hi, lo
    float s[2][4];
    uint64_t x[BLOCKS][2], m, l, o[DP / 16][2];

    static __device__ __forceinline__ int q_head(int lane) { return lane >> 2; }
    static __device__ __forceinline__ int out_head(int quad, int h) { return quad * 2 + h; }
    __device__ __forceinline__ void put(int k, const float4& v, int) { split_step(v, q[k][0], q[k][1]); }
    __device__ __forceinline__ void reset()
    {
        m = f2_bits(-INFINITY, -INFINITY);
        l = 0;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            o[d][0] = o[d][1] = 0;
    }
    __device__ __forceinline__ void begin_scores()
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[0][e] = s[1][e] = 0.0f;
    }
    // two chains, hi and lo
    __device__ __forceinline__ void score(int k, const uint32_t (&a)[4])
    {
        mma16816_free(s[0], a, q[k][0][0], q[k][0][1]);
        mma16816_free(s[1], a, q[k][1][0], q[k][1][1]);
    }
    __device__ __forceinline__ void end_scores(int b, float kc)
    {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            x[b][e] = mul2(fma2(f2_bits(s[1][2 * e], s[1][2 * e + 1]), f2_bits(0x1p-10f, 0x1p-10f),
                                f2_bits(s[0][2 * e], s[0][2 * e + 1])),
                           f2_bits(kc, kc));
    }
    __device__ __forceinline__ void set_score(int b, int e, float v) { x[b][e] = f2_bits(v, v); }
    __device__ __forceinline__ void weights()
    {
        float top0 = fmaxf(lo_f(x[0][0]), lo_f(x[0][1])), top1 = fmaxf(hi_f(x[0][0]), hi_f(x[0][1]));
#pragma unroll
        for (int b = 1; b < BLOCKS; ++b) {
            top0 = fmaxf(top0, fmaxf(lo_f(x[b][0]), lo_f(x[b][1])));
            top1 = fmaxf(top1, fmaxf(hi_f(x[b][0]), hi_f(x[b][1])));
        }
        const float m0 = fmaxf(lo_f(m), warp_max_of_places(top0)), m1 = fmaxf(hi_f(m), warp_max_of_places(top1));
        const float shift0 = m0 == -INFINITY ? 0.0f : m0, shift1 = m1 == -INFINITY ? 0.0f : m1;
        if (__any_sync(0xffffffffu, m0 > lo_f(m) || m1 > hi_f(m))) {
            const uint64_t alpha = f2_bits(ex2(lo_f(m) - shift0), ex2(hi_f(m) - shift1));
            l = mul2(l, alpha);
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                o[d][0] = mul2(o[d][0], alpha);
                o[d][1] = mul2(o[d][1], alpha);
            }
        }
        m = f2_bits(m0, m1);
        const uint64_t shift = f2_bits(-shift0, -shift1);
        uint64_t sum = 0;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint64_t y = add2(add2(x[b][e], shift), f2_bits(14.0f, 14.0f));
                const float w0 = ex2(lo_f(y)), w1 = ex2(hi_f(y));
                uint32_t hi, lo;
                split_p(w0, w1, hi, lo);
                pb[b][0][e] = transposed(hi);
                pb[b][1][e] = transposed(lo);
                sum = add2(sum, f2_bits(w0, w1));
            }
        l = add2(l, sum);
    }
    // hi and lo have no scale between them and add up in one product's sums
    __device__ __forceinline__ void value(int b, int d, const uint32_t (&a)[4], float vs)
    {
        float y[4] = {};
        mma16816_free(y, a, pb[b][1][0], pb[b][1][1]);
        mma16816_free(y, a, pb[b][0][0], pb[b][0][1]);
        o[d][0] = fma2(f2_bits(y[0], y[1]), f2_bits(vs, vs), o[d][0]);
        o[d][1] = fma2(f2_bits(y[2], y[3]), f2_bits(vs, vs), o[d][1]);
    }
    static __device__ __forceinline__ float part(uint64_t v, int h) { return h ? hi_f(v) : lo_f(v); }
    __device__ __forceinline__ float4 four(int j, int h) const
    {
        return make_float4(part(o[2 * j][0], h), part(o[2 * j][1], h), part(o[2 * j + 1][0], h),
                           part(o[2 * j + 1][1], h));
    }
    __device__ __forceinline__ void set_four(int j, int h, const float4& v)
    {
        const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint64_t& to = o[2 * j + e / 2][e % 2];
            to = h ? f2_bits(lo_f(to), y[e]) : f2_bits(y[e], hi_f(to));
        }
    }
    __device__ __forceinline__ float2 sums(int h) const { return make_float2(part(m, h), part(l, h)); }
    __device__ __forceinline__ void set_sum(int h, float v) { l = h ? f2_bits(lo_f(l), v) : f2_bits(v, hi_f(l)); }
};

template <int DP, int NT, int BLOCKS>
struct MathOf {
    using T = Eight<DP, BLOCKS>;
    static constexpr int kSets = NT / 2, kSetHeads = 8;
};

template <int DP, int BLOCKS>
struct MathOf<DP, 1, BLOCKS> {
    using T = Four<DP, BLOCKS>;
    static constexpr int kSets = 1, kSetHeads = 4;
};

// What a CTA's warps keep beside their tiles, each its own.
template <int DP, int NT>
struct Shared {
    uint64_t full[kWarps][2];                           // keys, values
    float scale[kWarps][2][Cfg<DP, NT>::kBlocks];
    int abort_flag[kWarps];
    float2 far[kWarps][NT][32];                         // maximum and sum of each head of a lane
};

// A pass over a warp's piece of the line; whether there is a result that may be a number
// and is not.  SMALL: the second one, with values of kDown times their size, which replaces
// those.  i: the tiles that went through the stages so far.
template <int DP, int NT, bool SMALL>
__device__ __forceinline__ bool go_over(const CUtensorMap& map_k, const CUtensorMap& map_v, const Params& p,
                                        const Cache8& c, Shared<DP, NT>& shared, uint8_t* const stages,
                                        const int piece, int& i)
{
    using C = Cfg<DP, NT>;
    constexpr int W = C::kWords, kDims = DP / 8;  // kDims: of a lane's output
    constexpr int kTileShift = C::kTileShift, kTile = C::kTile, kBlocks = C::kBlocks, kRun = kRunKeys / kTile;
    const int dim = p.dim;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t k_stage = smem_u32(stages), v_stage = k_stage + C::kPlane;
    uint64_t* const full = shared.full[warp];
    int begin, end;
    Place r;
    if (!find_piece(p, piece, begin, end, r))
        return false;

    // A lane has the codes of the key at place g (and 8 more) in the words quad + 4 j,
    // and for the values those of the keys at 2 quad and 2 quad + 1 (and 8 more),
    // dimensions g kDims on.
    const int g = lane >> 2, quad = lane & 3;
    const float c2 = p.scale * kAttnLog2E;
    const int my_key = key_of<DP>(g);
    const uint32_t k_at = swizzled<DP>(my_key, quad);
    uint32_t v_at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        v_at[e] = swizzled<DP>(key_of<DP>(quad * 2 + e), g * kDims / 16) + g * kDims % 16;

    // Loads.  The lanes hold the page numbers of a row's next tiles, fetched when it is
    // new, 32 of them; one that is not there: a place beyond the cache, which reads
    // zeros.  The first lanes have a block's scale each, and those whose block begins a
    // page (or the tile) a box.  A tile's keys are loaded when those of the tile before
    // have been read, and its values, from the place that `at_v` keeps, likewise.
    Place next = r;
    int pages = 0, page_tile = 0, loads_k = i, loads_v = i, ahead = begin;  // ahead: the next place of the line
    const int blocks_shift = p.page_shift - 4;
    const int box_shift = min(p.page_shift, kTileShift);
    const int split = kTileShift - box_shift;       // a tile is on 1 << split pages
    const int my_box = lane * 16 >> box_shift, my_block = (lane * 16 & ((1 << box_shift) - 1)) >> 4;
    struct {
        int unit, slot;
        bool there;
    } at_v;
    auto look_up = [&] {
        page_tile = next.tile;
        const int tile = next.tile + (lane >> split);
        const int col = (next.tile * kTile + lane * (kTile >> split)) >> p.page_shift;
        pages = tile < next.tiles && col < p.width ? p.table[next.b * p.width + col] : -1;
    };
    // A row's queries and angles, some tiles before they are needed: lines of 32 values.
    auto prefetch_row = [&](const Place& at) {
        const int head = at.unit / p.row_blocks, first_head = at.unit % p.row_blocks * (NT * 4);
        const int heads = min(NT * 4, p.group - first_head), lines = (dim + 31) / 32;
        for (int l = lane; l < heads * lines; l += 32)
            prefetch_l1(p.q + at.b * p.q_token + (head * p.group + first_head + l / lines) * p.q_head +
                        l % lines * 32);
        const float* const angles = c.rope.rot > 0 ? angles_of(c.rope, at.own - 1) : nullptr;
        if (angles && lane * 32 < c.rope.rot)
            prefetch_l1(angles + lane * 32);
    };
    auto issue = [&](int is_v) {
        if (lane == 0)
            mbar_arrive_expect_tx(&full[is_v], C::kPlane);
        __syncwarp();
        if (lane < kBlocks) {
            if (my_block == 0)
                tma_load_3d(stages + is_v * C::kPlane + lane * (C::kPlane / kBlocks), is_v ? &map_v : &map_k,
                            &full[is_v], 0, at_v.slot, at_v.there ? at_v.unit : p.pages * p.kv_heads);
            const int64_t scale = (static_cast<int64_t>(at_v.unit) << blocks_shift) + (at_v.slot >> 4) + my_block;
            copy4_async(smem_u32(&shared.scale[warp][is_v][lane]), (is_v ? c.v_scale : c.k_scale) + scale, at_v.there,
                        &full[is_v]);
        }
    };
    auto load_k = [&] {
        const int box = ((next.tile - page_tile) << split) + (my_box & ((1 << split) - 1));
        const int at = __shfl_sync(0xffffffffu, pages, box);
        at_v.there = at >= 0 && at < p.pages;
        at_v.slot = (next.tile * kTile) & ((1 << p.page_shift) - 1);
        at_v.unit = (at_v.there ? at : 0) * p.kv_heads + next.unit / p.row_blocks;
        issue(0);
        ++loads_k;
        ++ahead;
        if (++next.tile == next.tiles)
            ahead += kRowCost;
        if (ahead < end) {
            if (next.tile == next.tiles) {
                next_row(p, next);
                look_up();
                prefetch_row(next);
            } else if (next.tile == page_tile + (32 >> split)) {
                look_up();
            }
        }
    };
    auto load_v = [&] {
        issue(1);
        ++loads_v;
    };
    look_up();
    if (ahead < end) {
        load_k();
        load_v();
    }

    using Math = MathOf<DP, NT, kBlocks>;
    using Rows = typename Math::T;
    constexpr int kSets = Math::kSets;
    Rows rows[kSets];
    bool ok = true, lost = false;
    int fragment = 0;
    for (int at = begin; ok && at < end; ++fragment) {
        const int n = min(r.tiles - r.tile, end - at);
        const int head = r.unit / p.row_blocks, first_head = r.unit % p.row_blocks * (NT * 4);
        // The query heads, rotated and split.
        const float* const angles = c.rope.rot > 0 ? angles_of(c.rope, r.own - 1) : nullptr;
        // Halves of a head of DP that is all rotated: the partner of dimension d stands in
        // the lane's word 4 steps on (heads of 128), or in the lane 2 quads on (64).
        const bool paired = c.rope.rot == DP && !c.rope.interleaved && p.vec_q && c.wide && angles;
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            const int hg = first_head + set * Math::kSetHeads + Rows::q_head(lane);
            const float* const src = p.q + r.b * p.q_token + (head * p.group + hg) * p.q_head;
            float4 x[DP / 16];
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int d = (quad + 4 * (k / 4)) * 16 + k % 4 * 4;
                x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (hg < p.group && d < dim)
                    x[k] = paired ? __ldg(reinterpret_cast<const float4*>(src + d))
                                  : load_rotated(src, d, c.rope, angles, p.vec_q != 0, c.wide != 0);
            }
            if (paired) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int i = (DP == 128 ? quad : quad & 1) * 16 + w * 4;
                    const float4 a = load_angles(angles + 2 * i, true), b = load_angles(angles + 2 * i + 4, true);
                    if constexpr (DP == 128) {
                        const float4 y = x[w], z = x[w + 4];
                        x[w] = make_float4(turn(y.x, a.x, z.x, a.y, false), turn(y.y, a.z, z.y, a.w, false),
                                           turn(y.z, b.x, z.z, b.y, false), turn(y.w, b.z, z.w, b.w, false));
                        x[w + 4] = make_float4(turn(z.x, a.x, y.x, a.y, true), turn(z.y, a.z, y.y, a.w, true),
                                               turn(z.z, b.x, y.z, b.y, true), turn(z.w, b.z, y.w, b.w, true));
                    } else {
                        const float4 y = x[w];
                        const float4 z = make_float4(__shfl_xor_sync(0xffffffffu, y.x, 2),
                                                     __shfl_xor_sync(0xffffffffu, y.y, 2),
                                                     __shfl_xor_sync(0xffffffffu, y.z, 2),
                                                     __shfl_xor_sync(0xffffffffu, y.w, 2));
                        const bool second = quad >= 2;
                        x[w] = make_float4(turn(y.x, a.x, z.x, a.y, second), turn(y.y, a.z, z.y, a.w, second),
                                           turn(y.z, b.x, z.z, b.y, second), turn(y.w, b.z, z.w, b.w, second));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                rows[set].put(k, x[k], g);
            rows[set].reset();
        }
        const int part = 2 * piece + (fragment > 0 ? 1 : 0);
        const int o_dim = g * kDims;
        // where the sums of the runs before stand, and shared.far has what belongs to them
        float* const slot =
            p.part_o + static_cast<int64_t>(SMALL ? 2 * p.pieces + piece : part) * (NT * 4) * dim + o_dim;
        auto row_of = [&](int set, int h) { return set * Math::kSetHeads + Rows::out_head(quad, h); };
        auto ready = [&](int is_v) {
            ok = __all_sync(0xffffffffu, mbar_try_wait(&full[is_v], i & 1)) ||
                 attn_warp_wait(&full[is_v], i & 1, &shared.abort_flag[warp], kFaultDecode8);
            return ok;
        };
        for (int t0 = 0; ok && t0 < n; t0 += kRun) {
            const int t1 = min(n, t0 + kRun);
            for (int t = t0; t < t1; ++t, ++i) {
                if (!ready(0))
                    break;
                const int left = r.own - (r.tile + t) * kTile;  // keys of the tile that count
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    if (b > 0 && b * 16 >= left) {  // a block behind the end; its scale may be anything
#pragma unroll
                        for (int set = 0; set < kSets; ++set) {
                            rows[set].set_score(b, 0, -INFINITY);
                            rows[set].set_score(b, 1, -INFINITY);
                        }
                        continue;
                    }
#pragma unroll
                    for (int set = 0; set < kSets; ++set)
                        rows[set].begin_scores();
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        uint32_t word[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e)  // the swizzle leaves bit 2 of a chunk in its place
                            lds(k_stage + (k_at ^ (j * 64)) + (b * 16 + e * 8) * DP, word[e]);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t a[4] = {even_codes(word[0][w]), even_codes(word[1][w]),
                                                   odd_codes(word[0][w]), odd_codes(word[1][w])};
#pragma unroll
                            for (int set = 0; set < kSets; ++set)
                                rows[set].score(j * 4 + w, a);
                        }
                    }
                    const float ks = shared.scale[warp][0][b];
#pragma unroll
                    for (int set = 0; set < kSets; ++set)
                        rows[set].end_scores(b, fabsf(ks) * c2);
                    const int end_of = left - b * 16;  // keys of the block that count
                    if (end_of < 16 || has_odd(ks)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            unsigned odd = 0;  // four bits a place
                            if (has_odd(ks)) {
                                uint32_t any = 0;
#pragma unroll
                                for (int j = 0; j < W; ++j) {
                                    uint32_t word[4];
                                    lds(k_stage + (k_at ^ (j * 64)) + (b * 16 + e * 8) * DP, word);
                                    any |= odd_bytes(word[0]) | odd_bytes(word[1]) | odd_bytes(word[2]) |
                                           odd_bytes(word[3]);
                                }
                                odd = __ballot_sync(0xffffffffu, any != 0) >> (4 * g) & 0xfu;
                            }
                            const bool out = e * 8 + my_key >= end_of;
                            if (out || odd)
#pragma unroll
                                for (int set = 0; set < kSets; ++set)
                                    rows[set].set_score(b, e, out ? -INFINITY : __int_as_float(0x7fffffff));
                        }
                        __syncwarp();
                    }
                }
                __syncwarp();  // all lanes have read the keys
                if (ahead < end)
                    load_k();
#pragma unroll
                for (int set = 0; set < kSets; ++set)
                    rows[set].weights();
                if (!ready(1))
                    break;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    if (b > 0 && b * 16 >= left)
                        continue;
                    // the values: four keys' codes of kDims dimensions
                    constexpr int VW = DP / 32;
                    uint32_t v[4][VW];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        lds(v_stage + v_at[k & 1] + (b * 16 + (k >> 1) * 8) * DP, v[k]);
                    const float vs = shared.scale[warp][1][b], value_scale = SMALL ? fabsf(vs) * kDown : fabsf(vs);
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d) {
                        // dimensions 2 d and 2 d + 1 of two keys: bytes a0 a1 b0 b1
                        const uint32_t p01 = __byte_perm(v[0][d / 2], v[1][d / 2], d & 1 ? 0x7632 : 0x5410);
                        const uint32_t p23 = __byte_perm(v[2][d / 2], v[3][d / 2], d & 1 ? 0x7632 : 0x5410);
                        const uint32_t a[4] = {even_codes(p01), odd_codes(p01), even_codes(p23), odd_codes(p23)};
#pragma unroll
                        for (int set = 0; set < kSets; ++set)
                            rows[set].value(b, d, a, value_scale);
                    }
                    if (has_odd(vs)) {
                        // the components in which a key that counts is not a number: a bit for
                        // each of the lane's dimensions, of its four keys, then of all 16
                        uint32_t odd = 0;
                        for (int k = 0; k < 4; ++k)
                            if (key_of<DP>(quad * 2 + (k & 1)) + b * 16 + 8 * (k >> 1) < left)
                                for (int w = 0; w < VW; ++w) {
                                    const uint32_t word =
                                        lds(v_stage + v_at[k & 1] + (b * 16 + (k >> 1) * 8) * DP + w * 4);
                                    odd |= ((odd_bytes(word) >> 7) * 0x00204081u >> 21 & 0xfu) << (4 * w);
                                }
                        odd |= __shfl_xor_sync(0xffffffffu, odd, 1);
                        odd |= __shfl_xor_sync(0xffffffffu, odd, 2);
                        const float nan = __int_as_float(0x7fffffff);
#pragma unroll
                        for (int set = 0; set < kSets; ++set)
#pragma unroll
                            for (int h = 0; h < Rows::kHeads; ++h)
#pragma unroll
                                for (int j = 0; j < kDims / 4; ++j) {
                                    const float4 y = rows[set].four(j, h);
                                    const uint32_t bad = odd >> (4 * j);
                                    rows[set].set_four(j, h, make_float4(bad & 1 ? nan : y.x, bad & 2 ? nan : y.y,
                                                                         bad & 4 ? nan : y.z, bad & 8 ? nan : y.w));
                                }
                    }
                }
                __syncwarp();  // all lanes have read the values
                if (loads_v < loads_k)
                    load_v();
            }
            if (t0 == 0 && t1 == n)
                continue;
#pragma unroll
            for (int set = 0; set < kSets; ++set)
#pragma unroll
                for (int h = 0; h < Rows::kHeads; ++h) {
                    float2& far = shared.far[warp][set * Rows::kHeads + h][lane];
                    float* const sums = slot + row_of(set, h) * dim;
                    if (t0 > 0) {  // added to those of the runs before
                        const float2 now = rows[set].sums(h);
                        const float a = ex2(far.x - (now.x == -INFINITY ? 0.0f : now.x));
                        rows[set].set_sum(h, fmaf(far.y, a, now.y));
                        if (o_dim < dim)
#pragma unroll
                            for (int j = 0; j < kDims / 4; ++j) {
                                const float4 y = *reinterpret_cast<const float4*>(sums + 4 * j);
                                const float4 z = rows[set].four(j, h);
                                rows[set].set_four(j, h, make_float4(fmaf(y.x, a, z.x), fmaf(y.y, a, z.y),
                                                                     fmaf(y.z, a, z.z), fmaf(y.w, a, z.w)));
                            }
                    }
                    if (t1 < n) {  // and put there, to begin anew
                        far = rows[set].sums(h);
                        rows[set].set_sum(h, 0.0f);
#pragma unroll
                        for (int j = 0; j < kDims / 4; ++j) {
                            if (o_dim < dim)
                                *reinterpret_cast<float4*>(sums + 4 * j) = rows[set].four(j, h);
                            rows[set].set_four(j, h, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
                        }
                    }
                }
        }

        // the row, or this warp's part of it
        const bool whole = n == r.tiles;
#pragma unroll
        for (int set = 0; set < kSets; ++set)
#pragma unroll
            for (int h = 0; h < Rows::kHeads; ++h) {
                const float2 last = rows[set].sums(h);
                const float sum = warp_sum_of_places(last.y);
                const int row = row_of(set, h), hg = first_head + row;
                if (!ok || hg >= p.group)
                    continue;
                const int64_t at_row = static_cast<int64_t>(r.b) * p.heads + head * p.group + hg;
                float* const dst = (whole ? p.out + at_row * dim
                                          : p.part_o + (static_cast<int64_t>(part) * (NT * 4) + row) * dim) +
                                   o_dim;
                const float norm = sum == 0.0f ? 0.0f : (SMALL ? 1.0f / kDown : 1.0f) / sum;
                float top = 0.0f;
                if (o_dim < dim)
#pragma unroll
                    for (int j = 0; j < kDims / 4; ++j) {
                        const float4 z = rows[set].four(j, h);
                        float y[4] = {z.x * norm, z.y * norm, z.z * norm, z.w * norm};
                        if constexpr (SMALL) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (is_number(dst[4 * j + e]))
                                    y[e] = dst[4 * j + e];
                        } else {
                            top = largest(largest(top, y[0], y[1]), y[2], y[3]);
                        }
                        if (p.vec_out || !whole) {
                            *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(y[0], y[1], y[2], y[3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dst[4 * j + e] = y[e];
                        }
                    }
                lost = lost || (!is_number(top) && is_number(sum));
                if (!SMALL && g == 0) {
                    const float lse =
                        sum == 0.0f ? -INFINITY : fmaf(last.x, kAttnLn2, logf(sum * (1.0f / kAttnPScale)));
                    if (!whole)
                        p.part_lse[part * (NT * 4) + row] = lse;
                    else if (p.lse)
                        p.lse[at_row] = lse;
                }
            }
        at += n + kRowCost;
        if (at < end)
            next_row(p, r);
    }
    if (!ok) {  // what was issued lands before the warp leaves
        if (loads_k > 0)
            attn_drain_wait(&full[0], (loads_k - 1) & 1);
        if (loads_v > 0)
            attn_drain_wait(&full[1], (loads_v - 1) & 1);
    }
    return ok && __any_sync(0xffffffffu, lost);
}

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<DP, NT>::kCtas)
    attn_decode8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ Params p, const __grid_constant__ Cache8 c)
{
    using C = Cfg<DP, NT>;
    const int dim = p.dim;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared<DP, NT> shared;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* const stages =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
        warp * (2 * C::kPlane);
    if (lane == 0) {
        for (int i = 0; i < 2; ++i)
            mbar_init(&shared.full[warp][i], 1 + C::kBlocks);  // the TMA's bytes and the scales
        shared.abort_flag[warp] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    // What the first steps read one after the other comes into L2 meanwhile, a line a
    // thread: lengths, page tables, queries.
    {
        const int64_t thread = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
        const int64_t lines = (static_cast<int64_t>(p.batch) * p.width + 31) / 32;
        const int64_t q_lines = (static_cast<int64_t>(p.heads) * dim + 31) / 32, row = (thread - lines) / q_lines;
        if (thread < lines)
            prefetch_l2(p.table + thread * 32);
        else if (row < p.batch)
            prefetch_l2(p.q + row * p.q_token + (thread - lines) % q_lines * 32 / dim * p.q_head +
                        (thread - lines) % q_lines * 32 % dim);
        if (threadIdx.x == 0 && blockIdx.x * 32 < p.batch)
            prefetch_l2(p.lengths + blockIdx.x * 32);
    }
    grid_dependency_wait();
    grid_dependency_launch();  // the join relies on what came before

    // this warp's piece; consecutive ones are on different SMs
    const int ctas = p.pieces / kWarps;
    const int piece = warp * ctas + blockIdx.x;

    int i = 0;
    if (go_over<DP, NT, false>(map_k, map_v, p, c, shared, stages, piece, i))
        go_over<DP, NT, true>(map_k, map_v, p, c, shared, stages, piece, i);
}

// A cache's codes: rows are the tokens of one head on one page.
bool encode_codes(CUtensorMap* map, const int8_t* base, const comp_kv8_cache_t& c, int tile_shift)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const bool wide = c.head_dim > 64;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.pages * c.kv_heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_dim),
                                   static_cast<cuuint64_t>(c.page_size) * static_cast<cuuint64_t>(c.head_dim)};
    const cuuint32_t rows = c.page_size < 1 << tile_shift ? c.page_size : 1 << tile_shift;
    const cuuint32_t box[3] = {wide ? 128u : 64u, rows, 1}, estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, int NT>
comp_status_t launch_t(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, const Cache8& c,
                       const DeviceInfo& dev, cudaStream_t stream)
{
    using C = Cfg<DP, NT>;
    static std::mutex mu;
    static bool done[64] = {};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev.device < 0 || dev.device >= 64)
            return COMP_ERR_CUDA;
        if (!done[dev.device]) {
            if (cudaFuncSetAttribute(attn_decode8_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(C::kSmem)) != cudaSuccess) {
                (void)cudaGetLastError();
                return COMP_ERR_CUDA;
            }
            done[dev.device] = true;
        }
    }
    return launch_pdl(attn_decode8_kernel<DP, NT>, p.pieces / kWarps, kThreads, C::kSmem, stream, mk, mv, p, c);
}

// Pieces of the line of tiles: one for each warp that the SMs hold.  The
// workspace's size must not depend on the device, so their number is bounded.
constexpr int kMostSms = 160;

// Columns of four query heads that a warp takes at once.
int columns_at_once(int group)
{
    return group > 8 ? 4 : (group > 4 ? 2 : 1);
}

int ctas_an_sm(int nt)
{
    return nt == 4 ? Cfg<128, 4>::kCtas : Cfg<128, 1>::kCtas;
}

template <int DP>
int tile_shift_of_columns(int nt)
{
    return nt == 4 ? Cfg<DP, 4>::kTileShift : (nt == 2 ? Cfg<DP, 2>::kTileShift : Cfg<DP, 1>::kTileShift);
}

int tile_shift_for(int head_dim, int nt)
{
    return head_dim <= 64 ? tile_shift_of_columns<64>(nt) : tile_shift_of_columns<128>(nt);
}

// Floats of the workspace: for each piece two parts of rows and the sums of a second pass,
// and their lse.
int64_t slots_of(int nt)
{
    return 3 * static_cast<int64_t>(ctas_an_sm(nt)) * kMostSms * kWarps * 4 * nt;
}

}  // namespace

int64_t attn_decode8_bytes(const comp_kv8_cache_t& cache, int heads)
{
    return 4 * slots_of(columns_at_once(heads / cache.kv_heads)) * (cache.head_dim + 1);
}

comp_status_t launch_attn_decode8(const comp_kv8_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                  int heads, float scale, const int32_t* table, int64_t batch, int64_t width,
                                  const int32_t* lengths, const comp_rope_t* rope, float* out, float* lse,
                                  void* workspace, const DeviceInfo& dev, cudaStream_t stream)
{
    const int group = heads / cache.kv_heads, nt = columns_at_once(group);
    float* const ws = static_cast<float*>(workspace);
    Params p{};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.part_o = ws;
    p.part_lse = ws + slots_of(nt) * cache.head_dim;
    p.table = table;
    p.lengths = lengths;
    p.q_token = q_token;
    p.q_head = q_head;
    p.width = width;
    p.pages = static_cast<int>(cache.pages);
    p.batch = static_cast<int>(batch);
    p.heads = heads;
    p.kv_heads = cache.kv_heads;
    p.group = group;
    p.row_blocks = row_blocks(group);
    p.dim = cache.head_dim;
    while ((1 << p.page_shift) < cache.page_size)
        ++p.page_shift;
    p.most_keys = static_cast<int>(width * cache.page_size);
    p.pieces = (dev.sm_count < kMostSms ? dev.sm_count : kMostSms) * ctas_an_sm(nt) * kWarps;
    p.waves = 1;
    p.vec_q = aligned16(q) && q_token % 4 == 0 && q_head % 4 == 0;
    p.vec_out = aligned16(out);  // rows are multiples of 64 bytes
    p.scale = scale;
    p.tile_shift = tile_shift_for(cache.head_dim, nt);
    const Cache8 c{cache.k_scale, cache.v_scale, rope ? *rope : comp_rope_t{},
                   rope && angles_wide(*rope)};
    CUtensorMap mk{}, mv{};
    if (width > 0) {  // otherwise there are no tiles
        if (!encode_codes(&mk, cache.k, cache, p.tile_shift) || !encode_codes(&mv, cache.v, cache, p.tile_shift))
            return COMP_ERR_CUDA;
    }
    comp_status_t st;
    if (cache.head_dim <= 64)
        st = nt == 1   ? launch_t<64, 1>(mk, mv, p, c, dev, stream)
             : nt == 2 ? launch_t<64, 2>(mk, mv, p, c, dev, stream)
                       : launch_t<64, 4>(mk, mv, p, c, dev, stream);
    else
        st = nt == 1   ? launch_t<128, 1>(mk, mv, p, c, dev, stream)
             : nt == 2 ? launch_t<128, 2>(mk, mv, p, c, dev, stream)
                       : launch_t<128, 4>(mk, mv, p, c, dev, stream);
    if (st != COMP_OK)
        return st;
    const Join x{nullptr, nullptr, lse, 0, 4 * nt};
    return launch_pdl(attn_join_kernel, static_cast<int>((batch * heads + 7) / 8), 256, 0, stream, p, x);
}

comp_status_t read_and_clear_decode8_fault(cudaStream_t stream, uint32_t* where)
{
    return read_and_clear_word(&g_attn_fault_word, stream, where);
}

}  // namespace compfp32
