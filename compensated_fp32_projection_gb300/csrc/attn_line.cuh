// Attention of single tokens over pages, whatever the cache's type: the line of
// tiles, its pieces, and the join of the parts of rows that were cut.  Included
// by the decode kernels, each of which has its own copies and defines before:
//   kTileShift log2 of the keys of a tile, or 0 where Params says;
//   kLeastKeys keys of a piece at least, about;
//   kRowCost   tiles that the beginning of a row costs as much time as;
//   kJoinEarly whether the join lets the next kernel start before it has begun;
//   kJoinWeight the largest weight in the join's sums, a power of two: 1, or less where the
//              sums of some parts' values may leave binary32 and their mean does not.
#pragma once

#include "attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kLongKeys = 128;

struct Params {
    const float* q;
    float* out;
    float* lse;             // [batch, heads] (nullptr: none)
    float* part_o;          // [2 * pieces][NB * 8][dim]
    float* part_lse;        // [2 * pieces][NB * 8]
    const int32_t* table;
    const int32_t* lengths;
    int64_t q_token, q_head, width;
    int batch, heads, kv_heads, group, row_blocks, dim;
    int page_shift, pages, shared_keys, most_keys, pieces, waves, vec_q, vec_out, after_prefix;
    float scale;
    int tile_shift;         // where kTileShift is 0
};

__device__ __forceinline__ int tile_shift_of(const Params& p)
{
    return kTileShift > 0 ? kTileShift : p.tile_shift;
}

// Keys of a sequence beyond the shared pages, and their tiles.
__device__ __forceinline__ int own_keys(const Params& p, int b)
{
    const int n = p.lengths[b];
    return max(0, min(n, p.most_keys) - p.shared_keys);
}

__device__ __forceinline__ int tiles_of(const Params& p, int own)
{
    return (own + (1 << tile_shift_of(p)) - 1) >> tile_shift_of(p);
}

// What a row of this many tiles takes of the line.
__device__ __forceinline__ int line_of(int tiles)
{
    return tiles > 0 ? tiles + kRowCost : 0;
}

// What the sequences before `end` take of the line for each unit, by one warp.
__device__ __forceinline__ int sum_tiles(const Params& p, int end)
{
    int n = 0;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < end; b += 32)
        n += line_of(tiles_of(p, own_keys(p, b)));
    return __reduce_add_sync(0xffffffffu, n);
}

// The line of tiles: sequence by sequence, within one head unit by head unit
// (a key/value head and a block of its query heads), kRowCost empty places before
// each row, cut into pieces that
// differ by at most one tile: the first `rest` have one more.  A piece has about
// kLeastKeys at least: a part of a row costs its join more than a tile costs.
// There are `waves` times as many pieces where they have kLongKeys then.
struct Cut {
    int pieces, each, rest;
    __device__ __forceinline__ Cut(const Params& p, int total)
        : pieces(min((total + least(p, kLeastKeys) - 1) / least(p, kLeastKeys),
                     total / p.waves >= least(p, kLongKeys) * p.pieces ? p.waves * p.pieces : p.pieces)),
          each(pieces > 0 ? total / pieces : 0),
          rest(pieces > 0 ? total % pieces : 0)
    {
    }
    static __device__ __forceinline__ int least(const Params& p, int keys) { return max(keys >> tile_shift_of(p), 1); }
    __device__ __forceinline__ int begin(int piece) const { return piece * each + min(piece, rest); }
    __device__ __forceinline__ int piece_of(int tile) const
    {
        const int big = rest * (each + 1);
        return tile < big ? tile / (each + 1) : rest + (tile - big) / each;
    }
};

// A row of the line, and a tile of it.
struct Place {
    int b, unit, tile, own, tiles;
};

__device__ __forceinline__ void set_row(const Params& p, Place& r)
{
    r.own = r.b < p.batch ? own_keys(p, r.b) : 0;
    r.tiles = tiles_of(p, r.own);
}

// The next row that has tiles.
__device__ __forceinline__ void next_row(const Params& p, Place& r)
{
    r.tile = 0;
    if (++r.unit < p.kv_heads * p.row_blocks)
        return;
    r.unit = 0;
    do {
        ++r.b;
        set_row(p, r);
    } while (r.tiles == 0 && r.b < p.batch);
}

// A warp's piece of the line and the place where it begins; false if there is
// none.  A lane sums the tiles of consecutive sequences.
__device__ __forceinline__ bool find_piece(const Params& p, int piece, int& begin, int& end, Place& r)
{
    const int units = p.kv_heads * p.row_blocks, lane = threadIdx.x & 31;
    const int each = (p.batch + 31) / 32, first = lane * each, last = min(first + each, p.batch);
    int mine = 0;
#pragma unroll 8
    for (int b = first; b < last; ++b)
        mine += line_of(tiles_of(p, own_keys(p, b)));
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    const Cut cut(p, __shfl_sync(0xffffffffu, x, 31) * units);
    if (piece >= cut.pieces)
        return false;
    begin = cut.begin(piece);
    end = cut.begin(piece + 1);
    int at = begin - (x - mine) * units;
    r = Place{0, 0, 0, 0, 0};
    const bool here = at >= 0 && at < mine * units;
    if (here) {
        for (r.b = first;; ++r.b) {
            set_row(p, r);
            if (at < line_of(r.tiles) * units)
                break;
            at -= line_of(r.tiles) * units;
        }
        r.unit = at / line_of(r.tiles);
        r.tile = at % line_of(r.tiles) - kRowCost;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    r.b = __shfl_sync(0xffffffffu, r.b, src);
    r.unit = __shfl_sync(0xffffffffu, r.unit, src);
    r.tile = __shfl_sync(0xffffffffu, r.tile, src);
    r.own = __shfl_sync(0xffffffffu, r.own, src);
    r.tiles = __shfl_sync(0xffffffffu, r.tiles, src);
    if (kRowCost > 0) {  // a piece that begins with empty places begins behind them
        begin += max(-r.tile, 0);
        r.tile = max(r.tile, 0);
    }
    return true;
}

// c += a b: a 16 x 16, b 16 x 8, FP16 in, FP32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The parts of each row joined: the prefix's (splits of them), then those of
// the sequence's own keys, in order.  One warp for each row, four values of
// the head dimension a lane.  Four CTAs an SM: 36.2 -> 35.5 us for 64 sequences on
// 8192 tokens, whose rows have 17 parts and more.
struct Join {
    const float* pre_o;     // [splits][batch * heads][dim]
    const float* pre_lse;   // [splits][batch * heads]
    float* lse_out;         // the caller's (nullptr: none)
    int splits, rows_a_unit;
};

__global__ void __launch_bounds__(256, 4) attn_join_kernel(Params p, Join x)
{
    // Where the parts are follows from the lengths alone, which are complete:
    // this kernel starts when the decode kernel's CTAs run, and those start, or
    // go on, when what came before them is.
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t rows = static_cast<int64_t>(p.batch) * p.heads;
    if (row >= rows)
        return;
    const int b = static_cast<int>(row / p.heads), h = static_cast<int>(row % p.heads);
    const int head = h / p.group, block = h % p.group / x.rows_a_unit, in_block = h % p.group % x.rows_a_unit;
    const int units = p.kv_heads * p.row_blocks, tiles = tiles_of(p, own_keys(p, b));
    // the pieces that have this row's tiles
    int first_slot = 0, own_parts = 0;
    bool whole = false;
    if (tiles > 0) {
        const Cut cut(p, sum_tiles(p, p.batch) * units);
        const int t0 = sum_tiles(p, b) * units + (head * p.row_blocks + block) * line_of(tiles) + kRowCost;
        const int c0 = cut.piece_of(t0), c1 = cut.piece_of(t0 + tiles - 1);
        whole = c0 == c1;
        if (whole && x.splits == 0) {  // the output is there
            grid_dependency_wait();
            return;
        }
        own_parts = c1 - c0 + 1;
        first_slot = 2 * c0 + (cut.begin(c0) < t0 - kRowCost ? 1 : 0);  // that piece begins with another row
    }
    const int parts = x.splits + own_parts;
    if (kJoinEarly)
        grid_dependency_launch();
    grid_dependency_wait();
    // part i: its lse and where its sums are; slots first_slot, then 2 (c0 + 1), 2 (c0 + 2), ...
    auto find = [&](int i, const float*& o) {
        if (i < x.splits) {
            o = x.pre_o + (static_cast<int64_t>(i) * rows + row) * p.dim;
            return x.pre_lse[static_cast<int64_t>(i) * rows + row];
        }
        if (whole)  // its sums are read below
            return p.lse[row];
        const int64_t slot = i == x.splits ? first_slot : 2 * (first_slot / 2 + i - x.splits);
        o = p.part_o + (slot * x.rows_a_unit + in_block) * p.dim;
        return p.part_lse[slot * x.rows_a_unit + in_block];
    };
    float top = -INFINITY, acc[4] = {}, sum = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += 32) {  // a lane has one part's lse, all lanes share the sums
        const float* mine = nullptr;
        const float y = i0 + lane < parts ? find(i0 + lane, mine) : -INFINITY;
        float t = y;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        t = fmaxf(top, t);
        const float shift = t == -INFINITY ? 0.0f : t, a = expf(top - shift);
        top = t;
        float w = expf(y - shift);  // a part that sees nothing weighs nothing; NaN stays NaN
        float s = w;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        sum = fmaf(sum, a, s);
        w *= kJoinWeight;
        float run[4] = {};  // of these 32: see kRun
        // the caller's out, the last part of a whole row, may lie at any address
        const bool from_out = whole && i0 + 32 >= parts;
        const int n = min(32, parts - i0) - from_out;
#pragma unroll 16
        for (int i = 0; i < n; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const float* const o = reinterpret_cast<const float*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), i));
            if (lane * 4 < p.dim) {
                const float4 v = *reinterpret_cast<const float4*>(o + lane * 4);
                // where nothing was seen the sums are 0
                run[0] = fmaf(v.x, wi, run[0]);
                run[1] = fmaf(v.y, wi, run[1]);
                run[2] = fmaf(v.z, wi, run[2]);
                run[3] = fmaf(v.w, wi, run[3]);
            }
        }
        if (from_out) {
            const float wi = __shfl_sync(0xffffffffu, w, n);
            const float* const o = p.out + row * p.dim + lane * 4;
            if (lane * 4 < p.dim) {
                const float4 v =
                    p.vec_out ? *reinterpret_cast<const float4*>(o) : make_float4(o[0], o[1], o[2], o[3]);
                run[0] = fmaf(v.x, wi, run[0]);
                run[1] = fmaf(v.y, wi, run[1]);
                run[2] = fmaf(v.z, wi, run[2]);
                run[3] = fmaf(v.w, wi, run[3]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] = fmaf(acc[e], a, run[e]);
    }
    const float norm = sum == 0.0f ? 0.0f : 1.0f / kJoinWeight / sum;
    if (lane * 4 < p.dim) {
        float* const dst = p.out + row * p.dim + lane * 4;
        if (p.vec_out) {
            *reinterpret_cast<float4*>(dst) =
                make_float4(acc[0] * norm, acc[1] * norm, acc[2] * norm, acc[3] * norm);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dst[e] = acc[e] * norm;
        }
    }
    if (x.lse_out && lane == 0)
        x.lse_out[row] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

// Blocks of eight query heads that a warp takes at once, and how often a
// key/value head's keys are gone through.
inline int blocks_at_once(int group)
{
    return group > 8 ? 2 : 1;
}

inline int row_blocks(int group)
{
    return (group + 8 * blocks_at_once(group) - 1) / (8 * blocks_at_once(group));
}

}  // namespace
}  // namespace compfp32
