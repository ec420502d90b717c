// Attention of single tokens over a paged FP16 cache: each key and value of a
// sequence is read once for up to 16 query heads that share it (once more for each
// further 16), 4 D bytes for 4 D operations a head, so the bound is HBM.
//
// Tensor cores.  The m16n8k16 product has room for 16 rows; up to eight query
// heads of a key/value head come in twice, rows 0..7 hi = fp16(x) and rows
// 8..15 lo.  One product so does both halves of the compensated form, and a
// thread finds a row's hi sum and lo sum side by side in its own registers:
//   s = S_hi + 2^-10 S_lo        with q split as in the projections;
//   O' = O'_hi + O'_lo           with 2^14 p split into hi and lo (no scale on
//                                lo: see the packed kernel).
// O' of a tile is added to o = o 2^(m_old - m_new) + O' in FP32 registers, as
// in the packed kernel.  Memory, not these products, is the bound here, so the
// older warp-wide instructions serve: tcgen05's 128 rows would be empty.
//
// Work.  The tiles of all (sequence, key/value head) rows stand in one line
// that is cut into equal pieces, one for each warp: the lengths may differ as
// they like and no warp waits for the longest, nor for any other.  A warp
// goes through its piece row by row; a row that lies wholly in one piece is
// written to the output, the parts of a row that was cut go to the workspace
// and are joined by a second launch, in order, as are the parts of a shared
// prefix (computed for the whole batch by the packed kernel).  A warp loads
// its own tiles of 16 keys (TMA, a ring of stages).  An earlier form, four
// warps sharing tiles of 64 keys of a row and joining at its end, spent more
// on the joins than on the tiles where rows are short.
#include <cuda_fp16.h>

#include <cmath>

#include "attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kTile = 16;       // keys of a tile, the k of a product
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kLeast = 4;
constexpr int kLong = 8;
// Tiles that are added up before they are added to the sums so far: equal terms
// (identical, zero or padding keys) all round the same way, so that a running sum
// of every tile is off by 5e-5 after 65536 keys; with runs of 64 tiles, by 1e-6.
// The sums of the runs before lie in the warp's slot of the workspace, which it
// writes only later: 24 sequences of 8000 tokens, 64 heads over 4 of 128, take 77 us,
// 74 without runs, 113 with those sums in registers and 123 with them in shared
// memory, which leaves an SM one CTA.
constexpr int kRun = 64;
constexpr uint32_t kFaultDecode = 0xA01;

// DP: head dimension padded to 64 or 128; NB: blocks of eight query heads.
template <int DP, int NB>
struct Cfg {
    static constexpr int kBoxes = DP / 64;
    static constexpr uint32_t kPlane = kTile * DP * 2;
    static constexpr uint32_t kStage = 2 * kPlane;          // k, v
    static constexpr int NS = DP == 128 ? 3 : 6;            // 24 KB a warp
    static constexpr size_t kSmem = 1024 + kWarps * NS * kStage;
};

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
};

// Keys of a sequence beyond the shared pages, and their tiles.
__device__ __forceinline__ int own_keys(const Params& p, int b)
{
    const int n = p.lengths[b];
    return max(0, min(n, p.most_keys) - p.shared_keys);
}

__device__ __forceinline__ int tiles_of(int own)
{
    return (own + kTile - 1) / kTile;
}

// Sum of the tiles of the sequences before `end` by one warp.
__device__ __forceinline__ int sum_tiles(const Params& p, int end)
{
    int n = 0;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < end; b += 32)
        n += tiles_of(own_keys(p, b));
    return __reduce_add_sync(0xffffffffu, n);
}

// The line of tiles: sequence by sequence, within one head unit by head unit
// (a key/value head and a block of its query heads), cut into pieces that
// differ by at most one tile: the first `rest` have one more.  A piece has about
// kLeast tiles at least: a part of a row costs its join more than a tile costs.
// There are `waves` times as many pieces where they have kLong tiles then.
struct Cut {
    int pieces, each, rest;
    __device__ __forceinline__ Cut(const Params& p, int total)
        : pieces(min((total + kLeast - 1) / kLeast,
                     total / p.waves >= kLong * p.pieces ? p.waves * p.pieces : p.pieces)),
          each(pieces > 0 ? total / pieces : 0),
          rest(pieces > 0 ? total % pieces : 0)
    {
    }
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
    r.tiles = tiles_of(r.own);
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
        mine += tiles_of(own_keys(p, b));
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
            if (at < r.tiles * units)
                break;
            at -= r.tiles * units;
        }
        r.unit = at / r.tiles;
        r.tile = at % r.tiles;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    r.b = __shfl_sync(0xffffffffu, r.b, src);
    r.unit = __shfl_sync(0xffffffffu, r.unit, src);
    r.tile = __shfl_sync(0xffffffffu, r.tile, src);
    r.own = __shfl_sync(0xffffffffu, r.own, src);
    r.tiles = __shfl_sync(0xffffffffu, r.tiles, src);
    return true;
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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

template <int DP, int NB>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const Params p)
{
    using C = Cfg<DP, NB>;
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_of[kWarps][NS];
    __shared__ int abort_flag[kWarps];
    __shared__ float2 l_far_of[kWarps][NB][32];
    __shared__ float m_far_of[kWarps][NB][32];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* const stages =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
        warp * (NS * C::kStage);
    uint64_t* const full = full_of[warp];
    if (lane == 0) {
        for (int i = 0; i < NS; ++i)
            mbar_init(&full[i], 1);
        abort_flag[warp] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    // After a prefix's kernel this one need not wait for it, only for what came
    // before, which that kernel has waited for before it let this one start: the
    // SMs it leaves free, and those it is done with, work here meanwhile.  What
    // follows this kernel follows both, so its first CTA waits at its end.
    if (!p.after_prefix)
        grid_dependency_wait();
    grid_dependency_launch();  // the join relies on what came before

    // this warp's piece; consecutive ones are on different SMs
    const int ctas = p.pieces / kWarps, wave = static_cast<int>(blockIdx.x) >= ctas;
    const int piece = wave * (p.pieces - ctas) + warp * ctas + blockIdx.x;
    int begin, end;
    Place r;
    if (!find_piece(p, piece, begin, end, r)) {
        if (blockIdx.x == 0)
            grid_dependency_wait();
        return;
    }

    // Rows.  The query heads split: rows 0..7 of a block hi, 8..15 lo.
    const int g = lane >> 2, quad = lane & 3;
    const float c2 = p.scale * kAttnLog2E;
    bool ok = true;
    int i = 0, fragment = 0;
    float2 raw[NB][DP / 16][2];
    auto load_q = [&](const Place& at) {
        const int head = at.unit / p.row_blocks, first_head = at.unit % p.row_blocks * (NB * 8);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int hg = first_head + nb * 8 + g;
            const float* const src = p.q + at.b * p.q_token + (head * p.group + hg) * p.q_head;
            const bool there = hg < p.group && at.b < p.batch;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = k * 16 + e * 8 + quad * 2;  // the head dimension is a multiple of 8
                    float2 x = make_float2(0.0f, 0.0f);
                    if (there && d < p.dim) {
                        if (p.vec_q) {
                            x = __ldg(reinterpret_cast<const float2*>(src + d));
                        } else {
                            x.x = __ldg(src + d);
                            x.y = __ldg(src + d + 1);
                        }
                    }
                    raw[nb][k][e] = x;
                }
        }
    };
    // Loads run NS tiles ahead: lanes 0 .. 2 kBoxes - 1 have a box of each.  The
    // lanes hold the page numbers of 32 tiles of a row, fetched when the row
    // is new; one that is not there: a place beyond the cache, which reads
    // zeros.
    Place next = r;
    const int box = lane % C::kBoxes, is_v = lane / C::kBoxes;
    const bool mine = is_v < 2;
    const uint32_t to = is_v * C::kPlane + box * (kTile * 128);
    const CUtensorMap* const map = is_v ? &map_v : &map_k;
    int pages = 0, page_tile = 0, loads = 0;
    auto look_up = [&] {
        page_tile = next.tile;
        const int col = (p.shared_keys + (next.tile + lane) * kTile) >> p.page_shift;
        pages = next.tile + lane < next.tiles && col < p.width ? p.table[next.b * p.width + col] : -1;
    };
    auto load = [&] {
        const int s = loads % NS, at = __shfl_sync(0xffffffffu, pages, next.tile - page_tile);
        const int slot = (p.shared_keys + next.tile * kTile) & ((1 << p.page_shift) - 1);
        if (lane == 0)
            mbar_arrive_expect_tx(&full[s], C::kStage);
        __syncwarp();
        if (mine)
            tma_load_3d(stages + s * C::kStage + to, map, &full[s], box * 64, slot,
                        (at >= 0 && at < p.pages ? at : p.pages) * p.kv_heads + next.unit / p.row_blocks);
        if (begin + ++loads < end) {
            if (++next.tile == next.tiles) {
                next_row(p, next);
                look_up();
            } else if (next.tile == page_tile + 32) {
                look_up();
            }
        }
    };
    look_up();
    load_q(r);
    for (int i = 0; i < NS && begin + i < end; ++i)
        load();

    for (int at = begin; ok && at < end; ++fragment) {
        const int n = min(r.tiles - r.tile, end - at);
        const int head = r.unit / p.row_blocks, first_head = r.unit % p.row_blocks * (NB * 8);
        uint32_t q[NB][DP / 16][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split2(raw[nb][k][e].x, raw[nb][k][e].y, q[nb][k][2 * e], q[nb][k][2 * e + 1]);
        Place after = r;
        if (at + n < end) {
            next_row(p, after);
            if (NB == 1)  // with two blocks the registers do not suffice
                load_q(after);
        }
        // the running maximum and the sums of a run; slot, l_far_of, m_far_of: of the runs before
        float m[NB];
        uint64_t l2[NB], o[NB][DP / 8];
        const int part = 2 * piece + (fragment > 0 ? 1 : 0);
        float* const slot = p.part_o + (static_cast<int64_t>(part) * (NB * 8) + g) * p.dim + quad * 2;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb] = -INFINITY;
            l2[nb] = 0;
#pragma unroll
            for (int t = 0; t < DP / 8; ++t)
                o[nb][t] = 0;
        }
        for (int t0 = 0; ok && t0 < n; t0 += kRun) {
            const int t1 = min(n, t0 + kRun);
            for (int t = t0; t < t1; ++t, ++i) {
                const int s = i % NS;
                if (!attn_warp_wait(&full[s], (i / NS) & 1, &abort_flag[warp], kFaultDecode)) {
                    ok = false;
                    break;
                }
                uint8_t* const kt = stages + s * C::kStage;
                uint8_t* const vt = kt + C::kPlane;
                const int left = r.own - (r.tile + t) * kTile;  // keys of the tile that count
                if (left < kTile) {
                    // beyond the sequence's end v may hold anything: 0 times that must be 0
#pragma unroll
                    for (int x = 0; x < C::kBoxes; ++x)
                        for (int u = lane; u < kTile * 8; u += 32)
                            if (u / 8 >= left)
                                *reinterpret_cast<uint4*>(vt + x * (kTile * 128) + u * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();  // before the next load into this stage
                    __syncwarp();
                }
                // two chains for each eight keys, the even and the odd steps of the head dimension
                float c[NB][2][2][4] = {};
#pragma unroll
                for (int k = 0; k < DP / 16; k += 2)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        uint32_t b[4];
                        ldmatrix4(smem_u32(kt) + (k / 4) * (kTile * 128) +
                                      sw128(nt * 8 + (lane & 7), (k % 4) * 2 + (lane >> 3)),
                                  b);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            mma16816(c[nb][nt][0], q[nb][k], b[0], b[1]);
                            mma16816(c[nb][nt][1], q[nb][k + 1], b[2], b[3]);
                        }
                    }
                uint32_t pa[NB][4];
                uint64_t a2[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int nt = e >> 1, col = e & 1, key = nt * 8 + quad * 2 + col;
                        x[e] = fmaf(c[nb][nt][0][2 + col] + c[nb][nt][1][2 + col], 0x1p-10f,
                                    c[nb][nt][0][col] + c[nb][nt][1][col]);
                        x[e] = key < left ? x[e] : -INFINITY;
                    }
                    float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c2;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float m_new = fmaxf(m[nb], top), shift = m_new == -INFINITY ? 0.0f : m_new;
                    const float alpha = ex2(m[nb] - shift);
                    m[nb] = m_new;
                    a2[nb] = f2_bits(alpha, alpha);
                    // 2^14 p; the product rounded as the maximum is, or large scores would not
                    // end at 0 (see the packed kernel; a branch for them instead took 72 us
                    // where this takes 68: 16 sequences of 16000 tokens, 40 heads over 1 of 128)
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = ex2(__fadd_rn(__fsub_rn(__fmul_rn(x[e], c2), shift), 14.0f));
                    split_p(w[0], w[1], pa[nb][0], pa[nb][1]);
                    split_p(w[2], w[3], pa[nb][2], pa[nb][3]);
                    l2[nb] = fma2(l2[nb], a2[nb], add2(f2_bits(w[0], w[1]), f2_bits(w[2], w[3])));
                }
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    uint32_t b[4];
                    ldmatrix4_trans(
                        smem_u32(vt) + (d / 4) * (kTile * 128) + sw128(lane & 15, (d % 4) * 2 + (lane >> 4)), b);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y[4] = {};
                            mma16816(y, pa[nb], b[2 * e], b[2 * e + 1]);
                            const uint64_t both = add2(f2_bits(y[0], y[1]), f2_bits(y[2], y[3]));
                            o[nb][2 * d + e] = fma2(o[nb][2 * d + e], a2[nb], both);
                        }
                }
                __syncwarp();  // all lanes have read the stage
                if (begin + loads < end)
                    load();
            }
            if (t0 > 0) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float a = ex2(m_far_of[warp][nb][lane] - (m[nb] == -INFINITY ? 0.0f : m[nb]));
                    const uint64_t a2 = f2_bits(a, a);
                    const float2 l = l_far_of[warp][nb][lane];
                    l2[nb] = fma2(f2_bits(l.x, l.y), a2, l2[nb]);
#pragma unroll
                    for (int x = 0; x < DP / 8; ++x)
                        if (x * 8 < p.dim)
                            o[nb][x] = fma2(*reinterpret_cast<const uint64_t*>(slot + nb * 8 * p.dim + x * 8), a2,
                                            o[nb][x]);
                }
            }
            if (t1 < n) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    m_far_of[warp][nb][lane] = m[nb];
                    l_far_of[warp][nb][lane] = make_float2(lo_f(l2[nb]), hi_f(l2[nb]));
                    l2[nb] = 0;
#pragma unroll
                    for (int x = 0; x < DP / 8; ++x) {
                        if (x * 8 < p.dim)
                            *reinterpret_cast<uint64_t*>(slot + nb * 8 * p.dim + x * 8) = o[nb][x];
                        o[nb][x] = 0;
                    }
                }
            }
        }

        // the row, or this warp's part of it
        if (ok) {
            const bool whole = n == r.tiles;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float sum = lo_f(l2[nb]) + hi_f(l2[nb]);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int row = nb * 8 + g, hg = first_head + row;
                if (hg >= p.group)
                    continue;
                const int64_t at_row = static_cast<int64_t>(r.b) * p.heads + head * p.group + hg;
                float* const dst = whole ? p.out + at_row * p.dim
                                         : p.part_o + (static_cast<int64_t>(part) * (NB * 8) + row) * p.dim;
                const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (p.vec_out || !whole) {
#pragma unroll
                    for (int t = 0; t < DP / 8; ++t)
                        if (t * 8 < p.dim)
                            *reinterpret_cast<float2*>(dst + t * 8 + quad * 2) =
                                make_float2(lo_f(o[nb][t]) * norm, hi_f(o[nb][t]) * norm);
                } else {
#pragma unroll
                    for (int t = 0; t < DP / 8; ++t)
                        if (t * 8 < p.dim) {
                            dst[t * 8 + quad * 2] = lo_f(o[nb][t]) * norm;
                            dst[t * 8 + quad * 2 + 1] = hi_f(o[nb][t]) * norm;
                        }
                }
                if (quad == 0) {
                    const float lse =
                        sum == 0.0f ? -INFINITY : fmaf(m[nb], kAttnLn2, logf(sum * (1.0f / kAttnPScale)));
                    if (!whole)
                        p.part_lse[part * (NB * 8) + row] = lse;
                    else if (p.lse)
                        p.lse[at_row] = lse;
                }
            }
        }
        at += n;
        r = after;
        if (NB > 1 && at < end)
            load_q(r);
    }
    if (!ok)  // what was issued lands before the warp leaves
        for (int j = i; j < loads; ++j)
            attn_drain_wait(&full[j % NS], (j / NS) & 1);
    if (blockIdx.x == 0)
        grid_dependency_wait();
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
    const int units = p.kv_heads * p.row_blocks, tiles = tiles_of(own_keys(p, b));
    // the pieces that have this row's tiles
    int first_slot = 0, own_parts = 0;
    bool whole = false;
    if (tiles > 0) {
        const Cut cut(p, sum_tiles(p, p.batch) * units);
        const int t0 = sum_tiles(p, b) * units + (head * p.row_blocks + block) * tiles;
        const int c0 = cut.piece_of(t0), c1 = cut.piece_of(t0 + tiles - 1);
        whole = c0 == c1;
        if (whole && x.splits == 0) {  // the output is there
            grid_dependency_wait();
            return;
        }
        own_parts = c1 - c0 + 1;
        first_slot = 2 * c0 + (cut.begin(c0) < t0 ? 1 : 0);  // that piece begins with another row
    }
    const int parts = x.splits + own_parts;
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
        const float w = expf(y - shift);  // a part that sees nothing weighs nothing; NaN stays NaN
        float s = w;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        sum = fmaf(sum, a, s);
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
    const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;
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

template <int DP, int NB>
comp_status_t launch_t(const CUtensorMap& mk, const CUtensorMap& mv, const Params& p, const DeviceInfo& dev,
                       cudaStream_t stream)
{
    using C = Cfg<DP, NB>;
    static std::mutex mu;
    static bool done[64] = {};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev.device < 0 || dev.device >= 64)
            return COMP_ERR_CUDA;
        if (!done[dev.device]) {
            if (cudaFuncSetAttribute(attn_decode_kernel<DP, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(C::kSmem)) != cudaSuccess) {
                (void)cudaGetLastError();
                return COMP_ERR_CUDA;
            }
            done[dev.device] = true;
        }
    }
    return launch_pdl(attn_decode_kernel<DP, NB>, p.waves * p.pieces / kWarps, kThreads, C::kSmem, stream, mk, mv, p);
}

// Pieces of the line of tiles: one for each warp of two CTAs an SM.  The
// workspace's size must not depend on the device, so their number is bounded.
constexpr int kMostPieces = 320 * kWarps;
// Beside a prefix's kernel the CTAs start as SMs become free, and pieces half as
// long fill its end better, where they are still long enough: 256 sequences on a
// 32768-token prefix take 211 us instead of 230, 64 short ones on 8192 tokens 34.0
// instead of 34.3.  Without a prefix all pieces start together, and
// two waves of them cost 77 us where one takes 69 (48 ragged sequences).
constexpr int kPrefixWaves = 2;  // the kernel tells the second by one comparison

// How the shared pages' keys are split: into parts of at least kLeastTiles tiles of
// 128 keys, so that about one wave of the packed kernel's CTAs works on them (at
// least four tiles: 24.9 us instead of 21.1 for 8 sequences on 512 tokens).
// Where tiles are left then for twice as many parts, and a CTA has rows for one
// half only, each half takes a part of its own (64 sequences on 8192 tokens, 16
// heads of 64: 37.8 -> 34.0 us).  Heads wider than 64 gain nothing: their ring
// holds three tiles, too few for two halves apart (45.8 us against 44.7 with
// 16 rows on 16384 tokens).
constexpr int kLeastTiles = 2;

constexpr int kMostSms = 160;

struct Split {
    int parts;
    bool fold;
};

Split prefix_split(const comp_kv_cache_t& c, int64_t shared, int64_t batch, int heads, int sms, bool bound = false)
{
    const int64_t tiles = (shared * c.page_size + 127) / 128, rows = batch * (heads / c.kv_heads);
    const int64_t wave = sms / ((rows + 255) / 256 * c.kv_heads), most = tiles / kLeastTiles;
    const bool two = rows <= 128 && c.head_dim <= 64;
    const bool fold = two && wave > 0 && 2 * wave <= most;
    // the bound: what no smaller number of SMs exceeds
    int64_t n = fold || (bound && two) ? 2 * wave : wave;
    n = n < most ? n : most;
    n = n < 1 ? 1 : n;
    if (!bound && tiles > 0) {  // no part without tiles (folded: one at most)
        const int64_t each = (tiles + n - 1) / n;
        n = (tiles + each - 1) / each;
        n += fold ? n % 2 : 0;
    }
    return {static_cast<int>(n), fold};
}

// Blocks of eight query heads that a warp takes at once, and how often a
// key/value head's keys are gone through.
int blocks_at_once(int group)
{
    return group > 8 ? 2 : 1;
}

int row_blocks(int group)
{
    return (group + 8 * blocks_at_once(group) - 1) / (8 * blocks_at_once(group));
}

// Floats of the workspace: parts of rows, the prefix's parts, the rows' lse.
struct Layout {
    int64_t part_o, part_lse, pre_o, pre_lse, lse, total;
};

Layout layout_of(const comp_kv_cache_t& c, int64_t batch, int heads, int splits)
{
    const int group = heads / c.kv_heads;
    const int64_t pieces = splits > 0 ? kPrefixWaves * kMostPieces : kMostPieces;
    const int64_t slots = 2 * pieces * 8 * blocks_at_once(group), rows = batch * heads;
    Layout l;
    l.part_o = 0;
    l.part_lse = l.part_o + slots * c.head_dim;
    l.lse = l.part_lse + slots;
    l.pre_lse = l.lse + (rows + 3) / 4 * 4;
    l.pre_o = l.pre_lse + (splits * rows + 3) / 4 * 4;
    l.total = l.pre_o + splits * rows * c.head_dim;
    return l;
}

// Sharing pays from two sequences on.
int64_t effective_shared(int64_t batch, int64_t shared_pages)
{
    return batch > 1 ? shared_pages : 0;
}

}  // namespace

bool attn_decode_countable(const comp_kv_cache_t& cache, int64_t batch, int heads, int64_t width)
{
    const int64_t units = static_cast<int64_t>(cache.kv_heads) * row_blocks(heads / cache.kv_heads);
    return (width * cache.page_size / kTile + 1) * batch <= INT32_MAX / units;
}

int64_t attn_decode_bytes(const comp_kv_cache_t& cache, int64_t batch, int heads, int64_t shared_pages)
{
    const int64_t shared = effective_shared(batch, shared_pages);
    const int parts = shared > 0 ? prefix_split(cache, shared, batch, heads, kMostSms, true).parts : 0;
    return 4 * layout_of(cache, batch, heads, parts).total;
}

comp_status_t launch_attn_decode(const comp_kv_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                 int heads, float scale, const int32_t* table, int64_t batch, int64_t width,
                                 const int32_t* lengths, int64_t shared_pages, float* out, float* lse,
                                 void* workspace, const DeviceInfo& dev, cudaStream_t stream)
{
    const int64_t shared = effective_shared(batch, shared_pages);
    const int group = heads / cache.kv_heads;
    const Split split = shared > 0 ? prefix_split(cache, shared, batch, heads,
                                                  dev.sm_count < kMostSms ? dev.sm_count : kMostSms)
                                   : Split{0, false};
    const int splits = split.parts;
    const Layout at = layout_of(cache, batch, heads, splits);
    float* const ws = static_cast<float*>(workspace);
    if (splits > 0) {
        const comp_status_t st = launch_attn_prefix(cache, q, q_token, q_head, heads, scale, table, batch, lengths,
                                                    shared, splits, split.fold, ws + at.pre_o, ws + at.pre_lse, dev,
                                                    stream);
        if (st != COMP_OK)
            return st;
    }
    const int nb = blocks_at_once(group);
    Params p{};
    p.q = q;
    p.out = out;
    p.lse = splits > 0 ? ws + at.lse : lse;
    p.part_o = ws + at.part_o;
    p.part_lse = ws + at.part_lse;
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
    p.shared_keys = static_cast<int>(shared * cache.page_size);
    p.most_keys = static_cast<int>(width * cache.page_size);
    p.pieces = 2 * dev.sm_count * kWarps < kMostPieces ? 2 * dev.sm_count * kWarps : kMostPieces;
    p.waves = splits > 0 ? kPrefixWaves : 1;
    p.vec_q = (reinterpret_cast<uintptr_t>(q) & 7u) == 0 && q_token % 2 == 0 && q_head % 2 == 0;
    p.vec_out = aligned16(out);  // rows are multiples of 32 bytes
    p.scale = scale;
    p.after_prefix = splits > 0;
    CUtensorMap mk{}, mv{};
    if (width > 0) {  // otherwise there are no tiles
        if (!encode_pages(&mk, cache.k, cache, kTile) || !encode_pages(&mv, cache.v, cache, kTile))
            return COMP_ERR_CUDA;
    }
    comp_status_t st;
    if (cache.head_dim <= 64)
        st = nb == 1 ? launch_t<64, 1>(mk, mv, p, dev, stream) : launch_t<64, 2>(mk, mv, p, dev, stream);
    else
        st = nb == 1 ? launch_t<128, 1>(mk, mv, p, dev, stream) : launch_t<128, 2>(mk, mv, p, dev, stream);
    if (st != COMP_OK)
        return st;
    const Join x{ws + at.pre_o, ws + at.pre_lse, lse, splits, 8 * nb};
    return launch_pdl(attn_join_kernel, static_cast<int>((batch * heads + 7) / 8), 256, 0, stream, p, x);
}

comp_status_t read_and_clear_decode_fault(cudaStream_t stream, uint32_t* where)
{
    return read_and_clear_word(&g_attn_fault_word, stream, where);
}

}  // namespace compfp32
