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

namespace compfp32 {
namespace {
constexpr int kTileShift = 4;
constexpr int kTile = 1 << kTileShift;  // keys of a tile, the k of a product
constexpr int kLeastKeys = 64;
constexpr int kRowCost = 0;
constexpr bool kJoinEarly = true;
constexpr float kJoinWeight = 1.0f;
}
}  // namespace compfp32

#include "attn_line.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

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

bool attn_decode_countable(int kv_heads, int page_size, int64_t batch, int heads, int64_t width, int per_row)
{
    const int64_t units = static_cast<int64_t>(kv_heads) * row_blocks(heads / kv_heads);
    return (width * page_size / kTile + per_row) * batch <= INT32_MAX / units;
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
