// Attention of single tokens over a paged cache in 8 bits, with a scale for each
// 16 tokens of a head: 2 D bytes for 4 D operations a key and query head, so the
// bound is HBM, at half the FP16 cache's bytes.
//
// Arithmetic.  Codes are whole numbers up to 127, exact in FP16, so the products
// are those of the FP16 decode kernel over the codes, a block's scale applied
// once to what its 16 keys gave:
//   s = (S_hi + 2^-10 S_lo) (scale kscale)     q split into hi and lo;
//   o = o 2^(m_old - m_new) + vscale (O'_hi + O'_lo)   2^14 p split into hi and lo.
// A tile is a block, 16 keys, and its products are added up in FP32 registers.
//
// Layout.  The sum over the head dimension may go in any order, and so may the
// columns of the output: a lane's operands are 16 codes that stand side by side in
// a row, whole 16-byte words of memory.  So a lane copies with cp.async just the
// words that it will use itself, to places of its own in a ring of stages: no
// registers wait for memory, shared memory has no conflicts, and the only
// synchronisation is each lane's wait for its own copies (and one of the warp for
// the two scales).  Codes become FP16 two at a time, 1024 + 128 + code by a
// bitwise operation and one subtraction.
//
// Work is cut and joined as in the FP16 kernel (attn_line.cuh).
#include <cuda_fp16.h>

#include <cmath>

#include "attn.h"
#include "attn_line.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

static_assert(kTile == COMP_KV8_BLOCK, "a tile has one scale");

constexpr int kRun8 = 64;  // tiles that are added up before they are added to the sums so far, as in the FP16 kernel

// DP: head dimension padded to 64 or 128; NB: blocks of eight query heads.
template <int DP, int NB>
struct Cfg {
    static constexpr int kWords = DP / 64;                  // 16-byte words of a key that a lane has
    static constexpr uint32_t kPlane = kTile * DP;
    static constexpr uint32_t kStage = 2 * kPlane + 16;     // k, v, the two scales
    static constexpr int NS = DP == 128 ? 4 : 7;
    static constexpr int kCtas = NB == 1 ? 3 : 2;           // an SM
    static constexpr size_t kSmem = kWarps * NS * kStage;
};

struct Cache8 {
    const int8_t* k;
    const int8_t* v;
    const float* k_scale;
    const float* v_scale;
    comp_rope_t rope;
};

// Copies 16 or 8 bytes, or zeros where `there` is false (src is then any address).
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy8_async(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}

__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

__device__ __forceinline__ void copies_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bytes 0 and 2 of w, two codes, as FP16: 0x6400 + u is 1024 + u, u = code + 128.
__device__ __forceinline__ uint32_t even_codes(uint32_t w)
{
    const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u;
    return pack_h2(__hsub2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(1152.0f, 1152.0f)));
}

__device__ __forceinline__ uint32_t odd_codes(uint32_t w)
{
    return even_codes(w >> 8);
}

// NaN in the place of a code of -128.
__device__ __forceinline__ uint32_t odd_to_nan(uint32_t h2)
{
    const uint32_t odd = 0xd800d800u;  // -128
    return h2 | __heq2_mask(*reinterpret_cast<const __half2*>(&h2), *reinterpret_cast<const __half2*>(&odd));
}

__device__ __forceinline__ bool has_odd(uint32_t w)
{
    return __vcmpeq4(w, 0x80808080u) != 0;
}

template <int DP, int NB>
__global__ void __launch_bounds__(kThreads, Cfg<DP, NB>::kCtas)
    attn_decode8_kernel(const Params p, const Cache8 c)
{
    using C = Cfg<DP, NB>;
    constexpr int NS = C::NS, W = C::kWords;
    extern __shared__ __align__(16) uint8_t stages_of[];
    __shared__ float2 l_far_of[kWarps][NB][32];
    __shared__ float m_far_of[kWarps][NB][32];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* const stages = stages_of + warp * (NS * C::kStage);
    const uint32_t stages32 = smem_u32(stages);
    grid_dependency_wait();
    grid_dependency_launch();  // the join relies on what came before

    // this warp's piece; consecutive ones are on different SMs
    const int ctas = p.pieces / kWarps;
    const int piece = warp * ctas + blockIdx.x;
    int begin, end;
    Place r;
    if (!find_piece(p, piece, begin, end, r))
        return;

    // A lane has the codes of key g (and 8 + g) in the words quad + 4 j, and for the
    // values those of the keys 2 quad, 2 quad + 1 and 8 more, dimensions g DP/8 on.
    const int g = lane >> 2, quad = lane & 3;
    const float c2 = p.scale * kAttnLog2E;
    const int v_dim = g * (DP / 8);

    // Loads run NS - 1 tiles ahead.  The lanes hold the page numbers of 32 tiles of
    // a row, fetched when the row is new; one that is not there reads as zeros.
    Place next = r;
    int pages = 0, page_tile = 0, loads = 0;
    const int blocks_shift = p.page_shift - 4;
    auto look_up = [&] {
        page_tile = next.tile;
        const int col = ((next.tile + lane) * kTile) >> p.page_shift;
        pages = next.tile + lane < next.tiles && col < p.width ? p.table[next.b * p.width + col] : -1;
    };
    auto load = [&] {
        if (begin + loads < end) {
            const int at = __shfl_sync(0xffffffffu, pages, next.tile - page_tile);
            const bool there = at >= 0 && at < p.pages;
            const int slot = (next.tile * kTile) & ((1 << p.page_shift) - 1);
            const int64_t unit = (there ? at : 0) * static_cast<int64_t>(p.kv_heads) + next.unit / p.row_blocks;
            const int64_t from = ((unit << p.page_shift) + slot) * p.dim;
            const uint32_t to = stages32 + loads % NS * C::kStage;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int d = (quad + 4 * j) * 16;
                    const bool in = there && d < p.dim;
                    copy16_async(to + ((nt * W + j) * 32 + lane) * 16, c.k + from + (in ? (nt * 8 + g) * p.dim + d : 0),
                                 in);
                }
            const bool in = there && v_dim < p.dim;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = quad * 2 + (i & 1) + 8 * (i >> 1);
                const int8_t* const src = c.v + from + (in ? key * p.dim + v_dim : 0);
                if (DP == 128)
                    copy16_async(to + C::kPlane + (i * 32 + lane) * 16, src, in);
                else
                    copy8_async(to + C::kPlane + (i * 32 + lane) * 8, src, in);
            }
            if (lane < 2)
                copy4_async(to + 2 * C::kPlane + lane * 4,
                            (lane ? c.v_scale : c.k_scale) + (unit << blocks_shift) + (slot >> 4), there);
            if (begin + ++loads < end) {
                if (++next.tile == next.tiles) {
                    next_row(p, next);
                    look_up();
                } else if (next.tile == page_tile + 32) {
                    look_up();
                }
            }
        } else {
            ++loads;
        }
        copies_commit();
    };
    look_up();
    for (int i = 0; i < NS - 1; ++i)
        load();

    int i = 0, fragment = 0;
    for (int at = begin; at < end; ++fragment) {
        const int n = min(r.tiles - r.tile, end - at);
        const int head = r.unit / p.row_blocks, first_head = r.unit % p.row_blocks * (NB * 8);
        // The query heads, rotated and split: rows 0..7 of a block hi, 8..15 lo.  Step
        // 4 j + w of the head dimension takes word w of the lane's codes, whose four
        // stand in the order 0, 2, 1, 3.
        uint32_t q[NB][DP / 16][4];
        const float* const angles = c.rope.rot > 0 ? angles_of(c.rope, min(p.lengths[r.b], p.most_keys) - 1) : nullptr;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int hg = first_head + nb * 8 + g;
            const float* const src = p.q + r.b * p.q_token + (head * p.group + hg) * p.q_head;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int d = (quad + 4 * (k / 4)) * 16 + k % 4 * 4;
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (hg < p.group && d < p.dim)
                    x = load_rotated(src, d, c.rope, angles, p.vec_q != 0);
                split2(x.x, x.z, q[nb][k][0], q[nb][k][1]);
                split2(x.y, x.w, q[nb][k][2], q[nb][k][3]);
            }
        }
        // the running maximum and the sums of a run; slot, l_far_of, m_far_of: of the runs before
        float m[NB];
        uint64_t l2[NB], o[NB][DP / 8];
        const int part = 2 * piece + (fragment > 0 ? 1 : 0);
        // a lane's output: DP/8 dimensions from 2 quad DP/8 on, and the DP/8 after them
        const int o_dim = quad * (DP / 4);
        float* const slot = p.part_o + (static_cast<int64_t>(part) * (NB * 8) + g) * p.dim + o_dim;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb] = -INFINITY;
            l2[nb] = 0;
#pragma unroll
            for (int t = 0; t < DP / 8; ++t)
                o[nb][t] = 0;
        }
        for (int t0 = 0; t0 < n; t0 += kRun8) {
            const int t1 = min(n, t0 + kRun8);
            for (int t = t0; t < t1; ++t, ++i) {
                copies_wait<NS - 2>();
                __syncwarp();  // the scales; and all lanes have read the stage before
                load();
                const uint8_t* const stage = stages + i % NS * C::kStage;
                const float2 scales = *reinterpret_cast<const float2*>(stage + 2 * C::kPlane);
                const int left = r.own - (r.tile + t) * kTile;  // keys of the tile that count
                const float kc = fabsf(scales.x) * c2;
                // two chains for each eight keys, the even and the odd steps of the head dimension
                float s[NB][2][2][4] = {};
                unsigned odd_keys[2] = {0, 0};  // four bits a key
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    bool odd = false;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + ((nt * W + j) * 32 + lane) * 16);
                        const uint32_t word[4] = {x.x, x.y, x.z, x.w};
                        if (scales.x < 0.0f || __float_as_uint(scales.x) == 0x80000000u)
                            odd |= has_odd(x.x) || has_odd(x.y) || has_odd(x.z) || has_odd(x.w);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t b0 = even_codes(word[w]), b1 = odd_codes(word[w]);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma16816(s[nb][nt][w & 1], q[nb][j * 4 + w], b0, b1);
                        }
                    }
                    if (__float_as_int(scales.x) < 0)
                        odd_keys[nt] = __ballot_sync(0xffffffffu, odd);
                }
                uint32_t pa[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int nt = e >> 1, col = e & 1, key = quad * 2 + col;
                        x[e] = fmaf(s[nb][nt][0][2 + col] + s[nb][nt][1][2 + col], 0x1p-10f,
                                    s[nb][nt][0][col] + s[nb][nt][1][col]);
                        x[e] = __fmul_rn(x[e], kc);
                        if ((odd_keys[nt] >> (4 * key)) & 0xfu)
                            x[e] = __int_as_float(0x7fffffff);
                        x[e] = nt * 8 + key < left ? x[e] : -INFINITY;
                    }
                    float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float m_new = fmaxf(m[nb], top), shift = m_new == -INFINITY ? 0.0f : m_new;
                    if (__any_sync(0xffffffffu, m_new > m[nb])) {  // rare after some tiles
                        const float alpha = ex2(m[nb] - shift);
                        const uint64_t a2 = f2_bits(alpha, alpha);
                        l2[nb] = mul2(l2[nb], a2);
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d)
                            o[nb][d] = mul2(o[nb][d], a2);
                    }
                    m[nb] = m_new;
                    // 2^14 p; each step rounded as the maximum was, or large scores would not end at 0
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = ex2(__fadd_rn(__fsub_rn(x[e], shift), 14.0f));
                    split_p(w[0], w[1], pa[nb][0], pa[nb][1]);
                    split_p(w[2], w[3], pa[nb][2], pa[nb][3]);
                    l2[nb] = add2(l2[nb], add2(f2_bits(w[0], w[1]), f2_bits(w[2], w[3])));
                }
                // the values: four keys' codes of DP/8 dimensions
                constexpr int VW = DP / 32;
                uint32_t v[4][VW];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (DP == 128) {
                        const uint4 x =
                            *reinterpret_cast<const uint4*>(stage + C::kPlane + (k * 32 + lane) * 16);
                        v[k][0] = x.x;
                        v[k][1] = x.y;
                        v[k][VW - 2] = x.z;
                        v[k][VW - 1] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(stage + C::kPlane + (k * 32 + lane) * 8);
                        v[k][0] = x.x;
                        v[k][1] = x.y;
                    }
                }
                const bool odd_v = __float_as_int(scales.y) < 0;
                if (odd_v) {  // beyond the sequence's end 0 times a NaN must be 0
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (quad * 2 + (k & 1) + 8 * (k >> 1) >= left)
#pragma unroll
                            for (int w = 0; w < VW; ++w)
                                v[k][w] = 0;
                }
                const float vs = fabsf(scales.y);
                const uint64_t vs2 = f2_bits(vs, vs);
#pragma unroll
                for (int w = 0; w < VW; ++w)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // dimensions 4 w + 2 half and the next of two keys: bytes a0 a1 b0 b1
                        const uint32_t p01 = __byte_perm(v[0][w], v[1][w], half ? 0x7632 : 0x5410);
                        const uint32_t p23 = __byte_perm(v[2][w], v[3][w], half ? 0x7632 : 0x5410);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = 4 * w + 2 * half + e;
                            uint32_t b0 = e ? odd_codes(p01) : even_codes(p01);
                            uint32_t b1 = e ? odd_codes(p23) : even_codes(p23);
                            if (odd_v) {
                                b0 = odd_to_nan(b0);
                                b1 = odd_to_nan(b1);
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float y[4] = {};
                                mma16816(y, pa[nb], b0, b1);
                                o[nb][d] = fma2(f2_bits(y[0], y[1]), vs2,
                                                fma2(f2_bits(y[2], y[3]), vs2, o[nb][d]));
                            }
                        }
                    }
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
                        o[nb][x] = fma2(f2_bits(o_dim + x < p.dim ? slot[nb * 8 * p.dim + x] : 0.0f,
                                                o_dim + DP / 8 + x < p.dim ? slot[nb * 8 * p.dim + DP / 8 + x] : 0.0f),
                                        a2, o[nb][x]);
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
                        if (o_dim + x < p.dim)
                            slot[nb * 8 * p.dim + x] = lo_f(o[nb][x]);
                        if (o_dim + DP / 8 + x < p.dim)
                            slot[nb * 8 * p.dim + DP / 8 + x] = hi_f(o[nb][x]);
                        o[nb][x] = 0;
                    }
                }
            }
        }

        // the row, or this warp's part of it
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
            float* const dst = (whole ? p.out + at_row * p.dim
                                      : p.part_o + (static_cast<int64_t>(part) * (NB * 8) + row) * p.dim) +
                               o_dim;
            const float norm = sum == 0.0f ? 0.0f : 1.0f / sum;
            const bool vec = p.vec_out || !whole;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 0; d < DP / 8; d += 4) {
                    if (o_dim + e * (DP / 8) + d >= p.dim)
                        continue;
                    float y[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        y[x] = (e ? hi_f(o[nb][d + x]) : lo_f(o[nb][d + x])) * norm;
                    float* const to = dst + e * (DP / 8) + d;
                    if (vec) {
                        *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            to[x] = y[x];
                    }
                }
            if (quad == 0) {
                const float lse = sum == 0.0f ? -INFINITY : fmaf(m[nb], kAttnLn2, logf(sum * (1.0f / kAttnPScale)));
                if (!whole)
                    p.part_lse[part * (NB * 8) + row] = lse;
                else if (p.lse)
                    p.lse[at_row] = lse;
            }
        }
        at += n;
        if (at < end)
            next_row(p, r);
    }
    copies_wait<0>();
}

template <int DP, int NB>
comp_status_t launch_t(Params p, const Cache8& c, const DeviceInfo& dev, cudaStream_t stream)
{
    using C = Cfg<DP, NB>;
    static std::mutex mu;
    static bool done[64] = {};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev.device < 0 || dev.device >= 64)
            return COMP_ERR_CUDA;
        if (!done[dev.device]) {
            if (cudaFuncSetAttribute(attn_decode8_kernel<DP, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(C::kSmem)) != cudaSuccess) {
                (void)cudaGetLastError();
                return COMP_ERR_CUDA;
            }
            done[dev.device] = true;
        }
    }
    return launch_pdl(attn_decode8_kernel<DP, NB>, p.pieces / kWarps, kThreads, C::kSmem, stream, p, c);
}

// Pieces of the line of tiles: one for each warp that the SMs hold.  The
// workspace's size must not depend on the device, so their number is bounded.
constexpr int kMostSms = 160;

int ctas_an_sm(int nb)
{
    return nb == 1 ? Cfg<128, 1>::kCtas : Cfg<128, 2>::kCtas;
}

// Floats of the workspace: parts of rows, and their lse.
int64_t slots_of(int nb)
{
    return 2 * static_cast<int64_t>(ctas_an_sm(nb)) * kMostSms * kWarps * 8 * nb;
}

}  // namespace

int64_t attn_decode8_bytes(const comp_kv8_cache_t& cache, int heads)
{
    return 4 * slots_of(blocks_at_once(heads / cache.kv_heads)) * (cache.head_dim + 1);
}

comp_status_t launch_attn_decode8(const comp_kv8_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                  int heads, float scale, const int32_t* table, int64_t batch, int64_t width,
                                  const int32_t* lengths, const comp_rope_t* rope, float* out, float* lse,
                                  void* workspace, const DeviceInfo& dev, cudaStream_t stream)
{
    const int group = heads / cache.kv_heads, nb = blocks_at_once(group);
    float* const ws = static_cast<float*>(workspace);
    Params p{};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.part_o = ws;
    p.part_lse = ws + slots_of(nb) * cache.head_dim;
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
    p.pieces = (dev.sm_count < kMostSms ? dev.sm_count : kMostSms) * ctas_an_sm(nb) * kWarps;
    p.waves = 1;
    p.vec_q = aligned16(q) && q_token % 4 == 0 && q_head % 4 == 0;
    p.vec_out = aligned16(out);  // rows are multiples of 64 bytes
    p.scale = scale;
    const Cache8 c{cache.k, cache.v, cache.k_scale, cache.v_scale, rope ? *rope : comp_rope_t{}};
    comp_status_t st;
    if (cache.head_dim <= 64)
        st = nb == 1 ? launch_t<64, 1>(p, c, dev, stream) : launch_t<64, 2>(p, c, dev, stream);
    else
        st = nb == 1 ? launch_t<128, 1>(p, c, dev, stream) : launch_t<128, 2>(p, c, dev, stream);
    if (st != COMP_OK)
        return st;
    const Join x{nullptr, nullptr, lse, 0, 8 * nb};
    return launch_pdl(attn_join_kernel, static_cast<int>((batch * heads + 7) / 8), 256, 0, stream, p, x);
}

}  // namespace compfp32
