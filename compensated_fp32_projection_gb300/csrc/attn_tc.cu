// Attention on the fifth-generation tensor cores.
//
// A CTA computes up to 256 query rows of one key/value head, in two halves of
// 128 rows (the tensor cores' M); two CTAs may work as a pair on twice the
// rows (Cfg).  A row is a query token and one of the `group` query heads that
// share the key/value head, so that grouped heads share the loads and a tile
// of a causal prompt spans few tokens.  Keys and values pass once, in tiles of
// BN keys:
//
//   S  = q k^T        q is split as in the projections, hi = fp16(q) and
//                     lo = fp16((q - hi) 1024): the lo products first, into a
//                     fresh accumulator, then the hi products with that
//                     accumulator scaled by 2^-10 on input.  FP32 keys are
//                     split likewise: lo*hi, hi*lo, then hi*hi.
//   softmax           running maximum and sum of a row in one thread, in FP32
//                     and to base 2: p = 2^(s c - m), c = scale log2 e.
//   P                 to two FP16 values as well.  2^14 p, at most 16384, is
//                     split into hi = fp16(2^14 p) and lo = fp16(2^14 p - hi)
//                     with no further scale: values so small that lo falls
//                     among the subnormals lie 2^-24 and more below the
//                     row's largest, so the pair is exact to 2^-39 of it, and
//                     both halves add up in one accumulator.
//   O' = P v          of this tile alone, into a fresh accumulator; added in
//                     FP32 registers, o = o 2^(m_old - m_new) + O'.  The tensor
//                     cores' own sums so never run over more than BN keys, and
//                     rescaling costs the multiply of that addition.  One rounding
//                     a tile: 2^-24 at most for each BN keys, and that only where
//                     all of them go one way.
//
// Two products for FP16 keys and values, three for FP32 ones: the floor is
// 4 D operations for each visible pair and product, at the tensor cores' FP16
// rate.  One half's softmax runs while the tensor cores work for the other
// half.  S is overwritten in place by P (128 columns of 32 bits: hi and lo
// pairs), which the second product reads from tensor memory.  Measured: 16384
// causal tokens, 32 heads of 128 over 8 of FP16 keys, 2.26 ms, 1.94 PFLOP/s of
// products; 4096 FP32 tokens, 32 heads, 333 us, 1.24 PFLOP/s; 24 prompts of 23
// to 2011 tokens, 238 us, 1.04 PFLOP/s, where nearly half of a CTA's time passes
// before its first product and after its last.
//
// Warps: 0 loads tiles of k and v (TMA, a ring of stages), 1 and 2 issue the
// products of the two halves in turns, 3 sees to values that must not count
// (below), 4..7 and 8..11 own the rows of the two halves: thread =
// tensor-memory lane = row.
//
// Hidden keys: a score that its row may not see becomes -inf, whatever k held,
// so p = 0.  In the product with v a zero does not silence an infinity or a
// NaN.  Tiles that some row sees only in part are therefore looked through
// first: what is not finite there is set to zero in shared memory, and if a
// row of this CTA sees it, the rows that do add it afterwards, by hand.
#include <cuda_fp16.h>

#include <cmath>

#include "attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kThreads = 384;
// Registers a thread at launch, and after setmaxnreg: 128 x 56 + 256 x 224 is
// the launch's 384 x 168.  The row threads hold the D output sums of a row
// and 32 scores.  The build checks the 168.
constexpr int kCtrlRegs = 56;
constexpr int kRowRegs = 224;
static_assert(128 * kCtrlRegs + 256 * kRowRegs <= kThreads * 168, "register split");

// Fault codes of the waits.
constexpr uint32_t kFaultAttnLoad = 0x901;
constexpr uint32_t kFaultAttnMma = 0x902;
constexpr uint32_t kFaultAttnValues = 0x903;
constexpr uint32_t kFaultAttnRows = 0x904;
constexpr uint32_t kFaultAttnTmem = 0x905;

// DP: the head dimension padded to 64 or 128.  PL: planes of k and v, 1 (FP16)
// or 2 (FP32, split).  PAIR: two CTAs of a cluster work on the same keys, 512
// rows together: their products are issued as one (cta_group::2, M = 256), and
// each holds half of every tile, half the keys of k and half the head
// dimension of v.  FOLD: the two halves have the same 128 rows and each a part of
// the keys, for the few rows of a shared prefix: one half alone takes 3000 cycles
// a tile, most of them waiting for the step before, two halves 4100 for a tile
// of each.
template <int DP_, int PL_, bool PAIR_, bool FOLD_ = false>
struct Cfg {
    static constexpr int DP = DP_, PL = PL_;
    static constexpr int R = PAIR_ ? 2 : 1;                     // CTAs that share a tile
    // Keys of a tile.  With two planes at D = 128 a tile of 128 keys would take
    // 64 KB a stage beside the 128 KB of q: 64 keys leave three stages to one
    // CTA.  Products of 64 columns are bound by the shared memory that feeds
    // them (49 cycles instead of 32), so that a pair, which has room for 128,
    // takes 265 us where one CTA takes 321 (4096 FP32 tokens, 16 heads of 128, one
    // sequence without offsets; causal, 32 heads: 323 against 349, 1024 tokens of
    // them 58 against 62; in blocks of 512 rows 512 tokens took 36.4 against 36.2).
    // Its blocks of 512 rows want long sequences: it is used from 1024 rows on
    // average on.
    static constexpr int BN = DP == 128 && PL == 2 && !PAIR_ ? 64 : 128;
    static constexpr int kBoxes = DP / 64;                      // 64-wide boxes along D
    static constexpr uint32_t kQTile = 128 * DP * 2;            // one plane of one half
    static constexpr uint32_t kQBytes = 4 * kQTile;
    static constexpr uint32_t kPlane = BN * DP * 2 / R;
    static constexpr uint32_t kStage = PL * kPlane;
    static constexpr uint32_t kKBox = BN / R * 128;             // bytes of 64 values of a stage's keys
    static constexpr int NS = DP == 128 ? 3 : (PL == 2 ? 4 : 6);
    static constexpr int kLoads = FOLD_ ? 4 : 2;                // of a tile: k and v, of each half
    static_assert(!FOLD_ || (DP_ == 64 && PL_ == 1 && !PAIR_), "folded halves");
    static_assert(!PAIR_ || NS % 2 == 1, "a stage's turn among the values");
    // Buffers of O' a half: what tensor memory has left beside S (2 x 128 of
    // 512 columns).
    static constexpr int OB = DP == 128 ? 1 : 2;
    static constexpr size_t kSmem = 1024 + kQBytes + NS * kStage + 1024;
    static_assert(kSmem <= 232448, "shared memory");
    static constexpr uint32_t kIdescS = idesc_f16_f32(128 * R, BN);
    static constexpr uint32_t kIdescO = idesc_f16_f32(128 * R, DP) | kIdescBMnMajor;
};

struct Shared {
    uint64_t full[6], empty[6];  // a stage has landed; the products that read it and warp 3 are done with it
    uint64_t checked[6];         // warp 3 has looked through a stage (a barrier for each stage: it may be
                                 // several tiles ahead of the products)
    uint64_t qload[2];           // a half's q has landed, FP32
    uint64_t sfull[2];           // a half's S of a tile, and O' of the tile before, are complete
    uint64_t pfull[2][2];        // pairs: q, then the first part of each P, and the second, of both CTAs
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    int block;                   // this CTA's block of rows; < 0: none
    int q0, nq, k0, nk;          // its sequence's queries and keys
    int most[2], least[2];       // most and least keys that a row of a half sees
    int other[4];                // pairs: the other CTA's
    int hurt;                    // a looked-through tile has values that are not finite, and seen
};

struct Params {
    const float* q;
    float* out;
    float* lse;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const void* v;                // v as the caller has it
    int64_t v_token, v_head;
    const int32_t* table;         // pages of the keys (page_size > 0)
    const int32_t* lengths;       // keys that each query token sees (nullptr: by `causal`)
    int64_t q_token, q_head, out_token, out_head;
    int64_t out_split, lse_split; // elements between the outputs of two parts of the keys
    int n_seq, total_q, total_k, kv_heads, group, dim, causal, splits;
    int page_size, table_pages, pages;
    int v_f32, vec_q, vec_out;
    int q_tokens;                 // query tokens of a half, if q can be loaded by tensor map; else 0
    int out_tokens, out_part;     // query tokens of a warp's rows, if out can be written so, else 0; and of a part
    float scale;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi)
{
    return x < lo ? lo : (x > hi ? hi : x);
}

// The high half of every shared-memory descriptor here: 1024 bytes between
// groups of eight rows, version 1, 128-byte swizzle; and the low half: address
// and leading-dimension offset.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, uint32_t leading)
{
    return ((smem_addr & 0x3FFFFu) >> 4) | ((leading >> 4) << 16);
}

// The sign bits of the FP16 values of a pair that are infinite or NaN: an
// exponent of all ones carries into the sign's place.
__device__ __forceinline__ uint32_t not_finite(uint32_t pair)
{
    return ((pair & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// Named barriers of a half's four row warps and its issuing warp.
__device__ __forceinline__ void rows_sync(int id)
{
    asm volatile("bar.sync %0, 160;" ::"r"(id) : "memory");
}

__device__ __forceinline__ void rows_arrive(int id)
{
    asm volatile("bar.arrive %0, 160;" ::"r"(id) : "memory");
}

// This CTA's (or pair's) sequence and block of kRows rows: blocks are numbered
// sequence by sequence, the last of one, which sees most keys, first.  (All
// sequences' blocks by their number, highest first, end with many short blocks at
// once, which memory bounds: 245 us instead of 238 for the ragged prompts, 533
// instead of 506 for 40 of 300 to 1500 tokens.)  One warp; the offsets are read
// 32 sequences at a time.  Tokens beyond the last sequence are one more, without keys.
template <int kRows>
__device__ __forceinline__ void find_block(const Params& p, int block, Shared* sm)
{
    const int lane = threadIdx.x & 31;
    if (!p.cu_q) {
        if (lane == 0) {
            sm->block = static_cast<int>((static_cast<int64_t>(p.total_q) * p.group + kRows - 1) / kRows) - 1 - block;
            sm->q0 = sm->k0 = 0;
            sm->nq = p.total_q;
            sm->nk = p.total_k;
        }
        return;
    }
    for (int s0 = 0; s0 <= p.n_seq; s0 += 32) {
        const int s = s0 + lane;
        int n = 0, a = 0, b = 0, c = 0, d = 0;
        if (s <= p.n_seq) {
            a = clampi(p.cu_q[s], 0, p.total_q), b = p.total_q;
            if (s < p.n_seq) {
                b = clampi(p.cu_q[s + 1], a, p.total_q);
                c = clampi(p.cu_k[s], 0, p.total_k), d = clampi(p.cu_k[s + 1], c, p.total_k);
            }
            const unsigned rows = static_cast<unsigned>(b - a) * static_cast<unsigned>(p.group);
            n = static_cast<int>((rows + (kRows - 1u)) / kRows);
        }
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, x > block);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                sm->block = x - 1 - block;
                sm->q0 = a;
                sm->nq = b - a;
                sm->k0 = c;
                sm->nk = d - c;
            }
            return;
        }
        block -= __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0)
        sm->block = -1;
}

template <int DP, int PL, bool PAIR, bool FOLD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_k_lo, const __grid_constant__ CUtensorMap map_v_lo,
                   const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_out,
                   const Params p)
{
    using C = Cfg<DP, PL, PAIR, FOLD>;
    constexpr int BN = C::BN, NS = C::NS, OB = C::OB, R = C::R;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* const stages = smem + C::kQBytes;
    Shared* const sm = reinterpret_cast<Shared*>(stages + NS * C::kStage);
    static_assert(sizeof(Shared) <= 1024, "barrier area");
    // warp-uniform to the compiler, so that roles and loop counts stay in uniform registers
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // A dependent that starts early finds what this kernel waited for complete
    // (the decode kernel relies on it).
    grid_dependency_wait();
    grid_dependency_launch();
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const int item = blockIdx.x / R, head = item % p.kv_heads;
    const int cta_part = item / p.kv_heads % p.splits;
    if (warp == 0)
        find_block<256 * R>(p, item / p.kv_heads / p.splits, sm);
    if (threadIdx.x == 64) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sm->full[i], 1);
            mbar_init(&sm->empty[i], FOLD ? 2 : 3);
            mbar_init(&sm->checked[i], R);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&sm->qload[h], 1);
            mbar_init(&sm->sfull[h], 1);
            mbar_init(&sm->pfull[h][0], 4 * R);
            mbar_init(&sm->pfull[h][1], 4 * R);
        }
        mbar_init(&sm->drain[0], 1);
        mbar_init(&sm->drain[1], 1);
        sm->abort = 0;
        for (int h = 0; h < 2; ++h) {
            sm->most[h] = 0;
            sm->least[h] = INT32_MAX;
        }
        sm->hurt = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (sm->block < 0)
        return;  // the grid is an upper bound

    // A half's rows in blocks of 128: this CTA's block of them.
    const int half = (warp >> 2) - 1;
    const int rows128 = FOLD ? 0 : (2 * sm->block + half) * R + static_cast<int>(rank);
    // One load brings a half's rows of q, FP32, to where its planes will be
    // (tokens past the sequence's end too: rows that are not there).  Loads by
    // the threads would wait for each other in the small L1 that 227 KB of
    // shared memory leave.  The second half's is issued with the first keys', so
    // that the first half's lands, and is split, before.
    auto load_q = [&] {
        if (p.q_tokens > 0 && lane == 0) {
            mbar_arrive_expect_tx(&sm->qload[half], 128 * p.dim * 4);
            tma_load_3d(smem + half * 2 * C::kQTile, &map_q, &sm->qload[half], 0, head * p.group,
                        sm->q0 + rows128 * p.q_tokens);
        }
    };
    if (warp == 4)
        load_q();

    // the part of its sequence's keys that this CTA, or this half, goes through
    const int q0 = sm->q0, nq = sm->nq, k0 = sm->k0, nk = sm->nk;
    const int parts = FOLD ? 2 * p.splits : p.splits;
    const int part_keys = ((nk + BN - 1) / BN + parts - 1) / parts * BN;
    const int part = FOLD ? 2 * cta_part + max(half, 0) : cta_part;
    auto begin_of = [&](int i) -> int { return min(static_cast<int64_t>(nk), static_cast<int64_t>(i) * part_keys); };
    const int first = begin_of(part);
    const int keys = min(nk - first, part_keys);

    // rows: what each sees
    int64_t q_at = 0, out_at = 0, lse_at = 0;
    int lim = 0;
    bool valid = false;
    if (half >= 0) {
        // total_q * heads is an int
        const unsigned row = static_cast<unsigned>(rows128) * 128u + (threadIdx.x & 127);
        const unsigned group = static_cast<unsigned>(p.group);
        valid = row < static_cast<unsigned>(nq) * group;
        const int t = static_cast<int>(valid ? row / group : 0u), hq = head * p.group + static_cast<int>(row % group);
        int sees = nk;
        if (p.lengths)
            sees = valid ? clampi(p.lengths[q0 + t], 0, nk) : 0;
        else if (p.causal)
            sees = clampi(t + 1 - nq + nk, 0, nk);  // t < nq: no overflow
        lim = clampi(sees - first, 0, keys);
        const int64_t token = q0 + static_cast<int64_t>(t);
        q_at = token * p.q_token + hq * p.q_head;
        out_at = token * p.out_token + hq * p.out_head + part * p.out_split;
        lse_at = token * (p.kv_heads * p.group) + hq + part * p.lse_split;
        const int hi = __reduce_max_sync(0xffffffffu, valid ? lim : 0);
        const int lo = __reduce_min_sync(0xffffffffu, valid ? lim : INT32_MAX);
        if (lane == 0) {
            atomicMax(&sm->most[half], hi);
            atomicMin(&sm->least[half], lo);
        }
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(&sm->tmem_base, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&sm->tmem_base, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR) {
        // what the rows of either CTA see decides on the tiles of both
        cluster_sync();
        if (threadIdx.x < 4)
            st_cluster(mapa_shared(&sm->other[threadIdx.x], rank ^ 1),
                       threadIdx.x < 2 ? sm->most[threadIdx.x] : sm->least[threadIdx.x - 2]);
        cluster_sync();
        if (threadIdx.x < 2) {
            sm->most[threadIdx.x] = max(sm->most[threadIdx.x], sm->other[threadIdx.x]);
            sm->least[threadIdx.x] = min(sm->least[threadIdx.x], sm->other[threadIdx.x + 2]);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8)
        load_q();
    // All 512 columns are this CTA's, so they begin at 0: tensor-memory addresses
    // are constants to the issuing warp.
    const bool at_zero = sm->tmem_base == 0;
    if (!at_zero && threadIdx.x == 0)
        atomicCAS(&g_attn_fault_word, 0u, kFaultAttnTmem);
    const int n0 = __shfl_sync(0xffffffffu, at_zero ? (sm->most[0] + BN - 1) / BN : 0, 0);
    const int n1 = __shfl_sync(0xffffffffu, at_zero ? (sm->most[1] + BN - 1) / BN : 0, 0);
    const int n = max(n0, n1), most = max(sm->most[0], sm->most[1]);
    // tiles from this one on are seen only in part by some row
    const int edge = __shfl_sync(
        0xffffffffu, min(n0 > 0 ? sm->least[0] : INT32_MAX, n1 > 0 ? sm->least[1] : INT32_MAX) / BN, 0);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        if (warp == 0) {
            // ---------------- loads: K0, V0, K1, V1, ... (folded: each for one half, then the other)
            // A lane has one box of every tile (16 at most), and the page of one of its
            // pieces: looked up a tile ahead, or the ring would wait for it too (256 rows
            // on 32768 shared keys: 223 us instead of 212).  A page that is not there: a
            // place beyond the cache, which reads zeros.
            const int pieces = p.page_size ? BN / p.page_size : 1;
            const int piece = lane % pieces, box = lane / pieces % C::kBoxes, plane = lane / pieces / C::kBoxes;
            uint8_t* const to = stages + plane * C::kPlane + box * (BN * 128) + piece * p.page_size * 128;
            auto begin = [&](int i) { return FOLD ? begin_of(2 * cta_part + (i & 1)) : first; };
            auto look_up = [&](int i) {
                const int at = begin(i) / p.page_size + i / C::kLoads * pieces + piece;
                return at < p.table_pages ? p.table[at] : -1;
            };
            constexpr int kAhead = FOLD ? 2 : 1;  // tiles of a step
            int pages[kAhead] = {}, coming[kAhead] = {};
            if (p.page_size) {
#pragma unroll
                for (int h = 0; h < kAhead; ++h)
                    coming[h] = look_up(h);
            }
            int i = 0;
            for (; i < C::kLoads * n; ++i) {
                const int s = i % NS, j = i / C::kLoads, is_v = FOLD ? i >> 1 & 1 : i & 1;
                if (i >= NS && !attn_warp_wait(&sm->empty[s], ((i / NS) - 1) & 1, &sm->abort, kFaultAttnLoad))
                    break;
                // A pair's loads count on the first CTA's barrier, where the products are
                // issued; only values that are looked through, on their own CTA's.
                const bool looked = is_v && j >= edge;
                if (lane == 0) {
                    if (PAIR && !looked && rank == 1)
                        mbar_arrive(&sm->full[s]);
                    else
                        mbar_arrive_expect_tx(&sm->full[s], PAIR && !looked ? 2 * C::kStage : C::kStage);
                }
                __syncwarp();
                if (PAIR) {
                    // this CTA's half: keys of k in boxes along the head dimension, 64
                    // values of v in boxes of 64 keys
                    if (lane < 2 * PL) {
                        const uint32_t bar = mapa_shared(&sm->full[s], looked ? rank : 0);
                        const int plane = lane / 2, sub = lane % 2;
                        const CUtensorMap* const map =
                            plane ? (is_v ? &map_v_lo : &map_k_lo) : (is_v ? &map_v : &map_k);
                        const int key = k0 + first + j * BN;
                        tma_load_3d_pair(stages + s * C::kStage + plane * C::kPlane + sub * 8192, map, bar,
                                         (is_v ? rank : sub) * 64, key + (is_v ? sub : rank) * 64, head);
                    }
                    __syncwarp();
                    continue;
                }
                const int h = FOLD ? i & 1 : 0;
                if (p.page_size && !is_v) {
                    pages[h] = coming[h] >= 0 && coming[h] < p.pages ? coming[h] : p.pages;
                    coming[h] = look_up(i + C::kLoads);
                }
                if (plane < PL) {
                    const CUtensorMap* const map =
                        plane ? (is_v ? &map_v_lo : &map_k_lo) : (is_v ? &map_v : &map_k);
                    if (p.page_size)
                        tma_load_3d(to + s * C::kStage, map, &sm->full[s], box * 64, 0, pages[h] * p.kv_heads + head);
                    else
                        tma_load_3d(to + s * C::kStage, map, &sm->full[s], box * 64, k0 + begin(i) + j * BN, head);
                }
                __syncwarp();
            }
            if (i < C::kLoads * n) {  // abort: what was issued lands before the CTA leaves
                for (int j = max(0, i - NS); j < i; ++j)
                    attn_drain_wait(&sm->full[j % NS], (j / NS) & 1);
                if (PAIR) {  // those that count on the other CTA's barrier: time to land
                    const long long start = clock64();
                    while (clock64() - start < (1ll << 22)) {
                    }
                }
            }
        } else if (warp < 3 && rank == 0) {
            // ---------------- products: warp 1 issues those of the first half, warp 2 of the second
            // One lane issues in a branch of its own with constant accumulator
            // addresses: 65 cycles for a 128 x 128 x 16 product, the tensor
            // cores' rate (measured; 73 with the whole warp predicated, which
            // does not keep them busy).  The halves take turns, step by step
            // (named barriers 2 and 3): products of both mixed would leave the
            // two softmaxes at the same time, and the tensor cores idle then.
            // q and P arrive by named barriers too (4 to 7: half and part): a test of an
            // mbarrier takes hundreds of cycles while operands stream from shared
            // memory.  After an abort every warp still goes through its barriers.
            const int h = warp - 1, nh = h ? n1 : n0;
            const uint32_t qhi = desc_lo(smem_u32(smem), 16) + h * 2 * (C::kQTile >> 4), qlo = qhi + (C::kQTile >> 4);
            const uint32_t k_lo32 = desc_lo(smem_u32(stages), 16), v_lo32 = desc_lo(smem_u32(stages), BN * 128);
            constexpr uint32_t kKvPlane = C::kPlane >> 4, kKvStage = C::kStage >> 4;
            const uint32_t ds = h * 128;
            bool ok = true;
            auto wait = [&](uint64_t* bar, int phase) {
                ok = ok && attn_wait(bar, phase & 1, &sm->abort, kFaultAttnMma);
            };
            auto wait_cluster = [&](uint64_t* bar, int phase) {
                ok = ok && attn_wait_cluster(bar, phase & 1, &sm->abort, kFaultAttnMma);
            };
            // a stage's tile, in a pair both CTAs' halves of it (values that are looked
            // through: when both warps 3 are done; every NS-th of them has this stage)
            auto wait_tile = [&](int s, int load, bool looked_through) {
                if (PAIR && looked_through) {
                    wait_cluster(&sm->checked[s], (load / 2 - edge) / NS);
                } else {
                    wait(&sm->full[s], load / NS);
                    if (looked_through)
                        wait(&sm->checked[s], load / NS);
                }
            };
            auto commit = [&](uint64_t* bar) {
                if (PAIR)
                    umma_commit_pair_by(1, bar, 0x3);
                else
                    umma_commit_by(1, bar);
            };
            auto pv = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
                if (PAIR)
                    umma_pair_ta_w_by(1, d, a, b, kDescHi, C::kIdescO, add);
                else
                    umma_ta_w_by(1, d, a, b, kDescHi, C::kIdescO, add);
            };
            // S: a and b at q's and k's planes; how: 0 fresh, 1 added, 2 added to 2^-10 of what is there
            auto chain = [&](uint32_t qd, uint32_t kd, int how) {
#pragma unroll
                for (int t = 0; t < DP / 16; ++t) {
                    const uint32_t da = qd + (t / 4) * (128 * 128 >> 4) + (t % 4) * 2;
                    const uint32_t db = kd + (t / 4) * (C::kKBox >> 4) + (t % 4) * 2;
                    if (t == 0 && how == 2) {
                        if (PAIR)
                            umma_pair_w_scale10_by(1, ds, da, db, kDescHi, C::kIdescS);
                        else
                            umma_w_scale10_by(1, ds, da, db, kDescHi, C::kIdescS);
                    } else if (PAIR) {
                        umma_pair_w_by(1, ds, da, db, kDescHi, C::kIdescS, t > 0 || how > 0);
                    } else {
                        umma_w_by(1, ds, da, db, kDescHi, C::kIdescS, t > 0 || how > 0);
                    }
                }
            };
            // stages of K of tile j + 1 and V of tile j, and their next ones
            int sk = FOLD ? h : 0, sv = FOLD ? NS - 2 + h : NS - 1;
            auto next = [](int x) {
                x += C::kLoads % NS;
                return x >= NS ? x - NS : x;
            };
#pragma unroll 1
            for (int j = -1; j < n; ++j) {
                const int iv = FOLD ? 4 * j + 2 + h : 2 * j + 1, ik = FOLD ? 4 * j + 4 + h : 2 * j + 2;  // their loads
                if (j >= nh) {
                    // Stages that only the other half uses (folded: nobody) are given back
                    // too, but not before their load has landed: what the stage held
                    // before may still be read, and this arrival would count for that.
                    if (h == 1 || j >= 0)
                        asm volatile("bar.sync %0, 64;" ::"r"(3 - h) : "memory");
                    if (h == 0 || j + 1 < n)
                        asm volatile("bar.arrive %0, 64;" ::"r"(2 + h) : "memory");
                    if (elect_one()) {
                        if (j >= 0) {
                            wait(&sm->full[sv], iv / NS);
                            commit(&sm->empty[sv]);
                        }
                        if (j + 1 < n) {
                            wait(&sm->full[sk], ik / NS);
                            commit(&sm->empty[sk]);
                        }
                    }
                    __syncwarp();
                    sk = next(sk);
                    sv = next(sv);
                    continue;
                }
                const bool has_v = j >= 0, has_k = j + 1 < nh;
                if (elect_one()) {
                    if (has_v)
                        wait_tile(sv, iv, j >= edge);
                    if (PAIR && j < 0 && has_k)
                        wait_cluster(&sm->pfull[h][0], 0);
                    else if (PAIR && has_v)
                        wait(&sm->pfull[h][0], j + 1);
                }
                __syncwarp();
                if (!PAIR && (has_v || has_k))  // P's first half, before the first tile q
                    rows_sync(4 + 2 * h);
                // the turn: the second half waits for the first half's step, the first for the second's before
                if (h == 1 || j >= 0)
                    asm volatile("bar.sync %0, 64;" ::"r"(3 - h) : "memory");
                // P of 16 keys: 8 columns of hi pairs, then 8 of lo pairs.  The first
                // half of the keys, then, as soon as its P is there, the second.
                constexpr int kSteps = BN / 32;
                const uint32_t d = 256 + h * 128 + (OB == 2 ? (j & 1) * 64 : 0);
                const uint32_t vhi = v_lo32 + sv * kKvStage, vlo = vhi + kKvPlane;
                auto part = [&](int t0) {
                    tc_fence_after();
#pragma unroll
                    for (int t = t0; t < t0 + kSteps; ++t) {
                        if (PL == 1) {
                            pv(d, ds + t * 16 + 8, vhi + t * 128, t > 0);
                            pv(d, ds + t * 16, vhi + t * 128, 1);
                        } else {  // hi P with lo v, over all keys before the accumulator is scaled
                            pv(d, ds + t * 16, vlo + t * 128, t > 0);
                        }
                    }
                };
                if (has_v) {
                    if (elect_one() && ok)
                        part(0);
                    __syncwarp();
                    if (!PAIR)
                        rows_sync(5 + 2 * h);
                }
                if (elect_one()) {
                    if (PAIR && has_v)
                        wait(&sm->pfull[h][1], j);
                    if (has_v && ok) {
                        part(kSteps);
                        if (PL == 2) {
#pragma unroll
                            for (int t = 0; t < 2 * kSteps; ++t) {
                                if (t > 0)
                                    pv(d, ds + t * 16 + 8, vhi + t * 128, 1);
                                else if (PAIR)
                                    umma_pair_ta_w_scale10_by(1, d, ds + 8, vhi, kDescHi, C::kIdescO);
                                else
                                    umma_ta_w_scale10_by(1, d, ds + 8, vhi, kDescHi, C::kIdescO);
                                pv(d, ds + t * 16, vhi + t * 128, 1);
                            }
                        }
                    }
                    if (has_v)
                        commit(&sm->empty[sv]);
                    if (has_k)
                        wait_tile(sk, ik, false);
                    if (has_k && ok) {
                        tc_fence_after();
                        const uint32_t khi = k_lo32 + sk * kKvStage;
                        chain(qlo, khi, 0);
                        if (PL == 2)
                            chain(qhi, khi + kKvPlane, 1);
                        chain(qhi, khi, 2);
                    }
                    if ((has_v || has_k) && ok)
                        commit(&sm->sfull[h]);
                }
                __syncwarp();
                if (h == 0 || j + 1 < n)
                    asm volatile("bar.arrive %0, 64;" ::"r"(2 + h) : "memory");
                if (elect_one() && j + 1 < n) {
                    if (!has_k)
                        wait(&sm->full[sk], ik / NS);
                    commit(&sm->empty[sk]);
                }
                __syncwarp();
                sk = next(sk);
                sv = next(sv);
            }
            if (elect_one() && *reinterpret_cast<volatile int*>(&sm->abort)) {
                if (PAIR)
                    umma_commit_pair_by(1, &sm->drain[h], 0x1);
                else
                    umma_commit_by(1, &sm->drain[h]);
                attn_drain_wait(&sm->drain[h], 0);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ---------------- values that must not count
            for (int i = 0; i < C::kLoads * n; ++i) {
                const int s = i % NS, j = i / C::kLoads, is_v = FOLD ? i >> 1 & 1 : i & 1;
                const int seen_to = FOLD ? sm->most[i & 1] : most;
                if (!attn_warp_wait(&sm->full[s], (i / NS) & 1, &sm->abort, kFaultAttnValues))
                    break;
                if (is_v && j >= edge) {
                    uint8_t* const tile = stages + s * C::kStage;
                    bool seen = false;
                    constexpr int kBatch = 8;  // loads in flight a lane
#pragma unroll 1
                    for (uint32_t at = lane * 16; at < C::kStage; at += kBatch * 512) {
                        uint4 x[kBatch];
                        uint32_t odd = 0;
#pragma unroll
                        for (int b = 0; b < kBatch; ++b) {
                            x[b] = *reinterpret_cast<const uint4*>(tile + at + b * 512);
                            odd |= not_finite(x[b].x) | not_finite(x[b].y) | not_finite(x[b].z) | not_finite(x[b].w);
                        }
                        if (odd != 0) {
#pragma unroll
                            for (int b = 0; b < kBatch; ++b) {
                                uint32_t* const w = reinterpret_cast<uint32_t*>(&x[b]);
                                uint32_t here = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t f = not_finite(w[e]);
                                    here |= f;
                                    w[e] &= ~((f >> 15) * 0xffffu);
                                }
                                if (here) {
                                    *reinterpret_cast<uint4*>(tile + at + b * 512) = x[b];
                                    seen |= j * BN + static_cast<int>((at + b * 512) / 128 % BN) < seen_to;
                                }
                            }
                        }
                    }
                    if (__any_sync(0xffffffffu, seen) && lane == 0) {
                        *reinterpret_cast<volatile int*>(&sm->hurt) = 1;
                        if (PAIR)  // v's columns are the other CTA's rows' too
                            st_cluster(mapa_shared(&sm->hurt, rank ^ 1), 1);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (!PAIR)
                        mbar_arrive(&sm->checked[s]);
                    else if (is_v && j >= edge)
                        mbar_arrive_release_cluster(mapa_shared(&sm->checked[s], 0));
                    mbar_arrive(&sm->empty[s]);
                }
            }
        }
    } else {
        // ---------------- rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        const int nh = half ? n1 : n0, w4 = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
        bool ok = true;
        // q, or a part of P, to the issuing warp (a pair's is in its first CTA)
        auto hand_over = [&](int part_of_p, bool planes) {
            if (PAIR) {
                __syncwarp();
                const uint32_t to = mapa_shared(&sm->pfull[half][part_of_p], 0);
                if (lane == 0) {
                    // q's planes are shared memory; P is tensor memory, ordered by
                    // tcgen05's own fences, and a release over the cluster costs a
                    // thousand cycles a tile
                    if (planes)
                        mbar_arrive_release_cluster(to);
                    else
                        mbar_arrive_cluster(to);
                }
            } else {
                rows_arrive(4 + 2 * half + part_of_p);
            }
        };
        // q's planes: a warp splits its 32 rows
        if (nh > 0) {
            uint8_t* const hi_tile = smem + half * 2 * C::kQTile;
            constexpr int kLanes = DP / 4, kAtOnce = 32 / kLanes;  // lanes of a row, rows a load
            const int d0 = lane % kLanes * 4, sub = lane / kLanes;
            const unsigned rows_there = __ballot_sync(0xffffffffu, valid);
            auto split_row = [&](int i, float4 f) {
                if (!((rows_there >> i) & 1))
                    f = float4{};
                uint2 hi, lo;
                split2(f.x, f.y, hi.x, lo.x);
                split2(f.z, f.w, hi.y, lo.y);
                const uint32_t to = (d0 / 64) * (128 * 128) + sw128(w4 * 32 + i, (d0 % 64) / 8) + (d0 % 8) * 2;
                *reinterpret_cast<uint2*>(hi_tile + to) = hi;
                *reinterpret_cast<uint2*>(hi_tile + C::kQTile + to) = lo;
            };
            if (p.q_tokens > 0) {
                // the warps read all rows before one of them writes a plane
                ok = attn_warp_wait(&sm->qload[half], 0, &sm->abort, kFaultAttnRows);
                float4 x[32 / kAtOnce];
#pragma unroll
                for (int i = 0; i < 32 / kAtOnce; ++i)
                    x[i] = d0 < p.dim ? *reinterpret_cast<const float4*>(
                                            hi_tile + ((w4 * 32 + i * kAtOnce + sub) * p.dim + d0) * 4)
                                      : float4{};
                asm volatile("bar.sync %0, 128;" ::"r"(8 + half) : "memory");
#pragma unroll
                for (int i = 0; i < 32 / kAtOnce; ++i)
                    split_row(i * kAtOnce + sub, x[i]);
            } else if (p.vec_q) {
                // rows that are not there have the address of one that is
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += 8 * kAtOnce) {
                    float4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t at = __shfl_sync(0xffffffffu, q_at, i0 + i * kAtOnce + sub);
                        x[i] = __ldg(reinterpret_cast<const float4*>(p.q + at + (d0 < p.dim ? d0 : 0)));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        split_row(i0 + i * kAtOnce + sub, d0 < p.dim ? x[i] : float4{});
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < 32 / kAtOnce; ++i) {
                    const float* const src = p.q + __shfl_sync(0xffffffffu, q_at, i * kAtOnce + sub) + d0;
                    float4 f{};
                    f.x = d0 < p.dim ? __ldg(src) : 0.0f;
                    f.y = d0 + 1 < p.dim ? __ldg(src + 1) : 0.0f;
                    f.z = d0 + 2 < p.dim ? __ldg(src + 2) : 0.0f;
                    f.w = d0 + 3 < p.dim ? __ldg(src + 3) : 0.0f;
                    split_row(i * kAtOnce + sub, f);
                }
            }
            fence_proxy_async_smem();
            hand_over(0, true);
        } else if (p.q_tokens > 0) {
            // q lands before anything else is done where it goes, and before the CTA leaves
            ok = attn_warp_wait(&sm->qload[half], 0, &sm->abort, kFaultAttnRows);
        }

        const float c2 = p.scale * kAttnLog2E;
        const uint64_t c22 = f2_bits(c2, c2);
        const uint32_t st = lanes + half * 128;
        const int row_lim = valid ? lim : INT32_MAX;  // rows that are not there are not stored
        float m = -INFINITY;        // the running maximum of s * c2
        // The running sum of 2^14 p, and what its additions have rounded away: one
        // addition for each tile, of sums that begin at zero with the tile.  (Weights
        // added one by one to the running sum all round the same way where they are
        // equal: 4e-5 of it after 16384 keys, 2e-4 after 65536.)
        float l = 0.0f, l_low = 0.0f;
        float alpha = 0.0f;         // what the sums so far are to be scaled by with the next O'
        uint64_t o[DP / 2];
#pragma unroll
        for (int i = 0; i < DP / 2; ++i)
            o[i] = 0;

        // o = o alpha + O' of tile j, 32 values at a time; after each 32: done(c)
        auto take_and = [&](int j, auto done) {
            const uint64_t a2 = f2_bits(alpha, alpha);
            const uint32_t from = lanes + 256 + half * 128 + (OB == 2 ? (j & 1) * 64 : 0);
            uint32_t r[2][32];
            tmem_ld32(from, r[0]);
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t (&x)[32] = r[c & 1];
                tmem_ld_wait32(x);
                if (c + 1 < DP / 32)
                    tmem_ld32(from + (c + 1) * 32, r[(c + 1) & 1]);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[c * 16 + i] = fma2(o[c * 16 + i], a2, u2_bits(x[2 * i], x[2 * i + 1]));
                done(c);
            }
        };
        auto take = [&](int j) { take_and(j, [](int) {}); };

        // Tile j's scores become P, and O' of the tile before is taken: first
        // where there is one buffer for it (P's arrival frees it), else last,
        // while the tensor cores go on.
#pragma unroll 1
        for (int j = 0; j <= nh && nh > 0; ++j) {
            if (!attn_lane0_wait(&sm->sfull[half], j & 1, &sm->abort, kFaultAttnRows)) {
                ok = false;
                for (; !PAIR && j < nh; ++j) {  // the issuing warp waits for the rest of P
                    rows_sync(4 + 2 * half);
                    rows_sync(5 + 2 * half);
                }
                break;
            }
            tc_fence_after();
            // A pair takes the last O' below, while its output's stores are under way
            // (4096 FP32 tokens, 32 heads: 349 -> 343 us); alone the loop without
            // that step came out slower (16384 causal tokens: 2.26 -> 2.36 ms).
            if (!PAIR && j > 0 && (OB == 1 || j == nh))
                take(j - 1);
            if (j == nh)
                break;
            if (PAIR && j > 0)
                take(j - 1);
            {
                if (__any_sync(0xffffffffu, row_lim < (j + 1) * BN)) {
                    // hidden scores to -inf, in place
                    const int left = row_lim - j * BN;
#pragma unroll 1
                    for (int c = 0; c < BN; c += 16) {
                        uint32_t r[16];
                        tmem_ld16(st + c, r);
                        tmem_ld_wait16(r);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            r[i] = c + i < left ? r[i] : 0xff800000u;
                        tmem_st16(st + c, r);
                    }
                    tmem_st_wait();
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                {
                    uint32_t r[2][32];
                    tmem_ld32(st, r[0]);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        uint32_t (&x)[32] = r[c & 1];
                        tmem_ld_wait32(x);
                        if (c + 1 < BN / 32)
                            tmem_ld32(st + (c + 1) * 32, r[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            top[i / 2 & 3] =
                                fmaxf(top[i / 2 & 3], fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                    }
                }
                uint32_t x[32];
                tmem_ld32(st, x);
                const float m_new = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c2);
                const float shift = m_new == -INFINITY ? 0.0f : m_new;  // nothing seen yet: every p is 0
                const float alpha_new = ex2(m - shift);
                m = m_new;
                // 2^14 p in one operation: the sum's rounding, at most 2^-21 of 14,
                // is of the size of the scores' own.  Beyond kAttnLargeScore the two
                // roundings that s and 14 - m have apart would soon be whole units,
                // and 2^14 p no FP16 value (from 2^27 on): there s becomes s c - m in
                // place, the product rounded as the maximum is, so that it ends at 0.
                uint64_t by = c22, s2 = f2_bits(14.0f - shift, 14.0f - shift);
                const bool large = fabsf(shift) >= kAttnLargeScore;
                if (__any_sync(0xffffffffu, large)) {
                    tmem_ld_wait32(x);
#pragma unroll 1
                    for (int c = 0; c < BN; c += 16) {
                        uint32_t r[16];
                        tmem_ld16(st + c, r);
                        tmem_ld_wait16(r);
                        if (large) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                r[i] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(r[i]), c2), shift));
                        }
                        __syncwarp();
                        tmem_st16(st + c, r);
                    }
                    tmem_st_wait();
                    tmem_ld32(st, x);
                    if (large) {
                        by = f2_bits(1.0f, 1.0f);
                        s2 = f2_bits(14.0f, 14.0f);
                    }
                    __syncwarp();
                }
                uint64_t l2 = 0, l3 = 0;
#pragma unroll 1
                for (int c = 0; c < BN; c += 32) {
                    float w[32];
                    tmem_ld_wait32(x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t y = fma2(u2_bits(x[2 * i], x[2 * i + 1]), by, s2);
                        w[2 * i] = ex2(lo_f(y));
                        w[2 * i + 1] = ex2(hi_f(y));
                    }
                    // the last of these reads P, and is not used
                    tmem_ld32(st + (c + 32) % BN, x);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t out[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float w0 = w[e * 16 + 2 * i], w1 = w[e * 16 + 2 * i + 1];
                            (e ? l3 : l2) = add2(e ? l3 : l2, f2_bits(w0, w1));
                            split_p(w0, w1, out[i], out[8 + i]);
                        }
                        tmem_st16(st + c + e * 16, out);
                    }
                    if (c == BN / 2 - 32 || c == BN - 32) {
                        tmem_st_wait();
                        tc_fence_before();
                        hand_over(c >= BN / 2, false);
                    }
                }
                l2 = add2(l2, l3);
                {
                    const float before = l * alpha_new;
                    const float more = fmaf(l_low, alpha_new, lo_f(l2) + hi_f(l2));
                    l = before + more;
                    l_low = more - (l - before);
                }
                tmem_ld_wait32(x);
                if (OB == 2 && j > 0)
                    take(j - 1);
                alpha = alpha_new;
            }
        }
        // out, through shared memory (this warp's share of q's planes, which the
        // products of this half have read): a thread holds a row
        l *= 1.0f / kAttnPScale;
        // no key seen, or none that counts beside an infinite score (NaN stays NaN)
        const float norm = l == 0.0f ? 0.0f : (1.0f / kAttnPScale) / l;
        if (ok) {
            // Boxes of 32 values of the warp's 32 rows, 128-byte swizzled as the
            // tensor map wants them (and as free of bank conflicts either way).
            constexpr int kChunks = DP / 4;  // 16 bytes each
            uint8_t* const tile = smem + half * 2 * C::kQTile + w4 * (32 * DP * 4);
            const uint64_t norm2 = f2_bits(norm, norm);
            const unsigned rows_there = __ballot_sync(0xffffffffu, valid);
            const bool by_map = p.out_tokens > 0 && rows_there == 0xffffffffu;  // whole tokens, all there
            const int token = part * p.out_part + q0 + (rows128 * 4 + w4) * p.out_tokens;
            // a box is on its way while the next 32 values are taken
            auto put = [&](int c) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<ulonglong2*>(tile + c * 4096 + sw128(lane, i)) = make_ulonglong2(
                        mul2(o[c * 16 + 2 * i], norm2), mul2(o[c * 16 + 2 * i + 1], norm2));
                if (by_map && c * 32 < p.dim) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        tma_store_3d(&map_out, tile + c * 4096, c * 32, head * p.group, token);
                }
            };
            if (PAIR && nh > 0) {
                take_and(nh - 1, put);
            } else {
#pragma unroll
                for (int c = 0; c < DP / 32; ++c)
                    put(c);
            }
            constexpr int kRows = 32 / kChunks;  // rows a warp writes at once
            const int chunk = lane % kChunks, d = chunk * 4;
            if (by_map) {
                if (lane == 0) {
                    bulk_commit_group();
                    if (sm->hurt) {  // written before values are added below
                        bulk_wait_group0();
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                    } else {
                        bulk_wait_group_read0();
                    }
                }
                __syncwarp();
            } else if (__syncwarp(), p.vec_out && p.q_tokens > 0) {
                // rows are whole tokens of a power of two of heads: addresses by shifts
                // (exchanges between lanes queue behind the other half's operands)
                const int shift = 31 - __clz(p.group);
                float* const base = p.out + (static_cast<int64_t>(q0) + rows128 * p.q_tokens) * p.out_token +
                                    static_cast<int64_t>(head) * p.group * p.out_head + part * p.out_split + d;
#pragma unroll 8
                for (int i0 = 0; i0 < 32; i0 += kRows) {
                    const int i = i0 + lane / kChunks, row = w4 * 32 + i;
                    float* const to = base + (row >> shift) * p.out_token + (row & (p.group - 1)) * p.out_head;
                    const float4 x = *reinterpret_cast<const float4*>(tile + (chunk / 8) * 4096 + sw128(i, chunk % 8));
                    if (((rows_there >> i) & 1) && d < p.dim)
                        *reinterpret_cast<float4*>(to) = x;
                }
            } else {
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += kRows) {
                    const int i = i0 + lane / kChunks;
                    float* const to = p.out + __shfl_sync(0xffffffffu, out_at, i) + d;
                    const float4 x = *reinterpret_cast<const float4*>(tile + (chunk / 8) * 4096 + sw128(i, chunk % 8));
                    if (!((rows_there >> i) & 1))
                        continue;
                    if (p.vec_out && d < p.dim) {
                        *reinterpret_cast<float4*>(to) = x;
                        continue;
                    }
                    if (d < p.dim)
                        to[0] = x.x;
                    if (d + 1 < p.dim)
                        to[1] = x.y;
                    if (d + 2 < p.dim)
                        to[2] = x.z;
                    if (d + 3 < p.dim)
                        to[3] = x.w;
                }
            }
            __syncwarp();  // the rows are written before values are added below
        }
        if (ok && valid) {
            if (p.lse)
                p.lse[lse_at] = l == 0.0f ? -INFINITY : fmaf(m, kAttnLn2, logf(l));
            // values that are not finite were taken out of the tiles from
            // `edge` on: a row that sees one adds it (its weight is positive)
            if (*reinterpret_cast<volatile int*>(&sm->hurt)) {
                float* const out = p.out + out_at;
#pragma unroll 1
                for (int i = edge * BN; i < lim; ++i) {
                    const int key = first + i;
                    int64_t at = (static_cast<int64_t>(k0) + key) * p.v_token + head * p.v_head;
                    if (p.page_size) {
                        const int page = p.table[key / p.page_size];
                        if (page < 0 || page >= p.pages)
                            continue;
                        at = ((static_cast<int64_t>(page) * p.kv_heads + head) * p.page_size + key % p.page_size) *
                             p.dim;
                    }
#pragma unroll 1
                    for (int d = 0; d < p.dim; ++d) {
                        const float x = __half2float(p.v_f32 ? __float2half_rn(static_cast<const float*>(p.v)[at + d])
                                                             : static_cast<const __half*>(p.v)[at + d]);
                        if (!isfinite(x))
                            out[d] += x;
                    }
                }
            }
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync();  // neither CTA leaves while the other's products may read it or arrive on it
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if (PAIR)
            tmem_dealloc_pair(sm->tmem_base, 512);
        else
            tmem_dealloc(sm->tmem_base, 512);
    }
}

// FP32 keys and values as FP16 planes (hi = fp16(x), lo = fp16((x - hi) 1024)),
// or FP16 ones that the tensor maps cannot take (addresses or strides off 16
// bytes) as they are: rows of `dpad` values, zeros past the head dimension,
// head by head, so that a tile is one run of memory.
// Each value is read once; the kernel above then reads every row once for
// each 256 query rows.  Even CTAs: k, odd ones: v.
struct Stage {
    const void* src[2];
    int64_t token[2], head[2];
    uint16_t* hi[2];
    uint16_t* lo[2];
    int64_t tokens;
    int heads, dim, dpad, f32, vec;
};

__global__ void __launch_bounds__(256) attn_stage_kernel(Stage p)
{
    grid_dependency_launch();
    grid_dependency_wait();
    const int w = blockIdx.x & 1, parts = p.dpad / 8;
    const int64_t work = p.tokens * p.heads * parts;
    for (int64_t u = static_cast<int64_t>(blockIdx.x / 2) * blockDim.x + threadIdx.x; u < work;
         u += static_cast<int64_t>(gridDim.x / 2) * blockDim.x) {
        const int part = static_cast<int>(u % parts);
        const int64_t row = u / parts, at = row / p.heads * p.token[w] + row % p.heads * p.head[w] + part * 8;
        const int64_t to = (row % p.heads * p.tokens + row / p.heads) * p.dpad + part * 8;
        if (p.f32) {
            const float* const src = static_cast<const float*>(p.src[w]) + at;
            float x[8];
            if (p.vec && part * 8 + 8 <= p.dim) {
                const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = part * 8 + i < p.dim ? src[i] : 0.0f;
            }
            uint4 hi, lo;
            split2(x[0], x[1], hi.x, lo.x);
            split2(x[2], x[3], hi.y, lo.y);
            split2(x[4], x[5], hi.z, lo.z);
            split2(x[6], x[7], hi.w, lo.w);
            *reinterpret_cast<uint4*>(p.hi[w] + to) = hi;
            *reinterpret_cast<uint4*>(p.lo[w] + to) = lo;
        } else {
            const uint16_t* const src = static_cast<const uint16_t*>(p.src[w]) + at;
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = part * 8 + 2 * i < p.dim ? src[2 * i] : 0;
                const uint32_t b = part * 8 + 2 * i + 1 < p.dim ? src[2 * i + 1] : 0;
                x[i] = a | (b << 16);
            }
            *reinterpret_cast<uint4*>(p.hi[w] + to) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
}

// Whether a tensor map can describe [tokens, heads] rows with these strides.
bool map_legal(int64_t tokens, int64_t heads, int64_t token, int64_t head)
{
    const auto ok = [](int64_t extent, int64_t stride) {
        return extent <= 1 || (stride > 0 && stride % 8 == 0 && stride < (1ll << 38));
    };
    return ok(tokens, token) && ok(heads, head);
}

// FP32 [tokens, heads, dim] as boxes of `rows` rows that are whole tokens of
// `group` heads, `width` values of each: q's halves (dense) or out's warps (32
// values, 128-byte swizzled).  The box's tokens, or 0 if there is no such map.
int encode_tokens(CUtensorMap* map, const float* base, int dim, int heads, int group, int64_t tokens, int64_t token,
                  int64_t head, int rows, int width, bool vec)
{
    const auto ok = [](int64_t extent, int64_t stride) {
        return extent <= 1 || (stride > 0 && stride % 4 == 0 && stride < (1ll << 37));
    };
    EncodeTiledFn fn = encode_fn();
    if (!fn || !vec || rows % group != 0 || !ok(tokens, token) || !ok(heads, head))
        return 0;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head * 4 : 512),
                                   static_cast<cuuint64_t>(tokens > 1 ? token * 4 : 512)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(group),
                               static_cast<cuuint32_t>(rows / group)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const bool done = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         rows == 128 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    return done ? rows / group : 0;
}

template <int DP, int PL, bool PAIR = false, bool FOLD = false>
comp_status_t launch_t(const CUtensorMap (&maps)[6], const Params& p, int64_t grid, const DeviceInfo& dev,
                       cudaStream_t stream)
{
    using C = Cfg<DP, PL, PAIR, FOLD>;
    static std::mutex mu;
    static bool done[64] = {};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev.device < 0 || dev.device >= 64)
            return COMP_ERR_CUDA;
        if (!done[dev.device]) {
            if (cudaFuncSetAttribute(attn_tc_kernel<DP, PL, PAIR, FOLD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(C::kSmem)) != cudaSuccess) {
                (void)cudaGetLastError();
                return COMP_ERR_CUDA;
            }
            done[dev.device] = true;
        }
    }
    return launch_pdl_cluster(attn_tc_kernel<DP, PL, PAIR, FOLD>, C::R, static_cast<int>(grid) * C::R, kThreads,
                              C::kSmem, stream, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], p);
}

int64_t pad8(int64_t d)
{
    return (d + 7) / 8 * 8;
}

}  // namespace

// Planes that a call stages: k and v, two each if they are FP32; 0 if the
// caller's own FP16 rows can be loaded.
int64_t attn_stage_bytes(const comp_attn_t& a, int kv_bytes, const void* k, const void* v)
{
    if (a.total_k == 0 || a.n_seq == 0)
        return 0;
    if (kv_bytes == 2 && aligned16(k) && aligned16(v) && map_legal(a.total_k, a.kv_heads, a.k_token, a.k_head) &&
        map_legal(a.total_k, a.kv_heads, a.v_token, a.v_head))
        return 0;
    return (kv_bytes == 4 ? 4 : 2) * 2 * a.total_k * a.kv_heads * pad8(a.head_dim);
}

comp_status_t launch_attn(const comp_attn_t& a, const float* q, const void* k, const void* v, int kv_bytes,
                          const int32_t* cu_q, const int32_t* cu_k, float* out, float* lse, void* workspace,
                          const DeviceInfo& dev, cudaStream_t stream)
{
    Params p{};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.v = v;
    p.v_token = a.v_token;
    p.v_head = a.v_head;
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.out_token = a.out_token;
    p.out_head = a.out_head;
    p.n_seq = static_cast<int>(a.n_seq);
    p.total_q = static_cast<int>(a.total_q);
    p.total_k = static_cast<int>(a.total_k);
    p.kv_heads = a.kv_heads;
    p.group = a.heads / a.kv_heads;
    p.dim = a.head_dim;
    p.causal = a.causal;
    p.splits = 1;
    p.v_f32 = kv_bytes == 4;
    p.scale = a.scale;
    p.vec_q = a.q_token % 4 == 0 && a.q_head % 4 == 0 && a.head_dim % 4 == 0 && aligned16(q);
    p.vec_out = a.out_token % 4 == 0 && a.out_head % 4 == 0 && a.head_dim % 4 == 0 && aligned16(out);

    CUtensorMap maps[6] = {};
    const int box_rows = a.head_dim > 64 && kv_bytes == 4 ? 64 : 128;  // Cfg::BN
    if (a.total_k > 0) {
        const void* planes[4] = {k, v, nullptr, nullptr};
        int64_t token[2] = {a.k_token, a.v_token}, head[2] = {a.k_head, a.v_head}, dim = a.head_dim;
        if (attn_stage_bytes(a, kv_bytes, k, v) > 0) {
            const int64_t dpad = pad8(a.head_dim), plane = a.total_k * a.kv_heads * dpad;
            uint16_t* const ws = static_cast<uint16_t*>(workspace);
            Stage s{{k, v}, {a.k_token, a.v_token}, {a.k_head, a.v_head}, {ws, ws + plane},
                    {ws + 2 * plane, ws + 3 * plane}, a.total_k, a.kv_heads, a.head_dim, static_cast<int>(dpad),
                    kv_bytes == 4, 0};
            s.vec = aligned16(k) && aligned16(v) && a.k_token % 4 == 0 && a.v_token % 4 == 0 && a.k_head % 4 == 0 &&
                    a.v_head % 4 == 0;
            const int64_t work = a.total_k * a.kv_heads * (dpad / 8), most = dev.sm_count * 8;
            const int64_t blocks = (work + 255) / 256;
            const int grid = static_cast<int>(2 * (blocks < most ? blocks : most));
            const comp_status_t st = launch_pdl(attn_stage_kernel, grid, 256, 0, stream, s);
            if (st != COMP_OK)
                return st;
            for (int i = 0; i < 2; ++i) {
                planes[i] = s.hi[i];
                planes[2 + i] = s.lo[i];
                token[i] = dpad;
                head[i] = a.total_k * dpad;
            }
            dim = dpad;
        }
        for (int i = 0; i < (kv_bytes == 4 ? 4 : 2); ++i)
            if (!encode_rows(&maps[i], planes[i], dim, a.total_k, a.kv_heads, token[i % 2], head[i % 2], box_rows))
                return COMP_ERR_CUDA;
    }
    p.q_tokens = encode_tokens(&maps[4], q, p.dim, a.heads, p.group, a.total_q, a.q_token, a.q_head, 128, p.dim,
                               p.vec_q);
    p.out_tokens = encode_tokens(&maps[5], out, p.dim, a.heads, p.group, a.total_q, a.out_token, a.out_head, 32, 32,
                                 p.vec_out);
    const int64_t rows = a.total_q * p.group;
    // pairs of CTAs where the sequences fill their 512 rows on average (Cfg)
    const bool pair = a.head_dim > 64 && kv_bytes == 4 && rows >= 1024 * a.n_seq;
    const int64_t block = pair ? 512 : 256;
    // n rows have at most (n + block - 1) / block blocks; the tokens beyond the last sequence are one more
    const int64_t grid = (rows + (cu_q ? a.n_seq + 1 : 1) * (block - 1)) / block * a.kv_heads;
    if (pair)
        return launch_t<128, 2, true>(maps, p, grid, dev, stream);
    if (a.head_dim <= 64)
        return kv_bytes == 4 ? launch_t<64, 2>(maps, p, grid, dev, stream)
                             : launch_t<64, 1>(maps, p, grid, dev, stream);
    return kv_bytes == 4 ? launch_t<128, 2>(maps, p, grid, dev, stream)
                         : launch_t<128, 1>(maps, p, grid, dev, stream);
}

comp_status_t launch_attn_prefix(const comp_kv_cache_t& cache, const float* q, int64_t q_token, int64_t q_head,
                                 int heads, float scale, const int32_t* table, int64_t batch, const int32_t* lengths,
                                 int64_t shared, int splits, bool fold, float* out, float* lse, const DeviceInfo& dev,
                                 cudaStream_t stream)
{
    Params p{};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.v = cache.v;
    p.table = table;
    p.lengths = lengths;
    p.q_token = q_token;
    p.q_head = q_head;
    p.out_token = static_cast<int64_t>(heads) * cache.head_dim;
    p.out_head = cache.head_dim;
    p.lse_split = batch * heads;
    p.out_split = p.lse_split * cache.head_dim;
    p.n_seq = 1;
    p.total_q = static_cast<int>(batch);
    p.total_k = static_cast<int>(shared * cache.page_size);
    p.kv_heads = cache.kv_heads;
    p.group = heads / cache.kv_heads;
    p.dim = cache.head_dim;
    p.splits = fold ? splits / 2 : splits;
    p.page_size = cache.page_size;
    p.table_pages = static_cast<int>(shared);
    p.pages = static_cast<int>(cache.pages);
    p.scale = scale;
    p.vec_q = q_token % 4 == 0 && q_head % 4 == 0 && aligned16(q);
    p.vec_out = 1;
    CUtensorMap maps[6] = {};
    if (!encode_pages(&maps[0], cache.k, cache, cache.page_size) ||
        !encode_pages(&maps[1], cache.v, cache, cache.page_size))
        return COMP_ERR_CUDA;
    p.q_tokens = encode_tokens(&maps[4], q, p.dim, heads, p.group, batch, q_token, q_head, 128, p.dim, p.vec_q);
    p.out_tokens = encode_tokens(&maps[5], out, p.dim, heads, p.group, batch * splits, p.out_token, p.out_head, 32,
                                 32, true);
    p.out_part = static_cast<int>(batch);
    const int64_t grid = (batch * p.group + 255) / 256 * cache.kv_heads * p.splits;
    if (fold)
        return launch_t<64, 1, false, true>(maps, p, grid, dev, stream);
    return cache.head_dim <= 64 ? launch_t<64, 1>(maps, p, grid, dev, stream)
                                : launch_t<128, 1>(maps, p, grid, dev, stream);
}

comp_status_t read_and_clear_attn_fault(cudaStream_t stream, uint32_t* where)
{
    return read_and_clear_word(&g_attn_fault_word, stream, where);
}

}  // namespace compfp32
