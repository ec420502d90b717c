// Rotary positions: the table of angles and the rotation of packed heads.
//
// The table holds m (cos p f_i, sin p f_i) for pair i of rot / 2, angles and
// functions in 64 bits, rounded once: p f_i of a far position loses nothing that
// 32 bits show.  It is made once for a model: 131072 positions of 128 dimensions take
// 540 us, by the GPU's rate of 64-bit operations (to write them alone takes 10).
//
// The rotation streams: 8 bytes a value and no reuse, so HBM is the bound.  A
// thread holds the angles of a few pairs of one token in registers and goes
// through four of its heads, whose loads are all in flight together: the table
// is read once for four heads, and by all heads of a token in one CTA.  16384
// tokens of 40 heads of 128 take 97 us, 7.0 TB/s, and 4999 tokens of 20 heads of 96
// 14.3; with eight heads at once 98 and 18.8, with two 105 and 15.8.
#include <cmath>

#include "internal.h"
#include "rope.cuh"
#include "tc_util.cuh"

namespace compfp32 {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;       // heads that a thread goes through at once
constexpr int kMostThreads = 512;

struct Frequencies {
    double base, factor, context, low, high, magnitude;
};

__global__ void __launch_bounds__(kThreads) rope_table_kernel(Frequencies f, int half, int64_t first, int64_t positions,
                                                              float* table)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x / half;  // positions at once
    const int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int i = static_cast<int>(u % half);
    if (u / half >= step)
        return;
    double freq = pow(f.base, -static_cast<double>(i) / half);
    double keep = 0.0;
    if (f.context > 0.0) {
        const double turns = f.context * freq / 6.283185307179586;
        keep = fmin(fmax((turns - f.low) / (f.high - f.low), 0.0), 1.0);
    }
    freq *= keep + (1.0 - keep) / f.factor;
    for (int64_t p = u / half; p < positions; p += step) {
        double s, c;
        sincos(static_cast<double>(first + p) * freq, &s, &c);
        *reinterpret_cast<float2*>(table + (p * half + i) * 2) =
            make_float2(static_cast<float>(f.magnitude * c), static_cast<float>(f.magnitude * s));
    }
}

struct Params {
    comp_rope_t rope;
    const float* x;
    const int32_t* positions;
    float* out;
    int64_t x_token, x_head, out_token, out_head, tokens;
    int heads, dim, inverse, wide;
    int turning, units, chunks, tokens_a_cta;  // units of a head that turn, and all; of kHeads heads
};

template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&v)[N])
{
    if constexpr (N == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else if constexpr (N == 2) {  // of a half: on 8 bytes; of a pair: anywhere
        v[0] = p[0];
        v[1] = p[1];
    } else {
        v[0] = *p;
    }
}

template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&v)[N])
{
    if constexpr (N == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            p[e] = v[e];
    }
}

// A unit of work: REST values of a head that do not turn; P pairs that do, N values
// one after the other (interleaved, N = 2 P) or N = P from each half.  x and out
// may be the same, so loads are plain ones, all of a unit's before its stores.
template <int P, bool INTER, int REST>
__global__ void __launch_bounds__(kMostThreads) rope_kernel(const Params p)
{
    constexpr int N = INTER ? 2 * P : P;
    grid_dependency_launch();
    const int each = p.units * p.chunks;
    const int half = p.rope.rot / 2;
    for (int u = threadIdx.x; u < each * p.tokens_a_cta; u += blockDim.x) {
        const int64_t token = static_cast<int64_t>(blockIdx.x) * p.tokens_a_cta + u / each;
        if (token >= p.tokens)
            return;
        const int unit = u % each % p.units, h0 = u % each / p.units * kHeads;
        const int n = min(kHeads, p.heads - h0);
        const float* const x = p.x + token * p.x_token + h0 * p.x_head;
        float* const out = p.out + token * p.out_token + h0 * p.out_head;
        if (unit >= p.turning) {
            const int d = p.rope.rot + (unit - p.turning) * REST;
            float v[kHeads][REST];
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                if (h < n)
                    load_n<REST>(x + h * p.x_head + d, v[h]);
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                if (h < n)
                    store_n<REST>(out + h * p.out_head + d, v[h]);
            continue;
        }
        // the values first: what they turn by takes two loads, one after the other
        const int i = unit * P;  // the first pair
        float a[kHeads][N], b[kHeads][N];  // interleaved: a only
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
            if (h < n) {
                load_n<N>(x + h * p.x_head + (INTER ? 2 * i : i), a[h]);
                if constexpr (!INTER)
                    load_n<N>(x + h * p.x_head + half + i, b[h]);
            }
        const int64_t position = p.positions ? p.positions[token] : token;
        const float* const at = angles_of(p.rope, position);
        float c[P], s[P];
        const float nan = __int_as_float(0x7fffffff);
        if constexpr (P == 1) {
            const float2 cs = at ? __ldg(reinterpret_cast<const float2*>(at + 2 * i)) : make_float2(nan, nan);
            c[0] = cs.x;
            s[0] = p.inverse ? -cs.y : cs.y;
        } else {
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                const float4 cs = at ? load_angles(at + 2 * (i + e), p.wide) : make_float4(nan, nan, nan, nan);
                c[e] = cs.x;
                s[e] = p.inverse ? -cs.y : cs.y;
                c[e + 1] = cs.z;
                s[e + 1] = p.inverse ? -cs.w : cs.w;
            }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
            if (h < n) {
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    float& first = INTER ? a[h][2 * e] : a[h][e];
                    float& second = INTER ? a[h][2 * e + 1] : b[h][e];
                    const float y = first, z = second;
                    first = turn(y, c[e], z, s[e], false);
                    second = turn(z, c[e], y, s[e], true);
                }
                store_n<N>(out + h * p.out_head + (INTER ? 2 * i : i), a[h]);
                if constexpr (!INTER)
                    store_n<N>(out + h * p.out_head + half + i, b[h]);
            }
    }
}

template <int P, bool INTER, int REST>
comp_status_t launch_t(Params p, cudaStream_t stream)
{
    p.turning = p.rope.rot / 2 / P;
    p.units = p.turning + (p.dim - p.rope.rot) / REST;
    p.chunks = (p.heads + kHeads - 1) / kHeads;
    const int64_t each = static_cast<int64_t>(p.units) * p.chunks;
    p.tokens_a_cta = each >= kThreads ? 1 : static_cast<int>(kThreads / each);
    const int64_t ctas = (p.tokens + p.tokens_a_cta - 1) / p.tokens_a_cta;
    const int64_t work = each * p.tokens_a_cta;
    const int threads = static_cast<int>(work < kMostThreads ? (work + 31) / 32 * 32 : kMostThreads);
    rope_kernel<P, INTER, REST><<<static_cast<unsigned>(ctas), threads, 0, stream>>>(p);
    return launch_status();
}

}  // namespace
}  // namespace compfp32

using namespace compfp32;

extern "C" {

comp_status_t comp_rope_table(const comp_rope_angles_t* a, int32_t rot, int64_t first, int64_t positions,
                              float* table, comp_stream_t stream)
{
    int64_t values;
    if (!a || rot < 2 || rot % 2 != 0 || first < 0 || positions < 0 || first > INT32_MAX ||
        positions > INT32_MAX || !mul_ok(positions, rot, &values) || !std::isfinite(a->base) || !(a->base > 0.0) ||
        !std::isfinite(a->factor) || !(a->factor > 0.0) || !std::isfinite(a->magnitude) ||
        !std::isfinite(a->context) || a->context < 0.0 || rot > kMostRopeDim)
        return COMP_ERR_INVALID_VALUE;
    if (a->context > 0.0 && !(std::isfinite(a->low) && std::isfinite(a->high) && a->high > a->low))
        return COMP_ERR_INVALID_VALUE;
    if (positions == 0)
        return COMP_OK;
    if (!table || (reinterpret_cast<uintptr_t>(table) & 7u) != 0)
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    const int half = rot / 2;
    // at least one position at once
    const int64_t least = (half + kThreads - 1) / kThreads, want = (values / 2 + kThreads - 1) / kThreads;
    int64_t ctas = static_cast<int64_t>(dev.sm_count) * 8;
    ctas = want < ctas ? want : ctas;
    ctas = ctas < least ? least : ctas;
    rope_table_kernel<<<static_cast<unsigned>(ctas), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        Frequencies{a->base, a->factor, a->context, a->low, a->high, a->magnitude}, half, first, positions, table);
    return launch_status();
}

comp_status_t comp_rope_f32(const comp_rope_t* rope, const float* x, int64_t x_token, int64_t x_head, int64_t tokens,
                            int32_t heads, int32_t head_dim, const int32_t* positions, int inverse, float* out,
                            int64_t out_token, int64_t out_head, comp_stream_t stream)
{
    int64_t table, xb, ob;
    if (!rope || head_dim < 1 || head_dim > kMostRopeDim || heads < 1 || heads > 65535 || tokens < 0 ||
        tokens > INT32_MAX || !rope_ok(rope, head_dim, &table) ||
        !strided_bytes(tokens, heads, head_dim, x_token, x_head, 4, &xb) ||
        !strided_bytes(tokens, heads, head_dim, out_token, out_head, 4, &ob) ||
        !rows_apart(tokens, heads, head_dim, out_token, out_head))
        return COMP_ERR_INVALID_VALUE;
    if (tokens == 0)
        return COMP_OK;
    const bool in_place = out == x && out_token == x_token && out_head == x_head;
    const int64_t pb = positions ? 4 * tokens : 0;
    if (!x || !out || (!in_place && overlap(out, ob, x, xb)) || overlap(out, ob, positions, pb) ||
        overlap(out, ob, rope->table, table))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    Params p{};
    p.rope = *rope;
    p.x = x;
    p.positions = positions;
    p.out = out;
    p.x_token = x_token;
    p.x_head = x_head;
    p.out_token = out_token;
    p.out_head = out_head;
    p.tokens = tokens;
    p.heads = heads;
    p.dim = head_dim;
    p.inverse = inverse != 0;
    p.wide = angles_wide(*rope);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // four values at once where every row begins on 16 bytes and its parts are multiples
    // of four (of two for each half)
    const auto rows16 = [](const float* at, int64_t token, int64_t head) {
        return aligned16(at) && token % 4 == 0 && head % 4 == 0;
    };
    const bool vec = rows16(x, x_token, x_head) && rows16(out, out_token, out_head) && head_dim % 4 == 0 &&
                     rope->rot % 4 == 0;
    if (rope->interleaved)
        return vec ? launch_t<2, true, 4>(p, s) : launch_t<1, true, 1>(p, s);
    if (!vec)
        return launch_t<1, false, 1>(p, s);
    return rope->rot % 8 == 0 ? launch_t<4, false, 4>(p, s) : launch_t<2, false, 4>(p, s);
}

}  // extern "C"
