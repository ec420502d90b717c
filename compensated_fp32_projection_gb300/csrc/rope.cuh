// Rotary positions as the kernels apply them: the pair (a, b) turns into
// (a c - b s, b c + a s), each operation a binary32 operation rounded to nearest
// even and never fused, so that every kernel that rotates gives the same bits.
#pragma once

#include "internal.h"

namespace compfp32 {

constexpr int kMostRopeDim = 65536;

// The pair's first or second value: x c - y s, or x c + y s.
__device__ __forceinline__ float turn(float x, float c, float y, float s, bool second)
{
    const float a = __fmul_rn(x, c), b = __fmul_rn(y, s);
    return second ? __fadd_rn(a, b) : __fsub_rn(a, b);
}

// Where the angles of a position are (nullptr: the table does not have it).
__device__ __forceinline__ const float* angles_of(const comp_rope_t& r, int64_t position)
{
    return position >= 0 && position < r.positions ? r.table + position * r.rot : nullptr;
}

// The angles of two pairs that stand together, (c, s) each.  wide: on 16 bytes.
__device__ __forceinline__ float4 load_angles(const float* at, bool wide)
{
    if (wide)
        return __ldg(reinterpret_cast<const float4*>(at));
    const float2 a = __ldg(reinterpret_cast<const float2*>(at)), b = __ldg(reinterpret_cast<const float2*>(at + 2));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Whether a position's angles stand on 16 bytes.
inline bool angles_wide(const comp_rope_t& r)
{
    return (reinterpret_cast<uintptr_t>(r.table) & 15u) == 0 && r.rot % 4 == 0;
}

// Four values of a head from dimension d on (a multiple of 4), rotated: x is the
// head, `at` the position's angles.  vec: x is 16-byte aligned; wide: `at` is.
__device__ __forceinline__ float4 load_rotated(const float* x, int d, const comp_rope_t& r, const float* at, bool vec,
                                               bool wide)
{
    float v[4];
    if (vec) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(x + d));
        v[0] = f.x;
        v[1] = f.y;
        v[2] = f.z;
        v[3] = f.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = __ldg(x + d + e);
    }
    if (d < r.rot) {
        if (!at) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = d + e < r.rot ? __int_as_float(0x7fffffff) : v[e];
        } else if (r.interleaved) {
            // rot is even: a pair is rotated or not
            if (wide) {
                const float4 cs = load_angles(at + d, true);
                const float a = v[0], b = v[1], e = v[2], f = v[3];
                v[0] = turn(a, cs.x, b, cs.y, false);
                v[1] = turn(b, cs.x, a, cs.y, true);
                v[2] = turn(e, cs.z, f, cs.w, false);
                v[3] = turn(f, cs.z, e, cs.w, true);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    if (d + e < r.rot) {
                        const float2 cs = __ldg(reinterpret_cast<const float2*>(at + d + e));
                        const float a = v[e], b = v[e + 1];
                        v[e] = turn(a, cs.x, b, cs.y, false);
                        v[e + 1] = turn(b, cs.x, a, cs.y, true);
                    }
            }
        } else {
            const int half = r.rot / 2;
            if (half % 4 == 0) {  // d and its partners lie in one half each
                const bool second = d >= half;
                const int i = second ? d - half : d, partner = second ? i : d + half;
                float y[4];
                if (vec) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(x + partner));
                    y[0] = f.x;
                    y[1] = f.y;
                    y[2] = f.z;
                    y[3] = f.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __ldg(x + partner + e);
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float4 cs = load_angles(at + 2 * (i + e), wide);
                    v[e] = turn(v[e], cs.x, y[e], cs.y, second);
                    v[e + 1] = turn(v[e + 1], cs.z, y[e + 1], cs.w, second);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < r.rot) {
                        const bool second = d + e >= half;
                        const int i = second ? d + e - half : d + e;
                        const float2 cs = __ldg(reinterpret_cast<const float2*>(at + 2 * i));
                        v[e] = turn(v[e], cs.x, __ldg(x + (second ? i : i + half)), cs.y, second);
                    }
            }
        }
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// Whether a descriptor is one that the kernels take for heads of this size (NULL
// is, and rotates nothing), and the bytes of its table.
inline bool rope_ok(const comp_rope_t* r, int64_t head_dim, int64_t* bytes)
{
    *bytes = 0;
    if (!r)
        return true;
    if (r->rot < 2 || r->rot % 2 != 0 || r->rot > head_dim || r->positions < 0 ||
        !mul_ok(r->positions, 4 * static_cast<int64_t>(r->rot), bytes))
        return false;
    return *bytes == 0 || (r->table && (reinterpret_cast<uintptr_t>(r->table) & 7u) == 0);
}

}  // namespace compfp32
