// Attention: argument checks, dispatch, and a plain kernel for any case.
#include <cuda_fp16.h>

#include <cmath>

#include "internal.h"

namespace compfp32 {
namespace {

constexpr int kRowWarps = 4;

// Where a key or value row is: in a packed tensor or on a page.
struct Source {
    const void* k;
    const void* v;
    int64_t k_token, k_head, v_token, v_head;
    int f32;
    // paged: table row, page size (0: packed)
    const int32_t* table;
    int64_t width, pages;
    int page_size, kv_heads, dim;
};

__device__ __forceinline__ float load_at(const void* base, int64_t i, int f32)
{
    return f32 ? static_cast<const float*>(base)[i] : __half2float(static_cast<const __half*>(base)[i]);
}

struct Rows {
    const float* q;
    float* out;
    float* lse;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* lengths;  // decode: keys of each row
    int64_t n_seq, total_q, total_k, q_token, q_head, out_token, out_head;
    int heads, group, dim, causal;
    float scale;
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi)
{
    return x < lo ? lo : (x > hi ? hi : x);
}

// One warp for each query row; lanes hold the head dimension.
__global__ void __launch_bounds__(32 * kRowWarps) attn_rows_kernel(Rows p, Source s)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row >= p.total_q * p.heads)
        return;
    const int64_t t = row / p.heads;
    const int h = static_cast<int>(row % p.heads), g = h / p.group;
    int64_t first = 0, seen = 0;
    if (p.lengths) {
        seen = clamp64(p.lengths[t], 0, s.width * s.page_size);
    } else {
        int64_t q0 = 0, q1 = p.total_q, k1 = p.total_k;
        if (p.cu_q) {
            int64_t lo = 0, hi = p.n_seq - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) / 2;
                if (p.cu_q[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            q0 = clamp64(p.cu_q[lo], 0, p.total_q);
            q1 = clamp64(p.cu_q[lo + 1], 0, p.total_q);
            first = clamp64(p.cu_k[lo], 0, p.total_k);
            k1 = clamp64(p.cu_k[lo + 1], first, p.total_k);
        }
        seen = k1 - first;
        if (p.causal)
            seen = clamp64(t - q0 + 1 + seen - (q1 - q0), 0, seen);
        if (t < q0 || t >= q1)
            return;
    }
    float q[4], o[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = lane + 32 * i < p.dim ? p.q[t * p.q_token + h * p.q_head + lane + 32 * i] : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j < seen; ++j) {
        int64_t ka, va;
        bool there = true;
        if (s.page_size) {
            const int64_t page = s.table[t * s.width + j / s.page_size];
            there = page >= 0 && page < s.pages;
            ka = va = ((page * s.kv_heads + g) * s.page_size + j % s.page_size) * s.dim;
        } else {
            ka = (first + j) * s.k_token + g * s.k_head;
            va = (first + j) * s.v_token + g * s.v_head;
        }
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (there && lane + 32 * i < p.dim)
                x = fmaf(q[i], load_at(s.k, ka + lane + 32 * i, s.f32), x);
#pragma unroll
        for (int o2 = 16; o2; o2 >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, o2);
        x *= p.scale;
        const float m2 = fmaxf(m, x), a = m == -INFINITY ? 0.0f : expf(m - m2), e = expf(x - m2);
        l = l * a + e;
        m = m2;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = o[i] * a +
                   e * (there && lane + 32 * i < p.dim ? load_at(s.v, va + lane + 32 * i, s.f32) : 0.0f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < p.dim)
            p.out[t * p.out_token + h * p.out_head + lane + 32 * i] = seen > 0 ? o[i] / l : 0.0f;
    if (p.lse && lane == 0)
        p.lse[t * p.heads + h] = seen > 0 ? m + logf(l) : -INFINITY;
}

comp_status_t launch_rows(const Rows& p, const Source& s, cudaStream_t stream)
{
    const int64_t blocks = (p.total_q * p.heads + kRowWarps - 1) / kRowWarps;
    attn_rows_kernel<<<static_cast<unsigned>(blocks), 32 * kRowWarps, 0, stream>>>(p, s);
    return launch_status();
}

// Whether the rows of a [tokens, heads, dim] output do not overlap each other.
bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head)
{
    return (tokens <= 1 && (heads <= 1 || head >= dim)) || (heads <= 1 && token >= dim) ||
           (head >= dim && token >= (heads - 1) * head + dim) ||
           (token >= dim && head >= (tokens - 1) * token + dim);
}

struct AttnBytes {
    int64_t q, k, v, out, lse;
};

bool attn_ok(const comp_attn_t* a, int kv_bytes, AttnBytes* b)
{
    if (!a || a->n_seq < 0 || a->n_seq > INT32_MAX || a->total_q < 0 || a->total_q > INT32_MAX || a->total_k < 0 ||
        a->total_k > INT32_MAX || a->heads <= 0 || a->kv_heads <= 0 || a->heads > 65535 ||
        a->heads % a->kv_heads != 0 || a->head_dim < 1 || a->head_dim > 128 || !std::isfinite(a->scale) ||
        !(a->scale > 0.0f) || a->total_q * a->heads > INT32_MAX)
        return false;
    if (!strided_bytes(a->total_q, a->heads, a->head_dim, a->q_token, a->q_head, 4, &b->q) ||
        !strided_bytes(a->total_k, a->kv_heads, a->head_dim, a->k_token, a->k_head, kv_bytes, &b->k) ||
        !strided_bytes(a->total_k, a->kv_heads, a->head_dim, a->v_token, a->v_head, kv_bytes, &b->v) ||
        !strided_bytes(a->total_q, a->heads, a->head_dim, a->out_token, a->out_head, 4, &b->out) ||
        !rows_apart(a->total_q, a->heads, a->head_dim, a->out_token, a->out_head))
        return false;
    b->lse = 4 * a->total_q * a->heads;
    return true;
}

comp_status_t attn(const comp_attn_t* a, const float* q, const void* k, const void* v, int kv_bytes,
                   const int32_t* cu_q, const int32_t* cu_k, float* out, float* lse, void* workspace,
                   int64_t workspace_bytes, comp_stream_t stream)
{
    AttnBytes b;
    if (!attn_ok(a, kv_bytes, &b) || (cu_q == nullptr) != (cu_k == nullptr) || (!cu_q && a->n_seq > 1) ||
        workspace_bytes < 0)
        return COMP_ERR_INVALID_VALUE;
    if (a->total_q == 0 || a->n_seq == 0)
        return COMP_OK;
    if (!q || !out || (b.k > 0 && (!k || !v)))
        return COMP_ERR_INVALID_VALUE;
    const int64_t cu = cu_q ? 4 * (a->n_seq + 1) : 0;
    const struct {
        const void* p;
        int64_t n;
    } in[] = {{q, b.q}, {k, b.k}, {v, b.v}, {cu_q, cu}, {cu_k, cu}},
      outs[] = {{out, b.out}, {lse, lse ? b.lse : 0}, {workspace, workspace_bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& x : in)
            if (overlap(outs[i].p, outs[i].n, x.p, x.n))
                return COMP_ERR_INVALID_VALUE;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return COMP_ERR_INVALID_VALUE;
    }
    const int64_t need = comp_attn_workspace_bytes(a, kv_bytes, k, v);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    return launch_attn(*a, q, k, v, kv_bytes, cu_q, cu_k, out, lse, workspace, dev, static_cast<cudaStream_t>(stream));
}

bool decode_ok(const comp_kv_cache_t* c, int64_t batch, int32_t heads, int64_t width, int64_t shared_pages,
               int64_t* bytes, int64_t* entries)
{
    return kv_cache_ok(c, bytes) && batch >= 0 && heads > 0 && heads <= 65535 && heads % c->kv_heads == 0 &&
           width >= 0 && width <= INT32_MAX / (2 * c->page_size) && mul_ok(batch, width, entries) &&
           batch <= INT32_MAX / heads && *entries <= INT64_MAX / 8 && shared_pages >= 0 && shared_pages <= width;
}

}  // namespace
}  // namespace compfp32

using namespace compfp32;

extern "C" {

int64_t comp_attn_workspace_bytes(const comp_attn_t* a, int kv_bytes, const void* k, const void* v)
{
    AttnBytes b;
    if ((kv_bytes != 2 && kv_bytes != 4) || !attn_ok(a, kv_bytes, &b))
        return 0;
    return attn_stage_bytes(*a, kv_bytes, k, v);
}

comp_status_t comp_attn_f32x16(const comp_attn_t* a, const float* q, const uint16_t* k, const uint16_t* v,
                               const int32_t* cu_q, const int32_t* cu_k, float* out, float* lse, void* workspace,
                               int64_t workspace_bytes, comp_stream_t stream)
{
    return attn(a, q, k, v, 2, cu_q, cu_k, out, lse, workspace, workspace_bytes, stream);
}

comp_status_t comp_attn_f32(const comp_attn_t* a, const float* q, const float* k, const float* v,
                            const int32_t* cu_q, const int32_t* cu_k, float* out, float* lse, void* workspace,
                            int64_t workspace_bytes, comp_stream_t stream)
{
    return attn(a, q, k, v, 4, cu_q, cu_k, out, lse, workspace, workspace_bytes, stream);
}

int64_t comp_attn_decode_workspace_bytes(const comp_kv_cache_t* cache, int64_t batch, int32_t heads, int64_t width,
                                         int64_t shared_pages)
{
    int64_t bytes, entries;
    if (!decode_ok(cache, batch, heads, width, shared_pages, &bytes, &entries))
        return 0;
    return 0;
}

comp_status_t comp_attn_decode_f32x16(const comp_kv_cache_t* cache, const float* q, int64_t q_token, int64_t q_head,
                                      int32_t heads, float scale, const int32_t* table, int64_t batch,
                                      int64_t width, const int32_t* lengths, int64_t shared_pages, float* out,
                                      float* lse, void* workspace, int64_t workspace_bytes, comp_stream_t stream)
{
    int64_t bytes, entries, qb;
    if (!decode_ok(cache, batch, heads, width, shared_pages, &bytes, &entries) || !std::isfinite(scale) ||
        !(scale > 0.0f) || workspace_bytes < 0 ||
        !strided_bytes(batch, heads, cache->head_dim, q_token, q_head, 4, &qb))
        return COMP_ERR_INVALID_VALUE;
    if (batch == 0)
        return COMP_OK;
    if (!q || !lengths || !out || (entries > 0 && !table))
        return COMP_ERR_INVALID_VALUE;
    const struct {
        const void* p;
        int64_t n;
    } in[] = {{q, qb}, {cache->k, bytes}, {cache->v, bytes}, {table, 4 * entries}, {lengths, 4 * batch}},
      outs[] = {{out, 4 * batch * heads * cache->head_dim}, {lse, lse ? 4 * batch * heads : 0},
                {workspace, workspace_bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& x : in)
            if (overlap(outs[i].p, outs[i].n, x.p, x.n))
                return COMP_ERR_INVALID_VALUE;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return COMP_ERR_INVALID_VALUE;
    }
    const int64_t need = comp_attn_decode_workspace_bytes(cache, batch, heads, width, shared_pages);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    Rows p{q, out, lse, nullptr, nullptr, lengths, batch, batch, 0, q_token, q_head,
           static_cast<int64_t>(heads) * cache->head_dim, cache->head_dim, heads, heads / cache->kv_heads,
           cache->head_dim, 0, scale};
    Source s{cache->k, cache->v, 0, 0, 0, 0, 0, table, width, cache->pages, cache->page_size, cache->kv_heads,
             cache->head_dim};
    return launch_rows(p, s, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
