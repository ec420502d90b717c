// The C calls of the attention operators: argument checks.
#include <cmath>

#include "internal.h"
#include "rope.cuh"

namespace compfp32 {
namespace {

struct Range {
    const void* p;
    int64_t n;
};

// No output shares memory with an input or another output.
template <int N, int M>
bool apart(const Range (&in)[N], const Range (&outs)[M])
{
    for (int i = 0; i < M; ++i) {
        for (const Range& x : in)
            if (overlap(outs[i].p, outs[i].n, x.p, x.n))
                return false;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return false;
    }
    return true;
}

constexpr int64_t kMostAttnKeys = INT32_MAX - 255;  // a tile's end is an int too
constexpr int64_t kMostAttnUnits = 1 << 29;  // sequences times key/value heads: blocks are counted in ints

struct AttnBytes {
    int64_t q, k, v, out, lse;
};

bool attn_ok(const comp_attn_t* a, int kv_bytes, AttnBytes* b)
{
    if (!a || a->n_seq < 0 || a->n_seq > INT32_MAX || a->total_q < 0 || a->total_q > INT32_MAX || a->total_k < 0 ||
        a->total_k > kMostAttnKeys || a->heads <= 0 || a->kv_heads <= 0 || a->heads > 65535 ||
        a->heads % a->kv_heads != 0 || a->head_dim < 1 || a->head_dim > 128 || !std::isfinite(a->scale) ||
        !(a->scale > 0.0f) || a->total_q * a->heads > INT32_MAX ||
        a->n_seq * a->kv_heads > kMostAttnUnits)
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
    if (a->total_q == 0)
        return COMP_OK;
    comp_attn_t seen = *a;
    if (a->n_seq == 0)
        seen.total_k = 0;  // no sequence has the keys
    if (!q || !out || (seen.total_k > 0 && (!k || !v)))
        return COMP_ERR_INVALID_VALUE;
    const int64_t cu = cu_q ? 4 * (a->n_seq + 1) : 0;
    const Range in[] = {{q, b.q}, {k, b.k}, {v, b.v}, {cu_q, cu}, {cu_k, cu}};
    const Range outs[] = {{out, b.out}, {lse, lse ? b.lse : 0}, {workspace, workspace_bytes}};
    if (!apart(in, outs))
        return COMP_ERR_INVALID_VALUE;
    const int64_t need = comp_attn_workspace_bytes(a, kv_bytes, k, v);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    return launch_attn(seen, q, k, v, kv_bytes, cu_q, cu_k, out, lse, workspace, dev,
                       static_cast<cudaStream_t>(stream));
}

// The sizes of a decode call over a cache of either type, which is checked already;
// per_row: what a row takes of the line of tiles beside its tiles of 16.
template <typename Cache>
bool decode_sizes_ok(const Cache* c, int64_t batch, int32_t heads, int64_t width, int per_row, int64_t* entries)
{
    return batch >= 0 && heads > 0 && heads <= 65535 && heads % c->kv_heads == 0 &&
           width >= 0 && width <= INT32_MAX / (2 * c->page_size) && mul_ok(batch, width, entries) &&
           batch <= INT32_MAX / heads && *entries <= INT64_MAX / 8 &&
           attn_decode_countable(c->kv_heads, c->page_size, batch, heads, width, per_row);
}

bool decode_ok(const comp_kv_cache_t* c, int64_t batch, int32_t heads, int64_t width, int64_t shared_pages,
               int64_t* bytes, int64_t* entries)
{
    return kv_cache_ok(c, bytes) && decode_sizes_ok(c, batch, heads, width, 1, entries) && shared_pages >= 0 &&
           shared_pages <= width;
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
    if (!decode_ok(cache, batch, heads, width, shared_pages, &bytes, &entries) || batch == 0)
        return 0;
    return attn_decode_bytes(*cache, batch, heads, shared_pages);
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
    if (!q || !lengths || !out || (entries > 0 && (!table || cache->pages == 0)))
        return COMP_ERR_INVALID_VALUE;
    const Range in[] = {{q, qb}, {cache->k, bytes}, {cache->v, bytes}, {table, 4 * entries}, {lengths, 4 * batch}};
    const Range outs[] = {{out, 4 * batch * heads * cache->head_dim}, {lse, lse ? 4 * batch * heads : 0},
                {workspace, workspace_bytes}};
    if (!apart(in, outs))
        return COMP_ERR_INVALID_VALUE;
    const int64_t need = comp_attn_decode_workspace_bytes(cache, batch, heads, width, shared_pages);
    if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    return launch_attn_decode(*cache, q, q_token, q_head, heads, scale, table, batch, width, lengths, shared_pages,
                              out, lse, workspace, dev, static_cast<cudaStream_t>(stream));
}

int64_t comp_attn_decode_f32x8_workspace_bytes(const comp_kv8_cache_t* cache, int64_t batch, int32_t heads,
                                               int64_t width)
{
    int64_t bytes, scales, entries;
    if (!kv8_cache_ok(cache, &bytes, &scales) || !decode_sizes_ok(cache, batch, heads, width, 4, &entries) ||
        batch == 0)
        return 0;
    return attn_decode8_bytes(*cache, heads);
}

comp_status_t comp_attn_decode_f32x8(const comp_kv8_cache_t* cache, const float* q, int64_t q_token, int64_t q_head,
                                     int32_t heads, float scale, const int32_t* table, int64_t batch, int64_t width,
                                     const int32_t* lengths, const comp_rope_t* rope, float* out, float* lse,
                                     void* workspace, int64_t workspace_bytes, comp_stream_t stream)
{
    int64_t bytes, scales, entries, qb, rb;
    if (!kv8_cache_ok(cache, &bytes, &scales) || !decode_sizes_ok(cache, batch, heads, width, 4, &entries) ||
        !std::isfinite(scale) || !(scale > 0.0f) || workspace_bytes < 0 ||
        !strided_bytes(batch, heads, cache->head_dim, q_token, q_head, 4, &qb) ||
        !rope_ok(rope, cache->head_dim, &rb))
        return COMP_ERR_INVALID_VALUE;
    if (batch == 0)
        return COMP_OK;
    if (!q || !lengths || !out || (entries > 0 && (!table || cache->pages == 0)))
        return COMP_ERR_INVALID_VALUE;
    const Range in[] = {{q, qb}, {cache->k, bytes}, {cache->v, bytes}, {cache->k_scale, scales},
                        {cache->v_scale, scales}, {table, 4 * entries}, {lengths, 4 * batch},
                        {rope ? rope->table : nullptr, rb}};
    const Range outs[] = {{out, 4 * batch * heads * cache->head_dim}, {lse, lse ? 4 * batch * heads : 0},
                {workspace, workspace_bytes}};
    if (!apart(in, outs))
        return COMP_ERR_INVALID_VALUE;
    const int64_t need = attn_decode8_bytes(*cache, heads);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
        return COMP_ERR_INVALID_VALUE;
    DeviceInfo dev;
    const comp_status_t st = current_device(&dev);
    if (st != COMP_OK)
        return st;
    return launch_attn_decode8(*cache, q, q_token, q_head, heads, scale, table, batch, width, lengths, rope, out, lse,
                               workspace, dev, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
