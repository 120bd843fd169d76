// prompt_api.cu -- the prompt-side entry points of include/retopk.h (rotated
// append, cache copy, chunk attention): argument checks and launches.
#include <math.h>

#include "prompt.cuh"

using namespace retopk;

namespace {

constexpr int kMaxTokens = 1 << 22;
constexpr int kMaxBatch = 65535;
constexpr int kMaxHeads = 1024;
constexpr long long kMaxTokenHeads = 1ll << 30;   // heads of all tokens: 256 GB of rows

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_cache(const retopk_cache *c, int B)
{
    if (!c || !c->k || !c->v || c->n_pages < 1 || c->n_kv_heads < 1 || c->page_rows < 1)
        return RETOPK_ERR_INVALID;
    if (c->format != RETOPK_CACHE_BF16 && c->format != RETOPK_CACHE_MX8)
        return RETOPK_ERR_INVALID;
    if (c->format == RETOPK_CACHE_MX8 && (!c->k_scale || !c->v_scale))
        return RETOPK_ERR_INVALID;
    if (c->table ? c->table_width < 1 || c->page_rows % 16 != 0 : c->n_pages < B)
        return RETOPK_ERR_INVALID;
    if (c->n_kv_heads > kMaxHeads || cache_capacity(*c) > kMaxLen ||
        (long long)c->n_pages * c->n_kv_heads >= INT32_MAX)
        return RETOPK_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4) ||
        (c->format == RETOPK_CACHE_MX8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
        return RETOPK_ERR_ALIGN;
    return RETOPK_OK;
}

int check_tokens(int T, int B, int Hq, int Hkv, const int32_t *cu, const int32_t *seqlens)
{
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !seqlens || (!cu && T != B))
        return RETOPK_ERR_INVALID;
    if (T > kMaxTokens || B > kMaxBatch || Hq > kMaxHeads || Hq / Hkv > kMaxGroup ||
        (long long)T * (Hq + 2 * Hkv) > kMaxTokenHeads)
        return RETOPK_ERR_UNSUPPORTED;
    if (!aligned(cu, 4) || !aligned(seqlens, 4))
        return RETOPK_ERR_ALIGN;
    return RETOPK_OK;
}

// Bytes of a cache's keys (or values).
size_t pool_bytes(const retopk_cache &c)
{
    return (size_t)c.n_pages * c.n_kv_heads * c.page_rows * kD * (c.format == RETOPK_CACHE_MX8 ? 1 : 2);
}

// A strided [T, heads, 128] tensor.
int check_rows(const void *p, int64_t stride, int heads)
{
    if (!p || stride < (int64_t)heads * kD || stride > INT32_MAX)
        return RETOPK_ERR_INVALID;
    return aligned(p, 16) && stride % 8 == 0 ? RETOPK_OK : RETOPK_ERR_ALIGN;
}

// Bytes [p, p + n) and [q, q + m).
bool meet(const void *p, size_t n, const void *q, size_t m)
{
    return (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n;
}

// Whether two strided [T, heads, 128] tensors share an element; of two whose rows lie between each other's, those of one
// stride are told apart, others count as sharing.
bool rows_meet(const void *p, int64_t ps, int pheads, const void *q, int64_t qs, int qheads, int T)
{
    const int64_t pw = (int64_t)pheads * kD * 2, qw = (int64_t)qheads * kD * 2;   // bytes
    if (!meet(p, (T - 1) * ps * 2 + pw, q, (T - 1) * qs * 2 + qw))
        return false;
    if (ps != qs || T == 1)
        return true;
    const int64_t s = ps * 2, d = (((int64_t)((uintptr_t)q - (uintptr_t)p)) % s + s) % s;
    return d < pw || d + qw > s;
}

// An output of rows that are one of the inputs', row for row, or share nothing with it.
bool may_write(const void *out, int64_t out_stride, const void *in, int64_t in_stride, int heads, int T)
{
    return (out == in && (out_stride == in_stride || T == 1)) ||
           !rows_meet(out, out_stride, heads, in, in_stride, heads, T);
}

int check_rope(const retopk_rope *r)
{
    if (!r || r->rot_dim < 0 || (r->rot_dim > 0 && !r->inv_freq) || !(r->eps >= 0.f) || isinf(r->eps))
        return RETOPK_ERR_INVALID;
    if (r->rot_dim > kD || r->rot_dim % 16 != 0)
        return RETOPK_ERR_UNSUPPORTED;
    return aligned(r->q_weight, 16) && aligned(r->k_weight, 16) && aligned(r->inv_freq, 4) ? RETOPK_OK
                                                                                              : RETOPK_ERR_ALIGN;
}

}  // namespace

extern "C" {

int retopk_qk_rope(const retopk_rope *rope, const retopk_bf16 *q, int64_t q_stride, const retopk_bf16 *k,
                   int64_t k_stride, const int32_t *cu_tokens, int T, int B, int Hq, int Hkv,
                   const int32_t *seqlens, retopk_bf16 *q_out, retopk_bf16 *k_out, void *stream)
{
    int e;
    if ((e = check_rope(rope)) || (e = check_tokens(T, B, Hq, Hkv, cu_tokens, seqlens)))
        return e;
    if (T == 0)
        return RETOPK_OK;
    if ((e = check_rows(q, q_stride, Hq)) || (e = check_rows(k, k_stride, Hkv)))
        return e;
    if (!q_out || !k_out || (q_out == q && q_stride != (int64_t)Hq * kD) ||
        (k_out == k && k_stride != (int64_t)Hkv * kD))
        return RETOPK_ERR_INVALID;
    if (!aligned(q_out, 16) || !aligned(k_out, 16))
        return RETOPK_ERR_ALIGN;
    const int64_t qw = (int64_t)Hq * kD, kw = (int64_t)Hkv * kD;
    if (!may_write(q_out, qw, q, q_stride, Hq, T) || !may_write(k_out, kw, k, k_stride, Hkv, T) ||
        rows_meet(q_out, qw, Hq, k, k_stride, Hkv, T) || rows_meet(k_out, kw, Hkv, q, q_stride, Hq, T) ||
        rows_meet(q_out, qw, Hq, k_out, kw, Hkv, T))
        return RETOPK_ERR_INVALID;
    if ((e = ensure_configured()))
        return e;
    RopeArgs a{};
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.cu = cu_tokens;
    a.seqlens = seqlens;
    a.q_out = q_out;
    a.k_out = k_out;
    a.rope = *rope;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    return cuda_rc(launch_rope(a, (cudaStream_t)stream));
}

int retopk_qkv_append(const retopk_rope *rope, const retopk_bf16 *q, int64_t q_stride, const retopk_bf16 *k,
                      int64_t k_stride, const retopk_bf16 *v, int64_t v_stride, const int32_t *cu_tokens, int T,
                      int B, int Hq, const retopk_cache *cache, const int32_t *seqlens, int32_t *seqlens_out,
                      retopk_bf16 *q_out, uint32_t *d_status, void *stream)
{
    int e;
    if ((e = check_rope(rope)) || (e = check_cache(cache, B)) ||
        (e = check_tokens(T, B, Hq, cache->n_kv_heads, cu_tokens, seqlens)))
        return e;
    const int Hkv = cache->n_kv_heads;
    if (!seqlens_out)
        return RETOPK_ERR_INVALID;
    if (!aligned(seqlens_out, 4) || !aligned(d_status, 4))
        return RETOPK_ERR_ALIGN;
    if (T > 0) {
        if ((e = check_rows(q, q_stride, Hq)) || (e = check_rows(k, k_stride, Hkv)) ||
            (e = check_rows(v, v_stride, Hkv)))
            return e;
        if (!q_out || (q_out == q && q_stride != (int64_t)Hq * kD))
            return RETOPK_ERR_INVALID;
        if (!aligned(q_out, 16))
            return RETOPK_ERR_ALIGN;
        const int64_t qw = (int64_t)Hq * kD;
        if (!may_write(q_out, qw, q, q_stride, Hq, T) || rows_meet(q_out, qw, Hq, k, k_stride, Hkv, T) ||
            rows_meet(q_out, qw, Hq, v, v_stride, Hkv, T))
            return RETOPK_ERR_INVALID;
    }
    if (seqlens_out != seqlens && meet(seqlens_out, B * sizeof(int32_t), seqlens, B * sizeof(int32_t)))
        return RETOPK_ERR_INVALID;
    if ((e = ensure_configured()))
        return e;
    RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.cu = cu_tokens;
    a.seqlens = seqlens;
    a.q_out = q_out;
    a.status = d_status;
    a.rope = *rope;
    a.cache = *cache;
    a.capacity = cache_capacity(*cache);
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    const bool in_place = seqlens_out == seqlens;
    if (T > 0) {
        a.seqlens_out = in_place ? nullptr : seqlens_out;
        if ((e = cuda_rc(launch_rope(a, (cudaStream_t)stream))))
            return e;
    }
    // in place, the lengths advance once every block has read them
    if (T == 0 || in_place) {
        a.seqlens_out = seqlens_out;
        return cuda_rc(launch_advance(a, (cudaStream_t)stream));
    }
    return RETOPK_OK;
}

int retopk_cache_copy(const retopk_cache *src, const retopk_cache *dst, const int32_t *first, const int32_t *last,
                      int B, int max_rows, uint32_t *d_status, void *stream)
{
    int e;
    if (B < 1 || max_rows < 0 || !first || !last)
        return RETOPK_ERR_INVALID;
    if ((e = check_cache(src, B)) || (e = check_cache(dst, B)))
        return e;
    if (src->n_kv_heads != dst->n_kv_heads || src->k == dst->k || src->v == dst->v)
        return RETOPK_ERR_INVALID;
    if (B > kMaxBatch || max_rows > kMaxLen)
        return RETOPK_ERR_UNSUPPORTED;
    if (!aligned(first, 4) || !aligned(last, 4) || !aligned(d_status, 4))
        return RETOPK_ERR_ALIGN;
    if (max_rows == 0)
        return RETOPK_OK;
    for (const void *x : {src->k, src->v})
        for (const void *y : {dst->k, dst->v})
            if (meet(x, pool_bytes(*src), y, pool_bytes(*dst)))
                return RETOPK_ERR_INVALID;
    return cuda_rc(launch_cache_copy(*src, *dst, first, last, B, max_rows, d_status, (cudaStream_t)stream));
}

size_t retopk_chunk_attention_workspace_bytes(int T, int B, int Hq, int Hkv)
{
    if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || T > kMaxTokens || B > kMaxBatch ||
        Hq > kMaxHeads || Hq / Hkv > kMaxGroup)
        return 0;
    return chunk_attention_ws(T, Hq, Hkv);
}

int retopk_chunk_attention(const retopk_bf16 *q, int64_t q_stride, const retopk_cache *cache,
                           const int32_t *cu_tokens, int T, int B, int Hq, const int32_t *seqlens, float scale,
                           float softcap, int window, retopk_bf16 *out, int64_t out_stride, float *lse,
                           void *d_workspace, size_t bytes, uint32_t *d_status, void *stream)
{
    int e;
    if ((e = check_cache(cache, B)) || (e = check_tokens(T, B, Hq, cache->n_kv_heads, cu_tokens, seqlens)))
        return e;
    if (cache->format != RETOPK_CACHE_BF16)
        return RETOPK_ERR_UNSUPPORTED;
    if (!(scale >= 0.f) || isinf(scale) || !(softcap >= 0.f) || isinf(softcap) || window < 0)
        return RETOPK_ERR_INVALID;
    if (T == 0)
        return RETOPK_OK;
    if ((e = check_rows(q, q_stride, Hq)) || (e = check_rows(out, out_stride, Hq)))
        return e;
    if (!aligned(lse, 4) || !aligned(d_status, 4))
        return RETOPK_ERR_ALIGN;
    if (!d_workspace || !aligned(d_workspace, 256) ||
        bytes < retopk_chunk_attention_workspace_bytes(T, B, Hq, cache->n_kv_heads))
        return RETOPK_ERR_WORKSPACE;
    if (!may_write(out, out_stride, q, q_stride, Hq, T))
        return RETOPK_ERR_INVALID;
    if ((e = ensure_configured()))
        return e;
    AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.cu = cu_tokens;
    a.seqlens = seqlens;
    a.out = out;
    a.lse = lse;
    a.status = d_status;
    a.cache = *cache;
    a.capacity = (int)cache_capacity(*cache);
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.G = Hq / cache->n_kv_heads;
    a.window = window < kMaxLen ? window : 0;   // (a wider one hides nothing)
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)kD);
    a.softcap = softcap;
    a.ws = d_workspace;
    return cuda_rc(launch_chunk_attention(a, (cudaStream_t)stream));
}

}  // extern "C"
