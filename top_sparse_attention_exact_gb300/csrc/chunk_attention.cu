// chunk_attention.cu -- causal attention of ragged new tokens over a cache.
#include <algorithm>

#include "prompt.cuh"

namespace retopk {

// One warp takes one (token, query head): four elements of the head a lane,
// the running maximum and sum of the softmax over one key at a time.
__global__ void __launch_bounds__(128) chunk_attention_kernel(const AttnArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + threadIdx.x / 32, t = blockIdx.x;
    if (h >= a.Hq)
        return;
    int b = t, i = 0, n = 1;
    if (a.cu) {
        for (b = 0; b < a.B && a.cu[b + 1] <= t; ++b)
            ;
        if (b >= a.B || a.cu[b] > t)
            return;
        i = t - a.cu[b];
        n = a.cu[b + 1] - a.cu[b];
    }
    const int L = max(0, min(a.seqlens[b], a.capacity)), pos = L - n + i;
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const uint2 qu = *reinterpret_cast<const uint2 *>(a.q + t * a.q_stride + h * kD + lane * 4);
    const float q[4] = {bf16lo(qu.x), bf16hi(qu.x), bf16lo(qu.y), bf16hi(qu.y)};
    float m = -INFINITY, l = 0.f, o[4] = {};
    for (int j = lo; j <= pos; ++j) {
        const long long row = cache_row(a.cache, b, h / a.G, j, a.status);
        if (row < 0)
            continue;
        const uint2 k = *reinterpret_cast<const uint2 *>(static_cast<uint16_t *>(a.cache.k) + row * kD + lane * 4);
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<uint16_t *>(a.cache.v) + row * kD + lane * 4);
        float s = warp_sum(q[0] * bf16lo(k.x) + q[1] * bf16hi(k.x) + q[2] * bf16lo(k.y) + q[3] * bf16hi(k.y));
        s *= a.scale;
        if (a.softcap > 0.f)
            s = a.softcap * tanhf(s / a.softcap);
        const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * c + p;
        o[0] = o[0] * c + p * bf16lo(v.x);
        o[1] = o[1] * c + p * bf16hi(v.x);
        o[2] = o[2] * c + p * bf16lo(v.y);
        o[3] = o[3] * c + p * bf16hi(v.y);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + h * kD + lane * 4) =
        make_uint2(bf16x2(o[0] * inv, o[1] * inv), bf16x2(o[2] * inv, o[3] * inv));
    if (a.lse && lane == 0)
        a.lse[(size_t)t * a.Hq + h] = m + logf(l);
}

size_t chunk_attention_ws(int T, int B, int Hq, int Hkv)
{
    return 256;
}

cudaError_t launch_chunk_attention(const AttnArgs &a, cudaStream_t st)
{
    return launch_pdl(chunk_attention_kernel, dim3(a.T, (a.Hq + 3) / 4), dim3(128), 0, st, 1, a);
}

cudaError_t configure_chunk_attention() { return cudaSuccess; }

}  // namespace retopk
