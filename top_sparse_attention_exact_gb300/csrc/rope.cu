// rope.cu -- norm and rotation of the query and key heads of ragged new
// tokens, with the write of their key and value rows into a cache.
//
// Per head x (128 elements): x <- x * rsqrt(mean(x^2) + eps) * w, then the
// pairs (a, b) turn by t = pos * inv_freq: a cos t - b sin t, b cos t + a sin t.
// One block takes one token: its cosines and sines are made once, and every head
// of the token (16 lanes a head, 16 bytes a lane) uses them from shared memory.
// Memory bound: each element is read and written once.
#include <algorithm>

#include "prompt.cuh"

namespace retopk {

__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a)
{
    __shared__ float2 turn[kD / 2];   // (cos, sin)
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, n_thr = blockDim.x, t = blockIdx.x;
    // the lengths after this call (a separate buffer)
    if (a.seqlens_out)
        for (int b = blockIdx.x * n_thr + tid; b < a.B; b += gridDim.x * n_thr) {
            const int n = a.cu ? a.cu[b + 1] - a.cu[b] : 1, L = a.seqlens[b];
            a.seqlens_out[b] = L >= 0 && n >= 0 && (long long)L + n <= a.capacity ? L + n : L;
        }
    // the token's sequence
    int b = t, i = 0, n = 1;
    if (a.cu && !(t < a.B && a.cu[t] == t && a.cu[t + 1] == t + 1)) {
        b = 0;
        for (int base = 0; base < a.B; base += n_thr)
            b += __syncthreads_count(base + tid < a.B && a.cu[base + tid + 1] <= t);
        if (b >= a.B || a.cu[b] > t)
            return;
        i = t - a.cu[b];
        n = a.cu[b + 1] - a.cu[b];
        if (i >= n)   // offsets that decrease: the token is in no sequence
            return;
    }
    const int L = a.seqlens[b], pos = L + i;
    // angles: whole turns are taken off in 64 bits
    const int half = a.rope.rot_dim / 2;
    for (int j = tid; j < half; j += n_thr) {
        const double turns = (double)pos * ((double)a.rope.inv_freq[j] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        turn[j] = make_float2(c, s);
    }
    __syncthreads();
    const bool fits = L >= 0 && (long long)L + n <= a.capacity;
    if (a.v && !fits && i == 0 && tid == 0 && a.status)
        atomicOr(a.status, RETOPK_STATUS_KV_FULL);
    const int lane = tid & 15, rows = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
    const int step = n_thr / 16;
    // rounded up so that whole warps take part in the shuffles
    for (int r0 = tid / 16; r0 < (rows + 1) / 2 * 2; r0 += step) {
        const int r = min(r0, rows - 1);
        const bool isq = r < a.Hq, isv = r >= a.Hq + a.Hkv;
        const int h = isq ? r : isv ? r - a.Hq - a.Hkv : r - a.Hq;
        const uint16_t *src = isq ? a.q + t * a.q_stride : isv ? a.v + t * a.v_stride : a.k + t * a.k_stride;
        uint4 u = *reinterpret_cast<const uint4 *>(src + h * kD + lane * 8);
        float x[8];
        unpack8(u, x);
        const uint16_t *w = isv ? nullptr : isq ? a.rope.q_weight : a.rope.k_weight;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += x[e] * x[e];
#pragma unroll
        for (int o = 8; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (w) {
            const float f = rsqrtf(sum * (1.f / kD) + a.rope.eps);
            const uint4 wu = *reinterpret_cast<const uint4 *>(w + lane * 8);
            float wv[8];
            unpack8(wu, wv);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = x[e] * f * wv[e];
        }
        if (half) {
            const int first = lane * 8;
            if (a.rope.interleaved) {
                if (first < 2 * half && !isv) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 cs = turn[(first + e) / 2];
                        const float p = x[e], o = x[e + 1];
                        x[e] = p * cs.x - o * cs.y;
                        x[e + 1] = o * cs.x + p * cs.y;
                    }
                }
            } else {
                // the partner's 8 elements are half / 8 lanes away
                const bool low = first < half, in = first < 2 * half;
                const int other = (tid & 16) + (in ? (low ? lane + half / 8 : lane - half / 8) : lane);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = __shfl_sync(0xffffffffu, x[e], other);
                    if (in && !isv) {
                        const float2 cs = turn[low ? first + e : first + e - half];
                        x[e] = low ? x[e] * cs.x - y * cs.y : x[e] * cs.x + y * cs.y;
                    }
                }
            }
        }
        if (isq) {
            if (r0 < rows)
                *reinterpret_cast<uint4 *>(a.q_out + ((size_t)t * a.Hq + h) * kD + lane * 8) = pack8(x);
        } else if (!a.v) {
            if (r0 < rows)
                *reinterpret_cast<uint4 *>(a.k_out + ((size_t)t * a.Hkv + h) * kD + lane * 8) = pack8(x);
        }
        if (!a.v)
            continue;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (isq || !fits || r0 >= rows)
            continue;
        const long long row = cache_row(a.cache, b, h, pos, a.status);
        if (row < 0)
            continue;
        if (a.cache.format == RETOPK_CACHE_BF16) {
            uint16_t *dst = static_cast<uint16_t *>(isv ? a.cache.v : a.cache.k) + row * kD;
            *reinterpret_cast<uint4 *>(dst + lane * 8) = isv ? u : pack8(x);
        } else {
            const uint32_t sc = mx_scale(m);
            const float f = mx_inverse(sc);
            uint8_t *dst = static_cast<uint8_t *>(isv ? a.cache.v : a.cache.k) + row * kD;
            const uint32_t c0 = e4m3x2(x[0] * f, x[1] * f) | e4m3x2(x[2] * f, x[3] * f) << 16;
            const uint32_t c1 = e4m3x2(x[4] * f, x[5] * f) | e4m3x2(x[6] * f, x[7] * f) << 16;
            *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(c0, c1);
            if ((lane & 3) == 0)
                (isv ? a.cache.v_scale : a.cache.k_scale)[row * kMxScales + lane / 4] = (uint8_t)sc;
        }
    }
}

// seqlens_out from seqlens, in place or not, behind the rows' kernel.
__global__ void advance_kernel(const RopeArgs a)
{
    pdl_wait();
    pdl_trigger();
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x) {
        const int n = a.cu ? a.cu[b + 1] - a.cu[b] : 1, L = a.seqlens[b];
        a.seqlens_out[b] = L >= 0 && n >= 0 && (long long)L + n <= a.capacity ? L + n : L;
    }
}

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st)
{
    const int rows = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
    const int threads = std::min(256, (rows * 16 + 31) / 32 * 32);
    return launch_pdl(rope_kernel, dim3(a.T), dim3(threads), 0, st, 1, a);
}

cudaError_t launch_advance(const RopeArgs &a, cudaStream_t st)
{
    return launch_pdl(advance_kernel, dim3(std::min(64, (a.B + 127) / 128)), dim3(128), 0, st, 1, a);
}

}  // namespace retopk
