// rope.cu -- norm and rotation of the query and key heads of ragged new
// tokens, with the write of their key and value rows into a cache.
//
// Per head x (128 elements): x <- x * rsqrt(mean(x^2) + eps) * w, then the
// pairs (a, b) turn by t = pos * inv_freq: a cos t - b sin t, b cos t + a sin t.
// Each element is read and written once, so the memory bounds it; what has to be
// kept small is the work for each.  A warp takes a token (or, where tokens are
// few, some of a token's heads), two heads at a time, 16 lanes a head: a lane
// holds two runs of four elements that are each other's partners, so the rotation
// needs no exchange, its cosines and sines stay in registers for all heads of the token,
// and so do its norm weights.
//
// Angles.  pos is whole, so only the fraction of inv_freq / 2 pi counts: it is kept
// as a 64-bit fixed-point number, and pos times it, modulo 2^64, is the fraction of the
// turns, off by less than 2^-32 turns at the farthest position.
#include <algorithm>
#include <type_traits>

#include "prompt.cuh"

namespace retopk {

constexpr int kRopeWarps = 8;
constexpr int kRopeBatch = 4;   // pairs of heads in flight in a warp

// The sequence that token t belongs to: the number of sequences that end at or
// before t, found by the warp in steps of 32.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int B, int t, int lane)
{
    int lo = 0, n = B;
    while (n > 32) {
        const int step = (n + 31) / 32, i = lo + min((lane + 1) * step, n) - 1;
        const int whole = __popc(__ballot_sync(0xffffffffu, cu[i + 1] <= t));
        lo += min(whole * step, n);
        n = min(step, n - whole * step);
        if (n <= 0)
            return B;
    }
    return lo + __popc(__ballot_sync(0xffffffffu, lane < n && cu[lo + lane + 1] <= t));
}

__device__ __forceinline__ int advanced(const RopeArgs &a, int b)
{
    const int n = a.cu ? a.cu[b + 1] - a.cu[b] : 1, L = a.seqlens[b];
    return L >= 0 && n >= 0 && (long long)L + n <= a.capacity ? L + n : L;
}

// Where the keys and values go.
enum { TO_ROWS = 0, TO_BF16 = 1, TO_MX8 = 2 };   // k_out (no values), a bf16 cache, an 8-bit cache

// A lane's part of the norm and the rotation, with the weights in it: partners a, b
// become f (a ac - b bs) and f (b bc + a as), f the norm's factor.
struct Turn {
    float ac[4], bs[4], bc[4], as[4];
};

// Element numbers of a lane's partners: in its two runs, or side by side.
template <bool INTER>
__device__ __forceinline__ constexpr int first_of(int e)
{
    return INTER ? 2 * e : e;
}
template <bool INTER>
__device__ __forceinline__ constexpr int second_of(int e)
{
    return INTER ? 2 * e + 1 : e + 4;
}

__device__ __forceinline__ void unpack4(const uint2 (&u)[2], float (&x)[8])
{
    x[0] = bf16lo(u[0].x), x[1] = bf16hi(u[0].x), x[2] = bf16lo(u[0].y), x[3] = bf16hi(u[0].y);
    x[4] = bf16lo(u[1].x), x[5] = bf16hi(u[1].x), x[6] = bf16lo(u[1].y), x[7] = bf16hi(u[1].y);
}

// `groups` warps share a token's heads; a warp takes `tokens` tokens one after
// another: its share of the query heads, then of the keys', then of the values'.
template <bool INTER, int TO>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_kernel(const __grid_constant__ RopeArgs a, int groups, int tokens)
{
    __shared__ float2 turns[kRopeWarps][kD / 2];                  // (cos, sin) of the warp's token
    __shared__ __align__(16) uint32_t tops[kRopeWarps][2][32];    // largest |x| of runs of four, for the scales
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, second = lane >> 4;
    if (a.seqlens_out)   // the lengths after this call (a separate buffer)
        for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
            a.seqlens_out[b] = advanced(a, b);
    const int unit = blockIdx.x * kRopeWarps + warp;
    const int nq = (a.Hq + 1) / 2, nk = (a.Hkv + 1) / 2, all = nq + nk + (TO ? nk : 0), each = (all + groups - 1) / groups;
    const int p0 = unit % groups * each, p1 = min(all, p0 + each);   // pairs of heads
    const int t0 = unit / groups * tokens, t1 = min(a.T, t0 + tokens);
    // this lane's two runs of four: partners in the rotation
    const int half = a.rope.rot_dim / 2;
    const bool turned = 4 * l < half;
    const int c0 = INTER ? 2 * l : turned ? l : half / 4 + l;
    const int c1 = INTER ? 2 * l + 1 : turned ? l + half / 4 : l + 16;
    // turns of pairs lane and lane + 32 by one position
    uint64_t phase[2] = {0, 0};
    if (p0 < nq + nk)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < half) {
                const double f = (double)a.rope.inv_freq[lane + 32 * i] * 0.15915494309189533577;
                phase[i] = (uint64_t)(int64_t)((f - rint(f)) * 4611686018427387904.0) << 2;   // 2^62, then 2^2
            }
    int b = -1, begin = 0, end = -1, L = 0;
    bool fits = false;
    for (int t = t0; t < t1; ++t) {
        if (t >= end) {
            if (!a.cu || (t < a.B && a.cu[t] == t && a.cu[t + 1] == t + 1)) {
                b = begin = t;
                end = t + 1;
            } else {
                b = sequence_of(a.cu, a.B, t, lane);
                begin = b < a.B ? a.cu[b] : INT32_MAX;
                end = b < a.B ? a.cu[b + 1] : -1;
            }
            if (begin <= t && t < end) {
                L = a.seqlens[b];
                fits = L >= 0 && (long long)L + (end - begin) <= a.capacity;
            }
        }
        if (begin > t || t >= end) {   // in no sequence
            end = -1;
            continue;
        }
        const int pos = L + (t - begin);
        if (TO && !fits && t == begin && p0 == 0 && lane == 0 && a.status)
            atomicOr(a.status, RETOPK_STATUS_KV_FULL);
        if (p0 < nq + nk && half) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < half) {
                    float s, c;
                    sincospif((float)(int32_t)(phase[i] * (uint64_t)(int64_t)pos >> 32) * 0x1p-31f, &s, &c);
                    turns[warp][lane + 32 * i] = make_float2(c, s);
                }
            __syncwarp();
        }
        // the row of this token in the cache, of head 0
        long long at = -1;
        if (TO && fits && p1 > nq)
            at = cache_row(a.cache, b, 0, pos, a.status);

        // heads 2 lo .. 2 hi of the queries (0), keys (1) or values (2)
        auto heads = [&](auto kind_, int lo, int hi) {
            constexpr int kind = decltype(kind_)::value;
            constexpr bool cached = TO && kind > 0, mx8 = TO == TO_MX8 && kind > 0;
            const int H = kind ? a.Hkv : a.Hq;
            const uint16_t *const src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride);
            const uint16_t *const w = kind == 2 ? nullptr : kind == 0 ? a.rope.q_weight : a.rope.k_weight;
            Turn tn;
            if (kind < 2) {
                float wx[8];
                uint2 u[2] = {make_uint2(0x3f803f80u, 0x3f803f80u), make_uint2(0x3f803f80u, 0x3f803f80u)};   // ones
                if (w) {
                    u[0] = *reinterpret_cast<const uint2 *>(w + 4 * c0);
                    u[1] = *reinterpret_cast<const uint2 *>(w + 4 * c1);
                }
                unpack4(u, wx);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 cs = turned ? turns[warp][4 * l + e] : make_float2(1.f, 0.f);
                    const float wa = wx[first_of<INTER>(e)], wb = wx[second_of<INTER>(e)];
                    tn.ac[e] = wa * cs.x, tn.bs[e] = wb * cs.y, tn.bc[e] = wb * cs.x, tn.as[e] = wa * cs.y;
                }
            }
            for (int p = lo; p < hi; p += kRopeBatch) {
                uint2 u[kRopeBatch][2];
#pragma unroll
                for (int i = 0; i < kRopeBatch; ++i) {
                    const uint16_t *row = src + min(2 * (p + i) + second, H - 1) * kD;
                    u[i][0] = *reinterpret_cast<const uint2 *>(row + 4 * c0);
                    u[i][1] = *reinterpret_cast<const uint2 *>(row + 4 * c1);
                }
#pragma unroll
                for (int i = 0; i < kRopeBatch; ++i) {
                    const int h = 2 * (p + i) + second;
                    const bool real = p + i < hi && h < H;
                    float y[8];
                    if (kind < 2 || mx8) {
                        float x[8];
                        unpack4(u[i], x);
                        if (kind == 2) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                y[e] = x[e];
                        } else {
                            float f = 1.f;
                            if (w) {
                                float sum = x[0] * x[0];
#pragma unroll
                                for (int e = 1; e < 8; ++e)
                                    sum = fmaf(x[e], x[e], sum);
#pragma unroll
                                for (int o = 8; o; o >>= 1)
                                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                                f = rsqrtf(fmaf(sum, 1.f / kD, a.rope.eps));
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float xa = x[first_of<INTER>(e)], xb = x[second_of<INTER>(e)];
                                y[first_of<INTER>(e)] = f * fmaf(xa, tn.ac[e], -(xb * tn.bs[e]));
                                y[second_of<INTER>(e)] = f * fmaf(xb, tn.bc[e], xa * tn.as[e]);
                            }
                        }
                    }
                    if (mx8) {
                        // the largest of each 32 elements: eight runs of four
                        uint32_t m0 = 0, m1 = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            m0 = max(m0, __float_as_uint(y[e]) & 0x7fffffffu);
                            m1 = max(m1, __float_as_uint(y[4 + e]) & 0x7fffffffu);
                        }
                        __syncwarp();
                        tops[warp][second][c0] = m0;
                        tops[warp][second][c1] = m1;
                        __syncwarp();
                        auto scale = [&](int c) {
                            const uint4 *q = reinterpret_cast<const uint4 *>(&tops[warp][second][c & 24]);
                            const uint4 v = q[0], z = q[1];
                            return mx_scale(max(max(max(v.x, v.y), max(v.z, v.w)), max(max(z.x, z.y), max(z.z, z.w))));
                        };
                        const uint32_t s0 = scale(c0), s1 = scale(c1);
                        const float f0 = mx_inverse(s0), f1 = mx_inverse(s1);
                        if (real && at >= 0) {
                            const long long row = at + (long long)h * a.cache.page_rows;
                            uint8_t *dst = static_cast<uint8_t *>(kind == 2 ? a.cache.v : a.cache.k) + row * kD;
                            uint8_t *sc = (kind == 2 ? a.cache.v_scale : a.cache.k_scale) + row * kMxScales;
                            *reinterpret_cast<uint32_t *>(dst + 4 * c0) = e4m3x2(y[0] * f0, y[1] * f0) | e4m3x2(y[2] * f0, y[3] * f0) << 16;
                            *reinterpret_cast<uint32_t *>(dst + 4 * c1) = e4m3x2(y[4] * f1, y[5] * f1) | e4m3x2(y[6] * f1, y[7] * f1) << 16;
                            if ((c0 & 7) == 0)
                                sc[c0 / 8] = (uint8_t)s0;
                            if ((c1 & 7) == 0)
                                sc[c1 / 8] = (uint8_t)s1;
                        }
                    } else if (real && (!cached || at >= 0)) {
                        if (kind < 2) {
                            u[i][0] = make_uint2(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]));
                            u[i][1] = make_uint2(bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
                        }
                        uint16_t *dst = kind == 0 ? a.q_out + ((size_t)t * a.Hq + h) * kD
                                        : !cached ? a.k_out + ((size_t)t * a.Hkv + h) * kD
                                                  : static_cast<uint16_t *>(kind == 2 ? a.cache.v : a.cache.k) +
                                                        (at + (long long)h * a.cache.page_rows) * kD;
                        *reinterpret_cast<uint2 *>(dst + 4 * c0) = u[i][0];
                        *reinterpret_cast<uint2 *>(dst + 4 * c1) = u[i][1];
                    }
                }
            }
        };
        if (p0 < nq)
            heads(std::integral_constant<int, 0>{}, p0, min(p1, nq));
        if (p0 < nq + nk && p1 > nq)
            heads(std::integral_constant<int, 1>{}, max(p0, nq) - nq, min(p1, nq + nk) - nq);
        if (TO && p1 > nq + nk)
            heads(std::integral_constant<int, 2>{}, max(p0, nq + nk) - nq - nk, p1 - nq - nk);
    }
}

// seqlens_out from seqlens, in place or not, behind the rows' kernel.
__global__ void advance_kernel(const RopeArgs a)
{
    pdl_wait();
    pdl_trigger();
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
        a.seqlens_out[b] = advanced(a, b);
}

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st)
{
    const int all = (a.Hq + 1) / 2 + (a.Hkv + 1) / 2 * (a.v ? 2 : 1);
    // a warp a token once that fills the GPU; with fewer tokens, up to one warp for two heads
    const int fill = sm_count() * 32, groups = std::max(1, std::min(all, (fill + a.T - 1) / std::max(1, a.T)));
    const int tokens = std::max(1, std::min(8, a.T / (2 * fill)));
    const long long units = (long long)((a.T + tokens - 1) / tokens) * groups;
    const bool i = a.rope.interleaved != 0;
    auto kernel = !a.v ? (i ? rope_kernel<true, TO_ROWS> : rope_kernel<false, TO_ROWS>)
                  : a.cache.format == RETOPK_CACHE_MX8 ? (i ? rope_kernel<true, TO_MX8> : rope_kernel<false, TO_MX8>)
                                                       : (i ? rope_kernel<true, TO_BF16> : rope_kernel<false, TO_BF16>);
    return launch_pdl(kernel, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)), dim3(kRopeWarps * 32), 0, st, 1, a,
                      groups, tokens);
}

cudaError_t launch_advance(const RopeArgs &a, cudaStream_t st)
{
    return launch_pdl(advance_kernel, dim3(std::min(64, (a.B + 127) / 128)), dim3(128), 0, st, 1, a);
}

}  // namespace retopk
