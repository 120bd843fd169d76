// rope.cu -- norm and rotation of the query and key heads of ragged new
// tokens, with the write of their key and value rows into a cache.
//
// Per head x (128 elements): x <- x * rsqrt(mean(x^2) + eps) * w, then the
// pairs (a, b) turn by t = pos * inv_freq: a cos t - b sin t, b cos t + a sin t.
// Each element is read and written once, so the memory bounds it; what has to be
// kept small is the work for each, and what has to be kept large the bytes on
// their way.  Batches of eight heads are shared out evenly, in the order of tokens,
// queries, keys, values, over the warps that fit on the GPU.  A warp has a ring of its
// own in shared memory, into which bulk copies bring up to four batches ahead.  It
// takes four heads at once, 8 lanes a head: a lane holds two runs of eight elements
// that are each other's partners, so the rotation needs no exchange, and its
// factors, weights included, stay in registers for all heads of the token.  The factors
// of a token are made once, two pairs a lane, and pass to the lanes that turn those
// pairs through shared memory.
//
// Measured (28 query, 4 KV heads): 131072 tokens into 8-bit pages 366 us, 6.2 TB/s, 92 % of a
// plain copy; 8191 ragged tokens into bf16 pages 30 us, 5.0 TB/s (5 us of it start and end); one
// token 3.8 us.  The large call was 443 us while every lane made the factors that it used from the
// weights anew, 403 with the factors in rows of 128 bytes that share their banks.
//
// Angles.  pos is whole, so only the fraction of inv_freq / 2 pi counts: it is kept
// as a 64-bit fixed-point number, and pos times it, modulo 2^64, is the fraction of the
// turns, off by less than 2^-32 turns at the farthest position.
#include <algorithm>
#include <type_traits>

#include "prompt.cuh"

namespace retopk {

constexpr int kRopeWarps = 8, kRopeBlocks = 2;   // of a block; of an SM
constexpr int kRopeHeads = 8;    // heads of a batch
constexpr int kRopeStages = 4;   // batches of a warp's ring

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
    const long long n = a.cu ? (long long)a.cu[b + 1] - a.cu[b] : 1, L = a.seqlens[b];
    return (int)(L >= 0 && n >= 0 && L + n <= a.capacity ? L + n : L);
}

// Where the keys and values go.
enum { TO_ROWS = 0, TO_BF16 = 1, TO_MX8 = 2 };   // k_out (no values), a bf16 cache, an 8-bit cache

// A lane's part of the norm and the rotation, with the weights in it: partners a, b
// become f (a ac - b bs) and f (b bc + a as), f the norm's factor.
struct Turn {
    float ac[8], bs[8], bc[8], as[8];
};

// Element numbers of a lane's partners: side by side, or in its two runs.
template <bool INTER>
__device__ __forceinline__ constexpr int first_of(int e)
{
    return INTER ? 2 * e : e;
}
template <bool INTER>
__device__ __forceinline__ constexpr int second_of(int e)
{
    return INTER ? 2 * e + 1 : e + 8;
}

struct __align__(16) RopeWarp {
    uint8_t ring[kRopeStages][kRopeHeads * kD * 2];
    float4 turns[2][8][9];     // the token's factors for queries and keys, as in Turn: pair 8 l + e at [e][l] (rows of
                               // 144 bytes: 8 lanes that write one column meet no bank twice)
    uint2 weights[kD / 2];     // of a pair: of queries, of keys; in each the two elements'
    uint64_t phase[kD / 2];    // of a pair: turns by one position
    uint32_t tops[4][16];      // largest |x| of runs of eight, for the scales
    uint64_t full[kRopeStages];
};

__device__ __forceinline__ void unpack16(const uint4 &u, const uint4 &v, float (&x)[16])
{
    float lo[8], hi[8];
    unpack8(u, lo);
    unpack8(v, hi);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = lo[e], x[8 + e] = hi[e];
}

// A warp takes `each` batches of the tokens' `T * all`.  FULL: all 128 elements turn, and none is looked at for having
// no partner (131072 tokens into 8-bit pages 403 us, in the kernel for any part 418; both since faster).
template <bool INTER, bool FULL, int TO>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeBlocks) rope_kernel(const __grid_constant__ RopeArgs a, int each)
{
    extern __shared__ __align__(16) unsigned char rope_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, which = lane >> 3;
    RopeWarp &sh = reinterpret_cast<RopeWarp *>(rope_smem)[warp];
    if (lane == 0) {
        for (int i = 0; i < kRopeStages; ++i)
            mbar_init(&sh.full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    if (a.seqlens_out)   // the lengths after this call (a separate buffer)
        for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
            a.seqlens_out[b] = advanced(a, b);
    const int nq = (a.Hq + kRopeHeads - 1) / kRopeHeads, nk = (a.Hkv + kRopeHeads - 1) / kRopeHeads;
    const int all = nq + nk + (TO ? nk : 0);
    const int i0 = min((long long)(blockIdx.x * kRopeWarps + warp) * each, (long long)a.T * all), i1 = min((long long)i0 + each, (long long)a.T * all);
    if (i0 >= i1)
        return;
    // batch `p` of token `t` into the ring (one lane)
    int ahead_t = i0 / all, ahead_p = i0 % all;
    uint32_t ahead = 0;
    auto copy_next = [&] {
        if (i0 + (int)ahead >= i1)
            return;
        const int p = ahead_p, stage = ahead % kRopeStages;
        const int first = (p < nq ? p : p < nq + nk ? p - nq : p - nq - nk) * kRopeHeads;
        const uint16_t *src = (p < nq ? a.q + ahead_t * a.q_stride : p < nq + nk ? a.k + ahead_t * a.k_stride : a.v + ahead_t * a.v_stride);
        const uint32_t bytes = min(kRopeHeads, (p < nq ? a.Hq : a.Hkv) - first) * kD * 2;
        mbar_expect_tx(&sh.full[stage], bytes);
        bulk_load(sh.ring[stage], src + first * kD, bytes, &sh.full[stage]);
        ++ahead;
        if (++ahead_p == all) {
            ahead_p = 0;
            ++ahead_t;
        }
    };
    if (lane == 0)
        for (int i = 0; i < kRopeStages; ++i)
            copy_next();
    // this lane's two runs of eight: partners in the rotation
    const int half = FULL ? kD / 2 : a.rope.rot_dim / 2;
    const bool turned = FULL || 8 * l < half;
    const int c0 = INTER ? 2 * l : turned ? l : half / 8 + l;
    const int c1 = INTER ? 2 * l + 1 : turned ? l + half / 8 : l + 8;
    // Pairs lane and lane + 32 are this lane's to make factors for: their turns by one position (none past the
    // rotated elements) and their weights, of queries and keys
    {
        float freq[2];
        uint2 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = lane + 32 * i;
            const int ea = INTER ? 2 * j : j < half ? j : j + half, eb = INTER ? 2 * j + 1 : j < half ? j + half : j + kD / 2;
            auto pair = [&](const uint16_t *w) { return w ? w[ea] | (uint32_t)w[eb] << 16 : 0x3f803f80u; };
            freq[i] = j < half ? a.rope.inv_freq[j] : 0.f;
            w[i] = make_uint2(pair(a.rope.q_weight), pair(a.rope.k_weight));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double f = (double)freq[i] * 0.15915494309189533577;
            sh.phase[lane + 32 * i] = (uint64_t)(int64_t)((f - rint(f)) * 4611686018427387904.0) << 2;   // 2^62, then 2^2
            sh.weights[lane + 32 * i] = w[i];
        }
    }
    int b = -1, begin = 0, end = -1, L = 0;
    bool fits = false, ok = true;
    long long at = -1;     // the row of the token in the cache, of head 0
    int in_page = 0;       // its row in the page; 0: to be looked up
    uint32_t used = 0;
    for (int i = i0, t = i0 / all; i < i1 && ok; i = ++t * all) {
        const int p0 = i - t * all, p1 = min(all, i1 - t * all);   // batches of this token
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
                fits = L >= 0 && (long long)L + end - begin <= a.capacity;   // (whatever the offsets: no row outside is written)
            }
            in_page = 0;
        }
        const bool in = begin <= t && t < end;
        if (in) {
            const int pos = (int)((uint32_t)L + (uint32_t)t - (uint32_t)begin);   // (of a sequence that fits: within the capacity)
            if (TO && !fits && t == begin && p0 == 0 && lane == 0 && a.status)
                atomicOr(a.status, RETOPK_STATUS_KV_FULL);
            if (p0 < nq + nk) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float s = 0.f, c = 1.f;
                    const uint2 w = sh.weights[lane + 32 * i];
                    if (32 * i < half)
                        sincospif((float)(int32_t)(sh.phase[lane + 32 * i] * (uint64_t)(int64_t)pos >> 32) * 0x1p-31f, &s, &c);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float wa = bf16lo(k ? w.y : w.x), wb = bf16hi(k ? w.y : w.x);
                        sh.turns[k][lane & 7][lane / 8 + 4 * i] = make_float4(wa * c, wb * s, wb * c, wa * s);
                    }
                }
                __syncwarp();
            }
            if (TO && p1 > nq) {
                if (in_page == 0 || in_page == a.cache.page_rows) {
                    in_page = pos % a.cache.page_rows;
                    at = fits ? cache_row(a.cache, b, 0, pos, a.status) : -1;
                } else {
                    at += at >= 0;
                }
                ++in_page;
            }
        } else {
            end = -1;
        }

        // batches lo .. hi of the queries (0), keys (1) or values (2)
        auto heads = [&](auto kind_, int lo, int hi) {
            constexpr int kind = decltype(kind_)::value;
            constexpr bool cached = TO && kind > 0, mx8 = TO == TO_MX8 && kind > 0;
            const int H = kind ? a.Hkv : a.Hq;
            const bool there = in && (!cached || at >= 0);
            const bool norm = kind < 2 && (kind == 0 ? a.rope.q_weight : a.rope.k_weight) != nullptr;
            Turn tn;
            if (kind < 2 && there) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 x = sh.turns[kind][e][l];
                    tn.ac[e] = x.x, tn.bs[e] = x.y, tn.bc[e] = x.z, tn.as[e] = x.w;
                }
            }
            // four heads of a batch, one for each quarter of the warp
            auto four = [&](const uint8_t *from, uint8_t *to, uint8_t *sc, bool real) {
                const uint4 u = *reinterpret_cast<const uint4 *>(from), v = *reinterpret_cast<const uint4 *>(from + 16 * (c1 - c0));
                if (kind == 2 && !mx8) {
                    if (real) {
                        *reinterpret_cast<uint4 *>(to) = u;
                        *reinterpret_cast<uint4 *>(to + 16 * (c1 - c0)) = v;
                    }
                    return;
                }
                float y[16];
                unpack16(u, v, y);
                if (kind < 2) {
                    float f = 1.f;
                    if (norm) {
                        float sum[4] = {};
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            sum[e & 3] = fmaf(y[e], y[e], sum[e & 3]);
                        sum[0] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
                        for (int o = 4; o; o >>= 1)
                            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
                        f = rsqrtf(fmaf(sum[0], 1.f / kD, a.rope.eps));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xa = y[first_of<INTER>(e)], xb = y[second_of<INTER>(e)];
                        float pa = xa, pb = xb;
                        if (!FULL)   // elements that do not turn have no partner
                            pa = turned ? pa : 0.f, pb = turned ? pb : 0.f;
                        y[first_of<INTER>(e)] = fmaf(xa, tn.ac[e], -(pb * tn.bs[e])) * f;
                        y[second_of<INTER>(e)] = fmaf(xb, tn.bc[e], pa * tn.as[e]) * f;
                    }
                }
                if (mx8) {
                    // the largest of each 32 elements: four runs of eight
                    uint32_t m0 = 0, m1 = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        m0 = max(m0, __float_as_uint(y[e]) & 0x7fffffffu);
                        m1 = max(m1, __float_as_uint(y[8 + e]) & 0x7fffffffu);
                    }
                    __syncwarp();
                    sh.tops[which][c0] = m0;
                    sh.tops[which][c1] = m1;
                    __syncwarp();
                    auto scale = [&](int c) {
                        const uint4 m = *reinterpret_cast<const uint4 *>(&sh.tops[which][c & 12]);
                        return mx_scale(max(max(m.x, m.y), max(m.z, m.w)));
                    };
                    const uint32_t s0 = scale(c0), s1 = scale(c1);
                    const float f0 = mx_inverse(s0), f1 = mx_inverse(s1);
                    if (real) {
                        *reinterpret_cast<uint2 *>(to) =
                            make_uint2(e4m3x2(y[0] * f0, y[1] * f0) | e4m3x2(y[2] * f0, y[3] * f0) << 16,
                                       e4m3x2(y[4] * f0, y[5] * f0) | e4m3x2(y[6] * f0, y[7] * f0) << 16);
                        *reinterpret_cast<uint2 *>(to + 8 * (c1 - c0)) =
                            make_uint2(e4m3x2(y[8] * f1, y[9] * f1) | e4m3x2(y[10] * f1, y[11] * f1) << 16,
                                       e4m3x2(y[12] * f1, y[13] * f1) | e4m3x2(y[14] * f1, y[15] * f1) << 16);
                        if ((c0 & 3) == 0)
                            sc[c0 / 4] = (uint8_t)s0;
                        if ((c1 & 3) == 0)
                            sc[c1 / 4] = (uint8_t)s1;
                    }
                } else if (real) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
                    *reinterpret_cast<uint4 *>(to + 16 * (c1 - c0)) =
                        make_uint4(bf16x2(y[8], y[9]), bf16x2(y[10], y[11]), bf16x2(y[12], y[13]), bf16x2(y[14], y[15]));
                }
            };
            // where this lane's elements of the first four heads go, and the step to the next four
            constexpr int size = mx8 ? 1 : 2;
            const long long first_row = cached ? at + (long long)(lo * kRopeHeads + which) * a.cache.page_rows
                                               : (long long)t * H + lo * kRopeHeads + which;
            uint8_t *to = static_cast<uint8_t *>(kind == 0 ? a.q_out : kind == 2 ? a.cache.v : TO ? a.cache.k : a.k_out) +
                          first_row * (kD * size) + 8 * size * c0;
            uint8_t *sc = mx8 ? (kind == 2 ? a.cache.v_scale : a.cache.k_scale) + first_row * kMxScales : nullptr;
            const long long step = (cached ? a.cache.page_rows : 1) * 4ll * kD * size;
            for (int p = lo; p < hi; ++p) {
                const int stage = used % kRopeStages;
                ok = __all_sync(0xffffffffu, wait_full(&sh.full[stage], (used / kRopeStages) & 1, a.status));
                if (!ok)
                    return;
                ++used;
                const int left = min(kRopeHeads, H - p * kRopeHeads);   // heads of the batch
                const uint8_t *from = sh.ring[stage] + which * kD * 2 + 16 * c0;
                if (there) {
                    if (left == kRopeHeads) {
#pragma unroll
                        for (int i = 0; i < kRopeHeads / 4; ++i)
                            four(from + i * 8 * kD, to + i * step, sc + i * (step / (kD / kMxScales)), true);
                    } else {
                        for (int i = 0; 4 * i < left; ++i)
                            four(from + i * 8 * kD, to + i * step, sc + i * (step / (kD / kMxScales)), 4 * i + which < left);
                    }
                    to += kRopeHeads / 4 * step;
                    sc += kRopeHeads / 4 * (step / (kD / kMxScales));
                }
                __syncwarp();   // all lanes have read the batch
                if (lane == 0)
                    copy_next();
            }
        };
        if (p0 < nq)
            heads(std::integral_constant<int, 0>{}, p0, min(p1, nq));
        if (p0 < nq + nk && p1 > nq && ok)
            heads(std::integral_constant<int, 1>{}, max(p0, nq) - nq, min(p1, nq + nk) - nq);
        if (TO && p1 > nq + nk && ok)
            heads(std::integral_constant<int, 2>{}, max(p0, nq + nk) - nq - nk, p1 - nq - nk);
    }
    if (!ok && lane == 0) {   // a wait ran out: the copies in flight are waited for before the memory goes
        const long long from = clock64();
        for (uint32_t u = used; u < ahead; ++u)
            while (!mbar_try_wait(&sh.full[u % kRopeStages], (u / kRopeStages) & 1) && clock64() - from < kWaitCycles)
                ;
    }
    __syncwarp();
}

// seqlens_out from seqlens, in place or not, behind the rows' kernel.
__global__ void advance_kernel(const RopeArgs a)
{
    pdl_wait();
    pdl_trigger();
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < a.B; b += gridDim.x * blockDim.x)
        a.seqlens_out[b] = advanced(a, b);
}

template <bool INTER, bool FULL>
static const void *rope_kernel_to(int to)
{
    return to == TO_ROWS ? (const void *)rope_kernel<INTER, FULL, TO_ROWS>
         : to == TO_MX8  ? (const void *)rope_kernel<INTER, FULL, TO_MX8>
                         : (const void *)rope_kernel<INTER, FULL, TO_BF16>;
}

static const void *rope_kernel_for(bool inter, bool full, int to)
{
    return inter ? (full ? rope_kernel_to<true, true>(to) : rope_kernel_to<true, false>(to))
                 : (full ? rope_kernel_to<false, true>(to) : rope_kernel_to<false, false>(to));
}

constexpr size_t kRopeSmem = kRopeWarps * sizeof(RopeWarp);

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st)
{
    auto batches = [](int heads) { return (heads + kRopeHeads - 1) / kRopeHeads; };
    const long long total = (long long)a.T * (batches(a.Hq) + batches(a.Hkv) * (a.v ? 2 : 1));
    const int most = sm_count() * kRopeBlocks * kRopeWarps, each = (int)((total + most - 1) / most);
    const int blocks = (int)((total + (long long)each * kRopeWarps - 1) / ((long long)each * kRopeWarps));
    const void *kernel = rope_kernel_for(a.rope.interleaved != 0, a.rope.rot_dim == kD, !a.v ? TO_ROWS : a.cache.format == RETOPK_CACHE_MX8 ? TO_MX8 : TO_BF16);
    return launch_pdl(reinterpret_cast<void (*)(RopeArgs, int)>(const_cast<void *>(kernel)), dim3(blocks),
                      dim3(kRopeWarps * 32), kRopeSmem, st, 1, a, each);
}

cudaError_t configure_rope()
{
    cudaError_t e = cudaSuccess;
    for (int to : {TO_ROWS, TO_BF16, TO_MX8})
        for (int x = 0; x < 4; ++x)
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(rope_kernel_for(x & 1, x & 2, to), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRopeSmem);
    return e;
}

cudaError_t launch_advance(const RopeArgs &a, cudaStream_t st)
{
    return launch_pdl(advance_kernel, dim3(std::min(64, (a.B + 127) / 128)), dim3(128), 0, st, 1, a);
}

}  // namespace retopk
