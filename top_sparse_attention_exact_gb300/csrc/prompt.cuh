// prompt.cuh -- what the prompt-side kernels share (rotated append, cache
// copy, chunk attention): addressing of contiguous and paged caches, the
// 8-bit block format, and the lookup of a token's sequence.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace retopk {

constexpr int kMxBlock = 32;                    // elements that share a scale byte
constexpr int kMxScales = kD / kMxBlock;        // scale bytes of a row

// Capacity of a sequence in rows.
inline long long cache_capacity(const retopk_cache &c)
{
    return c.table ? (long long)c.table_width * c.page_rows : c.page_rows;
}

// Row (page, head, row in page) of sequence b, head hk, position pos, as an
// index into [n_pages, Hkv, page_rows]; -1 (and RETOPK_STATUS_BAD_PAGE) for a
// table entry outside the pool.  pos is within the capacity.
__device__ __forceinline__ long long cache_row(const retopk_cache &c, int b, int hk, int pos, uint32_t *status)
{
    int page = b, r = pos;
    if (c.table) {
        page = c.table[(long long)b * c.table_width + pos / c.page_rows];
        r = pos % c.page_rows;
        if ((uint32_t)page >= (uint32_t)c.n_pages) {
            if (status)
                atomicOr(status, RETOPK_STATUS_BAD_PAGE);
            return -1;
        }
    }
    return ((long long)page * c.n_kv_heads + hk) * c.page_rows + r;
}

// Bounded wait; false (and RETOPK_STATUS_TIMEOUT, where there is a status word) on expiry.
__device__ __forceinline__ bool wait_full(uint64_t *bar, uint32_t parity, uint32_t *status)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > kWaitCycles) {
            if (status)
                atomicOr(status, RETOPK_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// ---- 8-bit rows: e4m3 codes with one power-of-two scale for 32 elements -----
// Scale byte of a block from the largest |x| (its fp32 bits): the smallest e
// with amax <= 448 * 2^e, e = byte - 127.  448 = 1.75 * 2^8, so e is the
// exponent of amax less 8, plus one where its mantissa is above 1.75.  A power
// of two keeps the division by the scale exact: the only rounding is the
// code's own.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u)
        return 255u;
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 0);
}

// 2^(127 - byte): a normal number for every byte mx_scale gives (at most 247).
__device__ __forceinline__ float mx_inverse(uint32_t byte)
{
    return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float mx_value(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 0x00400000u : byte << 23);
}

// Two fp32 -> two e4m3 codes (lo in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8])
{
    x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
    x[4] = bf16lo(u.z), x[5] = bf16hi(u.z), x[6] = bf16lo(u.w), x[7] = bf16hi(u.w);
}

// ---- launchers ----------------------------------------------------------------
struct RopeArgs {
    const uint16_t *q, *k, *v;                 // v == NULL: no cache
    long long q_stride, k_stride, v_stride;    // elements
    const int32_t *cu, *seqlens;
    int32_t *seqlens_out;                      // NULL: not written by the kernel
    uint16_t *q_out, *k_out;
    uint32_t *status;
    retopk_rope rope;
    retopk_cache cache;
    long long capacity;
    int T, B, Hq, Hkv;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st);
cudaError_t launch_advance(const RopeArgs &a, cudaStream_t st);
cudaError_t launch_cache_copy(const retopk_cache &src, const retopk_cache &dst, const int32_t *first,
                              const int32_t *last, int B, int max_rows, uint32_t *status, cudaStream_t st);

struct AttnArgs {
    const uint16_t *q;
    long long q_stride, out_stride;            // elements
    const int32_t *cu, *seqlens;
    uint16_t *out;
    float *lse;
    uint32_t *status;
    retopk_cache cache;
    int capacity;                              // rows of a sequence
    int T, B, Hq, G, window;
    float scale, softcap;
    void *ws;
};
size_t chunk_attention_ws(int T, int Hq, int Hkv);
cudaError_t launch_chunk_attention(const AttnArgs &a, cudaStream_t st);

}  // namespace retopk
