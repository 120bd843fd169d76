// prompt.cuh -- what the prompt-side kernels share (rotated append, cache
// copy, chunk attention): addressing of contiguous and paged caches, the 8-bit
// and 4-bit block formats, and the lookup of a token's sequence.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace retopk {

constexpr int kMxBlock = 32;                    // elements that share a scale byte
constexpr int kMxScales = kD / kMxBlock;        // scale bytes of a row
constexpr int kFp4Block = 16;                   // the same of 4-bit rows
constexpr int kFp4Scales = kD / kFp4Block;

// Bytes of a row's elements, and of its scales.
__host__ __device__ constexpr int row_bytes(int format)
{
    return format == RETOPK_CACHE_FP4 ? kD / 2 : format == RETOPK_CACHE_MX8 ? kD : 2 * kD;
}
__host__ __device__ constexpr int row_scales(int format)
{
    return format == RETOPK_CACHE_FP4 ? kFp4Scales : format == RETOPK_CACHE_MX8 ? kMxScales : 0;
}

// Capacity of a sequence in rows.
inline long long cache_capacity(const retopk_cache &c)
{
    return c.table ? (long long)c.table_width * c.page_rows : c.page_rows;
}

// Place in the table of position pos, and its row there: a division by the page's rows as a product with 1 / rows.  Both
// are at most 2^23, so it is off by one at most.
__device__ __forceinline__ int page_of(int pos, int page_rows, float inverse, int &row)
{
    int i = (int)((float)pos * inverse);
    row = pos - i * page_rows;
    if (row < 0)
        row += page_rows, --i;
    else if (row >= page_rows)
        row -= page_rows, ++i;
    return i;
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

// ---- 4-bit rows: e2m1 codes with one scale for 16 elements --------------------
// A scale byte is the upper bits of an fp16 (5 of exponent, 3 of mantissa, no sign).
// With 3 mantissa bits a block's largest element lies within 2^-4 of the code 6 (a
// power of two would leave it anywhere in (3, 6]), without a second scale for the tensor,
// where that element is 6 * 2^-14 (3.7e-4) or more.  Below, scales are 2^-17 apart: byte n
// stands for largest elements of 6 n - 3 to 6 n + 3 times 2^-17, and a block of at most
// 6 * 2^-18 (2.3e-5) becomes zeros.  Code times scale has at
// most 6 significant bits and is exact in fp16 and in bf16.
constexpr uint32_t kFp4Top = 226;   // the largest that is written, 10240: six times it is an fp16

// Scale byte of a block from the largest |x| (its fp32 bits): a sixth of it, rounded to nearest even.
__device__ __forceinline__ uint32_t fp4_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u)
        return 255u;
    const float x = __uint_as_float(amax_bits);
    float s = x * (1.f / 6.f);
    s = fmaf(fmaf(-6.f, s, x), 1.f / 6.f, s);   // (a sixth itself, where it has one: see below)
    const uint32_t u = __float_as_uint(s);
    const uint32_t byte = s < 0x1p-14f ? (uint32_t)rintf(s * 0x1p17f) : ((u + 0x7ffffu + (u >> 20 & 1u)) >> 20) - (112u << 3);
    return min(byte, kFp4Top);
}

__device__ __forceinline__ float fp4_value(uint32_t byte)
{
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Eight codes as fp16, two a register.
__device__ __forceinline__ void e2m1x8_halves(uint32_t codes, uint32_t (&h)[4])
{
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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

// Eight elements as codes, the first in the low bits: x / s rounded once to the nearest
// code, ties to the even one.  s has 4 significant bits and a border between two codes at most 3,
// so bf16 elements do lie on borders, where a product with 1 / s would fall to either side.  What
// the product leaves, x - q s, is exact, and adding its quotient brings q to the border itself.  PACKED: two elements an
// instruction (7 x 40000 rows parked: 181 us, 212 one by one; in the append, whose warps have no registers to spare for
// pairs, 131072 tokens 415, 385 one by one).
template <bool PACKED>
__device__ __forceinline__ uint32_t e2m1x8(const float *x, float s)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = s > 0.f ? r : 0.f;
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PACKED) {
            const float2 y = make_float2(x[2 * i], x[2 * i + 1]), r2 = make_float2(r, r);
            q[i] = mul2(y, r2);
            q[i] = fma2(fma2(q[i], make_float2(-s, -s), y), r2, q[i]);
        } else {
            q[i] = make_float2(x[2 * i] * r, x[2 * i + 1] * r);
            q[i].x = fmaf(fmaf(-q[i].x, s, x[2 * i]), r, q[i].x);
            q[i].y = fmaf(fmaf(-q[i].y, s, x[2 * i + 1]), r, q[i].y);
        }
    }
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(w)
        : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
    return w;
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
size_t chunk_attention_ws(int T, int Hq, int Hkv, bool fp4);
cudaError_t launch_chunk_attention(const AttnArgs &a, cudaStream_t st);
// over 4-bit rows, where sequences have few of them
bool takes_rows(int T, int B, int G);
size_t row_attention_ws();
cudaError_t launch_row_attention(const AttnArgs &a, cudaStream_t st);

}  // namespace retopk
