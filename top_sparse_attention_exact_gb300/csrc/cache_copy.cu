// cache_copy.cu -- rows of one cache into another: 8-bit and 4-bit rows read back,
// bf16 rows quantised, pages gathered or scattered.  Memory bound: each row is
// read and written once.  4 heads: 1048576 8-bit rows read back 475 us, 6.8 TB/s, 4-bit ones 440 us, 6.2 TB/s, of which
// 4.9 are writes (a fill, which writes alone, reaches 4.05); 8 heads: 7 x 40000 rows quantised to 8 bits 187 us, 7.1 TB/s, to 4
// bits 181 us, 6.2 TB/s, issue slots 68 %; a plain copy reaches 6.8.  Between coded rows instructions bound it (issue slots 84 %): 1048576
// rows of 4 heads from 4 bits to 4 281 us, 4.3 TB/s, to 8 bits 482, from 8 bits to 4 543.
#include <algorithm>

#include "prompt.cuh"

namespace retopk {

constexpr int kCopyThreads = 128;
// rows in flight per 8 lanes (7 x 40000 rows quantised to 8 bits: 201 us with 3, 210 with 2, 206 with 4, to 4 bits 225 with 3, 221
// with 4, 230 with 6, all before pages were found by products; 1048576 8-bit rows read back: 474, with 3 488, with 4 489, 4-bit
// ones 454, 457, 451; small blocks also start sooner: 3 x 4099 rows 7.5 us, 10.1 in blocks of 128 rows)
__host__ __device__ constexpr int copy_rows(int src, int dst)
{
    return src == RETOPK_CACHE_BF16 && dst == RETOPK_CACHE_FP4 ? 4 : src == RETOPK_CACHE_BF16 && dst == RETOPK_CACHE_MX8 ? 3 : 2;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Sixteen elements of a row as they are read: bf16, 8-bit or 4-bit codes.
template <int FORMAT>
struct Piece {
    uint32_t w[FORMAT == RETOPK_CACHE_BF16 ? 8 : FORMAT == RETOPK_CACHE_MX8 ? 4 : 2];

    __device__ __forceinline__ void load(const char *row, int lane)
    {
        if constexpr (FORMAT == RETOPK_CACHE_FP4) {
            const uint2 x = reinterpret_cast<const uint2 *>(row)[lane];
            w[0] = x.x, w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(w) / 16; ++i) {
                const uint4 x = reinterpret_cast<const uint4 *>(row)[lane * ((int)sizeof(w) / 16) + i];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void store(char *row, int lane) const
    {
        if constexpr (FORMAT == RETOPK_CACHE_FP4) {
            reinterpret_cast<uint2 *>(row)[lane] = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(w) / 16; ++i)
                reinterpret_cast<uint4 *>(row)[lane * ((int)sizeof(w) / 16) + i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    // the largest size's fp32 bits
    __device__ __forceinline__ uint32_t top(const float (&x)[16]) const
    {
        uint32_t m = 0;
        if constexpr (FORMAT == RETOPK_CACHE_BF16) {   // two at a time, as they are
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max_u16x2(m, w[i] & 0x7fff7fffu);
            return max(m << 16, m & 0xffff0000u);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
            m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
        return m;
    }
    // the elements, with the scale byte that they share
    __device__ __forceinline__ void values(uint32_t scale, float (&x)[16]) const
    {
        if constexpr (FORMAT == RETOPK_CACHE_BF16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
        } else if constexpr (FORMAT == RETOPK_CACHE_MX8) {
            const float s = mx_value(scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = e4m3x2_value(w[i / 2] >> (i & 1) * 16 & 0xffffu);
                x[2 * i] = v.x * s, x[2 * i + 1] = v.y * s;
            }
        } else {
            const float s = fp4_value(scale);   // (not in fp16, where scales that no call writes overflow)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t h[4];
                e2m1x8_halves(w[i], h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 v = mul2(__half22float2(reinterpret_cast<const __half2 &>(h[k])), make_float2(s, s));
                    x[8 * i + 2 * k] = v.x, x[8 * i + 2 * k + 1] = v.y;
                }
            }
        }
    }
};

// cache_row with the page found by a product.
__device__ __forceinline__ long long row_of(const retopk_cache &c, float inverse, int b, int hk, int pos, uint32_t *status)
{
    int page = b, r = pos;
    if (c.table) {
        page = c.table[(long long)b * c.table_width + page_of(pos, c.page_rows, inverse, r)];
        if ((uint32_t)page >= (uint32_t)c.n_pages) {
            if (status)
                atomicOr(status, RETOPK_STATUS_BAD_PAGE);
            return -1;
        }
    }
    return ((long long)page * c.n_kv_heads + hk) * c.page_rows + r;
}

// 8 lanes a row, 16 elements a lane.
template <int SRC, int DST>
__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const retopk_cache src, const retopk_cache dst, const int32_t *first, const int32_t *last,
                      long long capacity, int max_rows, uint32_t *status)
{
    constexpr int kCopyRows = copy_rows(SRC, DST), kCopyTile = kCopyThreads / 8 * kCopyRows;   // rows of a block
    constexpr int kSrcScales = row_scales(SRC), kDstScales = row_scales(DST);
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.y >> 1, isv = blockIdx.y & 1, b = blockIdx.z;
    const int lane = threadIdx.x & 7;
    const int f = first[b], l = last[b];
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && f < l && (f < 0 || l > capacity) && status)
        atomicOr(status, RETOPK_STATUS_GATHER);
    const long long begin = f, end = min((long long)l, min((long long)f + max_rows, capacity));
    const long long base = begin + (long long)blockIdx.x * kCopyTile;
    if (base >= end)
        return;
    const char *sk = static_cast<const char *>(isv ? src.v : src.k);
    char *dk = static_cast<char *>(isv ? dst.v : dst.k);
    const uint8_t *ss = isv ? src.v_scale : src.k_scale;
    uint8_t *ds = isv ? dst.v_scale : dst.k_scale;
    const float src_inverse = 1.f / src.page_rows, dst_inverse = 1.f / dst.page_rows;
    // all rows of the block are on their way before the first is written
    long long rd[kCopyRows];
    Piece<SRC> in[kCopyRows];
    uint32_t sc[kCopyRows];
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        const long long pos = base + u * (kCopyThreads / 8) + threadIdx.x / 8;
        long long rs = -1;
        rd[u] = -1;
        if (pos >= 0 && pos < end) {
            rs = row_of(src, src_inverse, b, hk, (int)pos, status);
            rd[u] = row_of(dst, dst_inverse, b, hk, (int)pos, status);
        }
        if (rs < 0 || rd[u] < 0) {
            rd[u] = -1;
            rs = 0;   // (read for nothing: the pool's first row)
        }
        in[u].load(sk + rs * row_bytes(SRC), lane);
        // (bits are copied a scale a lane, values take the lane's own)
        if constexpr (kSrcScales > 0)
            sc[u] = ss[rs * kSrcScales + (SRC == DST ? lane % kSrcScales : lane * kSrcScales / 8)];
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        const bool ok = rd[u] >= 0;
        char *to = dk + rd[u] * row_bytes(DST);
        if constexpr (SRC == DST) {
            if (ok) {
                in[u].store(to, lane);
                if constexpr (kSrcScales > 0)
                    if (lane < kSrcScales)
                        ds[rd[u] * kDstScales + lane] = (uint8_t)sc[u];
            }
            continue;
        }
        float x[16];
        in[u].values(kSrcScales > 0 ? sc[u] : 0u, x);
        Piece<DST> out;
        if constexpr (DST == RETOPK_CACHE_BF16) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out.w[i] = bf16x2(x[2 * i], x[2 * i + 1]);
        } else {
            uint32_t m = in[u].top(x), s;
            if constexpr (DST == RETOPK_CACHE_MX8) {
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                s = mx_scale(m);
                const float q = mx_inverse(s);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out.w[i] = e4m3x2(x[4 * i] * q, x[4 * i + 1] * q) | e4m3x2(x[4 * i + 2] * q, x[4 * i + 3] * q) << 16;
            } else {
                s = fp4_scale(m);
                const float f = fp4_value(s);
                out.w[0] = e2m1x8<true>(x, f);
                out.w[1] = e2m1x8<true>(x + 8, f);
            }
            if (ok && lane % (8 / kDstScales) == 0)
                ds[rd[u] * kDstScales + lane / (8 / kDstScales)] = (uint8_t)s;
        }
        if (ok)
            out.store(to, lane);
    }
}

template <int SRC>
static auto copy_kernel_to(int dst)
{
    return dst == RETOPK_CACHE_BF16 ? cache_copy_kernel<SRC, RETOPK_CACHE_BF16>
           : dst == RETOPK_CACHE_MX8 ? cache_copy_kernel<SRC, RETOPK_CACHE_MX8>
                                     : cache_copy_kernel<SRC, RETOPK_CACHE_FP4>;
}

cudaError_t launch_cache_copy(const retopk_cache &src, const retopk_cache &dst, const int32_t *first,
                              const int32_t *last, int B, int max_rows, uint32_t *status, cudaStream_t st)
{
    const long long capacity = std::min(cache_capacity(src), cache_capacity(dst));
    const int tile = kCopyThreads / 8 * copy_rows(src.format, dst.format);
    const dim3 grid((max_rows + tile - 1) / tile, 2 * src.n_kv_heads, B), block(kCopyThreads);
    auto kernel = src.format == RETOPK_CACHE_BF16  ? copy_kernel_to<RETOPK_CACHE_BF16>(dst.format)
                  : src.format == RETOPK_CACHE_MX8 ? copy_kernel_to<RETOPK_CACHE_MX8>(dst.format)
                                                   : copy_kernel_to<RETOPK_CACHE_FP4>(dst.format);
    return launch_pdl(kernel, grid, block, 0, st, 1, src, dst, first, last, capacity, max_rows, status);
}

}  // namespace retopk
