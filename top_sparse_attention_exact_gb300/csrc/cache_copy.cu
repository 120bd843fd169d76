// cache_copy.cu -- rows of one cache into another: 8-bit rows read back,
// bf16 rows quantised, pages gathered or scattered.  Memory bound: each row is
// read and written once.  4 heads: 1048576 rows read back 476 us, 6.8 TB/s; 8 heads:
// 7 x 40000 rows quantised 202 us, 6.6 TB/s; a plain copy reaches 6.8.
#include <algorithm>

#include "prompt.cuh"

namespace retopk {

constexpr int kCopyThreads = 128;
// rows in flight per 8 lanes (7 x 40000 rows quantised: 201 us with 3, 210 with 2, 206 with 4; 1048576 rows read
// back: 474, with 3 488, with 4 489; small blocks also start sooner: 3 x 4099 rows 7.5 us, 10.1 in blocks of 128 rows)
__host__ __device__ constexpr int copy_rows(bool src8, bool dst8) { return !src8 && dst8 ? 3 : 2; }

// 8 lanes a row, 16 elements a lane.
template <bool SRC8, bool DST8>
__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const retopk_cache src, const retopk_cache dst, const int32_t *first, const int32_t *last,
                      long long capacity, int max_rows, uint32_t *status)
{
    constexpr int kCopyRows = copy_rows(SRC8, DST8), kCopyTile = kCopyThreads / 8 * kCopyRows;   // rows of a block
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
    // all rows of the block are on their way before the first is written
    long long rd[kCopyRows];
    uint4 in[kCopyRows][SRC8 ? 1 : 2];
    uint32_t sc[kCopyRows];
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        const long long pos = base + u * (kCopyThreads / 8) + threadIdx.x / 8;
        long long rs = -1;
        rd[u] = -1;
        if (pos >= 0 && pos < end) {
            rs = cache_row(src, b, hk, (int)pos, status);
            rd[u] = cache_row(dst, b, hk, (int)pos, status);
        }
        if (rs < 0 || rd[u] < 0) {
            rd[u] = -1;
            rs = 0;   // (read for nothing: the pool's first row)
        }
        if (SRC8) {
            in[u][0] = reinterpret_cast<const uint4 *>(sk + rs * kD)[lane];
            sc[u] = ss[rs * kMxScales + (DST8 ? lane & 3 : lane / 2)];
        } else {
            in[u][0] = (reinterpret_cast<const uint4 *>(sk + rs * 2 * kD) + 2 * lane)[0];
            in[u][SRC8 ? 0 : 1] = (reinterpret_cast<const uint4 *>(sk + rs * 2 * kD) + 2 * lane)[1];
        }
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        const bool ok = rd[u] >= 0;
        const uint4 v0 = in[u][0], v1 = in[u][SRC8 ? 0 : 1];
        if (SRC8 && DST8) {
            if (ok) {
                reinterpret_cast<uint4 *>(dk + rd[u] * kD)[lane] = v0;
                if (lane < kMxScales)
                    ds[rd[u] * kMxScales + lane] = (uint8_t)sc[u];
            }
        } else if (!DST8) {
            uint4 o0 = v0, o1 = v1;
            if (SRC8) {
                const float s = mx_value(sc[u]);
                const uint32_t w[4] = {v0.x, v0.y, v0.z, v0.w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 v = e4m3x2_value(w[i / 2] >> (i & 1) * 16 & 0xffffu);
                    o[i] = bf16x2(v.x * s, v.y * s);
                }
                o0 = make_uint4(o[0], o[1], o[2], o[3]);
                o1 = make_uint4(o[4], o[5], o[6], o[7]);
            }
            if (ok) {
                uint4 *d = reinterpret_cast<uint4 *>(dk + rd[u] * 2 * kD) + 2 * lane;
                d[0] = o0;
                d[1] = o1;
            }
        } else {
            float x[8], y[8];
            unpack8(v0, x);
            unpack8(v1, y);
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                m = max(m, max(__float_as_uint(x[e]) & 0x7fffffffu, __float_as_uint(y[e]) & 0x7fffffffu));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            if (ok) {
                const uint32_t s = mx_scale(m);
                const float q = mx_inverse(s);
                uint4 c;
                c.x = e4m3x2(x[0] * q, x[1] * q) | e4m3x2(x[2] * q, x[3] * q) << 16;
                c.y = e4m3x2(x[4] * q, x[5] * q) | e4m3x2(x[6] * q, x[7] * q) << 16;
                c.z = e4m3x2(y[0] * q, y[1] * q) | e4m3x2(y[2] * q, y[3] * q) << 16;
                c.w = e4m3x2(y[4] * q, y[5] * q) | e4m3x2(y[6] * q, y[7] * q) << 16;
                reinterpret_cast<uint4 *>(dk + rd[u] * kD)[lane] = c;
                if ((lane & 1) == 0)
                    ds[rd[u] * kMxScales + lane / 2] = (uint8_t)s;
            }
        }
    }
}

cudaError_t launch_cache_copy(const retopk_cache &src, const retopk_cache &dst, const int32_t *first,
                              const int32_t *last, int B, int max_rows, uint32_t *status, cudaStream_t st)
{
    const long long capacity = std::min(cache_capacity(src), cache_capacity(dst));
    const bool s8 = src.format == RETOPK_CACHE_MX8, d8 = dst.format == RETOPK_CACHE_MX8;
    const int tile = kCopyThreads / 8 * copy_rows(s8, d8);
    const dim3 grid((max_rows + tile - 1) / tile, 2 * src.n_kv_heads, B), block(kCopyThreads);
    auto kernel = s8 ? (d8 ? cache_copy_kernel<true, true> : cache_copy_kernel<true, false>)
                     : (d8 ? cache_copy_kernel<false, true> : cache_copy_kernel<false, false>);
    return launch_pdl(kernel, grid, block, 0, st, 1, src, dst, first, last, capacity, max_rows, status);
}

}  // namespace retopk
