// cache_copy.cu -- rows of one cache into another: 8-bit rows read back,
// bf16 rows quantised, pages gathered or scattered.  Memory bound: each row is
// read and written once.
#include <algorithm>

#include "prompt.cuh"

namespace retopk {

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 4;                                  // rows in flight per 8 lanes
constexpr int kCopyTile = kCopyThreads / 8 * kCopyRows;       // rows per block

// 8 lanes a row, 16 elements a lane.
template <bool SRC8, bool DST8>
__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const retopk_cache src, const retopk_cache dst, const int32_t *first, const int32_t *last,
                      long long capacity, int max_rows, uint32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int hk = blockIdx.y >> 1, isv = blockIdx.y & 1, b = blockIdx.z;
    const int lane = threadIdx.x & 7;
    const int f = first[b], l = last[b];
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && f < l && (f < 0 || l > capacity) && status)
        atomicOr(status, RETOPK_STATUS_GATHER);
    const long long begin = f, end = min((long long)l, min((long long)f + max_rows, capacity));
    const long long base = begin + (long long)blockIdx.x * kCopyTile;
    const char *sk = static_cast<const char *>(isv ? src.v : src.k);
    char *dk = static_cast<char *>(isv ? dst.v : dst.k);
    const uint8_t *ss = isv ? src.v_scale : src.k_scale;
    uint8_t *ds = isv ? dst.v_scale : dst.k_scale;
    for (int u = 0; u < kCopyRows; ++u) {
        const long long pos = base + u * (kCopyThreads / 8) + threadIdx.x / 8;
        const bool in = pos >= 0 && pos < end;
        long long rs = -1, rd = -1;
        if (in) {
            rs = cache_row(src, b, hk, (int)pos, status);
            rd = cache_row(dst, b, hk, (int)pos, status);
        }
        const bool ok = rs >= 0 && rd >= 0;
        if (SRC8 && DST8) {
            if (ok) {
                reinterpret_cast<uint4 *>(dk + rd * kD)[lane] = reinterpret_cast<const uint4 *>(sk + rs * kD)[lane];
                if (lane < kMxScales)
                    ds[rd * kMxScales + lane] = ss[rs * kMxScales + lane];
            }
        } else if (SRC8) {
            if (ok) {
                const uint4 c = reinterpret_cast<const uint4 *>(sk + rs * kD)[lane];
                const float s = mx_value(ss[rs * kMxScales + lane / 2]);
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 v = e4m3x2_value(w[i / 2] >> (i & 1) * 16 & 0xffffu);
                    o[i] = bf16x2(v.x * s, v.y * s);
                }
                uint4 *d = reinterpret_cast<uint4 *>(dk + rd * 2 * kD) + 2 * lane;
                d[0] = make_uint4(o[0], o[1], o[2], o[3]);
                d[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        } else {
            uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
            if (ok) {
                const uint4 *s = reinterpret_cast<const uint4 *>(sk + rs * 2 * kD) + 2 * lane;
                v0 = s[0];
                v1 = s[1];
            }
            if (!DST8) {
                if (ok) {
                    uint4 *d = reinterpret_cast<uint4 *>(dk + rd * 2 * kD) + 2 * lane;
                    d[0] = v0;
                    d[1] = v1;
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
                    const uint32_t sc = mx_scale(m);
                    const float q = mx_inverse(sc);
                    uint4 c;
                    c.x = e4m3x2(x[0] * q, x[1] * q) | e4m3x2(x[2] * q, x[3] * q) << 16;
                    c.y = e4m3x2(x[4] * q, x[5] * q) | e4m3x2(x[6] * q, x[7] * q) << 16;
                    c.z = e4m3x2(y[0] * q, y[1] * q) | e4m3x2(y[2] * q, y[3] * q) << 16;
                    c.w = e4m3x2(y[4] * q, y[5] * q) | e4m3x2(y[6] * q, y[7] * q) << 16;
                    reinterpret_cast<uint4 *>(dk + rd * kD)[lane] = c;
                    if ((lane & 1) == 0)
                        ds[rd * kMxScales + lane / 2] = (uint8_t)sc;
                }
            }
        }
    }
}

cudaError_t launch_cache_copy(const retopk_cache &src, const retopk_cache &dst, const int32_t *first,
                              const int32_t *last, int B, int max_rows, uint32_t *status, cudaStream_t st)
{
    const long long capacity = std::min(cache_capacity(src), cache_capacity(dst));
    const dim3 grid((max_rows + kCopyTile - 1) / kCopyTile, 2 * src.n_kv_heads, B), block(kCopyThreads);
    const bool s8 = src.format == RETOPK_CACHE_MX8, d8 = dst.format == RETOPK_CACHE_MX8;
    auto kernel = s8 ? (d8 ? cache_copy_kernel<true, true> : cache_copy_kernel<true, false>)
                     : (d8 ? cache_copy_kernel<false, true> : cache_copy_kernel<false, false>);
    return launch_pdl(kernel, grid, block, 0, st, 1, src, dst, first, last, capacity, max_rows, status);
}

}  // namespace retopk
