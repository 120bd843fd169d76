// row_attention.cu -- causal attention of a few query rows a sequence over a
// 4-bit cache: single tokens of a batch, and a few drafted ones.
//
// Mathematics.  As in chunk_attention.cu: s_j = scale q.k_j (capped: softcap tanh(s_j / softcap)), out = sum_j exp(s_j) v_j /
// sum_j exp(s_j) over the keys that a token sees, in one pass with a running maximum m and sum l of each row, parts
// joined by their (m, l).
//
// What bounds it.  144 bytes a key and head for keys and values, and the work of making 256 codes a key into
// numbers: each conversion gives two, at 64 lanes a cycle of an SM, so a key takes 2 cycles of that pipe where the
// memory takes 6.  The matrix work is small (rows: a group's query heads, times the tokens), so it is done
// by warps (mma.sync), in the transposed form whose rows are the keys: then 8 columns hold 8 query rows, codes become operands
// in the registers that they were loaded to, and nothing is written to shared memory but what the copies bring.
//   S^T = K Q^T     a lane's 32 codes of a key, 16 bytes, are its part of 8 steps of the contraction
//   O^T = V^T P^T   a lane's 16 codes of four keys, one scale block each; codes of two keys are brought side by side
//                   four bits at a time before they are converted; P^T is a transposed 8 x 8 of half words
// A warp takes 32 keys of every 128, with a ring of its own: copies bring 32 keys' codes and scales a tile ahead.  Four
// warps are a CTA, so that one CTA's end of an item lies beside the others' work.
//
// Rounding.  Code times scale is exact in fp16.  A query row is brought to fp16's range by a power of two, so
// its elements are exact down to 2^-28 of the largest.  P is rounded to fp16 (m lies 2^7 below the maximum when
// it is taken and is raised when that has grown by 2^8 more, so weights reach from 2^15 down to 2^-24).  All else has 32 bits.
//
// Measured (28 query heads over 4 KV heads but where said).  61 ragged sequences of up to 9000 keys, 32 over 8 heads: 80 us,
// 5.1 TB/s (over bf16 rows 217 us): the stream runs at nine tenths of a plain copy's rate, with ~5 us of start before it and ~5 of the
// slowest warps and the join behind.  One token over 131072 keys 26 us (bf16 51), over 500000 60 (153): 4 us of start, the
// stream, 6 of end and join.  128 sequences of 1500 keys, 32 over 8 heads, 40 us (130).  16 sequences of 2, 3 and 4 tokens
// over 20000 keys 44, 47 and 64 us (bf16 77, 79, 68): registers leave 12 and then 8 warps an SM, which issue in two
// cycles of five.  One token over 300 keys 7.2 us of a graph of such calls and 9.8 called from Python where the cache holds
// up to 512 rows; 9.9 and 11.3 where it holds more, as such a call is cut and joined whatever its length.
// Registers of a thread are 128, 168, 255 and 255 with one to four tiles of rows; 36, 8 and 108 bytes of it are spilled with two, three
// and four (capped: 44, 0 and 108).
// A tile of a warp, 32 keys, is 640 instructions: 128 conversions, 128 products with the scales, 32 matrix products, 32 to bring codes
// of two keys together, 24 loads, ~70 of softmax, the rest copies, scales and the loop.
// Not kept: one CTA of all the SM's warps (61 sequences 78 us, one token over 131072 27.5; with a limit on how far its groups of
// four run apart 80), the same only where items are few (16 x 3 47.4 of a graph, 45.0 as it is), codes made fp16 by shifts and masks
// (1.4 cycles of an SM for two codes of 32 lanes, a conversion takes 0.5).
#include <math.h>

#include <algorithm>

#include "attention_plan.cuh"

namespace retopk {

namespace {

constexpr int kRowWarps = 4, kRowThreads = kRowWarps * 32;
constexpr int kWarpKeys = kTile / kRowWarps;
constexpr int kCodeBytes = kWarpKeys * kD / 2, kScaleBytes = kWarpKeys * kFp4Scales;
constexpr int kStageBytes = 2 * (kCodeBytes + kScaleBytes);    // K's codes, V's codes, K's scales, V's scales
constexpr int kSumRow = kD + 4;                                // floats of a row where the warps' sums meet
constexpr float kLift = 7.f, kLazy = 8.f;                      // as in chunk_attention.cu
constexpr int kMaxRowShares = 1024;
constexpr int kMaxRowTiles = 4;                                // of 8 query rows

// CTAs of an SM, by the tiles of 8 query rows, and tiles of a warp's ring (61 ragged tokens 83.1 us with 2, 84.7 with 3; where
// few warps share an SM each has more on its way).
__host__ __device__ constexpr int row_blocks(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }
__host__ __device__ constexpr int row_stages(int nt) { return nt <= 2 ? 2 : 4; }
// The queries stay in registers, or, where the sums take those, in shared memory.
__host__ __device__ constexpr bool shared_queries(int nt) { return nt > 1; }

struct RowCost {
    static constexpr int kItem = 256;
    static __device__ __forceinline__ int grain(const Plan &p, int nt) { return nt > p.uncut ? 1 : p.uncut; }
};

// Parts of items, as in attention_plan.cuh, of `rows` rows: (m, l) pairs, and 128 sums a row.
struct RowParts {
    Bound *bound;
    float2 *ml;
    float *o;
    int rows;
};

struct RowLaunch {
    AttnArgs a;
    Plan plan;
    RowParts parts;
};

template <int NT>
struct RowShared {
    Share share;
    Walk walk;
    Segment segments[2];
    float2 ml[kRowWarps][8 * NT];
    int exponent[8 * NT];                                       // of the queries' rows
    uint4 q[shared_queries(NT) ? 4 : 1][shared_queries(NT) ? NT : 1][32];
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t mul_halves(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4])
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t (&w)[2])
{
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr)
{
    uint32_t x;
    asm volatile("{\n .reg .u16 h;\n ld.shared.u16 h, [%1];\n cvt.u32.u16 %0, h;\n}\n" : "=r"(x) : "r"(addr));
    return x;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr)
{
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr));
    return x;
}
template <int OFFSET>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(OFFSET) : "memory");
}
// Eight bytes, or zeros.
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}

// cap tanh(x / cap), up to half the cap by the polynomial of chunk_attention.cu (6.4e-7 of the value): a cap far above the
// scores leaves them as they are.
__device__ __forceinline__ float capped(float x, float cap, float inverse)
{
    const float y = x * inverse, t = y * y;
    const float small = x * fmaf(fmaf(fmaf(-0.04475064703577332f, t, 0.132053598066859f), t, -0.3332815934197915f), t, 1.f);
    const float large = fmaf(-2.f * cap, rcp(1.f + ex2(y * 2.885390081777927f)), cap);
    return fabsf(y) < 0.5f ? small : large;
}

}  // namespace

template <int NT, bool CAP>
__global__ void __launch_bounds__(kRowThreads, row_blocks(NT)) row_attention_kernel(const __grid_constant__ RowLaunch c)
{
    constexpr int kRowStages = row_stages(NT);
    constexpr bool kShared = shared_queries(NT);
    extern __shared__ __align__(16) unsigned char row_smem[];
    RowShared<NT> &sh = *reinterpret_cast<RowShared<NT> *>(row_smem + kRowWarps * kRowStages * kStageBytes);
    const AttnArgs &a = c.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3, G = a.G;
    const uint32_t ring = smem_u32(row_smem) + warp * kRowStages * kStageBytes;
    if (tid == 0) {
        sh.share.bound[0] = sh.share.bound[1] = Place{a.B, 0, 0, 0};
        sh.share.first_b = -1;
    }
    pdl_wait();
    pdl_trigger();
    find_share<RowCost, kRowThreads>(a, c.plan, sh.share);
    __syncthreads();
    if (tid == 0) {
        c.parts.bound[blockIdx.x] = Bound{sh.share.bound[0], sh.share.first.n, sh.share.first.t0};
        if (blockIdx.x == gridDim.x - 1)
            c.parts.bound[gridDim.x] = Bound{sh.share.bound[1], 0, 0};
        sh.walk = Walk{sh.share.bound[0], sh.share.bound[1], sh.share.first, sh.share.first_b};
        sh.segments[0].more = next_segment(a, c.plan, sh.walk, sh.segments[0]);
    }
    // Keys of a group of 16, by the number of the matrix' row: of rows 2 i and 2 i + 1 the first four and the second, so
    // that what 8 lanes (keys), or 16 (values), load lies in different banks
    auto key_of = [](int r) { return (r & 1 ? ((r >> 1 & 3) ^ 1) + 4 : r >> 1 & 3) + (r & 8); };
    const uint32_t k_at = key_of(g) * (kD / 2) + t4 * 16, ks_at = 2 * kCodeBytes + key_of(g) * kFp4Scales + t4 * 2;
    // values: the 16-byte pieces of keys 2, 3 of every four change places by two
    const uint32_t v_at = kCodeBytes + ((g >> 1 ^ (t4 >> 1) << 1) << 4) + (g & 1) * 8;
    const uint32_t va = key_of(2 * t4) * (kD / 2) + v_at, vb = key_of(2 * t4 + 1) * (kD / 2) + v_at;
    const uint32_t code_from = lane * 16, values_to = kCodeBytes + (g * 4 + (t4 ^ (g >> 1 & 1) << 1)) * 16;   // of the copies
    const uint32_t vs_at = 2 * kCodeBytes + kScaleBytes + g;
    const uint32_t vsa = key_of(2 * t4) * kFp4Scales + vs_at, vsb = key_of(2 * t4 + 1) * kFp4Scales + vs_at;

    for (int n = 0;; ++n) {
        __syncthreads();   // the segment is known, and the sums of the one before have been read
        const Segment &s = sh.segments[n & 1];
        if (!s.more)
            break;
        const int nt = s.j1 - s.j0, L = s.seq.L, tok0 = s.k * c.plan.tokens, tokens = min(c.plan.tokens, s.seq.n - tok0);
        const int first = L - s.seq.n + tok0, last = first + tokens - 1;   // positions of the tokens
        const int low = a.window > 0 ? first - a.window + 1 : 0;           // the first key that one sees
        const int pos0 = s.j0 * kTile + warp * kWarpKeys;

        // ---- the copies: this warp's keys of a tile.  Where 16 keys lie is looked up by a lane each, for 16 tiles at a
        // time: the byte of the pool where their codes begin; negative: nowhere
        long long place = -1;
        auto look = [&](int t) {
            t += lane >> 1;
            const int pos = pos0 + t * kTile + (lane & 1) * 16;
            place = -1;
            if (t < nt && pos < L && pos <= last && pos + 15 >= low) {
                int page = s.b, row = pos;
                if (a.cache.table)
                    page = a.cache.table[(long long)s.b * a.cache.table_width + page_of(pos, a.cache.page_rows, 1.f / a.cache.page_rows, row)];
                if ((uint32_t)page < (uint32_t)a.cache.n_pages)
                    place = (((long long)page * a.cache.n_kv_heads + s.hk) * a.cache.page_rows + row) * (kD / 2);
                else if (a.status)
                    atomicOr(a.status, RETOPK_STATUS_BAD_PAGE);
            }
        };
        uint32_t to = ring;
        auto issue = [&](int t) {
            if (t < nt) {
                if ((t & 15) == 0)
                    look(t);
                const int left = L - (pos0 + t * kTile);
                const long long from[2] = {__shfl_sync(0xffffffffu, place, (t & 15) * 2), __shfl_sync(0xffffffffu, place, (t & 15) * 2 + 1)};
                // rows that are not there keep what codes the place held, and get scales of zero
                constexpr int kEight = 8 * (kD / 2);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (from[i] < 0)
                        continue;
                    const char *k = static_cast<const char *>(a.cache.k) + from[i] + code_from;
                    const char *v = static_cast<const char *>(a.cache.v) + from[i] + code_from;
                    const uint32_t k_to = to + 2 * i * kEight + code_from, v_to = to + 2 * i * kEight + values_to;
                    if (16 * i + 16 <= left) {
                        copy16<0>(k_to, k);
                        copy16<kEight>(k_to, k);
                        copy16<0>(v_to, v);
                        copy16<kEight>(v_to, v);
                    } else {
                        if (16 * i + g < left) {
                            copy16<0>(k_to, k);
                            copy16<0>(v_to, v);
                        }
                        if (16 * i + 8 + g < left) {
                            copy16<kEight>(k_to, k);
                            copy16<kEight>(v_to, v);
                        }
                    }
                }
                const long long mine = lane >> 4 ? from[1] : from[0];
                const bool ok = mine >= 0 && lane < left;
                const long long x = ok ? (mine >> 3) + (lane & 15) * kFp4Scales : 0;
                copy8(to + 2 * kCodeBytes + lane * kFp4Scales, a.cache.k_scale + x, ok);
                copy8(to + 2 * kCodeBytes + kScaleBytes + lane * kFp4Scales, a.cache.v_scale + x, ok);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            to = to + kStageBytes == ring + kRowStages * kStageBytes ? ring : to + kStageBytes;
        };
        // ---- the queries: column g of each 8, this lane's 32 elements, as fp16 of at most 2^15
        uint32_t q[kShared ? 1 : NT][16];
        float factor[NT][2];             // of a column's scores, to be in powers of two
        int hi[NT][2];                   // the last key that a column sees
        auto ask = [&](int x, uint32_t (&w)[16]) {
            const int r = 8 * x + g, tok = r / G;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = 0;
            if (x < NT && tok < tokens) {
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (long long)(s.seq.t0 + tok0 + tok) * a.q_stride +
                                                                   (s.hk * G + r % G) * kD + t4 * 32);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 y = src[i];
                    w[4 * i] = y.x, w[4 * i + 1] = y.y, w[4 * i + 2] = y.z, w[4 * i + 3] = y.w;
                }
            }
        };
        auto scaled = [&](uint32_t (&q)[16]) {   // in place; the power of two
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = max(top, max(q[i] << 16 & 0x7fffffffu, q[i] & 0x7fff0000u));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = top == 0 ? 0 : max((int)(top >> 23) - 127 - 14, -100);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                q[i] = f16x2(bf16lo(q[i]) * down, bf16hi(q[i]) * down);
            return e;
        };
        auto columns = [&](int x, int k, int e) {
            const int col = 8 * x + 2 * t4 + k;
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
            // (never zero, as a hidden score is -inf and has to stay so)
            factor[x][k] = fmaxf(a.scale * 1.4426950408889634f * up, 1e-38f);
            hi[x][k] = min(first + col / G, last);
        };
        // they are asked for before the keys, whose copies would hold them up
        static_assert(NT <= kRowWarps, "a warp makes one tile of shared queries");
        if constexpr (kShared) {
            ask(warp, q[0]);
        } else {
#pragma unroll
            for (int x = 0; x < NT; ++x)
                ask(x, q[x]);
        }
#pragma unroll
        for (int t = 0; t < kRowStages - 1; ++t)
            issue(t);
        if (tid == 0)
            sh.segments[(n + 1) & 1].more = next_segment(a, c.plan, sh.walk, sh.segments[(n + 1) & 1]);

        if constexpr (kShared) {
            const int e = scaled(q[0]);
            if (warp < NT) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sh.q[i][warp][lane] = make_uint4(q[0][4 * i], q[0][4 * i + 1], q[0][4 * i + 2], q[0][4 * i + 3]);
                if (t4 == 0)
                    sh.exponent[8 * warp + g] = e;
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    columns(x, k, sh.exponent[8 * x + 2 * t4 + k]);
        } else {
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const int e = scaled(q[x]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    columns(x, k, __shfl_sync(0xffffffffu, e, (2 * t4 + k) * 4));
            }
        }

        // (capped scores have that factor before the softmax sees them)
        const float cap2 = a.softcap * 1.4426950408889634f, over_cap = fminf(1.f / cap2, 3e38f);
        auto unit = [&](int x, int k) { return CAP ? 1.f : factor[x][k]; };

        // ---- the tiles
        float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.f;
            m[x][0] = m[x][1] = -INFINITY;
            l[x][0] = l[x][1] = 0.f;
        }
        uint32_t from = ring;
        for (int t = 0; t < nt; ++t) {
            issue(t + kRowStages - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 1) : "memory");
            __syncwarp();
            const int pos = pos0 + t * kTile;
            if (pos <= last && pos + kWarpKeys > low) {
                float sc[2][NT][4];
                uint32_t w0[2][4], w1[2][4], s0[2], s1[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        sc[half][x][0] = sc[half][x][1] = sc[half][x][2] = sc[half][x][3] = 0.f;
                    const uint32_t base = from + half * 16 * (kD / 2), sbase = from + half * 16 * kFp4Scales;
                    lds128(base + k_at, w0[half]);
                    lds128(base + k_at + 8 * (kD / 2), w1[half]);
                    s0[half] = lds16(sbase + ks_at);
                    s1[half] = lds16(sbase + ks_at + 8 * kFp4Scales);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h0[2][4], h1[2][4];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t z0 = (i < 2 ? s0[half] & 255u : s0[half] >> 8) * 0x00800080u;   // fp16, twice
                        const uint32_t z1 = (i < 2 ? s1[half] & 255u : s1[half] >> 8) * 0x00800080u;
                        e2m1x8_halves(w0[half][i], h0[half]);
                        e2m1x8_halves(w1[half][i], h1[half]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            h0[half][k] = mul_halves(h0[half][k], z0);
                            h1[half][k] = mul_halves(h1[half][k], z1);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        uint4 b;
                        if constexpr (kShared)
                            b = sh.q[i][x][lane];
                        else
                            b = make_uint4(q[x][4 * i], q[x][4 * i + 1], q[x][4 * i + 2], q[x][4 * i + 3]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            mma_f16_16816(sc[half][x], h0[half][0], h1[half][0], h0[half][1], h1[half][1], b.x, b.y);
                            mma_f16_16816(sc[half][x], h0[half][2], h1[half][2], h0[half][3], h1[half][3], b.z, b.w);
                        }
                    }
                }
                // capped; hidden ones -inf
                if (CAP) {
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sc[i >> 2][x][i & 3] = capped(sc[i >> 2][x][i & 3] * factor[x][i & 1], cap2, over_cap);
                }
                if (pos + kWarpKeys - 1 > first || (a.window > 0 && pos < last - a.window + 1)) {
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int key = pos + (i >> 2) * 16 + key_of(g) + (i >> 1 & 1) * 8, h = hi[x][i & 1];
                            if (key > h || (a.window > 0 && key <= h - a.window))
                                sc[i >> 2][x][i & 3] = -INFINITY;
                        }
                }
                float top[NT][2];   // in powers of two
                bool grow = false;
#pragma unroll
                for (int x = 0; x < NT; ++x) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float y = max3(fmaxf(sc[0][x][k], sc[0][x][2 + k]), sc[1][x][k], sc[1][x][2 + k]);
                        top[x][k] = y * unit(x, k);
                        grow |= top[x][k] > m[x][k] + (kLift + kLazy);
                    }
                }
                if (__any_sync(0xffffffffu, grow)) {   // every column up to its maximum, and the sums with it
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        float down[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float y = top[x][k];
#pragma unroll
                            for (int d = 4; d < 32; d *= 2)
                                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                            y = fmaxf(m[x][k], y - kLift);
                            down[k] = m[x][k] == -INFINITY ? 1.f : ex2(m[x][k] - y);
                            m[x][k] = y;
                            l[x][k] *= down[k];
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[x][j][e] *= down[e & 1];
                    }
                }
                uint32_t p[2][NT][2];
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    const float b0 = m[x][0] == -INFINITY ? 0.f : m[x][0], b1 = m[x][1] == -INFINITY ? 0.f : m[x][1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y0 = ex2(fmaf(sc[i >> 1][x][(i & 1) * 2], unit(x, 0), -b0));
                        const float y1 = ex2(fmaf(sc[i >> 1][x][(i & 1) * 2 + 1], unit(x, 1), -b1));
                        l[x][0] += y0;
                        l[x][1] += y1;
                        p[i >> 1][x][i & 1] = transposed(f16x2(y0, y1));
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t base = from + half * 16 * (kD / 2), sbase = from + half * 16 * kFp4Scales;
                    uint32_t wa[2], wb[2], wc[2], wd[2];
                    lds64(base + va, wa);
                    lds64(base + vb, wb);
                    lds64(base + va + 8 * (kD / 2), wc);
                    lds64(base + vb + 8 * (kD / 2), wd);
                    const uint32_t s0 = lds8(sbase + vsa) << 7 | lds8(sbase + vsb) << 23;
                    const uint32_t s1 = lds8(sbase + vsa + 8 * kFp4Scales) << 7 | lds8(sbase + vsb + 8 * kFp4Scales) << 23;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        constexpr uint32_t kLow = 0x0f0f0f0fu;
                        uint32_t h[4][4];   // elements 0, 2, 4, 6 of the word of keys a and b; 1, 3, 5, 7; the same of c and d
                        e2m1x8_halves((wa[i] & kLow) | (wb[i] << 4 & ~kLow), h[0]);
                        e2m1x8_halves((wa[i] >> 4 & kLow) | (wb[i] & ~kLow), h[1]);
                        e2m1x8_halves((wc[i] & kLow) | (wd[i] << 4 & ~kLow), h[2]);
                        e2m1x8_halves((wc[i] >> 4 & kLow) | (wd[i] & ~kLow), h[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                h[y][k] = mul_halves(h[y][k], y < 2 ? s0 : s1);
#pragma unroll
                            for (int x = 0; x < NT; ++x)
                                mma_f16_16816(o[x][4 * i + k], h[0][k], h[1][k], h[2][k], h[3][k], p[half][x][0], p[half][x][1]);
                        }
                    }
                }
            }
            __syncwarp();   // all lanes have read the tile
            from = from + kStageBytes == ring + kRowStages * kStageBytes ? ring : from + kStageBytes;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();

        // ---- the warps' sums meet in shared memory: element 16 g + 2 j + e of a row at 16 j + 2 g + e
        float *sums = reinterpret_cast<float *>(row_smem + warp * kRowStages * kStageBytes);
        static_assert(8 * NT * kSumRow * 4 <= kRowStages * kStageBytes, "in the warp's ring");
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float *dst = sums + (8 * x + 2 * t4 + k) * kSumRow + 2 * g;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float2 *>(dst + 16 * j) = make_float2(o[x][j][k], o[x][j][2 + k]);
#pragma unroll
                for (int d = 4; d < 32; d *= 2)
                    l[x][k] += __shfl_xor_sync(0xffffffffu, l[x][k], d);
                if (g == 0)
                    sh.ml[warp][8 * x + 2 * t4 + k] = make_float2(m[x][k], l[x][k]);
            }
        }
        __syncthreads();
        const bool whole = s.j0 == s.lo && s.j1 == s.hi;
        const size_t part = 2 * blockIdx.x + (s.j0 == s.lo);
        for (int i = tid; i < tokens * G * (kD / 2); i += kRowThreads) {
            const int r = i / (kD / 2), x = i % (kD / 2);
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w)
                mm = fmaxf(mm, sh.ml[w][r].x);
            const float zero = mm == -INFINITY ? 0.f : mm;
            float2 y = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                const float2 ml = sh.ml[w][r];
                const float f = ex2(ml.x - zero);
                const float2 v = *reinterpret_cast<const float2 *>(row_smem + w * kRowStages * kStageBytes +
                                                                   4 * (r * kSumRow + 16 * (x & 7) + 2 * (x >> 3)));
                ll = fmaf(ml.y, f, ll);
                y.x = fmaf(v.x, f, y.x);
                y.y = fmaf(v.y, f, y.y);
            }
            if (whole) {
                const size_t t = s.seq.t0 + tok0 + r / G;
                const int head = s.hk * G + r % G;
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                *reinterpret_cast<uint32_t *>(a.out + t * a.out_stride + head * kD + 2 * x) = bf16x2(y.x * inv, y.y * inv);
                if (a.lse && x == 0)
                    a.lse[t * a.Hq + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float2 *>(c.parts.o + (part * c.parts.rows + r) * kD + 2 * x) = y;
                if (x == 0)
                    c.parts.ml[part * c.parts.rows + r] = make_float2(mm, ll);
            }
        }
    }
}

// One more part (m2, l2, o) of a row's sums.
__device__ __forceinline__ void add_part(float &m, float &l, float4 &acc, float m2, float l2, float4 o)
{
    const float mm = fmaxf(m, m2), zero = mm == -INFINITY ? 0.f : mm;
    const float f1 = ex2(m - zero), f2 = ex2(m2 - zero);
    l = l * f1 + l2 * f2;
    acc.x = fmaf(acc.x, f1, o.x * f2);
    acc.y = fmaf(acc.y, f1, o.y * f2);
    acc.z = fmaf(acc.z, f1, o.z * f2);
    acc.w = fmaf(acc.w, f1, o.w * f2);
    m = mm;
}

// A row's end: four columns a lane.
__device__ __forceinline__ void write_row(const AttnArgs &a, size_t t, int head, int lane, float m, float l, float4 acc)
{
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + head * kD + lane * 4) =
        make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0)
        a.lse[t * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Parts `from`, `from` + `step`, ... of n, kFlight of them on their way at once; part_of(i): its number, negative for none.
template <int kFlight, class Part>
__device__ __forceinline__ void add_parts(const RowParts &p, int row, int lane, int from, int step, int n, Part part_of, float &m, float &l,
                                          float4 &acc)
{
#pragma unroll 1
    for (int i0 = from; i0 < n; i0 += kFlight * step) {
        float2 ml[kFlight];
        float4 o[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int i = i0 + k * step, part = i < n ? part_of(i) : -1;
            ml[k] = make_float2(-INFINITY, 0.f);
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (part >= 0) {
                ml[k] = p.ml[(size_t)part * p.rows + row];
                o[k] = reinterpret_cast<const float4 *>(p.o + ((size_t)part * p.rows + row) * kD)[lane];
            }
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k)
            add_part(m, l, acc, ml[k].x, ml[k].y, o[k]);
    }
}

// Joins the parts of items.  An item's parts are the end of the share before the first bound in it, and the shares that
// begin at its bounds (but between two equal ones).  Few items, of many parts each: a block takes rows of a sequence
// and head, `crew` of its 32 warps a row, which share out the parts.
constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(kJoinWarps * 32) row_join_kernel(const __grid_constant__ RowLaunch c, int shares, int crew)
{
    __shared__ float4 sum[kJoinWarps][32];
    __shared__ float2 ml_of[kJoinWarps];
    __shared__ Place places[kMaxRowShares + 1];
    __shared__ int lowest, highest;
    pdl_wait();
    pdl_trigger();
    const AttnArgs &a = c.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.cache.n_kv_heads, hk = blockIdx.x % a.cache.n_kv_heads;
    for (int i = tid; i <= shares; i += kJoinWarps * 32)
        places[i] = c.parts.bound[i].at;
    const Seq s = sequence(a, b);
    for (int k = 0; k < blocks_of(c.plan, s); ++k) {
        if (tid == 0) {
            lowest = shares;
            highest = 0;
        }
        __syncthreads();
        for (int base = 0; base < shares; base += kJoinWarps * 32) {
            const int i = base + tid;
            const uint32_t in = __ballot_sync(0xffffffffu, i > 0 && i < shares && places[i].cut > 0 && same_item(places[i], Place{b, hk, k, 0}));
            if (in && lane == 0) {
                atomicMin(&lowest, i + __ffs(in) - 1);
                atomicMax(&highest, i + 31 - __clz(in));
            }
        }
        __syncthreads();
        const int x = lowest, n = highest - x + 2;   // bounds in the item, and one more part
        const int rows = min(c.plan.tokens, s.n - k * c.plan.tokens) * a.G;
        const int step = kJoinWarps / crew, mate = warp % crew;   // rows of the block at a time
        for (int base = blockIdx.y * step; base < rows && x < shares; base += gridDim.y * step) {
            const int r = base + warp / crew;
            float m = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            add_parts<5>(c.parts, r, lane, mate, crew, r < rows ? n : 0, [&](int i) {
                const int share = x - 1 + i;
                if (i == 0)
                    return 2 * share + 1;
                return same_item(places[share], places[share + 1]) && places[share].cut == places[share + 1].cut ? -1 : 2 * share;
            }, m, l, acc);
            sum[warp][lane] = acc;
            if (lane == 0)
                ml_of[warp] = make_float2(m, l);
            __syncthreads();
            if (mate == 0 && r < rows) {
                float top = -INFINITY;
#pragma unroll 4
                for (int i = 0; i < crew; ++i)
                    top = fmaxf(top, ml_of[warp + i].x);
                const float zero = top == -INFINITY ? 0.f : top;
                l = 0.f;
                acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int i = 0; i < crew; ++i) {
                    const float f = ex2(ml_of[warp + i].x - zero);
                    const float4 o = sum[warp + i][lane];
                    l = fmaf(ml_of[warp + i].y, f, l);
                    acc.x = fmaf(o.x, f, acc.x);
                    acc.y = fmaf(o.y, f, acc.y);
                    acc.z = fmaf(o.z, f, acc.z);
                    acc.w = fmaf(o.w, f, acc.w);
                }
                write_row(a, s.t0 + k * c.plan.tokens + r / a.G, hk * a.G + r % a.G, lane, top, l, acc);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// Many items, of few parts each: a block takes the item that its bound is the first in; a warp takes a row.
__global__ void __launch_bounds__(256) row_joins_kernel(const __grid_constant__ RowLaunch c, int shares)
{
    pdl_wait();
    pdl_trigger();
    const AttnArgs &a = c.a;
    const Bound *const bound = c.parts.bound;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x = blockIdx.x + 1;
    const Bound here = bound[x];
    const Place at = here.at, before = bound[x - 1].at;
    if (at.cut == 0 || (same_item(at, before) && before.cut > 0))
        return;
    int n = 2;   // parts: a lane looks at a bound
    for (int base = x + 1; base < shares; base += 32) {
        const int i = base + lane;
        const int more = __popc(__ballot_sync(0xffffffffu, i < shares && same_item(bound[min(i, shares)].at, at)));
        n += more;
        if (more < 32)
            break;
    }
    const int first = at.k * c.plan.tokens, rows = min(c.plan.tokens, here.n - first) * a.G;
    for (int r = warp; r < rows; r += 8) {
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        add_parts<4>(c.parts, r, lane, 0, 1, n, [&](int i) {
            const int share = x - 1 + i;
            if (i == 0)
                return 2 * share + 1;
            const Place p = bound[share].at, next = bound[share + 1].at;
            return same_item(p, next) && p.cut == next.cut ? -1 : 2 * share;
        }, m, l, acc);
        write_row(a, here.t0 + first + r / a.G, at.hk * a.G + r % a.G, lane, m, l, acc);
    }
}

// ---- host side ----------------------------------------------------------------
static size_t carve(int nt, char *ws, RowParts *p)
{
    const int n = std::min(sm_count() * row_blocks(nt), kMaxRowShares), rows = 8 * nt;
    const size_t o_ml = ((n + 1) * sizeof(Bound) + 255) / 256 * 256;
    const size_t o_o = o_ml + (2 * n * (size_t)rows * sizeof(float2) + 255) / 256 * 256;
    if (p) {
        p->bound = reinterpret_cast<Bound *>(ws);
        p->ml = reinterpret_cast<float2 *>(ws + o_ml);
        p->o = reinterpret_cast<float *>(ws + o_o);
        p->rows = rows;
    }
    return o_o + 2 * n * (size_t)rows * kD * sizeof(float);
}

size_t row_attention_ws()
{
    size_t n = 0;
    for (int nt = 1; nt <= kMaxRowTiles; ++nt)
        n = std::max(n, carve(nt, nullptr, nullptr));
    return n;
}

// Tiles of 8 rows that hold a sequence's tokens by the group's heads, by the mean of tokens (the lengths are the device's).  So a
// chunk among many single tokens comes here with them, in blocks of as few tokens, each of which reads every key that it sees
// again: 440 tokens beside 64 single ones over 1500 keys, 32 over 8 heads, 120 us, in a call of their own and one for the tokens 60; 3000
// beside 512, 933 against 282; 32 over 4000 beside 31 over 4000 49 against 63.
static int row_tiles(int T, int B, int G) { return (int)(((T + (long long)B - 1) / B * G + 7) / 8); }

bool takes_rows(int T, int B, int G) { return row_tiles(T, B, G) <= kMaxRowTiles; }

template <int NT>
static constexpr size_t row_smem_bytes()
{
    return kRowWarps * row_stages(NT) * kStageBytes + sizeof(RowShared<NT>);
}

template <int NT>
static cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st)
{
    RowLaunch c{};
    c.a = a;
    const int Hkv = a.cache.n_kv_heads;
    c.plan.tokens = 8 * NT / a.G;
    const long long items = std::min<long long>(a.T, a.T / c.plan.tokens + a.B) * Hkv;   // at most
    int n = std::min(sm_count() * row_blocks(NT), kMaxRowShares);
    // Where no sequence can have more than 4 tiles none is cut, and nothing joined (one token over 300 keys 7.3 us of a
    // graph, cut 9.8); else, as the join is launched anyway, all but those of two (128 sequences of 1500 keys, 32 over 8
    // heads, 39 us; up to 4 tiles uncut 40, up to 8 42).
    const bool cuts = a.capacity > 4 * kTile;
    c.plan.uncut = cuts ? 2 : 4;
    if (!cuts)
        n = (int)std::min<long long>(n, items);
    c.plan.inverse = ~0ull / (unsigned long long)n;
    carve(NT, static_cast<char *>(a.ws), &c.parts);
    cudaError_t e = launch_pdl(a.softcap > 0.f ? row_attention_kernel<NT, true> : row_attention_kernel<NT, false>, dim3(n),
                               dim3(kRowThreads), row_smem_bytes<NT>(), st, 1, c);
    if (e != cudaSuccess || n < 2 || !cuts)
        return e;
    if ((long long)a.B * Hkv <= sm_count()) {
        // (five parts of a warp are on their way at once)
        int crew = 1;
        while (crew < kJoinWarps && 5 * crew * a.B * Hkv < n)
            crew *= 2;
        return launch_pdl(row_join_kernel, dim3(a.B * Hkv, 8 * NT * crew / kJoinWarps + 1), dim3(kJoinWarps * 32), 0, st, 1, c, n, crew);
    }
    return launch_pdl(row_joins_kernel, dim3(n - 1), dim3(256), 0, st, 1, c, n);
}

cudaError_t launch_row_attention(const AttnArgs &a, cudaStream_t st)
{
    switch (row_tiles(a.T, a.B, a.G)) {
    case 1:
        return launch_rows<1>(a, st);
    case 2:
        return launch_rows<2>(a, st);
    case 3:
        return launch_rows<3>(a, st);
    default:
        return launch_rows<4>(a, st);
    }
}

template <int NT>
static cudaError_t configure_rows()
{
    for (const void *f : {(const void *)row_attention_kernel<NT, false>, (const void *)row_attention_kernel<NT, true>}) {
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)row_smem_bytes<NT>());
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t configure_row_attention()
{
    for (auto f : {configure_rows<1>, configure_rows<2>, configure_rows<3>, configure_rows<4>})
        if (cudaError_t e = f())
            return e;
    return cudaSuccess;
}

}  // namespace retopk
