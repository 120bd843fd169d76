// chunk_attention.cu -- causal attention of ragged new tokens over a cache.
//
// Mathematics.  Token i of sequence b (n_b tokens, L_b rows) at position
// p = L_b - n_b + i sees keys j in (p - window, p]:  s_j = scale q.k_j (capped:
// softcap tanh(s_j / softcap)), out = sum_j exp(s_j) v_j / sum_j exp(s_j).  One
// pass over the keys, 128 at a time, with a running maximum m and sum l of each
// row:  P = exp(S - m), O <- O exp(m_old - m) + P V, l likewise.  Parts of a
// row's keys are joined by sum_p exp(m_p - M) O_p / sum_p exp(m_p - M) l_p.
//
// Rows.  A tile has up to 128 rows, floor(128 / G) tokens by the G query heads of
// one KV head (the row of token t, head g is t G + g), so every head of the group uses
// the K / V rows that were loaded once.
//
// Roles (10 warps, one CTA per SM): two groups of four softmax warps, each
// thread one row of its tile; one thread that issues the matrix instructions
// (S = Q K^T from shared memory, O += P V with P in tensor memory); one warp that
// issues the copies.  Tensor memory: S_0, S_1 (P_i takes the first half of
// S_i's columns), O_0, O_1, 128 columns each.
//   two tiles    (TWO):  the groups hold neighbouring tiles of tokens and share
//                every K / V tile.  For prompts.
//   two streams  (!TWO): both groups hold the same tile; group i takes the K / V
//                tiles of its parity, joined through shared memory at the end.
//                For a few tokens over a long history.
// Either way the matrix unit works on one group while the other is in its softmax.
//
// Division of work.  Items are (sequence, KV head, block of tokens) and have
// one unit of weight per key; the CTAs take equal shares of the sum, so a share may begin
// and end inside an item.  A CTA then leaves its unnormalised rows in the
// workspace, and the join kernel adds them up.  Shares, and with them the order of
// every sum, depend on the lengths alone.
#include <algorithm>

#include "prompt.cuh"
#include "tensor_map.cuh"

namespace retopk {

constexpr int kTile = 128;                       // rows and keys of a tile
constexpr int kAttnStages = 5;                   // K / V tiles in flight
constexpr int kAttnStageBytes = kTile * kD * 2;  // 32 KiB: [half of d][key][64]
constexpr int kHalfBytes = kAttnStageBytes / 2;
constexpr int kAttnThreads = 10 * 32;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr size_t kAttnSmem = 1024 + (2 + kAttnStages) * (size_t)kAttnStageBytes;
constexpr float kLazy = 8.f;                     // growth of m, in powers of two, that is left to the accumulators

// Where a share begins: an item and the number of its K / V tiles that belong
// to earlier shares.
struct Place {
    int b, hk, k, cut;
};

__device__ __forceinline__ bool same_item(const Place &x, const Place &y)
{
    return x.b == y.b && x.hk == y.hk && x.k == y.k;
}

struct Plan {
    int tokens;      // tokens of a block (two tiles', or one tile's)
    int overhead;    // weight of an item beside its keys
};

// Tokens, first token and rows of a sequence.
struct Seq {
    int n, t0, L;
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b)
{
    Seq s;
    s.t0 = b;
    s.n = 1;
    if (a.cu) {
        s.t0 = min(max(a.cu[b], 0), a.T);
        s.n = min(max(a.cu[b + 1], s.t0), a.T) - s.t0;
    }
    s.L = max(0, min(a.seqlens[b], a.capacity));
    return s;
}

// K / V tiles [lo, hi) that the tokens of block k see; one (wholly masked) tile
// where they see none, so that their rows are written.
__device__ __forceinline__ void tiles_of(const AttnArgs &a, const Plan &p, const Seq &s, int k, int &lo, int &hi)
{
    const int first = s.L - s.n + k * p.tokens, last = s.L - s.n + min(s.n, (k + 1) * p.tokens) - 1;
    hi = last < 0 ? 1 : last / kTile + 1;
    lo = a.window > 0 ? min(max(0, first - a.window + 1) / kTile, hi - 1) : 0;
}

__device__ __forceinline__ int blocks_of(const Plan &p, const Seq &s) { return (s.n + p.tokens - 1) / p.tokens; }

// Weight of the first k blocks of a sequence, for one head: block i weighs its
// last key's position, bounded by the window.
__device__ __forceinline__ long long weight(const AttnArgs &a, const Plan &p, const Seq &s, int k)
{
    const long long first = (long long)max(0, s.L - s.n) + min(p.tokens, s.n) + p.overhead;
    const long long most = a.window > 0 ? (long long)a.window + p.tokens + kTile + p.overhead : 1ll << 40;
    const long long grow = most <= first ? 0 : min((long long)k, (most - first) / p.tokens + 1);
    return grow * first + p.tokens * (grow * (grow - 1) / 2) + (k - grow) * most;
}

// The place u units behind the beginning of sequence b.
__device__ Place place_in(const AttnArgs &a, const Plan &p, const Seq &s, int b, long long u)
{
    const int nb = blocks_of(p, s);
    const long long each = weight(a, p, s, nb);
    Place r{b, (int)(u / each), 0, 0};
    u -= r.hk * each;
    int top = nb - 1;
    while (r.k < top) {   // the last block that begins at or before u
        const int mid = (r.k + top + 1) / 2;
        if (weight(a, p, s, mid) <= u)
            r.k = mid;
        else
            top = mid - 1;
    }
    int lo, hi;
    tiles_of(a, p, s, r.k, lo, hi);
    const long long begin = weight(a, p, s, r.k), all = weight(a, p, s, r.k + 1) - begin;
    // short items are cut into no small parts: joining costs more than it gives
    const int nt = hi - lo, grain = nt >= 64 ? 1 : nt >= 16 ? 2 : 4;
    const int x = (int)((u - begin) * nt / all);
    r.cut = (x + grain / 2) / grain * grain;
    if (r.cut >= nt) {   // the beginning of the next item
        r.cut = 0;
        if (++r.k == nb) {
            r.k = 0;
            if (++r.hk == a.cache.n_kv_heads) {
                r.hk = 0;
                ++r.b;
            }
        }
    }
    return r;
}

struct AttnShared {
    uint64_t kv_full[kAttnStages], kv_empty[kAttnStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t x_full, x_empty;   // the streams' join in shared memory
    uint64_t drained;
    Place bound[2];
    long long sums[kAttnThreads / 32 + 1];
    uint32_t tmem;
    int failed;
    float ml[2][kTile];   // stream 1's maximum and sum, for the join in shared memory
};

// ---- waits -------------------------------------------------------------------
// Bounded; once one has run out every other gives up at once.
__device__ __forceinline__ bool wait(AttnShared &sh, uint64_t *bar, uint32_t parity, uint32_t *status)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(&sh.failed))
            return false;
        if (clock64() - t0 > kWaitCycles) {
            *reinterpret_cast<volatile int *>(&sh.failed) = 1;
            if (status)
                atomicOr(status, RETOPK_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(AttnShared &sh, uint64_t *bar, uint32_t parity, uint32_t *status)
{
    return __all_sync(0xffffffffu, wait(sh, bar, parity, status));
}

// ---- tensor memory and matrix instructions (inline PTX) -------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

#define R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define R16(x, i) R4(x, i), R4(x, i + 4), R4(x, i + 8), R4(x, i + 12)
#define W4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define W16(x, i) W4(x, i), W4(x, i + 4), W4(x, i + 8), W4(x, i + 12)

// 32 columns of this warp's 32 lanes (a lane of the warp is a lane of the memory).
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *x)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : R16(x, 0), R16(x, 16)
        : "r"(addr));
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *x)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        W16(x, 0), W16(x, 16)
        : "memory");
}
#undef R4
#undef R16
#undef W4
#undef W16

// Shared-memory operand descriptor, 128-byte swizzle.  K-major operands (Q, K:
// [half of d][row][64]) step 1024 bytes from one 8-row group to the next; V is read
// MN-major ([half of d][key][64], d being N): 1024 bytes from one group of 8 keys
// to the next, a half's size from one block of 64 columns to the next.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 |
           2ull << 61;
}

// fp32 accumulators, bf16 operands, M = N = 128.
constexpr uint32_t kIdescS = 1u << 4 | 1u << 7 | 1u << 10 | (kTile / 8) << 17 | (kTile / 16) << 24;
constexpr uint32_t kIdescO = kIdescS | 1u << 16;   // B (V) is MN-major

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(kIdescS), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(kIdescO), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

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

// softcap tanh(s / softcap) in powers of two, with tanh(y) = 1 - 2 / (1 + e^2y).
__device__ __forceinline__ float capped(float s, float in, float cap2)
{
    return fmaf(-2.f * cap2, rcp(1.f + ex2(s * in)), cap2);
}

// ---- the walk over a share ---------------------------------------------------------
struct Walk {
    Place at, end;
    Seq seq;
    int loaded;   // sequence that seq describes
};

struct Segment {
    int b, hk, k;
    int lo, j0, j1, hi;   // K / V tiles [j0, j1) of the item's [lo, hi)
};

__device__ __forceinline__ bool next_segment(const AttnArgs &a, const Plan &p, Walk &w, Segment &s)
{
    for (;;) {
        if (w.at.b > w.end.b || w.at.b >= a.B ||
            (w.at.b == w.end.b &&
             (w.at.hk > w.end.hk || (w.at.hk == w.end.hk && (w.at.k > w.end.k || (w.at.k == w.end.k && w.at.cut >= w.end.cut))))))
            return false;
        if (w.loaded != w.at.b) {
            w.seq = sequence(a, w.at.b);
            w.loaded = w.at.b;
        }
        const int nb = blocks_of(p, w.seq);
        if (nb == 0) {
            w.at = Place{w.at.b + 1, 0, 0, 0};
            continue;
        }
        s.b = w.at.b;
        s.hk = w.at.hk;
        s.k = w.at.k;
        tiles_of(a, p, w.seq, s.k, s.lo, s.hi);
        s.j0 = s.lo + w.at.cut;
        s.j1 = same_item(w.at, w.end) ? s.lo + w.end.cut : s.hi;
        w.at.cut = 0;
        if (++w.at.k == nb) {
            w.at.k = 0;
            if (++w.at.hk == a.cache.n_kv_heads) {
                w.at.hk = 0;
                ++w.at.b;
            }
        }
        if (s.j1 > s.j0)
            return true;
    }
}

// Order in which a segment's K and V tiles go through the ring.
template <bool TWO>
__device__ __forceinline__ int ring_k(int t)
{
    return TWO ? 2 * t : t < 2 ? t : 2 * t - 1;
}
template <bool TWO>
__device__ __forceinline__ int ring_v(int t, int nt)
{
    return TWO || nt == 1 ? 2 * t + 1 : 2 + t + min(t, nt - 2);
}

// ---- workspace ----------------------------------------------------------------------
// Places of the n + 1 bounds, then for each CTA two parts (0: of an item that began in an
// earlier share, 1: of an item that goes on in the next) of `rows` rows: (m, l) pairs and
// 128 accumulators each.
struct Parts {
    Place *bound;
    float2 *ml;
    float *o;
    int rows;
};

struct AttnLaunch {
    AttnArgs a;
    Plan plan;
    Parts parts;
    int chunk;   // rows of one K / V copy (a page's, 128 at most)
};

template <bool TWO, bool CAP>
__global__ void __launch_bounds__(kAttnThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const AttnLaunch c)
{
    extern __shared__ unsigned char attn_smem[];
    __shared__ AttnShared sh;
    const AttnArgs &a = c.a;
    const Plan &plan = c.plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t qbuf = (smem_u32(attn_smem) + 1023) & ~1023u;   // two Q tiles, then the ring
    const uint32_t ring = qbuf + 2 * kAttnStageBytes;
    const int G = a.G, tile_tokens = kTile / G, Hkv = a.cache.n_kv_heads;

    if (tid == 0) {
        for (int s = 0; s < kAttnStages; ++s) {
            mbar_init(&sh.kv_full[s], 1);
            mbar_init(&sh.kv_empty[s], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.x_full, 4);
        mbar_init(&sh.x_empty, 4);
        mbar_init(&sh.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.failed = 0;
        sh.bound[0] = sh.bound[1] = Place{a.B, 0, 0, 0};
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share: the sum of all weights, then the places of its two bounds
    long long total = 0;
    for (int base = 0; base < a.B; base += kAttnThreads) {
        const int b = base + tid;
        if (b < a.B) {
            const Seq s = sequence(a, b);
            total += Hkv * weight(a, plan, s, blocks_of(plan, s));
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0)
        sh.sums[warp] = total;
    __syncthreads();
    total = 0;
    for (int i = 0; i < kAttnThreads / 32; ++i)
        total += sh.sums[i];
    const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
    long long before = 0;
    for (int base = 0; base < a.B; base += kAttnThreads) {
        __syncthreads();
        const int b = base + tid;
        long long w = 0;
        Seq s{0, 0, 0};
        if (b < a.B) {
            s = sequence(a, b);
            w = Hkv * weight(a, plan, s, blocks_of(plan, s));
        }
        long long up = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o)
                up += y;
        }
        if (lane == 31)
            sh.sums[warp] = up;
        __syncthreads();
        long long off = before;
        for (int i = 0; i < kAttnThreads / 32; ++i) {
            if (i < warp)
                off += sh.sums[i];
            before += sh.sums[i];
        }
        const long long from = off + up - w;
        if (w > 0 && u0 >= from && u0 < from + w)
            sh.bound[0] = place_in(a, plan, s, b, u0 - from);
        if (w > 0 && u1 >= from && u1 < from + w)
            sh.bound[1] = place_in(a, plan, s, b, u1 - from);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (tid == 0) {
        c.parts.bound[blockIdx.x] = sh.bound[0];
        if (blockIdx.x == gridDim.x - 1)
            c.parts.bound[gridDim.x] = sh.bound[1];
    }
    Walk w{sh.bound[0], sh.bound[1], Seq{0, 0, 0}, -1};
    Segment s;
    uint32_t used = 0;   // ring slots before this segment
    uint32_t segs = 0;

    if (warp == kLoadWarp) {
        // ================= copies =================
        bool ok = true;
        uint32_t issued = 0, q_issued = 0;
        const int pieces = kTile / c.chunk;   // per half
        while (ok && next_segment(a, plan, w, s)) {
            const int nt = s.j1 - s.j0, L = w.seq.L;
            if (lane == 0) {
                ok = segs == 0 || wait(sh, &sh.q_empty, (segs - 1) & 1, a.status);
                if (ok) {
                    const int rows = tile_tokens * G, t0 = w.seq.t0 + s.k * plan.tokens;
                    mbar_expect_tx(&sh.q_full, (TWO ? 2 : 1) * rows * kD * 2);
                    for (int i = 0; i < (TWO ? 2 : 1); ++i)
                        for (int h = 0; h < 2; ++h)
                            load_3d(qbuf + i * kAttnStageBytes + h * kHalfBytes, &qmap, h * 64, s.hk * G,
                                    t0 + i * tile_tokens, &sh.q_full);
                    ++q_issued;
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            // the ring's order: K ahead of V by one tile (or two, one for each stream)
            const int ahead = TWO ? 1 : 2;
            for (int x = -ahead; x < nt && ok; ++x) {
#pragma unroll
                for (int isk = 0; isk < 2; ++isk) {
                    const int t = isk ? x + ahead : x;
                    if (t < 0 || t >= nt || !ok)
                        continue;
                    const uint32_t u = used + (isk ? ring_k<TWO>(t) : ring_v<TWO>(t, nt));
                    const int st = u % kAttnStages;
                    // rows of this lane's copy
                    const int half = lane & 1, piece = lane >> 1, pos = (s.j0 + t) * kTile + piece * c.chunk;
                    int z = a.cache.n_pages * Hkv, y = 0;   // outside: read as zeros
                    if (piece < pieces && pos < L) {
                        int page = s.b;
                        y = pos;
                        if (a.cache.table) {
                            page = a.cache.table[(long long)s.b * a.cache.table_width + pos / a.cache.page_rows];
                            y = pos % a.cache.page_rows;
                        }
                        if ((uint32_t)page < (uint32_t)a.cache.n_pages)
                            z = page * Hkv + s.hk;
                        else if (a.status)
                            atomicOr(a.status, RETOPK_STATUS_BAD_PAGE);
                    }
                    int good = 1;
                    if (lane == 0) {
                        if (u >= kAttnStages)
                            good = wait(sh, &sh.kv_empty[st], (u / kAttnStages - 1) & 1, a.status);
                        if (good)
                            mbar_expect_tx(&sh.kv_full[st], kAttnStageBytes);
                    }
                    ok = __shfl_sync(0xffffffffu, good, 0);
                    if (ok) {
                        issued = u + 1;
                        if (piece < pieces)
                            load_3d(ring + st * kAttnStageBytes + half * kHalfBytes + piece * c.chunk * 128,
                                    isk ? &kmap : &vmap, half * 64, y, z, &sh.kv_full[st]);
                    }
                }
            }
            used += 2 * nt;
            ++segs;
        }
        // a wait ran out: the copies in flight are waited for before the memory goes
        if (*reinterpret_cast<volatile int *>(&sh.failed) && lane == 0) {
            const long long t0 = clock64();
            for (uint32_t u = issued > kAttnStages ? issued - kAttnStages : 0; u < issued; ++u)
                while (!mbar_try_wait(&sh.kv_full[u % kAttnStages], (u / kAttnStages) & 1) && clock64() - t0 < kWaitCycles)
                    ;
            while (q_issued && !mbar_try_wait(&sh.q_full, (q_issued - 1) & 1) && clock64() - t0 < kWaitCycles)
                ;
        }
    } else if (warp == kMmaWarp) {
        // ================= matrix instructions =================
        if (lane == 0) {
            bool ok = true;
            uint32_t done[2] = {0, 0};   // tiles of each group before this segment
            // S_i of the segment's tile t
            auto scores = [&](int i, int t) {
                const uint32_t u = used + ring_k<TWO>(t);
                const int st = u % kAttnStages;
                if (!wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status))
                    return false;
                tc_fence_after();
                const uint32_t qa = qbuf + (TWO ? i * kAttnStageBytes : 0), ka = ring + st * kAttnStageBytes;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t o = (x >> 2) * kHalfBytes + (x & 3) * 32;
                    mma_ss(tmem + i * kTile, operand(qa + o, 0), operand(ka + o, 0), x > 0);
                }
                tc_commit(&sh.s_full[i]);
                if (!TWO || i == 1)
                    tc_commit(&sh.kv_empty[st]);
                return true;
            };
            while (ok && next_segment(a, plan, w, s)) {
                const int nt = s.j1 - s.j0;
                const int m[2] = {TWO ? nt : (nt + 1) / 2, TWO ? nt : nt / 2};
                auto tile = [&](int i, int t) { return TWO ? t : 2 * t + i; };
                ok = wait(sh, &sh.q_full, segs & 1, a.status);
                for (int i = 0; i < 2 && ok; ++i)
                    if (m[i] > 0)
                        ok = scores(i, tile(i, 0));
                if (ok && m[0] == 1)
                    tc_commit(&sh.q_empty);
                for (int t = 0; t < m[0] && ok; ++t) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (t >= m[i] || !ok)
                            continue;
                        const uint32_t u = used + ring_v<TWO>(tile(i, t), nt);
                        const int st = u % kAttnStages;
                        ok = wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status) &&
                             wait(sh, &sh.p_full[i], (done[i] + t) & 1, a.status);
                        if (!ok)
                            continue;
                        tc_fence_after();
                        const uint32_t va = ring + st * kAttnStageBytes;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            mma_ts(tmem + (2 + i) * kTile, tmem + i * kTile + x * 8, operand(va + x * 2048, kHalfBytes),
                                   t > 0 || x > 0);
                        tc_commit(&sh.o_full[i]);
                        if (!TWO || i == 1)
                            tc_commit(&sh.kv_empty[st]);
                        if (t + 1 < m[i])
                            ok = scores(i, tile(i, t + 1));
                    }
                    // the last use of Q
                    if (ok && t + 2 == m[0])
                        tc_commit(&sh.q_empty);
                }
                used += 2 * nt;
                done[0] += m[0];
                done[1] += m[1];
                ++segs;
            }
            if (!ok) {   // a wait ran out: the instructions in flight end before the tensor memory goes
                tc_commit(&sh.drained);
                const long long t0 = clock64();
                while (!mbar_try_wait(&sh.drained, 0) && clock64() - t0 < kWaitCycles)
                    ;
            }
        }
        __syncwarp();
    } else if (warp < kMmaWarp) {
        // ================= softmax =================
        const int i = warp >> 2, r = tid & (kTile - 1);
        const uint32_t quarter = (uint32_t)(warp & 3) << 21;   // this warp's lanes of the tensor memory
        const uint32_t s_addr = tmem + i * kTile + quarter, o_addr = tmem + (2 + i) * kTile + quarter;
        const float scale2 = a.scale * 1.4426950408889634f;     // scores in powers of two
        const float cap2 = a.softcap * 1.4426950408889634f;
        const float cap_in = CAP ? 2.f * scale2 / a.softcap : 0.f;   // e^2y = 2^(cap_in s)
        bool ok = true;
        uint32_t done = 0;
        while (ok && next_segment(a, plan, w, s)) {
            const int nt = s.j1 - s.j0, m_tiles = TWO ? nt : (nt + 1 - i) / 2;
            const int tok = s.k * plan.tokens + (TWO ? i * tile_tokens : 0) + r / G;   // in the sequence
            const bool valid = r < tile_tokens * G && tok < w.seq.n;
            const bool work = __any_sync(0xffffffffu, valid);
            const int pos = w.seq.L - w.seq.n + tok;
            const int low = a.window > 0 ? pos - a.window + 1 : 0;
            // every key of tiles [lowest / 128 rounded up, highest / 128) is seen by all rows of the warp
            const int all_hi = __reduce_min_sync(0xffffffffu, valid ? pos : INT32_MAX);
            const int all_lo = __reduce_max_sync(0xffffffffu, valid ? low : 0);
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < m_tiles && ok; ++t) {
                const int j = s.j0 + (TWO ? t : 2 * t + i);
                ok = warp_wait(sh, &sh.s_full[i], (done + t) & 1, a.status);
                if (!ok)
                    break;
                tc_fence_after();
                if (work) {
                    // The scores are read twice, half a row at a time (64 registers): for the maximum, then for the weights.
                    const bool part = j * kTile + kTile - 1 > all_hi || j * kTile < all_lo;
                    const int top = pos - j * kTile, bottom = low - j * kTile;
                    float mx = -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[64];
                        tc_ld32(s_addr + 64 * h, x);
                        tc_ld32(s_addr + 64 * h + 32, x + 32);
                        tc_wait_ld();
                        float *f = reinterpret_cast<float *>(x);
                        if (part) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                f[e] = 64 * h + e <= top && 64 * h + e >= bottom ? f[e] : -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 2)
                            mx = fmaxf(mx, fmaxf(f[e], f[e + 1]));
                    }
                    // (the cap does not change the order of scores)
                    mx = CAP && mx != -INFINITY ? capped(mx, cap_in, cap2) : mx * scale2;
                    // The maximum that the weights are taken against follows the true one only
                    // when it has grown by more than 2^8: until then the weights are at most 256, and the
                    // accumulators need no pass over them.
                    const bool grow = m != -INFINITY && mx > m + kLazy;
                    if (__any_sync(0xffffffffu, grow)) {
                        ok = warp_wait(sh, &sh.o_full[i], (done + t - 1) & 1, a.status);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const float f2 = grow ? ex2(m - mx) : 1.f;
                        l *= f2;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t o[32];
                            tc_ld32(o_addr + 32 * q, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f2);
                            tc_st32(o_addr + 32 * q, o);
                        }
                    }
                    if (grow || m == -INFINITY)
                        m = mx;
                    const float base = m == -INFINITY ? 0.f : m;
                    float sum[4] = {};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[64];
                        tc_ld32(s_addr + 64 * h, x);
                        tc_ld32(s_addr + 64 * h + 32, x + 32);
                        tc_wait_ld();
                        float *f = reinterpret_cast<float *>(x);
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            f[e] = CAP ? capped(f[e], cap_in, cap2) - base : fmaf(f[e], scale2, -base);
                        if (part) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                f[e] = 64 * h + e <= top && 64 * h + e >= bottom ? f[e] : -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            f[e] = ex2(f[e]);
                            f[e + 1] = ex2(f[e + 1]);
                            sum[(e >> 1) & 3] += f[e] + f[e + 1];
                            x[e >> 1] = bf16x2(f[e], f[e + 1]);
                        }
                        // P takes the columns of scores that are done with
                        tc_st32(s_addr + 32 * h, x);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc_wait_st();
                }
                // V rows past the length may hold anything, and 0 times that is not 0: they are
                // cleared where the tile is used first
                if ((!TWO || i == 0) && (j + 1) * kTile > w.seq.L) {
                    const uint32_t u = used + ring_v<TWO>(j - s.j0, nt);
                    const int st = u % kAttnStages;
                    ok = warp_wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status);
                    if (!ok)
                        break;
                    if (j * kTile + r >= w.seq.L) {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             ring + st * kAttnStageBytes + (q >> 3) * kHalfBytes + r * 128 + (q & 7) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.p_full[i]);
            }
            done += m_tiles;
            if (ok && m_tiles > 0)
                ok = warp_wait(sh, &sh.o_full[i], (done - 1) & 1, a.status);
            tc_fence_after();
            // ---- the rows' end: a share's part, or the output
            const bool whole = s.j0 == s.lo && s.j1 == s.hi;
            if (!TWO) {
                // stream 1's half joins stream 0's through shared memory, 64 columns at a time
                float *const other = reinterpret_cast<float *>(attn_smem + (qbuf - smem_u32(attn_smem)) + kAttnStageBytes);
                float f0 = 1.f, f1 = 0.f;
                for (int h = 0; h < 2; ++h) {
                    // (each of the two halves is one phase, so a segment takes two and the parities stay)
                    if (i == 1 && ok && (h == 1 || segs > 0))
                        ok = warp_wait(sh, &sh.x_empty, h ^ 1, a.status);
                    if (h == 0 && i == 1 && ok) {
                        sh.ml[0][r] = m;
                        sh.ml[1][r] = l;
                    }
                    if (i == 1 && work && ok) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t o[32];
                            tc_ld32(o_addr + h * 64 + 32 * q, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                other[(q * 32 + e) * kTile + r] = __uint_as_float(o[e]);
                        }
                    }
                    if (i == 1) {
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&sh.x_full);
                    } else if (ok) {
                        ok = warp_wait(sh, &sh.x_full, h, a.status);
                    }
                    if (i == 0 && work && ok) {
                        if (h == 0) {
                            const float m1 = sh.ml[0][r], mm = fmaxf(m, m1), b0 = mm == -INFINITY ? 0.f : mm;
                            f0 = ex2(m - b0);
                            f1 = ex2(m1 - b0);
                            l = l * f0 + (nt > 1 ? sh.ml[1][r] * f1 : 0.f);
                            m = mm;
                        }
                        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t o[32];
                            tc_ld32(o_addr + h * 64 + 32 * q, o);
                            tc_wait_ld();
                            float y[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                y[e] = __uint_as_float(o[e]) * f0;
                                if (nt > 1)
                                    y[e] = fmaf(other[(q * 32 + e) * kTile + r], f1, y[e]);
                                y[e] *= inv;
                            }
                            if (!valid)
                                continue;
                            const int col = h * 64 + q * 32;
                            if (whole) {
                                uint16_t *dst = a.out + (w.seq.t0 + tok) * a.out_stride + (s.hk * G + r % G) * kD + col;
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    *reinterpret_cast<uint4 *>(dst + e) =
                                        make_uint4(bf16x2(y[e], y[e + 1]), bf16x2(y[e + 2], y[e + 3]),
                                                   bf16x2(y[e + 4], y[e + 5]), bf16x2(y[e + 6], y[e + 7]));
                            } else {
                                float *dst = c.parts.o + ((size_t)(2 * blockIdx.x + (s.j0 == s.lo)) * c.parts.rows + r) * kD + col;
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4 *>(dst + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                            }
                        }
                    }
                    if (i == 0) {
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&sh.x_empty);
                    }
                }
            } else if (work && ok) {
                const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    tc_ld32(o_addr + 32 * q, o);
                    tc_wait_ld();
                    if (!valid)
                        continue;
                    float *y = reinterpret_cast<float *>(o);
                    if (whole) {
                        uint16_t *dst = a.out + (w.seq.t0 + tok) * a.out_stride + (s.hk * G + r % G) * kD + q * 32;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(dst + e) =
                                make_uint4(bf16x2(y[e] * inv, y[e + 1] * inv), bf16x2(y[e + 2] * inv, y[e + 3] * inv),
                                           bf16x2(y[e + 4] * inv, y[e + 5] * inv), bf16x2(y[e + 6] * inv, y[e + 7] * inv));
                    } else {
                        float *dst = c.parts.o +
                                     ((size_t)(2 * blockIdx.x + (s.j0 == s.lo)) * c.parts.rows + i * kTile + r) * kD + q * 32;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    }
                }
            }
            if (valid && ok && (TWO || i == 0)) {
                if (!whole)
                    c.parts.ml[(size_t)(2 * blockIdx.x + (s.j0 == s.lo)) * c.parts.rows + (TWO ? i * kTile : 0) + r] =
                        make_float2(m, l);
                else if (a.lse)
                    a.lse[(size_t)(w.seq.t0 + tok) * a.Hq + s.hk * G + r % G] =
                        l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
            used += 2 * nt;
            ++segs;
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the parts of the item that bound blockIdx.x + 1 cuts first: a warp a row.
template <bool TWO>
__global__ void __launch_bounds__(256) join_kernel(const AttnLaunch c, int shares)
{
    pdl_wait();
    pdl_trigger();
    const AttnArgs &a = c.a;
    const int x = blockIdx.x + 1, lane = threadIdx.x & 31;
    const Place at = c.parts.bound[x], prev = c.parts.bound[x - 1];
    if (at.cut == 0 || (same_item(at, prev) && prev.cut > 0))
        return;
    // parts: share x - 1's part 1, then part 0 of shares x, x + 1, ... while they begin in the item
    int end = x + 1;
    while (end < shares && same_item(c.parts.bound[end], at))
        ++end;
    const Seq s = sequence(a, at.b);
    const int tile_tokens = kTile / a.G, per_tile = tile_tokens * a.G;
    const int rows = TWO ? kTile + per_tile : per_tile;
    for (int r = blockIdx.y * 8 + threadIdx.x / 32; r < rows; r += gridDim.y * 8) {
        const int in = r & (kTile - 1);
        const int tok = at.k * c.plan.tokens + (r >= kTile ? tile_tokens : 0) + in / a.G;
        if (in >= per_tile || tok >= s.n)
            continue;
        auto index = [&](int i) { return (size_t)(2 * (x - 1 + i) + (i == 0)) * c.parts.rows + r; };
        // a share between two equal cuts has no part
        auto there = [&](int i) {
            const int y = x - 1 + i;
            return i == 0 || y + 1 > shares || !same_item(c.parts.bound[y + 1], at) ||
                   c.parts.bound[y + 1].cut > c.parts.bound[y].cut;
        };
        const int n = end - x + 1;
        float mm = -INFINITY;
        for (int i = lane; i < n; i += 32)
            if (there(i))
                mm = fmaxf(mm, c.parts.ml[index(i)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        const float base = mm == -INFINITY ? 0.f : mm;
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < n; i0 += 32) {
            float f = 0.f;
            if (i0 + lane < n && there(i0 + lane)) {
                const float2 ml = c.parts.ml[index(i0 + lane)];
                f = ex2(ml.x - base);
                l += f * ml.y;
            }
            const int most = min(32, n - i0);
#pragma unroll 8
            for (int i = 0; i < most; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                if (fi != 0.f) {   // (parts without a row's keys, and those that are not there)
                    const float4 o = reinterpret_cast<const float4 *>(c.parts.o + index(i0 + i) * kD)[lane];
                    acc.x = fmaf(fi, o.x, acc.x);
                    acc.y = fmaf(fi, o.y, acc.y);
                    acc.z = fmaf(fi, o.z, acc.z);
                    acc.w = fmaf(fi, o.w, acc.w);
                }
            }
        }
        l = warp_sum(l);
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t t = s.t0 + tok;
        const int h = at.hk * a.G + in % a.G;
        *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + h * kD + lane * 4) =
            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
        if (a.lse && lane == 0)
            a.lse[t * a.Hq + h] = l > 0.f ? (mm + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

// ---- host side ----------------------------------------------------------------
// Two tiles of tokens a block where the sequences have more tokens than a tile
// on average; else one tile and two streams of keys.
static bool two_tiles(int T, int B, int G) { return T / B > kTile / G; }

// Rows of a part.
static int part_rows(int T, int G, bool two)
{
    return two ? 2 * kTile : (int)std::min<long long>(kTile, ((long long)T * G + 7) / 8 * 8);
}

static size_t carve(int T, int B, int Hq, int Hkv, char *ws, Parts *p)
{
    const int G = Hq / Hkv, n = sm_count();
    const size_t rows = part_rows(T, G, two_tiles(T, B, G));
    const size_t o_ml = ((n + 1) * sizeof(Place) + 255) / 256 * 256;
    const size_t o_o = o_ml + (2 * n * rows * sizeof(float2) + 255) / 256 * 256;
    if (p) {
        p->bound = reinterpret_cast<Place *>(ws);
        p->ml = reinterpret_cast<float2 *>(ws + o_ml);
        p->o = reinterpret_cast<float *>(ws + o_o);
        p->rows = (int)rows;
    }
    return o_o + 2 * n * rows * kD * sizeof(float);
}

size_t chunk_attention_ws(int T, int B, int Hq, int Hkv) { return carve(T, B, Hq, Hkv, nullptr, nullptr); }

static bool make_map(CUtensorMap *map, const void *p, cuuint64_t d1, cuuint64_t d2, cuuint64_t s1, cuuint64_t s2, int b1,
                     int b2)
{
    EncodeTiledFn fn = encode_fn();
    const cuuint64_t dims[3] = {kD, d1, d2}, strides[2] = {s1, s2};
    const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, one[3] = {1, 1, 1};
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TWO>
static cudaError_t launch_mode(const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const AttnLaunch &c,
                               cudaStream_t st)
{
    const int n = sm_count();
    auto kernel = c.a.softcap > 0.f ? chunk_attention_kernel<TWO, true> : chunk_attention_kernel<TWO, false>;
    cudaError_t e = launch_pdl(kernel, dim3(n), dim3(kAttnThreads), kAttnSmem, st, 1, qm, km, vm, c);
    if (e != cudaSuccess || n < 2)
        return e;
    return launch_pdl(join_kernel<TWO>, dim3(n - 1, TWO ? 4 : (c.parts.rows + 7) / 8), dim3(256), 0, st, 1, c, n);
}

cudaError_t launch_chunk_attention(const AttnArgs &a, cudaStream_t st)
{
    AttnLaunch c{};
    c.a = a;
    const int Hkv = a.cache.n_kv_heads, tokens = kTile / a.G;
    const bool two = two_tiles(a.T, a.B, a.G);
    c.plan.tokens = two ? 2 * tokens : tokens;
    c.plan.overhead = two ? 128 : 256;
    carve(a.T, a.B, a.Hq, Hkv, static_cast<char *>(a.ws), &c.parts);
    c.chunk = kTile;
    if (a.cache.table)
        while (a.cache.page_rows % c.chunk)
            c.chunk /= 2;
    CUtensorMap qm, km, vm;
    const cuuint64_t page = (cuuint64_t)a.cache.page_rows * kD * 2, pages = (cuuint64_t)a.cache.n_pages * Hkv;
    if (!make_map(&qm, a.q, a.Hq, a.T, kD * 2, a.q_stride * 2, a.G, tokens) ||
        !make_map(&km, a.cache.k, a.cache.page_rows, pages, kD * 2, page, c.chunk, 1) ||
        !make_map(&vm, a.cache.v, a.cache.page_rows, pages, kD * 2, page, c.chunk, 1))
        return cudaErrorInvalidValue;
    return two ? launch_mode<true>(qm, km, vm, c, st) : launch_mode<false>(qm, km, vm, c, st);
}

cudaError_t configure_chunk_attention()
{
    cudaError_t e = cudaSuccess;
    auto set = [&](const void *f) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAttnSmem);
    };
    set((const void *)chunk_attention_kernel<true, true>);
    set((const void *)chunk_attention_kernel<true, false>);
    set((const void *)chunk_attention_kernel<false, true>);
    set((const void *)chunk_attention_kernel<false, false>);
    return e;
}

}  // namespace retopk
