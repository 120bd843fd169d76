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
// Roles (12 warps, one CTA per SM; one of them idle): two groups of four softmax
// warps, each thread one row of its tile, whose 128 scores stay in registers; one
// thread that issues the matrix instructions (S = Q K^T from shared memory, O += P V
// with P in tensor memory); one warp that issues the copies; one that walks the
// CTA's share and tells the others, ahead of time, the segments of items in it.  Shared
// memory leaves the L1 no room, so a spilled register costs a trip to the L2: what a
// warp keeps between tiles is small.  Tensor memory: S_0, S_1 (P_i takes the first half of
// S_i's columns), O_0, O_1, 128 columns each.
//   two tiles    (TWO):  the groups hold neighbouring tiles of tokens and share
//                every K / V tile.  For prompts.
//   two streams  (!TWO): both groups hold the same tile; group i takes the K / V
//                tiles of its parity, joined at the end.
//                For a few tokens over a long history.
// Either way the matrix unit works on one group while the other is in its softmax.
//
// Division of work.  Items are (sequence, KV head, block of tokens) and have
// one unit of weight per key; the CTAs take equal shares of the sum, so a share may begin
// and end inside an item.  A CTA then leaves its unnormalised rows in the
// workspace, and the join kernel adds them up.  Shares, and with them the order of
// every sum, depend on the lengths alone.
//
// Rounding.  Scores, maxima, sums, parts and accumulators have 32 bits.  P is rounded to bf16, as the matrix
// instruction takes both operands in one type and V is bf16: an output is off by up to 2^-8 sum_j p_j |v_j| for it
// (against 64 bits 0.0019 to 0.0023 of the outputs' size, where 32-bit weights give 0.0017, the output's own rounding).
//
// Measured (28 query heads over 4 KV heads but where said).  4096 tokens over 32768 keys: 1233 us,
// 1.47 PFLOP/s, held by the GPU's power limit (1133 us in short bursts, held by the chain softmax -> P V ->
// Q K of each group).  One token over 131072 keys: 51 us, 5.2 TB/s, of which the stream
// takes 40.  61 ragged sequences of 9000 keys, 32 over 8 heads: 219 us, 6.7 TB/s, 98 % of a plain copy's rate.  3 x 333
// tokens in windows of 4096 keys, 16 over 2 heads: 53 us; capped, 65 us, and 80 with scores past half the cap.
// What an item costs beside its tiles shows where items are short or shares small: a prompt of 2048 tokens 60 us and
// of 8192 388 (0.50 and 1.24 PFLOP/s), 128 sequences of 1500 keys, 32 over 8 heads, 130 us (3.9 TB/s), 36 tokens over
// 17663 keys, 16 over 2 heads, 39 us (0.13 PFLOP/s), one token over 300 keys 11.7 us.
#include <math.h>

#include <algorithm>

#include "prompt.cuh"
#include "tensor_map.cuh"

namespace retopk {

constexpr int kTile = 128;                       // rows and keys of a tile
constexpr int kAttnStages = 5;                   // K / V tiles in flight
constexpr int kAttnStageBytes = kTile * kD * 2;  // 32 KiB: [half of d][key][64]
constexpr int kHalfBytes = kAttnStageBytes / 2;
constexpr int kAttnThreads = 12 * 32;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kWalkWarp = 10;
constexpr int kSegments = 4;                     // known ahead
constexpr int kHalf = kTile / 2;                 // keys of half a tile
// registers of a thread after the split: 2 x 128 x 208 + 128 x 88 = 384 x 168, what the block is launched with
// (4096 tokens over 32768 keys in short bursts: 1133 us; with 216 and 72 or 224 and 56, 1190)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
// Weight of an item beside its keys: what beginning and ending it costs, in keys.  (A prompt
// of 8192 tokens: 494 us with 128, 386 with 512, 399 with 1024; 128 sequences of 1500 keys, 32 over 8 heads: 135 us
// with 256, 126 with 512, 128 with 1024.)
constexpr int kItemWeight = 512;
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
    int tokens;                    // tokens of a block (two tiles', or one tile's)
    unsigned long long inverse;    // 2^64 / shares
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
    const int first = max(0, s.L - s.n) + min(p.tokens, s.n) + kItemWeight;
    int grow = k;
    long long flat = 0;
    if (a.window > 0 && a.window < kMaxLen) {
        const int most = a.window + p.tokens + kTile + kItemWeight;
        grow = most <= first ? 0 : min(k, (most - first) / p.tokens + 1);
        flat = (long long)(k - grow) * most;
    }
    return (long long)grow * first + (long long)p.tokens * grow * (grow - 1) / 2 + flat;
}

// The place u units behind the beginning of sequence b.
__device__ __forceinline__ Place place_in(const AttnArgs &a, const Plan &p, const Seq &s, int b, long long u)
{
    const int nb = blocks_of(p, s);
    const long long each = weight(a, p, s, nb);
    Place r{b, 0, 0, 0};
    if (a.cache.n_kv_heads > 32) {
        r.hk = (int)(u / each);
        u -= r.hk * each;
    } else {
        for (; u >= each; u -= each)
            ++r.hk;
    }
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
    const long long begin = weight(a, p, s, r.k);
    // short items are cut into no small parts: joining costs more than it gives (8 sequences of 50 tokens over 1000
    // keys 29 us, cut anywhere 32); long ones anywhere (4 of 19 over 9000 keys 32 us, by fours 34)
    const int nt = hi - lo, grain = nt >= 64 ? 1 : nt >= 16 ? 2 : 4;
    // (half the item's own weight lies before its first tile, half behind its last)
    const int in = (int)(u - begin) - kItemWeight / 2, keys = (int)(weight(a, p, s, r.k + 1) - begin) - kItemWeight;
    const int x = (int)(__fdividef((float)max(in, 0), (float)keys) * nt);
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

// ---- the walk over a share ---------------------------------------------------------
struct Walk {
    Place at, end;
    Seq seq;
    int loaded;   // sequence that seq describes
};

struct Segment {
    int b, hk, k;
    int lo, j0, j1, hi;   // K / V tiles [j0, j1) of the item's [lo, hi)
    Seq seq;
    int more;             // 0: the share is done
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
        if (s.j1 > s.j0) {
            s.seq = w.seq;
            return true;
        }
    }
}

struct AttnShared {
    uint64_t kv_full[kAttnStages], kv_empty[kAttnStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2][2], o_full[2];
    uint64_t x_full, x_empty;   // the streams' join in shared memory
    uint64_t drained, nobody[2];
    Place bound[2];
    Seq first;                 // the sequence that bound[0] was found in
    int first_b;
    Segment segments[kSegments];
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    long long sums[kAttnThreads / 32 + 1];
    uint32_t tmem;
    int failed;
};
// two Q tiles, the ring, AttnShared; with one Q tile the second's place serves the streams' join (1 KB)
constexpr size_t kAttnSmem = (2 + kAttnStages) * (size_t)kAttnStageBytes + sizeof(AttnShared);
static_assert(kAttnSmem <= kMaxDynSmem, "one CTA's shared memory");

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

// Segment number n of the share; false when there is none (or a wait ran out).
__device__ __forceinline__ bool segment(AttnShared &sh, uint32_t n, uint32_t *status)
{
    const uint32_t k = n % kSegments;
    return warp_wait(sh, &sh.seg_full[k], (n / kSegments) & 1, status) && sh.segments[k].more;
}

// This warp is done with it.
__device__ __forceinline__ void segment_done(AttnShared &sh, uint32_t n)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sh.seg_empty[n % kSegments]);
}

// ---- the walk: one lane ------------------------------------------------------------
__device__ __forceinline__ void walk_share(const AttnArgs &a, const Plan &plan, AttnShared &sh)
{
    Walk w{sh.bound[0], sh.bound[1], sh.first, sh.first_b};
    for (uint32_t n = 0;; ++n) {
        const uint32_t k = n % kSegments;
        if (n >= kSegments && !wait(sh, &sh.seg_empty[k], (n / kSegments - 1) & 1, a.status))
            return;
        const int more = next_segment(a, plan, w, sh.segments[k]);
        sh.segments[k].more = more;
        mbar_arrive(&sh.seg_full[k]);
        if (!more)
            return;
    }
}

// ---- tensor memory and matrix instructions (inline PTX) -------------------------
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

#define R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define R16(x, i) R4(x, i), R4(x, i + 4), R4(x, i + 8), R4(x, i + 12)
#define RW4(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3])
#define RW16(x, i) RW4(x, i), RW4(x, i + 4), RW4(x, i + 8), RW4(x, i + 12)
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

// The wait for loads, with the registers that they fill: nothing may read these before it.
__device__ __forceinline__ void tc_wait_ld32(uint32_t *x)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RW16(x, 0), RW16(x, 16)::"memory");
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t *x)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RW16(x, 0)::"memory");
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *x)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        W16(x, 0), W16(x, 16)
        : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t *x)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : R16(x, 0)
                 : "r"(addr));
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *x)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            addr),
        W16(x, 0)
        : "memory");
}
#undef R4
#undef R16
#undef RW4
#undef RW16
#undef W4
#undef W16

// Shared-memory operand descriptor, 128-byte swizzle.  K-major operands (Q, K:
// [half of d][row][64]) step 1024 bytes from one 8-row group to the next; V is read
// MN-major ([half of d][key][64], d being N): 1024 bytes from one group of 8 keys
// to the next, a half's size from one block of 64 columns to the next.  The address
// is all that changes, in the low word.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDescLead = (uint32_t)(kHalfBytes >> 4) << 16;   // V's block of columns

// fp32 accumulators, bf16 operands, M = N = 128.
constexpr uint32_t kIdescS = 1u << 4 | 1u << 7 | 1u << 10 | (kTile / 8) << 17 | (kTile / 16) << 24;
constexpr uint32_t kIdescO = kIdescS | 1u << 16;   // B (V) is MN-major

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHigh), "r"(kIdescS), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHigh), "r"(kIdescO), "r"(accumulate)
        : "memory");
}

// One lane of the (converged) warp, the same each time.
__device__ __forceinline__ bool elected()
{
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
    return x != 0;
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], "
        "[%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
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

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The largest one, NaN where one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// softcap tanh(s / softcap) in powers of two, with tanh(y) = 1 - 2 / (1 + e^2y).
__device__ __forceinline__ float capped(float s, float in, float cap2)
{
    return fmaf(-2.f * cap2, rcp(1.f + ex2(s * in)), cap2);
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

constexpr int kMaxShares = 255;   // CTAs of a launch, one for each SM

// ---- workspace ----------------------------------------------------------------------
// Places of the n + 1 bounds, then for each CTA two parts (0: of an item that began in an
// earlier share, 1: of an item that goes on in the next) of `rows` rows: (m, l) pairs, and
// the accumulators as [column / 4][row][4], so that a warp's rows lie side by side.
struct Bound {
    Place at;
    int n, t0;   // of the place's sequence, where it is inside an item
};
struct Parts {
    Bound *bound;
    float2 *ml;
    float4 *o;
    int rows;
};

struct AttnLaunch {
    AttnArgs a;
    Plan plan;
    Parts parts;
    int chunk;    // rows of one K / V copy (a page's, 128 at most)
    int shares;   // CTAs
    long long items;   // at most
    // tanh(y) = y (1 + t (b_0 + b_1 t + b_2 t^2)), t = y^2, for |y| <= 1/2: b fitted at Chebyshev nodes for
    // the smallest largest error (6.4e-7 of the value).  Here for raw scores: y = s scale / softcap,
    // in powers of two, so cap_poly[i] = b_i (scale / softcap)^(2 i + 2) scale log2(e); cap_near: the largest |s|.
    float cap_poly[3], cap_near;
};

// ---- the copies --------------------------------------------------------------------
template <bool TWO>
__device__ __forceinline__ void copies(const AttnLaunch &c, AttnShared &sh, const CUtensorMap &qmap,
                                       const CUtensorMap &kmap, const CUtensorMap &vmap, uint32_t qbuf, uint32_t ring,
                                       int lane)
{
    const AttnArgs &a = c.a;
    const int Hkv = a.cache.n_kv_heads, tile_tokens = kTile / a.G;
    const int half = lane & 1, piece = lane >> 1, pieces = kTile / c.chunk;   // this lane's copy
    // a few tokens' keys and values pass through the L2 once: they are to leave it the rest, the
    // kernels' instructions among it
    uint64_t once;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    bool ok = true;
    uint32_t used = 0, issued = 0, segs = 0, q_copies = 0;   // ring slots before this segment, copied so far
    while (ok && segment(sh, segs, a.status)) {
        const Segment &s = sh.segments[segs % kSegments];
        const int nt = s.j1 - s.j0, L = s.seq.L, j0 = s.j0, hk = s.hk, b = s.b;
        if (lane == 0) {
            ok = segs == 0 || wait(sh, &sh.q_empty, (segs - 1) & 1, a.status);
            if (ok) {
                const int t0 = s.seq.t0 + s.k * c.plan.tokens;
                mbar_expect_tx(&sh.q_full, (TWO ? 2 : 1) * tile_tokens * a.G * kD * 2);
                for (int i = 0; i < (TWO ? 2 : 1); ++i)
                    for (int h = 0; h < 2; ++h)
                        load_3d(qbuf + i * kAttnStageBytes + h * kHalfBytes, &qmap, h * 64, hk * a.G, t0 + i * tile_tokens,
                                &sh.q_full);
                ++q_copies;
            }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        // where this lane's rows of tile t lie: the copy's coordinates in a page and among pages
        auto look = [&](int t) {
            int2 at = make_int2(0, a.cache.n_pages * Hkv);   // outside: read as zeros
            const int pos = (j0 + t) * kTile + piece * c.chunk;
            if (t < nt && piece < pieces && pos < L) {
                int page = b;
                at.x = pos;
                if (a.cache.table) {
                    page = a.cache.table[(long long)b * a.cache.table_width + pos / a.cache.page_rows];
                    at.x = pos % a.cache.page_rows;
                }
                if ((uint32_t)page < (uint32_t)a.cache.n_pages)
                    at.y = page * Hkv + hk;
                else if (a.status)
                    atomicOr(a.status, RETOPK_STATUS_BAD_PAGE);
            }
            return at;
        };
        // The ring's order: K ahead of V by one tile (or two, one for each stream).  A tile is looked up
        // one step before its K, and once for both.
        constexpr int ahead = TWO ? 1 : 2;
        int2 at[3] = {look(0), look(0), look(0)};   // of tiles x, x + 1, x + 2
        for (int x = -ahead; x < nt && ok; ++x) {
            const int2 next = look(x + ahead + 1);
#pragma unroll
            for (int isk = 0; isk < 2; ++isk) {
                const int t = isk ? x + ahead : x;
                if (t < 0 || t >= nt || !ok)
                    continue;
                const uint32_t u = used + (isk ? ring_k<TWO>(t) : ring_v<TWO>(t, nt));
                const int st = u % kAttnStages;
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
                    const uint32_t dst = ring + st * kAttnStageBytes + half * kHalfBytes + piece * c.chunk * 128;
                    const int2 from = at[isk ? ahead : 0];
                    if (piece < pieces) {
                        if (TWO)
                            load_3d(dst, isk ? &kmap : &vmap, half * 64, from.x, from.y, &sh.kv_full[st]);
                        else
                            load_3d(dst, isk ? &kmap : &vmap, half * 64, from.x, from.y, &sh.kv_full[st], once);
                    }
                }
            }
            at[0] = at[1];
            at[1] = TWO ? next : at[2];
            at[2] = next;
        }
        used += 2 * nt;
        segment_done(sh, segs++);
    }
    // a wait ran out: the copies in flight are waited for before the memory goes
    if (*reinterpret_cast<volatile int *>(&sh.failed) && lane == 0) {
        const long long t0 = clock64();
        for (uint32_t u = issued > kAttnStages ? issued - kAttnStages : 0; u < issued; ++u)
            while (!mbar_try_wait(&sh.kv_full[u % kAttnStages], (u / kAttnStages) & 1) && clock64() - t0 < kWaitCycles)
                ;
        while (q_copies && !mbar_try_wait(&sh.q_full, (q_copies - 1) & 1) && clock64() - t0 < kWaitCycles)
            ;
    }
    __syncwarp();
}

// ---- the matrix instructions ------------------------------------------------------------
// The whole warp walks and waits, one lane issues: what addresses the operands
// stays the same for all lanes, so that it can live in uniform registers (an
// instruction issued from a divergent branch cost 110 cycles in place of 64).
template <bool TWO>
__device__ __forceinline__ void matrices(const AttnLaunch &c, AttnShared &sh, uint32_t qbuf, uint32_t ring,
                                         uint32_t tmem_any)
{
    const AttnArgs &a = c.a;
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_any, 0);
    bool ok = true;
    uint32_t used = 0, segs = 0, done0 = 0, done1 = 0;   // done: tiles of each group before this segment
    // S_i of the segment's tile t
    auto scores = [&](int i, int t) {
        const uint32_t u = used + ring_k<TWO>(t), st = u % kAttnStages;
        if ((!TWO || i == 0) && !warp_wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status))
            return false;
        tc_fence_after();
        if (elected()) {
            const uint32_t q = (qbuf + (TWO ? i * kAttnStageBytes : 0)) >> 4, k = (ring + st * kAttnStageBytes) >> 4;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t o = ((x >> 2) * kHalfBytes + (x & 3) * 32) >> 4;
                mma_ss(tmem + i * kTile, q + o, k + o, x > 0);
            }
            tc_commit(&sh.s_full[i]);
            if (!TWO || i == 1)
                tc_commit(&sh.kv_empty[st]);
        }
        __syncwarp();
        return true;
    };
    while (ok && segment(sh, segs, a.status)) {
        const int nt = __shfl_sync(0xffffffffu, sh.segments[segs % kSegments].j1 - sh.segments[segs % kSegments].j0, 0);
        const int m0 = TWO ? nt : (nt + 1) / 2, m1 = TWO ? nt : nt / 2;
        auto tile = [&](int i, int t) { return TWO ? t : 2 * t + i; };
        ok = warp_wait(sh, &sh.q_full, segs & 1, a.status);
        if (ok)
            ok = scores(0, tile(0, 0));
        if (ok && m1 > 0)
            ok = scores(1, tile(1, 0));
        if (ok && m0 == 1 && elected())
            tc_commit(&sh.q_empty);
        for (int t = 0; t < m0 && ok; ++t) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (t >= (i ? m1 : m0) || !ok)
                    continue;
                const uint32_t u = used + ring_v<TWO>(tile(i, t), nt), st = u % kAttnStages;
                if (!TWO || i == 0)   // (both groups' product takes the tile)
                    ok = warp_wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status);
                // P comes in halves, so that the product begins while the second is made
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ok = ok && warp_wait(sh, &sh.p_full[i][h], ((i ? done1 : done0) + t) & 1, a.status);
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (elected()) {
                        const uint32_t v = (ring + st * kAttnStageBytes) >> 4 | kDescLead;
#pragma unroll
                        for (int x = 4 * h; x < 4 * h + 4; ++x)
                            mma_ts(tmem + (2 + i) * kTile, tmem + i * kTile + x * 8, v + (x * 2048 >> 4), t > 0 || x > 0);
                        if (h == 1) {
                            tc_commit(&sh.o_full[i]);
                            if (!TWO || i == 1)
                                tc_commit(&sh.kv_empty[st]);
                        }
                    }
                    __syncwarp();
                }
                if (ok && t + 1 < (i ? m1 : m0))
                    ok = scores(i, tile(i, t + 1));
            }
            // the last use of Q
            if (ok && t + 2 == m0 && elected())
                tc_commit(&sh.q_empty);
        }
        used += 2 * nt;
        done0 += m0;
        done1 += m1;
        segment_done(sh, segs++);
    }
    if (!ok && elected()) {   // a wait ran out: the instructions in flight end before the tensor memory goes
        tc_commit(&sh.drained);
        const long long t0 = clock64();
        while (!mbar_try_wait(&sh.drained, 0) && clock64() - t0 < kWaitCycles)
            ;
    }
    __syncwarp();
}

// ---- softmax: group i, row r --------------------------------------------------------------
template <bool TWO, bool CAP>
__device__ __forceinline__ void softmax(const AttnLaunch &c, AttnShared &sh, float *ml, uint32_t ring,
                                        uint32_t tmem, int warp, int lane)
{
    const AttnArgs &a = c.a;
    const int i = warp >> 2, r = (warp & 3) * 32 + lane, G = a.G;
    const uint32_t s_addr = tmem + i * kTile + ((uint32_t)(warp & 3) << 21), o_addr = s_addr + 2 * kTile;
    const float scale2 = a.scale * 1.4426950408889634f;     // scores in powers of two
    const float cap2 = a.softcap * 1.4426950408889634f;
    const float cap_in = CAP ? fminf(2.f * scale2 / a.softcap, 3e38f) : 0.f;   // e^2y = 2^(cap_in s)
    bool ok = true;
    uint32_t used = 0, done = 0, segs = 0, joins = 0;   // joins: of the two streams
    uint32_t done1 = 0;                               // tiles of stream 1
    bool near = !CAP;                                 // the last tile's scores were all far below the cap
    while (ok && segment(sh, segs, a.status)) {
        const Segment &s = sh.segments[segs % kSegments];
        const int nt = s.j1 - s.j0, m_tiles = TWO ? nt : (nt + 1 - i) / 2;
        const int tok = s.k * c.plan.tokens + (TWO ? i * (kTile / G) : 0) + r / G;   // in the sequence
        const bool valid = r < kTile / G * G && tok < s.seq.n;
        const bool work = __any_sync(0xffffffffu, valid);
        float m = -INFINITY, l = 0.f;
        {
            const int pos = s.seq.L - s.seq.n + tok;
            const int low = a.window > 0 ? pos - a.window + 1 : 0;
            // the positions up to which, and from which, all rows of the warp see every key
            const int all_hi = __reduce_min_sync(0xffffffffu, valid ? pos : INT32_MAX);
            const int all_lo = __reduce_max_sync(0xffffffffu, valid ? low : 0);
            // Before the first tile the steps are gone through once for nothing (P goes to where O will
            // be, and to no waiter): it brings their instructions in, 3 us when cold, while the first
            // keys are on their way.
            int t = segs == 0 && m_tiles > 0 ? -1 : 0, j = s.j0 + (TWO ? t : 2 * t + i);
            for (; t < m_tiles; ++t, j += TWO ? 1 : 2) {
                const bool live = t >= 0;
                if (live)
                    ok = warp_wait(sh, &sh.s_full[i], (done + t) & 1, a.status);
                if (!TWO && i == 1 && t == 0 && joins > 0 && ok)   // stream 0 has read the last accumulators
                    ok = warp_wait(sh, &sh.x_empty, (joins - 1) & 1, a.status);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t p_addr = live ? s_addr : o_addr;
                uint64_t *const p_bar = live ? sh.p_full[i] : sh.nobody;
                // V rows past the length may hold anything, and 0 times that is not 0: they are
                // cleared where the tile is used first
                if (live && (!TWO || i == 0) && (j + 1) * kTile > s.seq.L) {
                    const uint32_t u = used + ring_v<TWO>(j - s.j0, nt);
                    const int st = u % kAttnStages;
                    ok = warp_wait(sh, &sh.kv_full[st], (u / kAttnStages) & 1, a.status);
                    if (!ok)
                        break;
                    // 8 lanes side by side in a row meet no bank twice (1000 tokens over 33000 keys 316 us; a row a
                    // lane, 333); for the one tile that a single token's call clears a row a lane is sooner done
                    // (one over 300 keys 11.7 us; 8 lanes a row, 12.4)
                    if constexpr (TWO) {
#pragma unroll 2
                        for (int q = 0; q < 16; ++q) {
                            const int row = (r & ~31) + (q & 7) * 4 + lane / 8;
                            if (j * kTile + row >= s.seq.L)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 ring + st * kAttnStageBytes + (q >> 3) * kHalfBytes + row * 128 + (lane & 7) * 16),
                                             "r"(0)
                                             : "memory");
                        }
                    } else if (j * kTile + r >= s.seq.L) {
#pragma unroll 1
                        for (int q = 0; q < 16; ++q)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             ring + st * kAttnStageBytes + (q >> 3) * kHalfBytes + r * 128 + (q & 7) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                if (work) {
                    const bool part = j * kTile + kTile - 1 > all_hi || j * kTile < all_lo;
                    // first half of P to its place; handed over once the second is well under way
                    auto hand_over = [&] {
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(p_bar);
                    };
                    constexpr int kLead = 4, kPairs = kTile / 2;   // (1133 us as above; with 2, 3, 6: 1166, 1146, 1184)
                    uint32_t x[kTile];
                    float *f = reinterpret_cast<float *>(x);
                    float2 sum[2] = {};
                    float base;
                    // Two keys at a time, in three steps that overlap: the exponents of pair n + kLead, the
                    // exponentials of pair n, the sum and the rounding of pair n - kLead.
                    // (capped scores: by the polynomial, where all are far below the cap)
                    auto two = [](float y) { return make_float2(y, y); };
                    auto exponents = [&](int n) {
                        const float2 y = make_float2(f[2 * n], f[2 * n + 1]);
                        float2 factor = two(scale2);
                        if (CAP) {
                            const float2 t2 = mul2(y, y);
                            factor = fma2(fma2(fma2(two(c.cap_poly[2]), t2, two(c.cap_poly[1])), t2, two(c.cap_poly[0])), t2, factor);
                        }
                        const float2 z = fma2(y, factor, two(-base));
                        f[2 * n] = z.x, f[2 * n + 1] = z.y;
                    };
                    auto near_capped = [&](float y) {
                        const float t2 = y * y;
                        return y * fmaf(fmaf(fmaf(c.cap_poly[2], t2, c.cap_poly[1]), t2, c.cap_poly[0]), t2, scale2);
                    };
                    auto exponentials = [&](int n) {
                        f[2 * n] = ex2(f[2 * n]);
                        f[2 * n + 1] = ex2(f[2 * n + 1]);
                    };
                    auto rounding = [&](int n) {
                        sum[n & 1] = add2(sum[n & 1], make_float2(f[2 * n], f[2 * n + 1]));
                        x[n] = bf16x2(f[2 * n], f[2 * n + 1]);
                    };
                    // The maximum m that the weights are taken against follows the true one only when
                    // that has grown by more than 2^8: until then the weights are at most 256, and the
                    // accumulators need no pass over them.  So a tile that is neither the first nor cut by the
                    // mask begins with its weights and finds its maximum beside them; if it has grown too
                    // far after all, nothing has been stored and the tile is begun again.
                    // m up to the tile's maximum where that has grown too far, and the accumulators with it;
                    // false when a wait ran out
                    auto raise = [&](float top) {
                        const bool grow = valid && m != -INFINITY && top > m + kLazy;
                        if (__any_sync(0xffffffffu, grow)) {
                            if (!warp_wait(sh, &sh.o_full[i], (done + t - 1) & 1, a.status))
                                return ok = false;
                            tc_fence_after();
                            // every row goes up: the next tiles then find none just below the limit
                            const float up = fmaxf(m, top), f2 = m == -INFINITY ? 1.f : ex2(m - up);
                            m = up;
                            l *= f2;
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                uint32_t o[16];
                                tc_ld16(o_addr + 16 * q, o);
                                tc_wait_ld16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f2);
                                tc_st16(o_addr + 16 * q, o);
                            }
                        }
                        if (m == -INFINITY)
                            m = top;
                        return true;
                    };
                    bool made = false;
                    if (near && t > 0 && !part) {
                        base = m == -INFINITY ? 0.f : m;
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, big[2] = {};
                        auto seen = [&](int k, int e) {
                            mx[k & 3] = max3(mx[k & 3], f[e], f[e + 1]);
                            if (CAP)
                                big[k & 1] = max3(big[k & 1], fabsf(f[e]), fabsf(f[e + 1]));
                        };
                        tc_ld32(s_addr, x);
                        tc_ld32(s_addr + 32, x + 32);
                        tc_wait_ld32(x);
                        tc_wait_ld32(x + 32);
                        tc_ld32(s_addr + 64, x + 64);
                        tc_ld32(s_addr + 96, x + 96);
#pragma unroll
                        for (int n = -kLead; n < kPairs / 2 - kLead; ++n) {
                            seen(n, 2 * (n + kLead));
                            exponents(n + kLead);
                            if (n >= 0)
                                exponentials(n);
                            if (n >= kLead)
                                rounding(n - kLead);
                            if (n == 4) {
                                tc_wait_ld32(x + 64);
                                tc_wait_ld32(x + 96);
                            }
                            if (n >= 4 && n < 20) {   // the second half's maximum
                                const int e = kHalf + 4 * (n - 4);
                                seen(n, e);
                                seen(n + 1, e + 2);
                            }
                        }
                        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                        made = !__any_sync(0xffffffffu, valid && (CAP ? fmaxf(big[0], big[1]) > c.cap_near || near_capped(top) > m + kLazy
                                                                   : top * scale2 > m + kLazy));
                        if (made) {
#pragma unroll
                            for (int n = kPairs / 2 - kLead; n < kPairs + kLead; ++n) {
                                if (n + kLead < kPairs)
                                    exponents(n + kLead);
                                if (n < kPairs)
                                    exponentials(n);
                                rounding(n - kLead);
                                if (n == kPairs / 2 + kLead - 1)
                                    tc_st32(p_addr, x);
                                if (n == kPairs * 3 / 4)
                                    hand_over();
                            }
                            tc_st32(p_addr + 32, x + 32);
                        } else {
                            sum[0] = sum[1] = make_float2(0.f, 0.f);
                        }
                    }
                    if (CAP && !made) {
                        // Capped scores that the one pass above does not take (an item's first tile, one that the mask
                        // cuts, scores near the cap): a quarter of a row at a time, read once for the maximum (of the
                        // raw scores: the cap does not change their order) and once for the weights.  Small code
                        // matters here, as it is run now and then only: one token of each of 16 sequences over
                        // 5000 keys takes 35 us, by half rows 38; whole rows were slower again (3 x 333 tokens in
                        // windows of 4096 keys, 16 over 2 heads, 82 us, by half rows 76).
                        constexpr int kPiece = 32;
                        float top = -INFINITY, size = 0.f;
                        const int last = pos - j * kTile, first = low - j * kTile;
#pragma unroll 1
                        for (int h = 0; h < kTile / kPiece; ++h) {
                            tc_ld32(s_addr + kPiece * h, x);
                            tc_wait_ld32(x);
                            float mx[2] = {-INFINITY, -INFINITY}, big[2] = {};
                            if (part) {
#pragma unroll
                                for (int e = 0; e < kPiece; ++e) {
                                    const bool seen = kPiece * h + e <= last && kPiece * h + e >= first;
                                    mx[e & 1] = fmaxf(mx[e & 1], seen ? f[e] : -INFINITY);
                                    big[e & 1] = max3_nan(big[e & 1], big[e & 1], seen ? fabsf(f[e]) : 0.f);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < kPiece; e += 2) {
                                    mx[e >> 1 & 1] = max3(mx[e >> 1 & 1], f[e], f[e + 1]);
                                    big[e >> 1 & 1] = max3_nan(big[e >> 1 & 1], fabsf(f[e]), fabsf(f[e + 1]));
                                }
                            }
                            top = max3(top, mx[0], mx[1]);
                            size = max3_nan(size, big[0], big[1]);
                        }
                        // (a seen score that is NaN makes the row's sum NaN: by size, as the weights lose it)
                        if (size != size)
                            l = size;
                        // far below the cap throughout: tanh as a polynomial
                        near = !__any_sync(0xffffffffu, valid && size > c.cap_near);
                        // (their capped maximum by the form that the others take)
                        if (!raise(top == -INFINITY ? top : near ? near_capped(top) : capped(top, cap_in, cap2)))
                            break;
                        base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
                        for (int h = 0; h < kTile / kPiece; ++h) {
                            tc_ld32(s_addr + kPiece * h, x);
                            tc_wait_ld32(x);
                            if (near) {
#pragma unroll
                                for (int n = 0; n < kPiece / 2; ++n)
                                    exponents(n);
                            } else {
                                // two reciprocals from one (beyond 2^60 the cap is reached).  A hidden score may be
                                // NaN and is the partner of one that is seen, so NaN takes the bound here
#pragma unroll
                                for (int e = 0; e < kPiece; e += 2) {
                                    const float d0 = 1.f + ex2(fminf(f[e] * cap_in, 60.f)), d1 = 1.f + ex2(fminf(f[e + 1] * cap_in, 60.f));
                                    const float r = rcp(d0 * d1);
                                    f[e] = fmaf(-2.f * cap2, r * d1, cap2 - base);
                                    f[e + 1] = fmaf(-2.f * cap2, r * d0, cap2 - base);
                                }
                            }
                            if (part) {
#pragma unroll
                                for (int e = 0; e < kPiece; ++e)
                                    f[e] = kPiece * h + e <= last && kPiece * h + e >= first ? f[e] : -INFINITY;
                            }
#pragma unroll
                            for (int n = 0; n < kPiece / 2 + kLead; ++n) {
                                if (n < kPiece / 2)
                                    exponentials(n);
                                if (n >= kLead)
                                    rounding(n - kLead);
                            }
                            // P takes the columns of scores that are done with
                            tc_st16(p_addr + kPiece / 2 * h, x);
                            if (h == kTile / kPiece / 2 - 1)
                                hand_over();
                        }
                    }
                    if (!CAP && !made) {
                        // the maximum of the first half is taken while the second is on its way
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        const int last = pos - j * kTile, first = low - j * kTile;
                        tc_ld32(s_addr, x);
                        tc_ld32(s_addr + 32, x + 32);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tc_wait_ld32(x + 64 * q);
                            tc_wait_ld32(x + 64 * q + 32);
                            if (q == 0) {
                                tc_ld32(s_addr + 64, x + 64);
                                tc_ld32(s_addr + 96, x + 96);
                            }
                            if (part) {
#pragma unroll
                                for (int e = 64 * q; e < 64 * q + 64; ++e)
                                    f[e] = e <= last && e >= first ? f[e] : -INFINITY;
                            }
#pragma unroll
                            for (int e = 64 * q; e < 64 * q + 64; e += 8) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mx[k] = max3(mx[k], f[e + k], f[e + 4 + k]);
                            }
                        }
                        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * scale2;
                        if (!raise(top))
                            break;
                        base = m == -INFINITY ? 0.f : m;
#pragma unroll
                        for (int n = -kLead; n < kPairs + kLead; ++n) {
                            if (n + kLead < kPairs)
                                exponents(n + kLead);
                            if (n >= 0 && n < kPairs)
                                exponentials(n);
                            if (n >= kLead)
                                rounding(n - kLead);
                            // P takes the columns of scores that are in registers
                            if (n == kPairs / 2 + kLead - 1)
                                tc_st32(p_addr, x);
                            if (n == kPairs * 3 / 4)
                                hand_over();
                        }
                        tc_st32(p_addr + 32, x + 32);
                    }
                    const float2 both = add2(sum[0], sum[1]);
                    l = live ? l + both.x + both.y : 0.f;
                    m = live ? m : -INFINITY;
                    tc_wait_st();
                } else {
                    __syncwarp();   // every lane's rows past the length are clear (hand_over has its own)
                    if (lane == 0)
                        mbar_arrive(p_bar);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_bar + 1);
            }
        }
        done += m_tiles;
        done1 += nt / 2;
        if (ok && m_tiles > 0 && (TWO || i == 0))
            ok = warp_wait(sh, &sh.o_full[i], (done - 1) & 1, a.status);
        tc_fence_after();
        // ---- the rows' end: a share's part, or the output
        const bool whole = s.j0 == s.lo && s.j1 == s.hi;
        const size_t part = 2 * blockIdx.x + (s.j0 == s.lo);
        const int row = (TWO ? i * kTile : 0) + r;
        const size_t t = s.seq.t0 + tok;
        const int head = s.hk * G + r % G;
        // Stream 1's rows join stream 0's: its maxima and sums through shared memory, its accumulators straight
        // from the tensor memory, whose lanes are the same rows.
        const bool pair = !TWO && nt > 1;   // stream 1 had a tile
        float f0 = 1.f, f1 = 0.f;
        if (pair && i == 1) {
            ml[r] = m;
            ml[kTile + r] = l;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.x_full);
        } else if (pair) {
            if (ok)
                ok = warp_wait(sh, &sh.x_full, joins & 1, a.status) && warp_wait(sh, &sh.o_full[1], (done1 - 1) & 1, a.status);
            tc_fence_after();
            const float m1 = ml[r], mm = fmaxf(m, m1), b0 = mm == -INFINITY ? 0.f : mm;
            f0 = ex2(m - b0);
            f1 = ex2(m1 - b0);
            l = l * f0 + ml[kTile + r] * f1;
            m = mm;
        }
#pragma unroll 1
        for (int h = 0; h < 4 && (TWO || i == 0); ++h) {   // 32 columns
            uint32_t x[32];
            float *y = reinterpret_cast<float *>(x);
            if (work) {
                tc_ld32(o_addr + 32 * h, x);
                tc_wait_ld32(x);
            }
            if (pair && work) {
                uint32_t z[32];
                tc_ld32(o_addr + kTile + 32 * h, z);
                tc_wait_ld32(z);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    y[e] = fmaf(__uint_as_float(z[e]), f1, y[e] * f0);
            }
            if (valid && ok) {
                if (whole) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    uint16_t *const dst = a.out + t * a.out_stride + head * kD + h * 32;
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>(dst + e) =
                            make_uint4(bf16x2(y[e] * inv, y[e + 1] * inv), bf16x2(y[e + 2] * inv, y[e + 3] * inv),
                                       bf16x2(y[e + 4] * inv, y[e + 5] * inv), bf16x2(y[e + 6] * inv, y[e + 7] * inv));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        c.parts.o[(part * (kD / 4) + h * 8 + e / 4) * c.parts.rows + row] =
                            make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                }
            }
        }
        if (valid && ok && (TWO || i == 0)) {
            if (!whole)
                c.parts.ml[part * c.parts.rows + row] = make_float2(m, l);
            else if (a.lse)
                a.lse[t * a.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
        used += 2 * nt;
        if (pair && i == 0) {   // stream 1 may accumulate again
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.x_empty);
        }
        joins += pair;
        segment_done(sh, segs++);
        tc_fence_before();
    }
}

template <bool TWO, bool CAP>
__global__ void __launch_bounds__(kAttnThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const AttnLaunch c)
{
    extern __shared__ __align__(1024) unsigned char attn_smem[];
    AttnShared &sh = *reinterpret_cast<AttnShared *>(attn_smem + (2 + kAttnStages) * kAttnStageBytes);
    const AttnArgs &a = c.a;
    const Plan &plan = c.plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t qbuf = smem_u32(attn_smem);   // 1024-byte aligned, as the swizzle wants it
    const uint32_t ring = qbuf + 2 * kAttnStageBytes;
    const int Hkv = a.cache.n_kv_heads;

    if (tid == 0) {
        for (int s = 0; s < kAttnStages; ++s) {
            mbar_init(&sh.kv_full[s], 1);
            mbar_init(&sh.kv_empty[s], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 4);
            mbar_init(&sh.p_full[i][1], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        for (int s = 0; s < kSegments; ++s) {
            mbar_init(&sh.seg_full[s], 1);
            mbar_init(&sh.seg_empty[s], kLoadWarp + 1);
        }
        mbar_init(&sh.x_full, 4);
        mbar_init(&sh.x_empty, 4);
        mbar_init(&sh.drained, 1);
        mbar_init(&sh.nobody[0], 1 << 16);
        mbar_init(&sh.nobody[1], 1 << 16);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.failed = 0;
        sh.bound[0] = sh.bound[1] = Place{a.B, 0, 0, 0};
        sh.first_b = -1;
        for (const CUtensorMap *map : {&qmap, &kmap, &vmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share: the sum of all weights, then the places of its two
    //      bounds.  Up to 384 sequences stay in the threads' registers.
    auto of_sequence = [&](int b, Seq &q) {
        if (b >= a.B)
            return 0ll;
        q = sequence(a, b);
        return Hkv * weight(a, plan, q, blocks_of(plan, q));
    };
    Seq mine{0, 0, 0};
    const long long my_weight = of_sequence(tid, mine);
    long long total = my_weight;
    for (int b = tid + kAttnThreads; b < a.B; b += kAttnThreads) {
        Seq q;
        total += of_sequence(b, q);
    }
    long long up = my_weight;   // of the first round: the running sum within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o)
            up += y;
    }
    if (a.B > kAttnThreads) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0)
            sh.sums[warp] = total;
        __syncthreads();
        total = 0;
        for (int i = 0; i < kAttnThreads / 32; ++i)
            total += sh.sums[i];
        __syncthreads();
    }
    if (lane == 31)
        sh.sums[warp] = up;
    __syncthreads();
    long long off = 0, round = 0;
#pragma unroll
    for (int i = 0; i < kAttnThreads / 32; ++i) {
        const long long x = sh.sums[i];
        off += i < warp ? x : 0;
        round += x;
    }
    if (a.B <= kAttnThreads)
        total = round;
    const long long share = (long long)__umul64hi((unsigned long long)total, plan.inverse) + 1;
    const long long u0 = min(share * blockIdx.x, total), u1 = min(share * (blockIdx.x + 1), total);
    auto find = [&](int b, const Seq &q, long long from, long long weight_of) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const long long u = k ? u1 : u0;
            if (weight_of > 0 && u >= from && u < from + weight_of) {
                sh.bound[k] = place_in(a, plan, q, b, u - from);
                if (k == 0) {
                    sh.first = q;
                    sh.first_b = b;
                }
            }
        }
    };
    find(tid, mine, off + up - my_weight, my_weight);
    for (int base = kAttnThreads; base < a.B; base += kAttnThreads) {
        const long long before = round;
        Seq q{0, 0, 0};
        const long long x = of_sequence(base + tid, q);
        up = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o)
                up += y;
        }
        __syncthreads();
        if (lane == 31)
            sh.sums[warp] = up;
        __syncthreads();
        off = before;
        for (int i = 0; i < kAttnThreads / 32; ++i) {
            off += i < warp ? sh.sums[i] : 0;
            round += sh.sums[i];
        }
        find(base + tid, q, off + up - x, x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (tid == 0) {
        c.parts.bound[blockIdx.x] = Bound{sh.bound[0], sh.first.n, sh.first.t0};
        if (blockIdx.x == gridDim.x - 1)
            c.parts.bound[gridDim.x] = Bound{sh.bound[1], 0, 0};
    }
    if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax<TWO, CAP>(c, sh, reinterpret_cast<float *>(attn_smem + kAttnStageBytes), ring, tmem, warp, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kLoadWarp)
            copies<TWO>(c, sh, qmap, kmap, vmap, qbuf, ring, lane);
        else if (warp == kMmaWarp)
            matrices<TWO>(c, sh, qbuf, ring, tmem);
        else if (warp == kWalkWarp && lane == 0)
            walk_share(a, plan, sh);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the parts of an item.  With two tiles the grid's columns are the cut items (few
// items of many rows then have many blocks each: 36 tokens over 17663 keys, 16 over 2 heads, 48 -> 38 us);
// with one, where that search costs more than it gives, they are the bounds, and the first
// that cuts an item has it.  One, two, four or eight warps of a block take a row and share
// out its parts: as many as leave the item's blocks about one pass over the rows.
template <bool TWO>
__global__ void __launch_bounds__(256) join_kernel(const AttnLaunch c, int shares)
{
    __shared__ float4 sum[8][32];
    __shared__ float2 ml_of[8];
    __shared__ Bound bounds[kMaxShares + 1];
    __shared__ uint16_t list[kMaxShares + 1];   // the item's parts
    __shared__ int counts[8], first_cut;
    pdl_wait();
    pdl_trigger();
    const AttnArgs &a = c.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid <= shares)
        bounds[tid] = c.parts.bound[tid];
    if (tid == 0)
        first_cut = 0;
    __syncthreads();
    // the bounds that are the first to cut their item, counted up to this thread's
    const Place mine = tid <= shares ? bounds[tid].at : Place{0, 0, 0, 0};
    const Place prev = tid > 0 && tid <= shares ? bounds[tid - 1].at : Place{0, 0, 0, 0};
    const bool cuts = tid > 0 && tid < shares && mine.cut > 0 && !(same_item(mine, prev) && prev.cut > 0);
    auto rank = [&](bool flag, int &total) {
        const uint32_t votes = __ballot_sync(0xffffffffu, flag);
        if (lane == 0)
            counts[warp] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1));
        total = 0;
        for (int w = 0; w < 8; ++w) {
            before += w < warp ? counts[w] : 0;
            total += counts[w];
        }
        __syncthreads();
        return before;
    };
    int n, x;
    if constexpr (TWO) {
        if (rank(cuts, n) == (int)blockIdx.x && cuts)
            first_cut = tid;
        __syncthreads();
        x = first_cut;
        if (x == 0)
            return;
    } else {
        x = blockIdx.x + 1;
        const Place p = bounds[x].at, q = bounds[x - 1].at;
        if (p.cut == 0 || (same_item(p, q) && q.cut > 0))
            return;
    }
    const Bound here = bounds[x];
    const Place at = here.at;
    // parts: share x - 1's part 1, then part 0 of shares x, x + 1, ... while they begin in the item (a
    // share between two equal cuts has none)
    bool in = tid == x - 1;
    if (tid >= x && tid < shares) {
        const Place next = bounds[tid + 1].at;
        in = same_item(mine, at) && (!same_item(next, at) || next.cut > mine.cut);
    }
    const int slot = rank(in, n);
    if (in)
        list[slot] = (uint16_t)(2 * tid + (tid == x - 1));
    __syncthreads();
    const int tile_tokens = kTile / a.G, per_tile = tile_tokens * a.G, first = at.k * c.plan.tokens;
    const int rows = min(TWO ? 2 * per_tile : per_tile, (here.n - first) * a.G);
    int crew = 1;   // warps of a row
    while (crew < 8 && 4 * crew < n && 2 * crew * rows <= 8 * (int)gridDim.y)
        crew *= 2;
    const int mate = warp % crew, step = 8 / crew;   // rows of the block at a time
    for (int base = blockIdx.y * step; base < rows; base += gridDim.y * step) {
        const int r0 = base + warp / crew;
        const bool real = r0 < rows;
        const int second = r0 >= per_tile, in_tile = r0 - second * per_tile;
        const int r = second * kTile + in_tile;
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float m2, float l2, float4 o) {
            const float mm = fmaxf(m, m2), zero = mm == -INFINITY ? 0.f : mm;
            const float f1 = ex2(m - zero), f2 = m2 == -INFINITY ? 0.f : ex2(m2 - zero);
            l = l * f1 + l2 * f2;
            // (a part without a row's keys may hold anything)
            acc.x = fmaf(acc.x, f1, f2 != 0.f ? o.x * f2 : 0.f);
            acc.y = fmaf(acc.y, f1, f2 != 0.f ? o.y * f2 : 0.f);
            acc.z = fmaf(acc.z, f1, f2 != 0.f ? o.z * f2 : 0.f);
            acc.w = fmaf(acc.w, f1, f2 != 0.f ? o.w * f2 : 0.f);
            m = mm;
        };
#pragma unroll 1
        for (int i0 = mate; i0 < n && real; i0 += 4 * crew) {   // four parts on their way at once
            float2 ml[4];
            float4 o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * crew;
                ml[k] = make_float2(-INFINITY, 0.f);
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    const size_t part = list[i];
                    ml[k] = c.parts.ml[part * c.parts.rows + r];
                    o[k] = c.parts.o[(part * (kD / 4) + lane) * c.parts.rows + r];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                add(ml[k].x, ml[k].y, o[k]);
        }
        if (crew > 1) {
            sum[warp][lane] = acc;
            if (lane == 0)
                ml_of[warp] = make_float2(m, l);
            __syncthreads();
            if (mate == 0)
#pragma unroll 1
                for (int i = 1; i < crew; ++i)
                    add(ml_of[warp + i].x, ml_of[warp + i].y, sum[warp + i][lane]);
            __syncthreads();
        }
        if (mate != 0 || !real)
            continue;
        const int tok = first + second * tile_tokens + in_tile / a.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t t = here.t0 + tok;
        const int h = at.hk * a.G + in_tile % a.G;
        *reinterpret_cast<uint2 *>(a.out + t * a.out_stride + h * kD + lane * 4) =
            make_uint2(bf16x2(acc.x * inv, acc.y * inv), bf16x2(acc.z * inv, acc.w * inv));
        if (a.lse && lane == 0)
            a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

// ---- host side ----------------------------------------------------------------
// Two tiles of tokens a block where the sequences have more tokens than one and a half tiles
// on average; else one tile and two streams of keys.  (18 tokens a tile.  40 sequences over 1500 keys, streams against
// two tiles: of 12 tokens 39 us against 45, of 24 51 against 54, of 36 63 against 59, of 72 100 against 79;
// 4 over 9000: of 24 30 against 32, of 36 35 against 38, of 72 47 against 48.)  The mean stands for all sequences, as
// the lengths are the device's: a prompt among many single tokens takes the streams.  Against two calls, the prompt
// in one and the tokens in the other, 4096 tokens over 32768 keys beside 200 single tokens over 9000 take 2064 us
// (two calls 1729), 4096 over 4096 beside 200 over 1500 274 (259); with fewer tokens beside it one call is the faster:
// 512 over 9000 beside 63 over 9000 221 (254), 4096 over 32768 beside 63 over 9000 1350 (1382, in two tiles).
static bool two_tiles(int T, int B, int G) { return T / B > kTile / G * 3 / 2; }

// Rows of a part.
static int part_rows(int T, int G, bool two)
{
    return two ? 2 * kTile : (int)std::min<long long>(kTile, ((long long)T * G + 7) / 8 * 8);
}

static size_t carve(int rows, char *ws, Parts *p)
{
    const int n = std::min(sm_count(), kMaxShares);
    const size_t o_ml = ((n + 1) * sizeof(Bound) + 255) / 256 * 256;
    const size_t o_o = o_ml + (2 * n * (size_t)rows * sizeof(float2) + 255) / 256 * 256;
    if (p) {
        p->bound = reinterpret_cast<Bound *>(ws);
        p->ml = reinterpret_cast<float2 *>(ws + o_ml);
        p->o = reinterpret_cast<float4 *>(ws + o_o);
        p->rows = rows;
    }
    return o_o + 2 * n * (size_t)rows * kD * sizeof(float);
}

// Enough for fewer tokens and any number of sequences as well: of all batches of T tokens, the one of a single sequence
// has the most rows a part.
size_t chunk_attention_ws(int T, int Hq, int Hkv)
{
    const int G = Hq / Hkv;
    return carve(part_rows(T, G, two_tiles(T, 1, G)), nullptr, nullptr);
}

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
    // no item of four tiles or fewer is cut, so a cache that holds no more needs no join
    // (and no more CTAs than there may be items)
    const bool cuts = c.a.capacity > 4 * kTile;
    const int n = c.shares;
    auto kernel = c.a.softcap > 0.f ? chunk_attention_kernel<TWO, true> : chunk_attention_kernel<TWO, false>;
    cudaError_t e = launch_pdl(kernel, dim3(n), dim3(kAttnThreads), kAttnSmem, st, 1, qm, km, vm, c);
    if (e != cudaSuccess || n < 2 || !cuts)
        return e;
    // the items that may be cut, and blocks for each: few items have many parts
    const int cut = TWO ? (int)std::min<long long>(n - 1, c.items) : n - 1;
    const int each = TWO ? std::max(8, std::min(64, 1216 / cut)) : 8;
    return launch_pdl(join_kernel<TWO>, dim3(cut, each), dim3(256), 0, st, 1, c, n);
}

cudaError_t launch_chunk_attention(const AttnArgs &a, cudaStream_t st)
{
    AttnLaunch c{};
    c.a = a;
    const int Hkv = a.cache.n_kv_heads, tokens = kTile / a.G;
    const bool two = two_tiles(a.T, a.B, a.G);
    c.plan.tokens = two ? 2 * tokens : tokens;
    c.shares = std::min(sm_count(), kMaxShares);
    c.items = std::min<long long>(a.T, a.T / c.plan.tokens + a.B) * Hkv;
    if (a.capacity <= 4 * kTile)
        c.shares = (int)std::min<long long>(c.shares, c.items);
    c.plan.inverse = ~0ull / (unsigned long long)c.shares;
    carve(part_rows(a.T, a.G, two), static_cast<char *>(a.ws), &c.parts);
    if (a.softcap > 0.f) {
        const double b[3] = {-0.3332815934197915, 0.132053598066859, -0.04475064703577332};
        const double y = (double)a.scale / a.softcap;
        for (int i = 0; i < 3; ++i)
            c.cap_poly[i] = (float)(b[i] * pow(y, 2 * i + 2) * a.scale * 1.4426950408889634);
        // (a cap so small that the powers overflow: the other form for all but no scores)
        c.cap_near = isfinite(c.cap_poly[2]) ? (float)(0.5 / y) : -1.f;
    }
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
