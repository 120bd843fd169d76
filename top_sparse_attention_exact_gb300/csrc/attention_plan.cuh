// attention_plan.cuh -- how the attention kernels divide their work.
//
// Items are (sequence, KV head, block of tokens) and weigh one unit per key beside a
// weight of their own; the CTAs take equal shares of the sum, so a share may begin
// and end inside an item.  Each CTA finds its own share from the lengths, which stay on
// the device.  A CTA that has a part of an item leaves its rows, unnormalised, in the
// workspace for a join.  Shares, and with them the order of every sum, depend on the lengths alone.
//
// `Cost` is the kernel's: kItem, the weight of an item beside its keys, and grain(plan, tiles), the number
// of tiles that an item of so many is cut by.
#pragma once

#include "prompt.cuh"

namespace retopk {

constexpr int kTile = 128;                       // rows and keys of a tile

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
    int uncut;                     // tiles of an item that is not cut (row attention)
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
template <class Cost>
__device__ __forceinline__ long long weight(const AttnArgs &a, const Plan &p, const Seq &s, int k)
{
    const int first = max(0, s.L - s.n) + min(p.tokens, s.n) + Cost::kItem;
    int grow = k;
    long long flat = 0;
    if (a.window > 0 && a.window < kMaxLen) {
        const int most = a.window + p.tokens + kTile + Cost::kItem;
        grow = most <= first ? 0 : min(k, (most - first) / p.tokens + 1);
        flat = (long long)(k - grow) * most;
    }
    return (long long)grow * first + (long long)p.tokens * grow * (grow - 1) / 2 + flat;
}

// The place u units behind the beginning of sequence b.
template <class Cost>
__device__ __forceinline__ Place place_in(const AttnArgs &a, const Plan &p, const Seq &s, int b, long long u)
{
    const int nb = blocks_of(p, s);
    const long long each = weight<Cost>(a, p, s, nb);
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
        if (weight<Cost>(a, p, s, mid) <= u)
            r.k = mid;
        else
            top = mid - 1;
    }
    int lo, hi;
    tiles_of(a, p, s, r.k, lo, hi);
    const long long begin = weight<Cost>(a, p, s, r.k);
    const int nt = hi - lo, grain = Cost::grain(p, nt);
    // (half the item's own weight lies before its first tile, half behind its last)
    const int in = (int)(u - begin) - Cost::kItem / 2, keys = (int)(weight<Cost>(a, p, s, r.k + 1) - begin) - Cost::kItem;
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

// ---- a CTA's share -------------------------------------------------------------------
struct Share {
    Place bound[2];
    Seq first;                 // the sequence that bound[0] was found in
    int first_b;
    long long sums[17];
};

// The sum of all weights, then the places of the share's two bounds (set to the end of the work before), by all THREADS
// of the CTA.  Up to so many sequences stay in the threads' registers.
template <class Cost, int THREADS>
__device__ __forceinline__ void find_share(const AttnArgs &a, const Plan &plan, Share &sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto of_sequence = [&](int b, Seq &q) {
        if (b >= a.B)
            return 0ll;
        q = sequence(a, b);
        return a.cache.n_kv_heads * weight<Cost>(a, plan, q, blocks_of(plan, q));
    };
    Seq mine{0, 0, 0};
    const long long my_weight = of_sequence(tid, mine);
    long long total = my_weight;
    for (int b = tid + THREADS; b < a.B; b += THREADS) {
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
    if (a.B > THREADS) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0)
            sh.sums[warp] = total;
        __syncthreads();
        total = 0;
        for (int i = 0; i < THREADS / 32; ++i)
            total += sh.sums[i];
        __syncthreads();
    }
    if (lane == 31)
        sh.sums[warp] = up;
    __syncthreads();
    long long off = 0, round = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const long long x = sh.sums[i];
        off += i < warp ? x : 0;
        round += x;
    }
    if (a.B <= THREADS)
        total = round;
    const long long share = (long long)__umul64hi((unsigned long long)total, plan.inverse) + 1;
    const long long u0 = min(share * blockIdx.x, total), u1 = min(share * (blockIdx.x + 1), total);
    auto find = [&](int b, const Seq &q, long long from, long long weight_of) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const long long u = k ? u1 : u0;
            if (weight_of > 0 && u >= from && u < from + weight_of) {
                sh.bound[k] = place_in<Cost>(a, plan, q, b, u - from);
                if (k == 0) {
                    sh.first = q;
                    sh.first_b = b;
                }
            }
        }
    };
    find(tid, mine, off + up - my_weight, my_weight);
    for (int base = THREADS; base < a.B; base += THREADS) {
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
        for (int i = 0; i < THREADS / 32; ++i) {
            off += i < warp ? sh.sums[i] : 0;
            round += sh.sums[i];
        }
        find(base + tid, q, off + up - x, x);
    }
}

// ---- workspace ----------------------------------------------------------------------
// Places of the n + 1 bounds, then for each CTA two parts (0: of an item that began in an
// earlier share, 1: of an item that goes on in the next).
struct Bound {
    Place at;
    int n, t0;   // of the place's sequence, where it is inside an item
};

}  // namespace retopk
