// paged_select.cuh -- the k highest of n 64-bit keys in shared memory, in
// ascending order of their places; equal keys go to the lower place.
//
// The k-th highest key is found by bisection on the keys' upper words (then
// the lower ones where the upper words tie): a step counts the keys at or
// above the middle, one compare a key and one warp reduction, and the search
// ends as soon as a count is k.  Its cost does not grow with k.  One warp
// holds up to 512 keys in registers; more keys are first thinned by the
// CTA's warps, each keeping the k highest of its part.
#pragma once

#include <stdint.h>

namespace hga {
namespace paged {

// A float64 as an integer of the same order; NaN above everything, and
// every number above 0.
__device__ __forceinline__ unsigned long long ordered(double x)
{
    if (x != x) return ~0ull;
    const unsigned long long u = __double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Keys of one warp: in registers (M of them a lane), or read where they are.
template <int M> struct WarpKeys {
    unsigned long long v[M];
    __device__ __forceinline__ void load(const unsigned long long* keys, int n, int lane)
    {
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] = lane + 32 * m < n ? keys[lane + 32 * m] : 0ull;
    }
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int m = 0; m < M; ++m) f(m, v[m]);
    }
};
template <> struct WarpKeys<0> {
    const unsigned long long* at;
    int n, lane;
    __device__ __forceinline__ void load(const unsigned long long* keys, int n_, int lane_)
    {
        at = keys;
        n = n_;
        lane = lane_;
    }
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
        for (int m = 0; 32 * m < n; ++m) f(m, lane + 32 * m < n ? at[lane + 32 * m] : 0ull);
    }
};

// The largest t in [lo, up] with count(t) >= k, or the first t met with
// count(t) = k (then `exact`).  count(lo) >= k.
template <typename Count>
__device__ __forceinline__ uint32_t bisect(uint32_t lo, uint32_t up, int k, Count count, bool& exact)
{
    exact = false;
    while (lo < up) {
        const uint32_t mid = lo + ((up - lo) >> 1) + ((up - lo) & 1u);
        const int c = count(mid);
        if (c == k) {
            exact = true;
            return mid;
        }
        if (c > k) lo = mid;
        else up = mid - 1;
    }
    return lo;
}

// One warp: emit(place, rank) for the k highest of n keys, k < n; rank
// ascends with the place.
template <int M, typename Emit>
__device__ __forceinline__ void warp_select(const unsigned long long* keys, int n, int k, int lane, Emit emit)
{
    WarpKeys<M> w;
    w.load(keys, n, lane);
    uint32_t mx = 0u, mn = ~0u;
    w.each([&](int, unsigned long long v) {
        const uint32_t hi = uint32_t(v >> 32);
        mx = max(mx, hi);
        if (v) mn = min(mn, hi);
    });
    mx = __reduce_max_sync(0xFFFFFFFFu, mx);
    mn = __reduce_min_sync(0xFFFFFFFFu, mn);
    auto total = [](int c) { return __reduce_add_sync(0xFFFFFFFFu, c); };
    bool exact;
    const uint32_t t = bisect(mn, mx, k, [&](uint32_t mid) {
        int c = 0;
        w.each([&](int, unsigned long long v) { c += uint32_t(v >> 32) >= mid; });
        return total(c);
    }, exact);
    uint32_t t2 = 0;
    int ties = 0;                                    // keys equal to (t, t2) that are kept, lowest places first
    if (!exact) {
        int above = 0;
        w.each([&](int, unsigned long long v) { above += uint32_t(v >> 32) > t; });
        const int r = k - total(above);
        t2 = bisect(0u, ~0u, r, [&](uint32_t mid) {
            int c = 0;
            w.each([&](int, unsigned long long v) { c += uint32_t(v >> 32) == t && uint32_t(v) >= mid; });
            return total(c);
        }, exact);
        if (!exact) {
            int over = 0;
            w.each([&](int, unsigned long long v) { over += uint32_t(v >> 32) == t && uint32_t(v) > t2; });
            ties = r - total(over);
        }
    }
    const unsigned long long T = ((unsigned long long)t << 32) | t2;
    const unsigned below = (1u << lane) - 1u;
    int at = 0;
    w.each([&](int m, unsigned long long v) {
        bool keep = exact ? v >= T : v > T;
        if (!exact) {
            const unsigned eq = __ballot_sync(0xFFFFFFFFu, v == T);
            keep = keep || (v == T && __popc(eq & below) < ties);
            ties = max(0, ties - __popc(eq));
        }
        const unsigned kept = __ballot_sync(0xFFFFFFFFu, keep);
        if (keep) emit(lane + 32 * m, at + __popc(kept & below));
        at += __popc(kept);
    });
}

constexpr int kThin = 512;                           // keys that one warp takes at once

template <int Warps> struct SelectScratch {
    unsigned long long keys[kThin];
    int32_t ids[kThin];
};

// The whole CTA (synchronised before; synchronise after): emit(place, rank)
// for the k highest of n keys, from any thread, each once.
template <int Warps, typename Emit>
__device__ __forceinline__ void select(const unsigned long long* keys, int n, int k, SelectScratch<Warps>* sc, int tid,
                                       Emit emit)
{
    const int lane = tid & 31, warp = tid >> 5;
    if (k >= n) {
        for (int i = tid; i < n; i += 32 * Warps) emit(i, i);
        return;
    }
    if (n <= 256) {
        if (warp == 0) warp_select<8>(keys, n, k, lane, emit);
        return;
    }
    if (n <= kThin) {
        if (warp == 0) warp_select<16>(keys, n, k, lane, emit);
        return;
    }
    if (k * Warps > kThin) {                         // too many to thin: one warp over shared memory
        if (warp == 0) warp_select<0>(keys, n, k, lane, emit);
        return;
    }
    // Each warp keeps the k highest of its part (all parts hold at least k:
    // n > kThin >= k Warps, parts of n / Warps rounded down or up).
    const int a = int((int64_t)n * warp / Warps), z = int((int64_t)n * (warp + 1) / Warps);
    auto keep = [&](int i, int at) {
        sc->keys[warp * k + at] = keys[a + i];
        sc->ids[warp * k + at] = a + i;
    };
    if (z - a == k) {
        for (int i = lane; i < k; i += 32) keep(i, i);
    } else if (z - a <= kThin) {
        warp_select<16>(keys + a, z - a, k, lane, keep);
    } else {
        warp_select<0>(keys + a, z - a, k, lane, keep);
    }
    __syncthreads();
    if (warp == 0)
        warp_select<16>(sc->keys, k * Warps, k, lane, [&](int i, int at) { emit(sc->ids[i], at); });
}

}  // namespace paged
}  // namespace hga
