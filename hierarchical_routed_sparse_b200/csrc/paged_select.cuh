// paged_select.cuh -- the k highest of n 64-bit keys in shared memory, in
// ascending order of their places; equal keys go to the lower place.
//
// Up to 128 keys: every key counts the keys that beat it, all threads at
// once.  Up to 512, k <= 32: one warp holds them, up to 16 a lane; the k-th
// highest of the lanes' maxima bounds the k-th highest key from below, and the
// few keys at or above that bound (seldom more than 32) are ranked against
// each other by shuffles.  Where that does not apply, the k-th highest key is
// found by bisection, one count a step.  More than 512 keys are first thinned
// by the CTA's warps, each keeping the k highest of its part.
//
// What bounds these is the length of a warp's instruction chain (a lone warp
// issues one in about 4 cycles): 256 keys, k 8 take 1.5 us and 64 keys, k 32
// about 1 us, barriers included; a bisection over the same 256 keys 2.5 us, and a histogram of 256
// bins by all threads (five barriers) 2 us.
#pragma once

#include <stdint.h>

namespace hga {
namespace paged {

typedef unsigned long long Key;

// A float64 as an integer of the same order; NaN above everything, and
// every number above 0.
__device__ __forceinline__ Key ordered(double x)
{
    if (x != x) return ~0ull;
    const Key u = __double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

constexpr int kThin = 512;                           // keys that one warp takes at once
constexpr int kCount = 128;                          // keys that are ranked by counting

// (ids and keys are for more than kThin keys only.)
template <int Warps> struct SelectScratch {
    uint32_t room[Warps][32];
    int32_t place[Warps][32], count[(Warps + 3) / 4 * 4], ids[kThin];
    Key keys[kThin];
    static constexpr size_t kSmall = 4 * (64 * Warps + (Warps + 3) / 4 * 4);     // bytes before ids
};

// How many lanes below have their bit.
__device__ __forceinline__ int below(unsigned m, int lane) { return __popc(m & ((1u << lane) - 1u)); }

// One warp, bisection over shared memory: the places of the k highest of n
// keys, k < n, into out, ascending.
static __device__ __noinline__ void bisect_select(const Key* keys, int n, int k, int lane, int32_t* out)
{
    auto count = [&](Key t) {
        int c = 0;
        for (int i = lane; i < n; i += 32) c += keys[i] >= t;
        return __reduce_add_sync(0xFFFFFFFFu, c);
    };
    // The largest t with count(t) >= k.  Keys are above 0.
    Key lo = 1, up = ~0ull;
    while (lo < up) {
        const Key mid = lo + ((up - lo) >> 1) + ((up - lo) & 1ull);
        const int c = count(mid);
        if (c >= k) lo = mid;
        else up = mid - 1;
        if (c == k) break;
    }
    // All above lo, and of its equals the lowest places.
    int over = 0;
    for (int i = lane; i < n; i += 32) over += keys[i] > lo;
    int ties = k - __reduce_add_sync(0xFFFFFFFFu, over), at = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const Key v = i < n ? keys[i] : 0ull;
        const unsigned eq = __ballot_sync(0xFFFFFFFFu, v == lo);
        const bool keep = v > lo || (v == lo && below(eq, lane) < ties);
        ties -= min(ties, __popc(eq));
        const unsigned kept = __ballot_sync(0xFFFFFFFFu, keep);
        if (keep) out[at + below(kept, lane)] = i;
        at += __popc(kept);
    }
}

// One warp: as bisect_select, for n <= 32 M and k <= 32; false (and nothing
// written that counts) where it does not apply.  Works on the keys' upper
// words, and on whole keys where two of the few candidates tie there (one
// selection in a thousand; by bisection that one took 14 us instead of 4).
template <int M>
__device__ __forceinline__ bool warp_try(const Key* keys, int n, int k, int lane, uint32_t* room, int32_t* place, int32_t* out)
{
    const uint32_t* upper = reinterpret_cast<const uint32_t*>(keys) + 1;
    uint32_t v[M], mine = 0u;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        v[m] = lane + 32 * m < n ? upper[2 * (lane + 32 * m)] : 0u;
        mine = max(mine, v[m]);
    }
    // At least k lanes' maxima, so at least k keys, are at or above the bound:
    // the highest maximum that k - 1 others reach.
    int reach = 0;
#pragma unroll
    for (int o = 1; o < 32; ++o) reach += __shfl_sync(0xFFFFFFFFu, mine, lane + o) >= mine;
    const uint32_t bound = __reduce_max_sync(0xFFFFFFFFu, reach >= k - 1 ? mine : 0u);
    int got = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const bool is = v[m] >= bound;
        const unsigned b = __ballot_sync(0xFFFFFFFFu, is);
        const int at = got + below(b, lane);
        if (is && at < 32) {
            room[at] = v[m];
            place[at] = lane + 32 * m;
        }
        got += __popc(b);
    }
    if (got > 32 || bound == 0u) return false;
    __syncwarp();
    const uint32_t x = lane < got ? room[lane] : 0u;             // places ascend with the lane
    int beat = 0;
    bool tie = false;
#pragma unroll
    for (int o = 1; o < 32; ++o) {
        const uint32_t w = __shfl_sync(0xFFFFFFFFu, x, lane + o);
        beat += w > x;
        tie = tie || w == x;
    }
    if (__any_sync(0xFFFFFFFFu, tie && lane < got)) {            // whole keys, of equal ones the lower place
        const Key whole = lane < got ? keys[place[lane]] : 0ull;
        beat = 0;
#pragma unroll 1
        for (int o = 1; o < 32; ++o) {
            const Key w = __shfl_sync(0xFFFFFFFFu, whole, lane + o);
            beat += w > whole || (w == whole && ((lane + o) & 31) < lane);
        }
    }
    const bool keep = lane < got && beat < k;
    const unsigned kept = __ballot_sync(0xFFFFFFFFu, keep);
    if (keep) out[below(kept, lane)] = place[lane];
    __syncwarp();
    return true;
}

static __device__ __noinline__ void warp_select(const Key* keys, int n, int k, int lane, uint32_t* room, int32_t* place,
                                                int32_t* out)
{
    if (k <= 32) {
        if (n <= 256 ? warp_try<8>(keys, n, k, lane, room, place, out) : warp_try<16>(keys, n, k, lane, room, place, out))
            return;
    }
    bisect_select(keys, n, k, lane, out);
}

// The whole CTA of Warps warps (synchronised before; synchronise after): the
// places of the k highest of n keys into out, ascending.
template <int Warps>
__device__ __forceinline__ void select(const Key* keys, int n, int k, SelectScratch<Warps>* sc, int tid, int32_t* out)
{
    static_assert(32 * Warps >= kCount, "one thread a key");
    const int lane = tid & 31, warp = tid >> 5;
    if (k >= n) {
        for (int i = tid; i < n; i += 32 * Warps) out[i] = i;
        return;
    }
    if (n <= kCount) {
        // 2^e threads count for one key, each over the pairs of keys of its own
        // turn.  Upper words first; where two keys tie there, whole keys (and
        // of equal ones the lower place wins).
        const int e = n <= 8 * Warps ? 2 : n <= 16 * Warps ? 1 : 0;
        const int i = tid >> e, turn = tid & ((1 << e) - 1);
        const Key x = i < n ? keys[i] : 0ull;
        const uint32_t upper = uint32_t(x >> 32);
        int beat = 0, same = 0;
#pragma unroll 4
        for (int j = 2 * turn; j + 1 < n; j += 2 << e) {
            const uint4 w = *reinterpret_cast<const uint4*>(keys + j);
            beat += w.y > upper;
            beat += w.w > upper;
            same += w.y == upper;
            same += w.w == upper;
        }
        if ((n & 1) && turn == 0) {
            const uint32_t w = uint32_t(keys[n - 1] >> 32);
            beat += w > upper;
            same += w == upper;
        }
        if (e > 0) same += __shfl_xor_sync(0xFFFFFFFFu, same, 1);
        if (e > 1) same += __shfl_xor_sync(0xFFFFFFFFu, same, 2);
        if (__syncthreads_or(i < n && same > 1)) {   // (a key ties with itself)
            beat = 0;
            for (int j = turn; j < n; j += 1 << e) beat += keys[j] > x || (keys[j] == x && j < i);
        }
        if (e > 0) beat += __shfl_xor_sync(0xFFFFFFFFu, beat, 1);
        if (e > 1) beat += __shfl_xor_sync(0xFFFFFFFFu, beat, 2);
        const bool keep = i < n && beat < k && (tid & ((1 << e) - 1)) == 0;
        const unsigned kept = __ballot_sync(0xFFFFFFFFu, keep);
        if (lane == 0) sc->count[warp] = __popc(kept);
        __syncthreads();
        int at = below(kept, lane);
        for (int w = 0; w < warp; ++w) at += sc->count[w];
        if (keep) out[at] = i;
        return;
    }
    if (n <= kThin) {
        if (warp == 0) warp_select(keys, n, k, lane, sc->room[0], sc->place[0], out);
        return;
    }
    if (k * Warps > kThin) {                         // too many to thin: one warp over shared memory
        if (warp == 0) bisect_select(keys, n, k, lane, out);
        return;
    }
    // Each warp keeps the k highest of its part (n > kThin >= k Warps, so
    // every part holds at least k).
    const int a = int((int64_t)n * warp / Warps), z = int((int64_t)n * (warp + 1) / Warps);
    int32_t* ids = sc->ids + warp * k;
    if (z - a == k) {
        for (int i = lane; i < k; i += 32) ids[i] = i;
    } else if (z - a <= kThin) {
        warp_select(keys + a, z - a, k, lane, sc->room[warp], sc->place[warp], ids);
    } else {
        bisect_select(keys + a, z - a, k, lane, ids);
    }
    __syncwarp();
    for (int i = lane; i < k; i += 32) {
        ids[i] += a;
        sc->keys[warp * k + i] = keys[ids[i]];
    }
    __syncthreads();
    if (warp == 0) {
        warp_select(sc->keys, k * Warps, k, lane, sc->room[0], sc->place[0], out);
        __syncwarp();
        for (int i = lane; i < k; i += 32) out[i] = sc->ids[out[i]];
    }
}

}  // namespace paged
}  // namespace hga
