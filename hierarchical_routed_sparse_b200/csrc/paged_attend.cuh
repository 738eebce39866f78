// paged_attend.cuh -- one warp's attention over 16 keys at a time, for the up
// to 8 q-heads of a kv-head.
//
// The products run as mma.sync m16n8k16 with the keys (scores) or the head
// dimension (outputs) as M and the heads as N = 8: S^T = K Q^T, O^T = V^T P^T.
// A decode step does 2 x 8 multiply-adds for each code it reads, a
// hundredth of what tcgen05 could do and far below what its 128-row tiles
// would have to be fed, so the tensor work must be cheap to feed, not fast:
// with these fragments a code is loaded from shared memory once, straight into
// the register it is used from.  Which d an MMA's k index means and which key
// its column is are free as long as both operands agree, so the lanes' pieces
// are chosen as whole 16-byte loads:
//   lane = 4 g + t (g < 8, t < 4).
//   K   lane takes rows g of both groups, d = 64 j + 16 t .. + 15
//   Q   lane holds head g at the same d
//   V   lane takes rows 2t, 2t + 1 of both groups, d = (D/8) g .. + D/8 - 1
//   S   lane gets heads 2t, 2t + 1 of rows g; O: the same heads at its V d's.
// The weights pass from the S lanes to the P^T operand's by movmatrix.
//
// A tile is four groups (32 keys), two such products side by side.  Its keys
// and its values wait in halves of the warp's own ring of shared memory,
// filled by cp.async: while the scores of tile i are formed, its values and
// the keys of tile i + 1 are on their way.  A warp orders its ring by itself,
// so the loop has no barrier.  Rows of 128 bytes are swizzled so that neither
// the K nor the V loads meet bank conflicts.
//
// Precision.  Codes are exact in float16 (int8: at most 127; e4m3: 4
// significant bits).  A bf16 query is exact in float16 too once its row is
// scaled by a power of two (elements 2^-27 below the row's largest lose
// bits: their products are below the sum's rounding; so do rows below
// 2^-120, where the scaling ends); a float32 query, and
// every weight, is the sum of two float16 parts, which carry 2^-24 of it.
// Sums are float32.
//
// Running softmax, in units of log2.  With s the score and v the group's value
// scale, the normalising sum collects e = 2^(s - R), and a weight enters the
// products as e (v 2^-W): R is a score that has been met, W a whole number.
// They are two numbers, not their sum, because a score can be so large that
// a float32 next to it cannot say how large the values are, and because the
// sum of all e must not depend on the values' size (one tile of zeros
// beside one of 2^40).
// Both move when a tile's largest e max(v 2^-W, 1) is above 2^15, so e stays
// below that and so does e v 2^-W, which float16 has to hold.  W is
// then 12 below the largest s - R + log2 v so far, so most tiles find both as
// they should be and weights down to 2^-24 of the largest keep all their bits,
// whatever the values' sizes.  (Open rows take the largest of their values for
// v, for W alone.)  log2 v counts as at least -90; values below 2^-90 lose
// bits.  Parts of a head (warps, CTAs) are joined as means by their shares of
// the common sum, so W stays a warp's own.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "hga_internal.cuh"

namespace hga {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// R of a warp that has met no key, and a score like any other: the lowest of
// float32, so that no key is missed for being far below zero.
constexpr float kFloor = -3.402823466e38f;
constexpr float kBelow = 12.f, kAbove = 32768.f;      // of W in log2; of a weight
constexpr int kLeastV = -90;                         // log2 of the smallest values that W follows
// Keys further below R than this count as if they were there, so that v 2^-W
// stays a float32 however large the values of such keys are.
constexpr float kFar = -64.f, kFarWeight = 1.f / 18446744073709551616.f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from a zero sum.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Transpose of an 8 x 8 matrix of 16-bit elements, two of a row in each lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Float16 pair = hi + lo of two float32 values.
__device__ __forceinline__ void split_half2(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    hi = half2_bits(h);
    lo = half2_bits(__floats2half2_rn(x0 - f.x, x1 - f.y));
}

// Codes to float16.  four(): the codes of a word, two and two.
template <int CACHE> struct Codes;
template <> struct Codes<HGA_INT8> {
    // 0x64 above a byte u is the float16 1024 + u; u = code + 128.
    static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w ^ 0x80808080u; }
    static __device__ __forceinline__ uint32_t low(uint32_t u)
    {
        const uint32_t m = __byte_perm(u, 0x64646464u, 0x4140), k = 0x64806480u;
        return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&k)));
    }
    static __device__ __forceinline__ uint32_t high(uint32_t u)
    {
        const uint32_t m = __byte_perm(u, 0x64646464u, 0x4342), k = 0x64806480u;
        return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&k)));
    }
};
template <> struct Codes<HGA_E4M3> {
    static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w; }
    static __device__ __forceinline__ uint32_t low(uint32_t u)
    {
        uint32_t h;
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(h) : "r"(u));
        return h;
    }
    static __device__ __forceinline__ uint32_t high(uint32_t u)
    {
        uint32_t h;
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(h) : "r"(u));
        return h;
    }
};

// 1 / x, off by 2^-23 of it.
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a positive value rounded up (or one more): at least kLeastV; 0 where
// the value is not finite.
__device__ __forceinline__ int log2_above(float v)
{
    const int e = int(__float_as_uint(v) >> 23) - 126;
    return e > 128 ? 0 : max(e, kLeastV);
}

// Running state of a warp: references and sums of heads 2t, 2t + 1 (the sum
// over this lane's rows only), their outputs, and 2^-W of both as bfloat16
// halves of a word (a register less than two floats, where the 128-register
// kernels spill).
template <int D> struct Running {
    static constexpr int kM = D / 16;
    float acc[kM][4];                                // [i]: d = (D/8) g + 2i, head 2t, 2t + 1; then d + 1
    float R0, R1, l0, l1;
    uint32_t down;                                   // head 2t in the upper half

    __device__ __forceinline__ float down0() const { return __uint_as_float(down & 0xFFFF0000u); }
    __device__ __forceinline__ float down1() const { return __uint_as_float(down << 16); }

    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        R0 = R1 = kFloor;
        l0 = l1 = 0.f;
        down = 0x00010001u * (uint32_t)((127 + 12 - kLeastV) << 7);
        static_assert(kBelow == 12.f, "W starts at its least");
    }
    // R and W of one head from a tile's largest score m and log2 v; returns the
    // factor for the outputs, and 2^-W in place of c.  W stays in [-102, 116].
    __device__ __forceinline__ static float move(float& R, float& l, float& c, float m, float lv)
    {
        const float n = fmaxf(R, m), fall = R - n, W = float(127 - int(__float_as_uint(c) >> 23));
        const float w = ceilf(fmaxf(W + fall, fmaxf(m - n, kFar) + (lv - kBelow)));
        c = __uint_as_float(uint32_t(127 - int(w)) << 23);
        l *= ex2(fall);
        R = n;
        return ex2(fall + (W - w));
    }
    // Move them where a tile's largest scores of this lane and its largest v
    // ask for it.
    __device__ __forceinline__ void follow(float m0, float m1, float v)
    {
        float c0 = down0(), c1 = down1();
        const float x0 = fmaxf(ex2(m0 - R0), kFarWeight) * fmaxf(v * c0, 1.f);
        const float x1 = fmaxf(ex2(m1 - R1), kFarWeight) * fmaxf(v * c1, 1.f);
        if (!__any_sync(0xFFFFFFFFu, x0 > kAbove || x1 > kAbove)) return;
        const float lv = (float)log2_above(v);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
        }
        const float f0 = move(R0, l0, c0, m0, lv), f1 = move(R1, l1, c1, m1, lv);
        down = __float_as_uint(c0) | __float_as_uint(c1) >> 16;
#pragma unroll
        for (int i = 0; i < kM; ++i) {
            acc[i][0] *= f0;
            acc[i][1] *= f1;
            acc[i][2] *= f0;
            acc[i][3] *= f1;
        }
    }
    // Out of the registers into shared memory (kParked floats), and back.
    static constexpr int kParked = 32 * (4 * kM + 5);
    __device__ __forceinline__ void park(float* p, int lane) const
    {
#pragma unroll
        for (int i = 0; i < 4 * kM; ++i) p[32 * i + lane] = acc[i / 4][i % 4];
        p += 32 * 4 * kM + lane;
        p[0] = R0;
        p[32] = R1;
        p[64] = l0;
        p[96] = l1;
        p[128] = __uint_as_float(down);
    }
    __device__ __forceinline__ void unpark(const float* p, int lane)
    {
#pragma unroll
        for (int i = 0; i < 4 * kM; ++i) acc[i / 4][i % 4] = p[32 * i + lane];
        p += 32 * 4 * kM + lane;
        R0 = p[0];
        R1 = p[32];
        l0 = p[64];
        l1 = p[96];
        down = __float_as_uint(p[128]);
    }
    // o [G][D], r [G], l [G] of this warp, and f [G] that make means of o.
    __device__ __forceinline__ void store(float* o, float* r, float* l, float* f, int G, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, x);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, x);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (2 * t + e >= G) continue;
            float* row = o + (2 * t + e) * D + (D / 8) * g;
#pragma unroll
            for (int i = 0; i < kM; ++i)
                *reinterpret_cast<float2*>(row + 2 * i) = make_float2(acc[i][e], acc[i][2 + e]);
            if (g == 0) {
                r[2 * t + e] = e ? R1 : R0;
                const float sum = e ? l1 : l0;       // at least 1 where a key was met
                l[2 * t + e] = sum;
                f[2 * t + e] = sum == 0.f ? 0.f : __uint_as_float(0x7F000000u - __float_as_uint(e ? down1() : down0())) * rcp(sum);
            }
        }
    }
};

__device__ __forceinline__ void load4(const float* p, float (&y)[4])
{
    const float4 w = __ldg(reinterpret_cast<const float4*>(p));
    y[0] = w.x; y[1] = w.y; y[2] = w.z; y[3] = w.w;
}
__device__ __forceinline__ void widen4(uint2 w, float (&y)[4])
{
    y[0] = __uint_as_float(w.x << 16); y[1] = __uint_as_float(w.x & 0xFFFF0000u);
    y[2] = __uint_as_float(w.y << 16); y[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&y)[4])
{
    widen4(__ldg(reinterpret_cast<const uint2*>(p)), y);
}
__device__ __forceinline__ void load4_shared(const float* p, float (&y)[4])
{
    const float4 w = *reinterpret_cast<const float4*>(p);
    y[0] = w.x; y[1] = w.y; y[2] = w.z; y[3] = w.w;
}
__device__ __forceinline__ void load4_shared(const __nv_bfloat16* p, float (&y)[4])
{
    widen4(*reinterpret_cast<const uint2*>(p), y);
}

// The references and sums of one head's parts, one part a lane of N neighbours
// (a power of two): r becomes the common reference, l the sum for it; returns
// the part's share of that sum.  A sum of zero (no part has met a key) has
// shares of zero, or of NaN when these were the last parts: all scores were
// below float32.  The whole warp takes part.
template <int N> __device__ __forceinline__ float join_parts(float& r, float& l, bool last)
{
    float M = r;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    const float mine = l * ex2(r - M);
    l = mine;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    r = M;
    return l == 0.f && !last ? 0.f : mine * rcp(l);
}

// The query as the products' B operand, and what turns a product into a
// score in log2 units, for heads 2t, 2t + 1.
template <typename TIn, int D> struct Query {
    static constexpr bool kTwo = sizeof(TIn) == 4;   // float32: two float16 parts
    uint32_t b[D / 16][2], c[kTwo ? D / 16 : 1][2];
    float f0, f1;

    __device__ __forceinline__ Query(const TIn* q, int G, float scale, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        float x[D / 16][4], top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
            {
                float (&y)[4] = x[4 * j + k];
                y[0] = y[1] = y[2] = y[3] = 0.f;
                if (g < G) load4(q + g * D + 64 * j + 16 * t + 4 * k, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(y[e]));
            }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^(13 - floor(log2 top)), by the exponent's bits, at most 2^120 (its
        // inverse times `scale` is to stay a normal float32); 1 for rows of
        // zeros and of infinities.
        const int ex = int(__float_as_uint(top) >> 23);
        const int sh = ex == 0 || ex == 255 ? 0 : min(max(13 - (ex - 127), -126), 120);
        const float up = __uint_as_float(uint32_t(127 + sh) << 23), down = __uint_as_float(uint32_t(127 - sh) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t lo;
                split_half2(x[k][2 * e] * up, x[k][2 * e + 1] * up, b[k][e], lo);
                if constexpr (kTwo) c[k][e] = lo;
            }
        // Head n's factor sits in the lanes of g = n.
        f0 = __shfl_sync(0xFFFFFFFFu, down, 8 * t) * scale;
        f1 = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4) * scale;
    }
};

// Half of a tile's data: the codes and scales of the keys, or of the values, of
// four groups.  A group that is missing has a scale of -1 (keys) or 0.
constexpr int kTileGroups = 4, kTileKeys = kTileGroups * kGroup;
constexpr int kHalves = 3;                           // halves in a warp's ring
template <int D> struct alignas(16) Half {
    uint8_t code[kTileKeys * D];
    alignas(16) float scale[kTileGroups];
};

// 16-byte pieces of a row change places: K by the row's parity (eight lanes
// read four pieces of two neighbouring rows), V by the row pair (four lanes
// read the same two pieces of rows 0, 2, 4, 6).
template <int D, bool V> __device__ __forceinline__ int piece(int row, int c)
{
    if (V) return D == 128 ? c ^ (2 * ((row >> 1) & 3)) : c ^ ((row >> 1) & 3);
    return D == 128 ? c ^ (4 * (row & 1)) : c;
}

// 16 bytes from src + kFrom to dst + kTo of shared memory; bytes = 0 fills zeros.
template <int kTo, int kFrom> __device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0+%3], [%1+%4], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(kTo),
                 "n"(kFrom)
                 : "memory");
}

// Start the copy of a half: lanes 8 x .. 8 x + 7 copy group x, whose number
// (over page, kv-head and group; -1: none) they hold in `at`.
template <int D, bool V>
__device__ __forceinline__ void fetch(Half<D>& s, const uint8_t* codes, const float* scales, int64_t at, int lane)
{
    const int x = lane >> 3, c = lane & 7;
    const bool there = at >= 0;
    const int bytes = there ? 16 : 0;
    const uint8_t* from = codes + (there ? at : 0) * (kGroup * D) + 16 * c;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(s.code) + x * (kGroup * D);
    if constexpr (D == 128) {                        // a row at a time, its piece c
        const uint32_t even = to + 16 * c;
        const uint32_t r2 = to + 16 * (V ? c ^ 2 : c), r4 = to + 16 * (V ? c ^ 4 : c), r6 = to + 16 * (V ? c ^ 6 : c);
        const uint32_t odd = V ? even : to + 16 * (c ^ 4);       // piece<D, V>(row, c)
        cp16<0, 0>(even, from, bytes);
        cp16<128, 128>(odd, from, bytes);
        cp16<256, 256>(r2, from, bytes);
        cp16<384, 384>(V ? r2 : odd, from, bytes);
        cp16<512, 512>(r4, from, bytes);
        cp16<640, 640>(V ? r4 : odd, from, bytes);
        cp16<768, 768>(r6, from, bytes);
        cp16<896, 896>(V ? r6 : odd, from, bytes);
    } else {                                         // two rows at a time
        const uint32_t at0 = to + 64 * (c >> 2);
        const int p = c & 3;
        cp16<0, 0>(at0 + 16 * p, from, bytes);
        cp16<128, 128>(at0 + 16 * (V ? p ^ 1 : p), from, bytes);
        cp16<256, 256>(at0 + 16 * (V ? p ^ 2 : p), from, bytes);
        cp16<384, 384>(at0 + 16 * (V ? p ^ 3 : p), from, bytes);
    }
    if (c == 0) {
        if (there)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(s.scale + x)),
                         "l"(scales + at)
                         : "memory");
        else
            s.scale[x] = V ? 0.f : -1.f;
    }
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of the warp's copies but the newest two halves have landed, for all its lanes.
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kHalves - 1) : "memory");
    __syncwarp();
}

__device__ __forceinline__ void fetch_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// Scores of a tile in log2 units: s[x][0..1] of row g of group 2x for heads 2t,
// 2t + 1, s[x][2..3] of group 2x + 1.
template <typename TIn, int D, int CACHE>
__device__ __forceinline__ void held_scores(float (&s)[2][4], const Query<TIn, D>& q, const Half<D>& k, int lane)
{
    using C = Codes<CACHE>;
    const int g = lane >> 2, t = lane & 3;
    float r[2][4];                                   // two chains of products for each half of the tile
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint8_t* row = k.code + (16 * x + g) * D + 16 * piece<D, false>(g, 4 * j + t);
            const uint4 ka = *reinterpret_cast<const uint4*>(row), kz = *reinterpret_cast<const uint4*>(row + 8 * D);
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wz[4] = {kz.x, kz.y, kz.z, kz.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t ua = C::prep(wa[i]), uz = C::prep(wz[i]);
                const uint32_t a0 = C::low(ua), a1 = C::low(uz), a2 = C::high(ua), a3 = C::high(uz);
                const uint32_t b0 = q.b[4 * j + i][0], b1 = q.b[4 * j + i][1];
                if (j == 0 && i < 2) mma_f16_first(i ? r[x] : s[x], a0, a1, a2, a3, b0, b1);
                else mma_f16(i & 1 ? r[x] : s[x], a0, a1, a2, a3, b0, b1);
                if constexpr (Query<TIn, D>::kTwo)
                    mma_f16(i & 1 ? r[x] : s[x], a0, a1, a2, a3, q.c[4 * j + i][0], q.c[4 * j + i][1]);
            }
        }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const float ks = k.scale[y], none = ks < 0.f ? -INFINITY : 0.f;      // (a NaN scale is there)
        const float f0 = q.f0 * ks, f1 = q.f1 * ks;
        float* v = s[y / 2] + 2 * (y % 2);
        v[0] = fmaf(v[0] + r[y / 2][2 * (y % 2)], f0, none);
        v[1] = fmaf(v[1] + r[y / 2][2 * (y % 2) + 1], f1, none);
    }
}

// The tile's weights and outputs, given its scores.
template <int D, int CACHE>
__device__ __forceinline__ void held_outputs(Running<D>& run, const float (&s)[2][4], const Half<D>& v, int lane)
{
    using C = Codes<CACHE>;
    const int g = lane >> 2, t = lane & 3;
    const float4 scales = *reinterpret_cast<const float4*>(v.scale);
    const float vs[4] = {scales.x, scales.y, scales.z, scales.w};
    // (fmaxf passes a NaN scale over.)
    run.follow(fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2])),
               fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3])),
               fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3])));
    const float w0 = run.down0(), w1 = run.down1();
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const float e0 = ex2(s[y / 2][2 * (y % 2)] - run.R0), e1 = ex2(s[y / 2][2 * (y % 2) + 1] - run.R1);
        run.l0 += e0;
        run.l1 += e1;
        split_half2(e0 * (vs[y] * w0), e1 * (vs[y] * w1), hi[y], lo[y]);
        hi[y] = transpose8(hi[y]);
        lo[y] = transpose8(lo[y]);
    }
    // The tile's outputs are formed from zero and then added: a tensor-core sum
    // cuts its last bit off, which over thousands of keys would show.  p: the
    // words of rows 2t, 2t + 1 of the four groups at d .. d + 3.
    auto four = [&](int i, const uint32_t (&p)[4][2]) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            // Bytes d, d + 1 (then d + 2, d + 3) of two keys side by side.
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) w[y] = __byte_perm(C::prep(p[y][0]), C::prep(p[y][1]), m ? 0x7362 : 0x5140);
            uint32_t a[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                a[x][0] = C::low(w[2 * x]);
                a[x][1] = C::high(w[2 * x]);
                a[x][2] = C::low(w[2 * x + 1]);
                a[x][3] = C::high(w[2 * x + 1]);
            }
            float o[4];
            mma_f16_first(o, a[0][0], a[0][1], a[0][2], a[0][3], lo[0], lo[1]);
            mma_f16(o, a[1][0], a[1][1], a[1][2], a[1][3], lo[2], lo[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) mma_f16(o, a[x][0], a[x][1], a[x][2], a[x][3], hi[2 * x], hi[2 * x + 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) run.acc[i + m][e] += o[e];
        }
    };
    // A lane's piece of a row: D/8 bytes.
    const int c = D == 128 ? 16 * piece<D, true>(2 * t, g) : 16 * piece<D, true>(2 * t, g / 2) + 8 * (g % 2);
    const uint8_t* row = v.code + 2 * t * D + c;
    if constexpr (D == 128) {
        uint4 w[4][2];
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y / 2][y % 2] = *reinterpret_cast<const uint4*>(row + (8 * (y / 2) + y % 2) * D);
        const uint32_t p0[4][2] = {{w[0][0].x, w[0][1].x}, {w[1][0].x, w[1][1].x}, {w[2][0].x, w[2][1].x}, {w[3][0].x, w[3][1].x}};
        const uint32_t p1[4][2] = {{w[0][0].y, w[0][1].y}, {w[1][0].y, w[1][1].y}, {w[2][0].y, w[2][1].y}, {w[3][0].y, w[3][1].y}};
        const uint32_t p2[4][2] = {{w[0][0].z, w[0][1].z}, {w[1][0].z, w[1][1].z}, {w[2][0].z, w[2][1].z}, {w[3][0].z, w[3][1].z}};
        const uint32_t p3[4][2] = {{w[0][0].w, w[0][1].w}, {w[1][0].w, w[1][1].w}, {w[2][0].w, w[2][1].w}, {w[3][0].w, w[3][1].w}};
        four(0, p0);
        four(2, p1);
        four(4, p2);
        four(6, p3);
    } else {
        uint2 w[4][2];
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y / 2][y % 2] = *reinterpret_cast<const uint2*>(row + (8 * (y / 2) + y % 2) * D);
        const uint32_t p0[4][2] = {{w[0][0].x, w[0][1].x}, {w[1][0].x, w[1][1].x}, {w[2][0].x, w[2][1].x}, {w[3][0].x, w[3][1].x}};
        const uint32_t p1[4][2] = {{w[0][0].y, w[0][1].y}, {w[1][0].y, w[1][1].y}, {w[2][0].y, w[2][1].y}, {w[3][0].y, w[3][1].y}};
        four(0, p0);
        four(2, p1);
    }
}

// Attention over n tiles of held keys: group_of(i) is the number of this
// lane's group (lane / 8) of tile i, called once for each i in order by the
// whole warp.  Halves K0 V0 K1 V1 ... go round the ring; a copy that is not
// wanted is an empty group, so that the count of groups says what has landed.
// start() begins the first copies; other work of the warp may come between.
template <typename TIn, int D, int CACHE, typename GroupOf> struct HeldTiles {
    Half<D>* ring;
    const hga_paged_cache& c;
    GroupOf group_of;
    int n, lane;
    int64_t at;                                      // the newest tile's group

    __device__ __forceinline__ HeldTiles(Half<D>* ring_, const hga_paged_cache& c_, GroupOf group_of_, int n_, int lane_)
        : ring(ring_), c(c_), group_of(group_of_), n(n_), lane(lane_), at(-1)
    {
    }
    __device__ __forceinline__ void keys(int slot) { fetch<D, false>(ring[slot], static_cast<const uint8_t*>(c.k_pages), c.k_scale, at, lane); }
    __device__ __forceinline__ void values(int slot) { fetch<D, true>(ring[slot], static_cast<const uint8_t*>(c.v_pages), c.v_scale, at, lane); }
    __device__ __forceinline__ void start()
    {
        if (n <= 0) return;
        at = group_of(0);
        keys(0);
        fetch_commit();
        values(1);
        fetch_commit();
        if (n > 1) {
            at = group_of(1);
            keys(2);
        }
        fetch_commit();
    }
    __device__ __forceinline__ void attend(Running<D>& run, const TIn* q, int G, float scale)
    {
        if (n <= 0) return;
        const Query<TIn, D> qf(q, G, scale, lane);
        int slot = 0;                                // of K_i; V_i is in the next
        for (int i = 0; i < n; ++i) {
            const int vslot = slot == 2 ? 0 : slot + 1;
            float s[2][4];
            fetch_wait();
            held_scores<TIn, D, CACHE>(s, qf, ring[slot], lane);
            __syncwarp();
            if (i + 1 < n) values(slot);
            fetch_commit();
            fetch_wait();
            held_outputs<D, CACHE>(run, s, ring[vslot], lane);
            __syncwarp();
            if (i + 2 < n) {
                at = group_of(i + 2);
                keys(vslot);
            }
            fetch_commit();
            slot = vslot == 2 ? 0 : vslot + 1;
        }
    }
};

// ---- open rows: float32 keys, values in their own type --------------------------------
// Scores by tf32 products (m16n8k8): a float32 is the sum of two tf32 parts,
// 11 bits and 11 of the other 13, a bfloat16 is one.  Weights times values by
// bfloat16 products: a float32 is exactly the sum of three bfloat16 (its bits
// 8 and 8 and 8).  Products of parts below 2^-22 and 2^-24 of the whole are
// left out.
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo)
{
    hi = __float_as_uint(x) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// The upper halves of two words, the first in the low half.
__device__ __forceinline__ uint32_t upper(float x0, float x1) { return __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632); }

__device__ __forceinline__ void split3(float x0, float x1, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = upper(x0, x1);
        if (i == 2) break;
        x0 -= __uint_as_float(p[i] << 16);
        x1 -= __uint_as_float(p[i] & 0xFFFF0000u);
    }
}

// 16 open rows from row0 on, of which those below `rows` are there; the others
// count as zero.  key(), value(): a 16-byte piece of the tile's row.
template <typename TIn, int D> struct OpenGlobal {
    const float* k;
    const TIn* v;
    const TIn* q;                                    // the kv-head's queries
    int row0, rows;
    __device__ __forceinline__ void query(int head, int e, float (&y)[4]) const { load4(q + head * D + e, y); }
    __device__ __forceinline__ float4 key(int row, int piece) const
    {
        return row0 + row < rows ? __ldg(reinterpret_cast<const float4*>(k + (row0 + row) * D) + piece)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ uint4 value(int row, int piece) const
    {
        return row0 + row < rows ? __ldg(reinterpret_cast<const uint4*>(v + (row0 + row) * D) + piece)
                                 : make_uint4(0u, 0u, 0u, 0u);
    }
};

// The same from a slot of shared memory that cp.async has filled (values of 4
// bytes stay in global memory).  Pieces change places so that a quarter of a
// warp reads eight different ones: keys by the row's parity, values by the row
// pair.
template <typename TIn, int D> struct OpenSlot {
    static constexpr bool kValues = sizeof(TIn) == 2;
    static constexpr int kKeyBytes = 16 * D * 4, kBytes = kKeyBytes + (kValues ? 16 * D * (int)sizeof(TIn) : 0);
    static constexpr int N = D / 8 * (int)sizeof(TIn) / 16;      // pieces of a row that a lane takes
    static constexpr int kQueryRow = D + 16;         // elements; the eight heads' pieces lie in different banks
    const uint8_t* slot;
    TIn* qs;                                         // the queries' place, common to the CTA's warps
    OpenGlobal<TIn, D> rest;
    __device__ __forceinline__ void query(int head, int e, float (&y)[4]) const { load4_shared(qs + head * kQueryRow + e, y); }
    // By the whole warp (every warp that reads them writes all of them).
    __device__ __forceinline__ void fetch_queries(int G, int lane) const
    {
        constexpr int kPieces = D * (int)sizeof(TIn) / 16, kEach = 16 / (int)sizeof(TIn);
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(qs);
        for (int i = lane; i < G * kPieces; i += 32)
            cp16<0, 0>(to + (i / kPieces * kQueryRow + i % kPieces * kEach) * (int)sizeof(TIn), rest.q + i * kEach, 16);
    }

    static __device__ __forceinline__ int key_at(int row, int piece) { return 16 * (row * (D / 4) + (piece ^ (4 * (row & 1)))); }
    static __device__ __forceinline__ int value_at(int row, int piece)
    {
        const int p = row >> 1;
        return kKeyBytes + 16 * (row * (D / 8) + (piece ^ (N == 1 ? 2 * (p & 3) : 4 * (p & 1) + ((p >> 1) & 1))));
    }
    // By the whole warp; the copies are the warp's own, not committed yet.
    __device__ __forceinline__ void fetch(int lane) const
    {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const int row = (32 * i + lane) / (D / 4), piece = (32 * i + lane) % (D / 4);
            const bool there = rest.row0 + row < rest.rows;
            cp16<0, 0>(to + key_at(row, piece), rest.k + (there ? (rest.row0 + row) * D + 4 * piece : 0), there ? 16 : 0);
        }
        if constexpr (kValues) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int row = (32 * i + lane) / (D / 8), piece = (32 * i + lane) % (D / 8);
                const bool there = rest.row0 + row < rest.rows;
                cp16<0, 0>(to + value_at(row, piece), rest.v + (there ? (rest.row0 + row) * D + 8 * piece : 0), there ? 16 : 0);
            }
        }
    }
    __device__ __forceinline__ float4 key(int row, int piece) const
    {
        return *reinterpret_cast<const float4*>(slot + key_at(row, piece));
    }
    __device__ __forceinline__ uint4 value(int row, int piece) const
    {
        if constexpr (kValues) return *reinterpret_cast<const uint4*>(slot + value_at(row, piece));
        else return rest.value(row, piece);
    }
};

// A lane's values of 16 open rows: rows 2t, 2t + 1 and 8 + 2t, 8 + 2t + 1,
// d = (D/8) g .. + D/8 - 1.
template <typename TIn, int D> struct OpenValues {
    static constexpr int N = D / 8 * (int)sizeof(TIn) / 16;      // 16-byte pieces of a row
    uint4 w[4][N];
    template <typename Open> __device__ __forceinline__ void load(const Open& open, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < N; ++i) w[x][i] = open.value(8 * (x / 2) + 2 * t + x % 2, N * g + i);
    }
    __device__ __forceinline__ uint32_t word(int x, int i) const
    {
        const uint4 q = w[x][i / 4];
        return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
    }
    // The tile's largest value.
    __device__ __forceinline__ float most() const
    {
        float top = 0.f;
        if constexpr (sizeof(TIn) == 2) {
            __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4 * N; ++i) {
                    const uint32_t u = word(x, i);
                    m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u)));
                }
            top = fmaxf(__low2float(m), __high2float(m));
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4 * N; ++i) top = fmaxf(top, fabsf(__uint_as_float(word(x, i))));
        }
        return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
    }
};

// One tile of open rows (OpenGlobal, OpenSlot), of which the first `rows` are there.
template <typename TIn, int D, typename Open>
__device__ __forceinline__ void attend_open(Running<D>& run, int G, const Open& open, int rows, float scale, int lane)
{
    constexpr bool kF32 = sizeof(TIn) == 4;
    const int g = lane >> 2, t = lane & 3;
    const bool ha = g < rows, hz = 8 + g < rows;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
    // All of the tile's loads at once, where the registers reach (a tile is one
    // round trip and a chain of a few hundred instructions).
    OpenValues<TIn, D> val;
    if constexpr (!kF32) val.load(open, lane);
    float4 ka[D / 16], kz[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        ka[i] = open.key(g, 4 * i + t);
        kz[i] = open.key(8 + g, 4 * i + t);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {               // d = 16 i + 4 t .. + 3: two products of 8
        const float4 xa = ka[i], xz = kz[i];
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (g < G) open.query(g, 16 * i + 4 * t, y);
        uint32_t h[8], l[8];
        split_tf32(xa.x, h[0], l[0]);
        split_tf32(xz.x, h[1], l[1]);
        split_tf32(xa.y, h[2], l[2]);
        split_tf32(xz.y, h[3], l[3]);
        split_tf32(xa.z, h[4], l[4]);
        split_tf32(xz.z, h[5], l[5]);
        split_tf32(xa.w, h[6], l[6]);
        split_tf32(xz.w, h[7], l[7]);
        uint32_t b[4], c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kF32) split_tf32(y[e], b[e], c[e]);
            else b[e] = __float_as_uint(y[e]);
        }
        mma_tf32(r, l[0], l[1], l[2], l[3], b[0], b[1]);
        mma_tf32(r, l[4], l[5], l[6], l[7], b[2], b[3]);
        if constexpr (kF32) {
            mma_tf32(r, h[0], h[1], h[2], h[3], c[0], c[1]);
            mma_tf32(r, h[4], h[5], h[6], h[7], c[2], c[3]);
        }
        mma_tf32(s, h[0], h[1], h[2], h[3], b[0], b[1]);
        mma_tf32(s, h[4], h[5], h[6], h[7], b[2], b[3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = (e < 2 ? ha : hz) ? (s[e] + r[e]) * scale : -INFINITY;
    if constexpr (kF32) val.load(open, lane);
    run.follow(fmaxf(s[0], s[2]), fmaxf(s[1], s[3]), val.most());
    const float e0 = ex2(s[0] - run.R0), e1 = ex2(s[1] - run.R1), e2 = ex2(s[2] - run.R0), e3 = ex2(s[3] - run.R1);
    run.l0 += e0 + e2;
    run.l1 += e1 + e3;
    const float c0 = run.down0(), c1 = run.down1();
    uint32_t w0[3], w1[3];
    split3(e0 * c0, e1 * c1, w0);
    split3(e2 * c0, e3 * c1, w1);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        w0[i] = transpose8(w0[i]);
        w1[i] = transpose8(w1[i]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {               // d = (D/8) g + 2i, + 1
        if constexpr (!kF32) {
            const uint32_t w[4] = {val.word(0, i), val.word(1, i), val.word(2, i), val.word(3, i)};
#pragma unroll
            for (int x = 2; x >= 0; --x)
                mma_bf16(run.acc[i], __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                         __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632), w0[x], w1[x]);
        } else {
            uint32_t a[4][3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {            // d even, odd
                split3(__uint_as_float(val.word(0, 2 * i + e)), __uint_as_float(val.word(1, 2 * i + e)), a[e]);
                split3(__uint_as_float(val.word(2, 2 * i + e)), __uint_as_float(val.word(3, 2 * i + e)), a[2 + e]);
            }
#pragma unroll
            for (int n = 2; n >= 0; --n)             // parts x of V and n - x of the weights, the smallest first
#pragma unroll
                for (int x = 0; x <= n; ++x) mma_bf16(run.acc[i], a[0][x], a[1][x], a[2][x], a[3][x], w0[n - x], w1[n - x]);
        }
    }
}

}  // namespace paged
}  // namespace hga
