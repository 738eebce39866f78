// rope.cuh -- the position rotation of one row piece, shared by the rotation
// calls (rope.cu) and the paged cache's append (paged_append.cu).
//
// The pair (x1, x2) of frequency i at position t becomes
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s,   c = table[t][i], s = table[t][rot/2 + i],
// each product and each sum rounded to float32 by itself (no contraction to
// FMA), so the result is the same bit for bit wherever a row is rotated: in
// a training segment, in a prompt or as a single token.
// Pairs are (i, i + rot/2), or (2i, 2i + 1) when interleaved; elements from
// rot on pass unchanged.
//
// A row of d elements is cut into d/16 units of 16 elements that hold whole
// pairs: unit u < rot/16 of the half layout is elements 8u .. 8u+7 and their
// partners rot/2 + 8u .., an interleaved or unrotated unit 16 neighbours.
// Either way a unit is two 8-element vectors (16 bytes of bf16, 32 of
// float32) and needs the 8 cosines and sines from 8u on.
#pragma once

#include "hga_internal.cuh"

namespace hga {
namespace rope {

struct Unit {
    int a, b;          // first elements of its two vectors
    bool turned;
};

__device__ __forceinline__ Unit unit_of(int u, int rot, bool interleaved)
{
    Unit r;
    r.turned = 16 * u < rot;
    if (r.turned && !interleaved) {
        r.a = 8 * u;
        r.b = 8 * u + rot / 2;
    } else {
        r.a = 16 * u;
        r.b = 16 * u + 8;
    }
    return r;
}

// Raw bits of 8 elements (16 bytes of bf16, two times 16 of float32).
// load_plain: for rows that the same kernel also writes.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_plain(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void widen(float* o) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Raw8<float> {
    uint4 v, w;
    __device__ __forceinline__ void load(const float* p)
    {
        v = __ldg(reinterpret_cast<const uint4*>(p));
        w = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void load_plain(const float* p)
    {
        v = reinterpret_cast<const uint4*>(p)[0];
        w = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const
    {
        reinterpret_cast<uint4*>(p)[0] = v;
        reinterpret_cast<uint4*>(p)[1] = w;
    }
    __device__ __forceinline__ void widen(float* o) const
    {
        const uint32_t r[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(r[i]);
    }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 elements rounded once (to nearest even) and stored.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x)
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x)
{
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The cosines and sines of unit u at a table row.
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void load(const float* __restrict__ row, int u, int rot)
    {
        const float4* pc = reinterpret_cast<const float4*>(row + 8 * u);
        const float4* ps = reinterpret_cast<const float4*>(row + rot / 2 + 8 * u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 a = __ldg(pc + i), b = __ldg(ps + i);
            c[4 * i] = a.x; c[4 * i + 1] = a.y; c[4 * i + 2] = a.z; c[4 * i + 3] = a.w;
            s[4 * i] = b.x; s[4 * i + 1] = b.y; s[4 * i + 2] = b.z; s[4 * i + 3] = b.w;
        }
    }
};

// x[0..7] the unit's first vector, x[8..15] its second.  BACK turns by the
// opposite angle (the rotation's transpose, which is its gradient).
template <bool BACK>
__device__ __forceinline__ void turn(float (&x)[16], const Angles& t, bool interleaved)
{
    auto pair = [](float& x1, float& x2, float c, float s) {
        if (BACK) s = -s;
        const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
        x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
        x1 = y1;
    };
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) pair(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) pair(x[i], x[8 + i], t.c[i], t.s[i]);
    }
}

}  // namespace rope
}  // namespace hga
