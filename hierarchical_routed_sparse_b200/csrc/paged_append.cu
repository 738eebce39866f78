// paged_append.cu -- tokens of a ragged batch join the paged cache, rotated on
// the way.
//
// A call gets N packed tokens, some for each sequence.  It rotates their
// queries into q_out, writes rotated keys (float32) and values into the
// open rows of the sequence's last chunk, and closes every chunk that the
// tokens complete: keys and values as 8-bit codes with one scale for each
// 8-token group and kv-head, and the chunk and group summaries, into the
// chunk's page.  For a group x (8 rows of one head), with a = max |x| and
// L = 127 (int8) or 448 (e4m3):
//     a' = max(a, L 2^-126),  scale = a' / L,  code = round(x * (L * (1 / a')))
// to nearest even, each operation in float32.  A group with a value that is
// not finite gets a NaN scale, so that what reads it shows the fault.
//
// Work is cut into items: a chunk that the call touches, of one sequence.  A
// CTA takes one kv-head of an item (warp w holds group w in registers, so a
// group's maximum is one warp reduction and nothing passes through shared
// memory but the chunk summary) or some q-heads of it.  The kernel is bound
// by the bytes of q, k, v and what it writes for prompts (16384 tokens, 32
// q-heads, 8 kv-heads, d 128: 387 MB in 62 us, 6.2 TB/s, in a captured graph, 67
// us, 5.8 TB/s, called on ever new tokens), and by a launch and three
// dependent loads for single tokens (2 us for one sequence, 7 us for 64 of
// which eight complete a chunk, in a captured graph; a call from Python takes
// the host 9.5 us).  For 64 single tokens the grid is 576 CTAs on the 444 places
// that three CTAs an SM leave, and 8 of a CTA's threads a row at work where no
// chunk closes; for ragged prompts one CTA does two chunks in a row wherever a
// call closes one and opens the next.
//
// Positions are moved by a call of their own, behind the rule that the append
// itself goes by (sequence()): by what it took, so that an empty slot stays
// empty and a position never counts a token that is not in the cache.
//
// Rows of the open chunk that were there before are read when the chunk
// closes.  Where the same call also fills a later chunk, whose rows take
// their place, one CTA does both, in this order.
#include <cuda_fp8.h>

#include <algorithm>

#include "paged.cuh"
#include "rope.cuh"

namespace hga {
namespace {

using namespace rope;

constexpr int kThreads = 256;
// q-heads that a thread runs on one row's angles.
template <typename TIn> constexpr int kQHeads = sizeof(TIn) == 2 ? 4 : 2;
constexpr int kSitePage = 411, kSiteOffsets = 412, kSiteLength = 413;

struct Args {
    PagedShape s;
    hga_paged_cache c;
    PagedAppend a;
    int slots;                                      // CTAs of an item: one a kv-head, then those of the q-heads
    bool few;                                       // about a token a sequence: q-heads side by side, not rows
};

// The tokens that a sequence gets: n of them from `token` on, at positions
// pos .. pos + n - 1.
struct Seq {
    int32_t pos, token, n;                          // pos + n <= 64 max_chunks < 2^31
    __device__ __forceinline__ int first() const { return pos / kChunk; }
    __device__ __forceinline__ int last() const { return (pos + n - 1) / kChunk; }
    __device__ __forceinline__ int chunks() const { return n > 0 ? last() - first() + 1 : 0; }
};

__device__ __forceinline__ Seq sequence(const Args& g, int b)
{
    Seq q;
    q.pos = g.a.pos[b];
    q.token = b;
    q.n = 1;
    if (g.a.cu) {
        q.token = g.a.cu[b];
        const int32_t end = g.a.cu[b + 1];
        q.n = end - q.token;
        if (q.token < 0 || end < q.token || end > g.a.N) {
            paged::flag(kSiteOffsets);
            q.n = 0;
        }
    }
    if (q.pos < 0) q.n = 0;                         // an empty slot of the batch
    int64_t limit = (int64_t)g.s.max_chunks * kChunk;
    if (g.a.rot > 0) limit = limit < g.a.rope_rows ? limit : g.a.rope_rows;
    if (q.n > 0 && (int64_t)q.pos + q.n > limit) {
        paged::flag(kSiteLength);
        q.n = limit > q.pos ? int(limit - q.pos) : 0;
    }
    return q;
}

// Sequence and chunk of an item, by one warp: the items are the touched chunks,
// sequence by sequence.  A lane counts the chunks of `each` neighbouring
// sequences, a prefix sum over the lanes finds the lane, and that lane the
// sequence.  Returns -1 past the last item.
__device__ __forceinline__ int locate(const Args& g, int item, Seq& q, int& chunk)
{
    const int lane = threadIdx.x & 31;
    const int each = (g.s.B + 31) / 32, b0 = lane * each, b1 = min(b0 + each, g.s.B);
    int64_t count = 0;
    Seq mine{0, 0, 0};
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        mine = sequence(g, b);
        count += mine.chunks();
    }
    int64_t upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, item < upto);
    if (!hit) return -1;
    const int who = __ffs(hit) - 1;
    int at = 0, found = -1;
    if (lane == who) {
        int64_t rest = item - (upto - count);
        for (int b = b0; b < b1; ++b) {
            const Seq c = each == 1 ? mine : sequence(g, b);
            if (rest < c.chunks()) {
                q = c;
                at = c.first() + (int)rest;
                found = b;
                break;
            }
            rest -= c.chunks();
        }
    }
    q.pos = __shfl_sync(0xFFFFFFFFu, q.pos, who);
    q.token = __shfl_sync(0xFFFFFFFFu, q.token, who);
    q.n = __shfl_sync(0xFFFFFFFFu, q.n, who);
    chunk = __shfl_sync(0xFFFFFFFFu, at, who);
    return __shfl_sync(0xFFFFFFFFu, found, who);
}

// Rows of the open chunk are written by this kernel too: no read-only path.
__device__ __forceinline__ void load8(const float* p, float* x)
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// 8 codes of values already scaled to the code's range.
template <int CACHE> __device__ __forceinline__ uint2 codes8(const float* y)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (CACHE == HGA_INT8) {
            // Added to 1.5 * 2^23 a value is rounded to a whole number, to nearest
            // even, whose two's complement is in the sum's lowest byte.
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = __float_as_uint(__fadd_rn(y[4 * i + e], 12582912.f));
            w[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi =
                __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The warp's group (R rows of 16 elements a thread): codes into the page's
// rows and the scale.
template <int CACHE, int D, int R>
__device__ __forceinline__ void close_group(const float (&x)[R][16], uint8_t* page_rows, float* scale, const Unit& un,
                                            int rl, int RL, int lane)
{
    constexpr float kLevel = CACHE == HGA_INT8 ? 127.f : 448.f;
    float most = 0.f;                                // NaN once any value is
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) most = max_nan(most, fabsf(x[j][e]));
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    const bool finite = top < 0x7F800000u;
    const float a = fmaxf(__uint_as_float(top), kLevel * 1.17549435e-38f);
    const float f = __fmul_rn(__frcp_rn(a), kLevel);
    if (lane == 0) *scale = finite ? __fdiv_rn(a, kLevel) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        uint8_t* row = page_rows + (rl + RL * j) * D;
        uint2 lo = make_uint2(0u, 0u), hi = lo;
        if (finite) {                                // the same for the whole warp
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __fmul_rn(x[j][e], f);
            lo = codes8<CACHE>(y);
            hi = codes8<CACHE>(y + 8);
        }
        *reinterpret_cast<uint2*>(row + un.a) = lo;
        *reinterpret_cast<uint2*>(row + un.b) = hi;
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// One kv-head of one touched chunk.
template <typename TIn, int D, int CACHE>
__device__ __forceinline__ void append_chunk(const Args& g, const Seq& q, int b, int h, int chunk, float (*part)[D])
{
    constexpr int U = D / 16, RL = 32 / U, R = kGroup / RL;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = lane % U, rl = lane / U;
    const Unit un = unit_of(u, g.a.rot, g.a.interleaved);
    const int r0 = chunk == q.first() ? int(q.pos % kChunk) : 0;
    const int r1 = chunk == q.last() ? int((q.pos + q.n - 1) % kChunk) + 1 : kChunk;
    const bool closing = r1 == kChunk, open = chunk == q.last();
    const int64_t open_row = ((int64_t)b * g.s.Hkv + h) * kChunk;
    float* kt = g.c.k_tail + open_row * D;
    TIn* vt = static_cast<TIn*>(g.c.v_tail) + open_row * D;
    int64_t page = -1;
    if (closing) page = g.c.table[(int64_t)b * g.s.max_chunks + chunk];

    // Keys first and values after them, which wait as they were loaded.
    float k[R][16];
    Raw8<TIn> va[R], vb[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int r = warp * kGroup + rl + RL * j;
        if (r >= r0 && r < r1) {
            const int64_t p = (int64_t)chunk * kChunk + r, i = q.token + (p - q.pos);
            const TIn* pk = static_cast<const TIn*>(g.a.k.ptr) + i * g.a.k.token + h * g.a.k.head;
            const TIn* pv = static_cast<const TIn*>(g.a.v.ptr) + i * g.a.v.token + h * g.a.v.head;
            Raw8<TIn> ka, kb;
            ka.load(pk + un.a);
            kb.load(pk + un.b);
            va[j].load(pv + un.a);
            vb[j].load(pv + un.b);
            Angles ang;
            if (un.turned) ang.load(g.a.rope + p * g.a.rot, u, g.a.rot);
            ka.widen(k[j]);
            kb.widen(k[j] + 8);
            if (un.turned) turn<false>(k[j], ang, g.a.interleaved);
            if (open) {
                store8(kt + r * D + un.a, k[j]);
                store8(kt + r * D + un.b, k[j] + 8);
                va[j].store(vt + r * D + un.a);
                vb[j].store(vt + r * D + un.b);
            }
        } else if (closing) {
            load8(kt + r * D + un.a, k[j]);
            load8(kt + r * D + un.b, k[j] + 8);
            va[j].load_plain(vt + r * D + un.a);
            vb[j].load_plain(vt + r * D + un.b);
        }
    }
    if (!closing) return;                            // the same for the whole CTA
    page = paged::page_or_none((int32_t)page, g.s.n_pages, kSitePage);
    if (page < 0) return;

    const int64_t ph = page * g.s.Hkv + h;
    const int64_t rows = (ph * kChunk + warp * kGroup) * D;
    close_group<CACHE, D, R>(k, static_cast<uint8_t*>(g.c.k_pages) + rows, g.c.k_scale + ph * kGroupsPerChunk + warp, un,
                             rl, RL, lane);
    // Summaries: the group's mean over its 8 rows, then the chunk's over 8 groups.
    // Each term is divided (by a power of two) before it is added: a mean of
    // finite keys is finite where their sum is not.
    float mean[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float t = k[0][e] * (1.0f / kGroup);
#pragma unroll
        for (int j = 1; j < R; ++j) t = fmaf(k[j][e], 1.0f / kGroup, t);
#pragma unroll
        for (int o = U; o < 32; o <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        mean[e] = t;
    }
    if (rl == 0) {
        store8(&part[warp][un.a], mean);
        store8(&part[warp][un.b], mean + 8);
        float* dst = g.c.gsum + (ph * kGroupsPerChunk + warp) * D;
        store8(dst + un.a, mean);
        store8(dst + un.b, mean + 8);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
        va[j].widen(k[j]);
        vb[j].widen(k[j] + 8);
    }
    close_group<CACHE, D, R>(k, static_cast<uint8_t*>(g.c.v_pages) + rows, g.c.v_scale + ph * kGroupsPerChunk + warp, un,
                             rl, RL, lane);
    __syncthreads();
    for (int e = tid; e < D; e += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kGroupsPerChunk; ++w) t = fmaf(part[w][e], 1.0f / kGroupsPerChunk, t);
        g.c.csum[ph * D + e] = t;
    }
}

// q-heads of one touched chunk's new tokens: a few of them, rows side by side
// (Heads > 1), or as many as there are threads for, one each.
template <typename TIn, int D, int Heads>
__device__ __forceinline__ void rotate_queries(const Args& g, const Seq& q, int slot, int chunk)
{
    constexpr int U = D / 16, kSide = kThreads / U;
    const int u = threadIdx.x % U, side = threadIdx.x / U;
    const int h0 = Heads > 1 ? slot * Heads : slot * kSide + side;
    const Unit un = unit_of(u, g.a.rot, g.a.interleaved);
    const int r0 = chunk == q.first() ? int(q.pos % kChunk) : 0;
    const int r1 = chunk == q.last() ? int((q.pos + q.n - 1) % kChunk) + 1 : kChunk;
#pragma unroll (Heads > 1 ? 1 : 2)
    for (int r = r0 + (Heads > 1 ? side : 0); r < r1; r += Heads > 1 ? kSide : 1) {
        const int64_t p = (int64_t)chunk * kChunk + r, i = q.token + (p - q.pos);
        const TIn* src = static_cast<const TIn*>(g.a.q.ptr) + i * g.a.q.token;
        Raw8<TIn> ra[Heads], rb[Heads];
#pragma unroll
        for (int j = 0; j < Heads; ++j)
            if (h0 + j < g.s.Hq) {
                ra[j].load(src + (h0 + j) * g.a.q.head + un.a);
                rb[j].load(src + (h0 + j) * g.a.q.head + un.b);
            }
        Angles ang;
        if (un.turned) ang.load(g.a.rope + p * g.a.rot, u, g.a.rot);
        TIn* dst = static_cast<TIn*>(g.a.q_out) + i * g.s.Hq * D;
#pragma unroll
        for (int j = 0; j < Heads; ++j)
            if (h0 + j < g.s.Hq) {
                float x[16];
                ra[j].widen(x);
                rb[j].widen(x + 8);
                if (un.turned) turn<false>(x, ang, g.a.interleaved);
                store8(dst + (h0 + j) * D + un.a, x);
                store8(dst + (h0 + j) * D + un.b, x + 8);
            }
    }
}

template <typename TIn, int D, int CACHE>
__global__ void __launch_bounds__(kThreads, sizeof(TIn) * D < 512 ? 3 : 2) paged_append_kernel(const __grid_constant__ Args g)
{
    __shared__ __align__(16) float part[kGroupsPerChunk][D];
    __shared__ Seq s_q;
    __shared__ int s_b, s_chunk;
    pdl_wait();
    pdl_trigger();
    const int item = blockIdx.x / g.slots, slot = blockIdx.x % g.slots;
    Seq q{0, 0, 0};
    int b = -1, chunk = 0;
    if (!g.a.cu || g.s.B == 1) {                     // every warp for itself
        b = g.a.cu ? 0 : item;
        q = sequence(g, b);
        chunk = q.first() + (g.a.cu ? item : 0);
        if (q.n == 0 || chunk > q.last()) return;
    } else {
        if (threadIdx.x < 32) {
            b = locate(g, item, q, chunk);
            if (threadIdx.x == 0) {
                s_q = q;
                s_b = b;
                s_chunk = chunk;
            }
        }
        __syncthreads();
        q = s_q;
        b = s_b;
        chunk = s_chunk;
        if (b < 0) return;
    }
    if (slot >= g.s.Hkv) {
        if (g.few) rotate_queries<TIn, D, 1>(g, q, slot - g.s.Hkv, chunk);
        else rotate_queries<TIn, D, kQHeads<TIn>>(g, q, slot - g.s.Hkv, chunk);
        return;
    }
    // The first chunk's older rows are where the last chunk's rows will be.
    const bool both = q.pos % kChunk != 0 && q.first() != q.last();
    if (both && chunk == q.last()) return;
    if (both) {                                      // the last chunk's rows on their way to L2 meanwhile
        const int r = threadIdx.x / 4, rows = (q.pos + q.n - 1) % kChunk + 1, line = threadIdx.x % 4;
        if (r < rows && line * 128 < D * (int)sizeof(TIn)) {
            const int64_t i = (int64_t)q.token + q.n - rows + r;
            prefetch_l2(static_cast<const TIn*>(g.a.k.ptr) + i * g.a.k.token + slot * g.a.k.head + line * (128 / sizeof(TIn)));
            prefetch_l2(static_cast<const TIn*>(g.a.v.ptr) + i * g.a.v.token + slot * g.a.v.head + line * (128 / sizeof(TIn)));
        }
    }
    append_chunk<TIn, D, CACHE>(g, q, b, slot, chunk, part);
    if (both && chunk == q.first()) {
        __syncthreads();
        append_chunk<TIn, D, CACHE>(g, q, b, slot, q.last(), part);
    }
}

// pos[b] moves by the tokens that an append of the same arguments takes; last[b]
// (where wanted) is the position of the last of them, or -1.
__global__ void __launch_bounds__(kThreads) paged_advance_kernel(const __grid_constant__ Args g, int32_t* pos, int32_t* last)
{
    pdl_wait();
    pdl_trigger();
    const int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (b >= g.s.B) return;
    const Seq q = sequence(g, (int)b);
    if (q.n > 0) pos[b] = q.pos + q.n;
    if (last) last[b] = q.n > 0 ? q.pos + q.n - 1 : -1;
}

int64_t items_of(const PagedShape& s, const PagedAppend& a)
{
    // A sequence's n tokens touch at most n / 64 + 2 chunks, and at most n.
    return a.cu ? std::min<int64_t>(a.N, a.N / kChunk + 2 * (int64_t)s.B) : a.N;
}

template <typename TIn, int D, int CACHE>
cudaError_t launch(const Args& g, int64_t items, cudaStream_t st)
{
    return launch_pdl(paged_append_kernel<TIn, D, CACHE>, dim3((unsigned)(items * g.slots)), dim3(kThreads), 0, st, g);
}

template <typename TIn, int D>
cudaError_t by_cache(const Args& g, int64_t items, cudaStream_t st)
{
    return g.s.cache_dtype == HGA_INT8 ? launch<TIn, D, HGA_INT8>(g, items, st) : launch<TIn, D, HGA_E4M3>(g, items, st);
}

// Tokens are few where a sequence gets less than four on average: then a row's
// heads are side by side in a CTA, not a head's rows.
bool few_tokens(const PagedShape& s, const PagedAppend& a) { return a.N < 4 * (int64_t)s.B; }
int slots_of(const PagedShape& s, const PagedAppend& a)
{
    const int side = s.dtype == HGA_BF16 ? kQHeads<__nv_bfloat16> : kQHeads<float>;
    const int heads = few_tokens(s, a) ? kThreads / (s.d / 16) : side;
    return s.Hkv + (a.q.ptr ? (s.Hq + heads - 1) / heads : 0);
}

}  // namespace

bool paged_append_grid_fits(const PagedShape& s, const PagedAppend& a) { return items_of(s, a) <= INT32_MAX / slots_of(s, a); }

cudaError_t launch_paged_append(const PagedShape& s, const hga_paged_cache& c, const PagedAppend& a, cudaStream_t st)
{
    const Args g{s, c, a, slots_of(s, a), few_tokens(s, a)};
    const int64_t items = items_of(s, a);
    if (s.dtype == HGA_BF16)
        return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, items, st) : by_cache<__nv_bfloat16, 64>(g, items, st);
    return s.d == 128 ? by_cache<float, 128>(g, items, st) : by_cache<float, 64>(g, items, st);
}

cudaError_t launch_paged_advance(const PagedShape& s, const PagedAppend& a, int32_t* pos, int32_t* last, cudaStream_t st)
{
    const Args g{s, {}, a, 0, false};
    return launch_pdl(paged_advance_kernel, dim3((unsigned)(((int64_t)s.B + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, g,
                      pos, last);
}

HGA_CHECK_WORD_READER(check_word_paged_append)

}  // namespace hga
