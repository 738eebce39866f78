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
// memory but the chunk summary) or four q-heads of it.  The kernel is bound
// by the bytes of q, k, v and what it writes for prompts, and by a launch
// and three dependent loads for single tokens.
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
constexpr int kQHeads = 4;                          // q-heads of a CTA
constexpr int kSitePage = 411, kSiteOffsets = 412, kSiteLength = 413;

struct Args {
    PagedShape s;
    hga_paged_cache c;
    PagedAppend a;
    int slots, q_slots;                             // CTAs of an item: Hkv + q_slots
};

// The tokens that a sequence gets: n of them from `token` on, at positions
// pos .. pos + n - 1.
struct Seq {
    int64_t pos, token, n;
    __device__ __forceinline__ int64_t first() const { return pos / kChunk; }
    __device__ __forceinline__ int64_t last() const { return (pos + n - 1) / kChunk; }
    __device__ __forceinline__ int64_t chunks() const { return n > 0 ? last() - first() + 1 : 0; }
};

__device__ __forceinline__ Seq sequence(const Args& g, int b)
{
    Seq q;
    q.pos = g.a.pos[b];
    q.token = b;
    q.n = 1;
    if (g.a.cu) {
        q.token = g.a.cu[b];
        const int64_t end = g.a.cu[b + 1];
        q.n = end - q.token;
        if (q.token < 0 || q.n < 0 || end > g.a.N) {
            paged::flag(kSiteOffsets);
            q.n = 0;
        }
    }
    if (q.pos < 0) q.n = 0;                         // an empty slot of the batch
    int64_t limit = (int64_t)g.s.max_chunks * kChunk;
    if (g.a.rot > 0) limit = limit < g.a.rope_rows ? limit : g.a.rope_rows;
    if (q.n > 0 && q.pos + q.n > limit) {
        paged::flag(kSiteLength);
        q.n = limit > q.pos ? limit - q.pos : 0;
    }
    return q;
}

// Sequence and chunk of an item: the items are the touched chunks, sequence
// by sequence.  Every warp looks for itself (a prefix sum of 32 sequences at
// a time).  Returns -1 past the last item.
__device__ __forceinline__ int locate(const Args& g, int64_t item, Seq& q, int64_t& chunk)
{
    const int lane = threadIdx.x & 31;
    if (!g.a.cu) {
        q = sequence(g, (int)item);
        chunk = q.first();
        return q.n > 0 ? (int)item : -1;
    }
    for (int b0 = 0; b0 < g.s.B; b0 += 32) {
        Seq mine{0, 0, 0};
        if (b0 + lane < g.s.B) mine = sequence(g, b0 + lane);
        const int64_t count = mine.chunks();
        int64_t upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, item < upto);
        if (hit) {
            const int at = __ffs(hit) - 1;
            q.pos = __shfl_sync(0xFFFFFFFFu, mine.pos, at);
            q.token = __shfl_sync(0xFFFFFFFFu, mine.token, at);
            q.n = __shfl_sync(0xFFFFFFFFu, mine.n, at);
            chunk = q.first() + item - __shfl_sync(0xFFFFFFFFu, upto - count, at);
            return b0 + at;
        }
        item -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    return -1;
}

// Rows of the open chunk are written by this kernel too: no read-only path.
__device__ __forceinline__ void load8(const float* p, float* x)
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x)
{
    Raw8<__nv_bfloat16> r;
    r.v = *reinterpret_cast<const uint4*>(p);
    r.widen(x);
}

// 8 codes of values already scaled to the code's range.
template <int CACHE> __device__ __forceinline__ uint2 codes8(const float* y)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (CACHE == HGA_INT8) {
            const uint32_t c0 = __float2int_rn(y[4 * i]), c1 = __float2int_rn(y[4 * i + 1]),
                           c2 = __float2int_rn(y[4 * i + 2]), c3 = __float2int_rn(y[4 * i + 3]);
            w[i] = __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi =
                __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
    }
    return make_uint2(w[0], w[1]);
}

// The warp's group (R rows of 16 elements a thread): codes into the page's
// rows and the scale.
template <int CACHE, int D, int R>
__device__ __forceinline__ void close_group(const float (&x)[R][16], uint8_t* page_rows, float* scale, const Unit& un,
                                            int rl, int RL, int lane)
{
    constexpr float kLevel = CACHE == HGA_INT8 ? 127.f : 448.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[j][e]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const bool finite = top < 0x7F800000u;
    const float a = fmaxf(__uint_as_float(top), kLevel * 1.17549435e-38f);
    const float f = __fmul_rn(__frcp_rn(a), kLevel);
    if (lane == 0) *scale = finite ? __fdiv_rn(a, kLevel) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = finite ? __fmul_rn(x[j][e], f) : 0.f;
        uint8_t* row = page_rows + (rl + RL * j) * D;
        *reinterpret_cast<uint2*>(row + un.a) = codes8<CACHE>(y);
        *reinterpret_cast<uint2*>(row + un.b) = codes8<CACHE>(y + 8);
    }
}

// One kv-head of one touched chunk.
template <typename TIn, int D, int CACHE>
__device__ __forceinline__ void append_chunk(const Args& g, const Seq& q, int b, int h, int64_t chunk, float (*part)[D])
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

    float k[R][16], v[R][16];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int r = warp * kGroup + rl + RL * j;
        if (r >= r0 && r < r1) {
            const int64_t p = chunk * kChunk + r, i = q.token + (p - q.pos);
            const TIn* pk = static_cast<const TIn*>(g.a.k.ptr) + i * g.a.k.token + h * g.a.k.head;
            const TIn* pv = static_cast<const TIn*>(g.a.v.ptr) + i * g.a.v.token + h * g.a.v.head;
            Raw8<TIn> ka, kb, va, vb;
            ka.load(pk + un.a);
            kb.load(pk + un.b);
            va.load(pv + un.a);
            vb.load(pv + un.b);
            Angles ang;
            if (un.turned) ang.load(g.a.rope + p * g.a.rot, u, g.a.rot);
            ka.widen(k[j]);
            kb.widen(k[j] + 8);
            va.widen(v[j]);
            vb.widen(v[j] + 8);
            if (un.turned) turn<false>(k[j], ang, g.a.interleaved);
            if (open) {
                store8(kt + r * D + un.a, k[j]);
                store8(kt + r * D + un.b, k[j] + 8);
                store8(vt + r * D + un.a, v[j]);
                store8(vt + r * D + un.b, v[j] + 8);
            }
        } else if (closing) {
            load8(kt + r * D + un.a, k[j]);
            load8(kt + r * D + un.b, k[j] + 8);
            load8(vt + r * D + un.a, v[j]);
            load8(vt + r * D + un.b, v[j] + 8);
        }
    }
    if (!closing) return;                            // the same for the whole CTA
    page = paged::page_or_none((int32_t)page, g.s.n_pages, kSitePage);
    if (page < 0) return;

    const int64_t ph = page * g.s.Hkv + h;
    const int64_t rows = (ph * kChunk + warp * kGroup) * D;
    close_group<CACHE, D, R>(k, static_cast<uint8_t*>(g.c.k_pages) + rows, g.c.k_scale + ph * kGroupsPerChunk + warp, un,
                             rl, RL, lane);
    close_group<CACHE, D, R>(v, static_cast<uint8_t*>(g.c.v_pages) + rows, g.c.v_scale + ph * kGroupsPerChunk + warp, un,
                             rl, RL, lane);
    // Summaries: the group's sum over its 8 rows, then the chunk's over 8 groups.
    float sum[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float t = k[0][e];
#pragma unroll
        for (int j = 1; j < R; ++j) t += k[j][e];
#pragma unroll
        for (int o = U; o < 32; o <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        sum[e] = t;
    }
    if (rl == 0) {
        store8(&part[warp][un.a], sum);
        store8(&part[warp][un.b], sum + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] *= 1.0f / kGroup;
        float* dst = g.c.gsum + (ph * kGroupsPerChunk + warp) * D;
        store8(dst + un.a, sum);
        store8(dst + un.b, sum + 8);
    }
    __syncthreads();
    for (int e = tid; e < D; e += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kGroupsPerChunk; ++w) t += part[w][e];
        g.c.csum[ph * D + e] = t * (1.0f / kChunk);
    }
}

// Up to kQHeads q-heads of one touched chunk's new tokens.
template <typename TIn, int D>
__device__ __forceinline__ void rotate_queries(const Args& g, const Seq& q, int h0, int64_t chunk)
{
    constexpr int U = D / 16;
    const int u = threadIdx.x % U;
    const Unit un = unit_of(u, g.a.rot, g.a.interleaved);
    const int r0 = chunk == q.first() ? int(q.pos % kChunk) : 0;
    const int r1 = chunk == q.last() ? int((q.pos + q.n - 1) % kChunk) + 1 : kChunk;
    for (int r = r0 + threadIdx.x / U; r < r1; r += kThreads / U) {
        const int64_t p = chunk * kChunk + r, i = q.token + (p - q.pos);
        const TIn* src = static_cast<const TIn*>(g.a.q.ptr) + i * g.a.q.token;
        Raw8<TIn> ra[kQHeads], rb[kQHeads];
#pragma unroll
        for (int j = 0; j < kQHeads; ++j)
            if (h0 + j < g.s.Hq) {
                ra[j].load(src + (h0 + j) * g.a.q.head + un.a);
                rb[j].load(src + (h0 + j) * g.a.q.head + un.b);
            }
        Angles ang;
        if (un.turned) ang.load(g.a.rope + p * g.a.rot, u, g.a.rot);
        TIn* dst = static_cast<TIn*>(g.a.q_out) + i * g.s.Hq * D;
#pragma unroll
        for (int j = 0; j < kQHeads; ++j)
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
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ Args g)
{
    __shared__ __align__(16) float part[kGroupsPerChunk][D];
    pdl_wait();
    pdl_trigger();
    const int64_t item = blockIdx.x / g.slots;
    const int slot = blockIdx.x % g.slots;
    Seq q;
    int64_t chunk;
    const int b = locate(g, item, q, chunk);
    if (b < 0) return;
    if (slot >= g.s.Hkv) {
        rotate_queries<TIn, D>(g, q, (slot - g.s.Hkv) * kQHeads, chunk);
        return;
    }
    // The first chunk's older rows are where the last chunk's rows will be.
    const bool both = q.pos % kChunk != 0 && q.first() != q.last();
    if (both && chunk == q.last()) return;
    append_chunk<TIn, D, CACHE>(g, q, b, slot, chunk, part);
    if (both && chunk == q.first()) {
        __syncthreads();
        append_chunk<TIn, D, CACHE>(g, q, b, slot, q.last(), part);
    }
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

int q_slots_of(const PagedShape& s, const PagedAppend& a) { return a.q.ptr ? (s.Hq + kQHeads - 1) / kQHeads : 0; }

}  // namespace

bool paged_append_grid_fits(const PagedShape& s, const PagedAppend& a)
{
    return items_of(s, a) <= INT32_MAX / (s.Hkv + q_slots_of(s, a));
}

cudaError_t launch_paged_append(const PagedShape& s, const hga_paged_cache& c, const PagedAppend& a, cudaStream_t st)
{
    const Args g{s, c, a, s.Hkv + q_slots_of(s, a), q_slots_of(s, a)};
    const int64_t items = items_of(s, a);
    if (s.dtype == HGA_BF16)
        return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, items, st) : by_cache<__nv_bfloat16, 64>(g, items, st);
    return s.d == 128 ? by_cache<float, 128>(g, items, st) : by_cache<float, 64>(g, items, st);
}

HGA_CHECK_WORD_READER(check_word_paged_append)

}  // namespace hga
