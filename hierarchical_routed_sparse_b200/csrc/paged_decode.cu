// paged_decode.cu -- one query per sequence over the paged 8-bit cache: routed
// (or dense) attention.
//
// The sequence's query stands at position p = pos[b] (its key and value are
// in the open rows already).  With u = the sum of the kv-head's q-heads'
// queries, chunk c < p / 64 scores u . csum[c]; the k_c highest are kept, then
// the k_g highest of their groups by u . gsum.  Scores are formed in float64:
// products of float32 values are exact there and a sum of 128 of them keeps
// 2^-46, so which of two near candidates is kept is what the definition says
// and not what an order of summation makes of it.  Every q-head attends the
// kept groups' dequantised rows and the open rows 0 .. p % 64:
//     O = softmax(scale q K^T) V,  lse = log sum exp (scale q K^T).
//
// One CTA takes one (batch, kv-head).  Warps take keys in turn, each with a
// running maximum and sum for each head; the warps' results meet in shared
// memory.
#include <cuda_fp8.h>

#include "paged.cuh"

namespace hga {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxG = 8;
constexpr int kSitePage = 421, kSiteLength = 422;

struct Args {
    PagedShape s;
    hga_paged_cache c;
    const int32_t* pos;
    const void* q;
    float* O;
    float* lse;
    int32_t* cidx;
    int32_t* gidx;
};

// float64 scores of the chunks and of the group candidates (as ordered
// integers), the candidates' ids and the kept rows.
struct Layout {
    size_t keys, ids, crow, grow, total;
};
__host__ __device__ inline Layout layout(const PagedShape& s)
{
    Layout L;
    const size_t cand = (size_t)s.wc * kGroupsPerChunk;
    L.keys = 0;
    L.ids = L.keys + 8 * (cand > (size_t)s.max_chunks ? cand : (size_t)s.max_chunks);
    L.crow = L.ids + 4 * cand;
    L.grow = L.crow + 4 * (size_t)s.wc;
    L.total = (L.grow + 4 * (size_t)s.wg + 15) & ~size_t(15);
    return L;
}

// A float64 as an integer of the same order; NaN above everything.
__device__ __forceinline__ unsigned long long ordered(double x)
{
    if (x != x) return ~0ull;
    const unsigned long long u = __double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double warp_sum_f64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Of the n keys, those that fewer than k beat (equal keys: the lower index
// wins) in ascending order into row, -1 up to width; id(i) names candidate i.
template <typename Id>
__device__ __forceinline__ void select(const unsigned long long* keys, int n, int k, int32_t* row, int width, Id id,
                                       int* count)
{
    __shared__ int s_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int s_warp[kWarps];
    if (tid == 0) s_base = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        bool keep = false;
        if (i < n) {
            int beat = 0;
            if (k < n) {
                const unsigned long long mine = keys[i];
                for (int j = 0; j < n; ++j) beat += keys[j] > mine || (keys[j] == mine && j < i);
            }
            keep = beat < k;
        }
        const unsigned m = __ballot_sync(0xFFFFFFFFu, keep);
        if (lane == 0) s_warp[warp] = __popc(m);
        __syncthreads();
        int at = s_base;
        for (int w = 0; w < warp; ++w) at += s_warp[w];
        if (keep) row[at + __popc(m & ((1u << lane) - 1u))] = id(i);
        __syncthreads();
        if (tid == 0)
            for (int w = 0; w < kWarps; ++w) s_base += s_warp[w];
        __syncthreads();
    }
    const int got = s_base;
    for (int i = got + tid; i < width; i += kThreads) row[i] = -1;
    if (tid == 0) *count = got;
    __syncthreads();
}

template <int CACHE> __device__ __forceinline__ float value_of(uint8_t code)
{
    if constexpr (CACHE == HGA_INT8) return (float)(int8_t)code;
    __nv_fp8_e4m3 x;
    x.__x = code;
    return float(x);
}

template <typename TIn> __device__ __forceinline__ float to_f32(TIn x) { return (float)x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename TIn, int D, int CACHE>
__global__ void __launch_bounds__(kThreads) paged_decode_kernel(const __grid_constant__ Args g)
{
    constexpr int P = D / 32;
    extern __shared__ __align__(16) uint8_t sm[];
    const Layout L = layout(g.s);
    auto* keys = reinterpret_cast<unsigned long long*>(sm + L.keys);
    auto* ids = reinterpret_cast<int32_t*>(sm + L.ids);
    auto* crow = reinterpret_cast<int32_t*>(sm + L.crow);
    auto* grow = reinterpret_cast<int32_t*>(sm + L.grow);
    __shared__ double us[D];
    __shared__ float pm[kWarps][kMaxG], pl[kWarps][kMaxG], po[kWarps][D];
    __shared__ int s_nc, s_ng;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / g.s.Hkv, h = blockIdx.x % g.s.Hkv;
    const int G = g.s.G;
    int64_t p = g.pos[b];
    if (p >= (int64_t)g.s.max_chunks * kChunk) {
        paged::flag(kSiteLength);
        p = -1;
    }
    const int c0 = p < 0 ? 0 : int(p / kChunk);
    const int rows = p < 0 ? 0 : int(p % kChunk) + 1;
    const int32_t* table = g.c.table + (int64_t)b * g.s.max_chunks;
    const TIn* q = static_cast<const TIn*>(g.q) + ((int64_t)b * g.s.Hq + h * G) * D;

    const bool dense = !g.gidx;                       // HGA_ALL without index rows
    if (!dense) {
        for (int e = tid; e < D; e += kThreads) {
            double a = 0.0;
            for (int i = 0; i < G; ++i) a += (double)to_f32<TIn>(q[i * D + e]);
            us[e] = a;
        }
        __syncthreads();
        auto score = [&](const float* row) {
            double a = 0.0;
#pragma unroll
            for (int e = 0; e < P; ++e) a += us[lane * P + e] * (double)row[lane * P + e];
            return warp_sum_f64(a);
        };
        const int kc = g.s.k_c > 0 ? g.s.k_c : c0;
        if (kc < c0)
            for (int c = warp; c < c0; c += kWarps) {
                const int64_t page = paged::page_or_none(table[c], g.s.n_pages, kSitePage);
                const double a = page < 0 ? -INFINITY : score(g.c.csum + (page * g.s.Hkv + h) * D);
                if (lane == 0) keys[c] = ordered(a);
            }
        __syncthreads();
        select(keys, c0, kc, crow, g.s.wc, [](int i) { return i; }, &s_nc);
        const int n = s_nc * kGroupsPerChunk;
        const int kg = g.s.k_g > 0 ? g.s.k_g : n;
        for (int i = tid; i < n; i += kThreads) ids[i] = crow[i / kGroupsPerChunk] * kGroupsPerChunk + i % kGroupsPerChunk;
        __syncthreads();
        if (kg < n)
            for (int i = warp; i < n; i += kWarps) {
                const int64_t page = paged::page_or_none(table[ids[i] / kGroupsPerChunk], g.s.n_pages, kSitePage);
                const double a = page < 0 ? -INFINITY
                                          : score(g.c.gsum + ((page * g.s.Hkv + h) * kGroupsPerChunk +
                                                              ids[i] % kGroupsPerChunk) * D);
                if (lane == 0) keys[i] = ordered(a);
            }
        __syncthreads();
        select(keys, n, kg, grow, g.s.wg, [&](int i) { return ids[i]; }, &s_ng);
        for (int i = tid; i < g.s.wc; i += kThreads) g.cidx[(int64_t)blockIdx.x * g.s.wc + i] = crow[i];
        for (int i = tid; i < g.s.wg; i += kThreads) g.gidx[(int64_t)blockIdx.x * g.s.wg + i] = grow[i];
    }
    const int ng = dense ? c0 * kGroupsPerChunk : s_ng;

    // Keys in units of a group: the open rows first, then the kept groups.
    float qv[kMaxG][P], acc[kMaxG][P], m[kMaxG], l[kMaxG];
#pragma unroll
    for (int i = 0; i < kMaxG; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            qv[i][e] = i < G ? to_f32<TIn>(q[i * D + lane * P + e]) * g.s.scale : 0.f;
            acc[i][e] = 0.f;
        }
    }
    auto attend = [&](const float* k, const float* v) {
#pragma unroll
        for (int i = 0; i < kMaxG; ++i) {
            if (i >= G) break;
            float a = 0.f;
#pragma unroll
            for (int e = 0; e < P; ++e) a = fmaf(qv[i][e], k[e], a);
            a = warp_sum(a);
            const float mn = fmaxf(m[i], a);
            const float f = expf(m[i] - mn), w = expf(a - mn);
            m[i] = mn;
            l[i] = l[i] * f + w;
#pragma unroll
            for (int e = 0; e < P; ++e) acc[i][e] = fmaf(acc[i][e], f, w * v[e]);
        }
    };
    const int64_t open_row = ((int64_t)b * g.s.Hkv + h) * kChunk;
    for (int r = warp; r < rows; r += kWarps) {
        float k[P], v[P];
        const float* kr = g.c.k_tail + (open_row + r) * D + lane * P;
        const TIn* vr = static_cast<const TIn*>(g.c.v_tail) + (open_row + r) * D + lane * P;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            k[e] = kr[e];
            v[e] = to_f32<TIn>(vr[e]);
        }
        attend(k, v);
    }
    for (int i = warp; i < ng; i += kWarps) {
        const int grp = dense ? i : grow[i];
        const int64_t page = paged::page_or_none(table[grp / kGroupsPerChunk], g.s.n_pages, kSitePage);
        if (page < 0) continue;
        const int64_t at = (page * g.s.Hkv + h) * kGroupsPerChunk + grp % kGroupsPerChunk;
        const float ks = g.c.k_scale[at], vs = g.c.v_scale[at];
        const uint8_t* kr = static_cast<const uint8_t*>(g.c.k_pages) + at * kGroup * D + lane * P;
        const uint8_t* vr = static_cast<const uint8_t*>(g.c.v_pages) + at * kGroup * D + lane * P;
        for (int r = 0; r < kGroup; ++r) {
            float k[P], v[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                k[e] = value_of<CACHE>(kr[r * D + e]) * ks;
                v[e] = value_of<CACHE>(vr[r * D + e]) * vs;
            }
            attend(k, v);
        }
    }
#pragma unroll
    for (int i = 0; i < kMaxG; ++i) {
        if (i >= G) break;
        if (lane == 0) {
            pm[warp][i] = m[i];
            pl[warp][i] = l[i];
        }
#pragma unroll
        for (int e = 0; e < P; ++e) po[warp][lane * P + e] = acc[i][e];
        __syncthreads();
        float M = -INFINITY, l_all = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, pm[w][i]);
        float f[kWarps];
        for (int w = 0; w < kWarps; ++w) {
            f[w] = pm[w][i] == -INFINITY ? 0.f : expf(pm[w][i] - M);
            l_all = fmaf(pl[w][i], f[w], l_all);
        }
        const int64_t row = (int64_t)b * g.s.Hq + h * G + i;
        for (int e = tid; e < D; e += kThreads) {
            float o = 0.f;
            for (int w = 0; w < kWarps; ++w) o = fmaf(po[w][e], f[w], o);
            g.O[row * D + e] = rows > 0 ? o / l_all : 0.f;
        }
        if (tid == 0) g.lse[row] = rows > 0 ? M + logf(l_all) : -INFINITY;
        __syncthreads();
    }
}

template <typename TIn, int D, int CACHE>
cudaError_t launch(const Args& g, cudaStream_t st)
{
    const size_t smem = g.gidx ? layout(g.s).total : 16;     // dense: no routing state
    auto k = paged_decode_kernel<TIn, D, CACHE>;
    if (cudaError_t e = allow_smem(k, (int)smem)) return e;
    return launch_pdl(k, dim3((unsigned)(g.s.B * g.s.Hkv)), dim3(kThreads), smem, st, g);
}

template <typename TIn, int D>
cudaError_t by_cache(const Args& g, cudaStream_t st)
{
    return g.s.cache_dtype == HGA_INT8 ? launch<TIn, D, HGA_INT8>(g, st) : launch<TIn, D, HGA_E4M3>(g, st);
}

}  // namespace

size_t paged_decode_smem(const PagedShape& s) { return layout(s).total + 8 * 1024; }
size_t paged_workspace(const PagedShape&) { return 0; }

cudaError_t launch_paged_decode(const PagedShape& s, const hga_paged_cache& c, const int32_t* pos, const void* q,
                                float* O, float* lse, int32_t* cidx, int32_t* gidx, void*, cudaStream_t st)
{
    const Args g{s, c, pos, q, O, lse, cidx, gidx};
    if (s.dtype == HGA_BF16) return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, st) : by_cache<__nv_bfloat16, 64>(g, st);
    return s.d == 128 ? by_cache<float, 128>(g, st) : by_cache<float, 64>(g, st);
}

HGA_CHECK_WORD_READER(check_word_paged_decode)

}  // namespace hga
