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
// kept groups' held values and the open rows 0 .. p % 64:
//     O = softmax(scale q K^T) V,  lse = log sum exp (scale q K^T).
//
// A cluster of S CTAs (4 warps each) takes one (batch, kv-head).
//   * Scoring: CTA r scores the r-th part of the candidates and writes their
//     keys into every peer's shared memory; each CTA then makes the same
//     selection (paged_select.cuh).
//   * Attention: a warp takes tiles of two groups (16 keys), tile i going to
//     warp i mod 4 S of the cluster.  Codes go from global memory to the
//     registers of mma.sync fragments without passing shared memory
//     (paged_attend.cuh), the next tile's loads issued before the current
//     tile's products.
//   * Merge: every warp has a running reference, sum and unnormalised output
//     for each head; the CTA's four meet in shared memory, and each CTA
//     combines a 1/S part of the outputs of all S (distributed shared memory).
#include "paged.cuh"
#include "paged_attend.cuh"
#include "paged_select.cuh"
#include "sm100.cuh"

namespace hga {
namespace {

using namespace paged;
using sm100::cluster_rank;
using sm100::peer_addr;
using sm100::smem_u32;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxS = 16;                            // CTAs per (batch, kv-head)
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
    int S;
};

// Dynamic shared memory.  Routing: keys of the chunks, then of the group
// candidates; the kept chunks and their pages, the kept groups and theirs.
// The warps' outputs take the routing keys' place when these are done with;
// what peers write (inbox) has a place of its own.
struct Layout {
    size_t ckeys, gkeys, crow, cpage, grow, gpage, scratch, merge, inbox, total;
};
__host__ __device__ inline size_t up16(size_t x) { return (x + 15) & ~size_t(15); }
__host__ __device__ inline Layout layout(const PagedShape& s, bool dense, int S)
{
    Layout L;
    const size_t nc = dense ? 0 : (size_t)s.max_chunks, wc = dense ? 0 : (size_t)s.wc, wg = dense ? 0 : (size_t)s.wg;
    L.ckeys = 0;
    L.gkeys = up16(L.ckeys + 8 * nc);
    L.scratch = up16(L.gkeys + 8 * 8 * wc);
    L.merge = 0;
    const size_t keys_end = L.scratch + (dense ? 0 : sizeof(SelectScratch<kWarps>));
    const size_t merge_end = 4 * (size_t)kWarps * s.G * (s.d + 2);
    L.crow = up16(keys_end > merge_end ? keys_end : merge_end);
    L.cpage = L.crow + 4 * wc;
    L.grow = L.cpage + 4 * wc;
    L.gpage = L.grow + 4 * wg;
    L.inbox = up16(L.gpage + 4 * wg);
    // From each peer: 1/S of its G x d outputs, its G references and sums.
    L.total = up16(L.inbox + 4 * ((size_t)s.G * s.d + 2 * (size_t)s.G * S));
    return L;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename TIn> __device__ __forceinline__ float widen(TIn x);
template <> __device__ __forceinline__ float widen<float>(float x) { return x; }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Scores of candidates [c0, c1) as ordered keys: eight lanes take a
// candidate (four 16-byte pieces of its row each at d = 128), a warp eight
// candidates at a time.  row(c) is null for one that cannot be read.
template <int D, typename Row>
__device__ __forceinline__ void score(const double* us, int c0, int c1, Row row, unsigned long long* keys, int warp,
                                      int lane)
{
    constexpr int J = D / 32;
    const int sub = lane & 7, slot = lane >> 3;
    double u[4 * J];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[4 * j + e] = us[4 * (sub + 8 * j) + e];
    for (int base = c0 + 8 * warp; base < c1; base += 8 * kWarps) {
        float4 x[2][J];
        bool have[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = base + 4 * i + slot;
            const float* r = c < c1 ? row(c) : nullptr;
            have[i] = r != nullptr;
#pragma unroll
            for (int j = 0; j < J; ++j)
                x[i][j] = have[i] ? __ldg(reinterpret_cast<const float4*>(r) + sub + 8 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            double a = 0.0, b = 0.0;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                a = fma(u[4 * j], (double)x[i][j].x, a);
                b = fma(u[4 * j + 1], (double)x[i][j].y, b);
                a = fma(u[4 * j + 2], (double)x[i][j].z, a);
                b = fma(u[4 * j + 3], (double)x[i][j].w, b);
            }
            a += b;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            const int c = base + 4 * i + slot;
            if (sub == 0 && c < c1) keys[c] = ordered(have[i] ? a : -INFINITY);
        }
    }
}

// keys[c0, c1) of this CTA into the same slots of its peers.
__device__ __forceinline__ void push(unsigned long long* keys, int c0, int c1, int S, int rank, int tid)
{
    const int n = c1 - c0;
    for (int i = tid; i < n * S; i += kThreads) {
        const int p = i / n, c = c0 + i % n;
        if (p != rank) sm100::st_cluster_u64(peer_addr(smem_u32(keys + c), p), keys[c]);
    }
}

template <typename TIn, int D, int CACHE>
__global__ void __launch_bounds__(kThreads, 3) paged_decode_kernel(const __grid_constant__ Args g)
{
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ double us[D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = g.S, rank = S > 1 ? (int)cluster_rank() : 0;
    const int64_t bh = blockIdx.x / S;
    const int b = int(bh / g.s.Hkv), h = int(bh % g.s.Hkv), G = g.s.G;
    const bool dense = !g.gidx;                      // HGA_ALL without index rows
    const Layout L = layout(g.s, dense, S);
    if (S > 1) cluster_arrive();                     // waited for before the first write to a peer
    pdl_wait();
    pdl_trigger();

    int64_t p = g.pos[b];
    if (p >= (int64_t)g.s.max_chunks * kChunk) {
        flag(kSiteLength);
        p = -1;
    }
    const int64_t head0 = (int64_t)b * g.s.Hq + h * G;   // first of the kv-head's q-heads
    if (p < 0) {                                     // an empty sequence: all CTAs of the cluster alike
        if (rank == 0) {
            for (int i = tid; i < G * D; i += kThreads) g.O[head0 * D + i] = 0.f;
            for (int i = tid; i < G; i += kThreads) g.lse[head0 + i] = -INFINITY;
            if (!dense) {
                for (int i = tid; i < g.s.wc; i += kThreads) g.cidx[bh * g.s.wc + i] = -1;
                for (int i = tid; i < g.s.wg; i += kThreads) g.gidx[bh * g.s.wg + i] = -1;
            }
        }
        if (S > 1) cluster_wait();
        return;
    }
    const int c0 = int(p / kChunk), rows = int(p % kChunk) + 1;
    const int32_t* table = g.c.table + (int64_t)b * g.s.max_chunks;
    const TIn* q = static_cast<const TIn*>(g.q) + head0 * D;
    auto page_of = [&](int c) { return (int32_t)page_or_none(__ldg(table + c), g.s.n_pages, kSitePage); };

    int ng = 0;
    int32_t* gpage = reinterpret_cast<int32_t*>(sm + L.gpage);
    int32_t* grow = reinterpret_cast<int32_t*>(sm + L.grow);
    if (!dense) {
        auto* ckeys = reinterpret_cast<unsigned long long*>(sm + L.ckeys);
        auto* gkeys = reinterpret_cast<unsigned long long*>(sm + L.gkeys);
        auto* scratch = reinterpret_cast<SelectScratch<kWarps>*>(sm + L.scratch);
        int32_t* crow = reinterpret_cast<int32_t*>(sm + L.crow);
        int32_t* cpage = reinterpret_cast<int32_t*>(sm + L.cpage);
        for (int e = tid; e < D; e += kThreads) {
            double a = 0.0;
            for (int i = 0; i < G; ++i) a += (double)widen<TIn>(q[i * D + e]);
            us[e] = a;
        }
        __syncthreads();
        const int kc = g.s.k_c > 0 ? min(g.s.k_c, c0) : c0;
        if (kc < c0) {
            const int b0 = int((int64_t)rank * c0 / S), b1 = int((int64_t)(rank + 1) * c0 / S);
            score<D>(us, b0, b1, [&](int c) -> const float* {
                const int32_t page = page_of(c);
                return page < 0 ? nullptr : g.c.csum + ((int64_t)page * g.s.Hkv + h) * D;
            }, ckeys, warp, lane);
            __syncthreads();
            if (S > 1) {
                cluster_wait();
                push(ckeys, b0, b1, S, rank, tid);
                cluster_arrive();
                cluster_wait();
                cluster_arrive();                    // for the groups' push
            }
        }
        select<kWarps>(ckeys, c0, kc, scratch, tid, [&](int i, int at) {
            crow[at] = i;
            cpage[at] = page_of(i);
        });
        __syncthreads();
        const int n = kc * kGroupsPerChunk;
        const int kg = g.s.k_g > 0 ? min(g.s.k_g, n) : n;
        if (kg < n) {
            const int b0 = int((int64_t)rank * n / S), b1 = int((int64_t)(rank + 1) * n / S);
            score<D>(us, b0, b1, [&](int i) -> const float* {
                const int32_t page = cpage[i / kGroupsPerChunk];
                return page < 0 ? nullptr
                                : g.c.gsum + (((int64_t)page * g.s.Hkv + h) * kGroupsPerChunk + i % kGroupsPerChunk) * D;
            }, gkeys, warp, lane);
            __syncthreads();
            if (S > 1) {
                cluster_wait();
                push(gkeys, b0, b1, S, rank, tid);
                cluster_arrive();
                cluster_wait();
                cluster_arrive();                    // for the merge
            }
        }
        select<kWarps>(gkeys, n, kg, scratch, tid, [&](int i, int at) {
            grow[at] = crow[i / kGroupsPerChunk] * kGroupsPerChunk + i % kGroupsPerChunk;
            gpage[at] = cpage[i / kGroupsPerChunk];
        });
        __syncthreads();
        ng = kg;
        if (rank == 0) {
            for (int i = tid; i < g.s.wc; i += kThreads) g.cidx[bh * g.s.wc + i] = i < kc ? crow[i] : -1;
            for (int i = tid; i < g.s.wg; i += kThreads) g.gidx[bh * g.s.wg + i] = i < ng ? grow[i] : -1;
        }
    }

    // Attention.
    const int wid = rank * kWarps + warp, n_workers = S * kWarps;
    Running<D> run;
    run.init();
    {
        const int tiles = (rows + 15) / 16;
        const int64_t row0 = (bh * kChunk) * D;
        for (int i = n_workers - 1 - wid; i < tiles; i += n_workers)
            attend_open<TIn, D>(run, q, G, g.c.k_tail + row0, static_cast<const TIn*>(g.c.v_tail) + row0, 16 * i, rows,
                                g.s.scale * kLog2e, lane);
    }
    {
        const Query<TIn, D> qf(q, G, g.s.scale * kLog2e, lane);
        const uint8_t* kp = static_cast<const uint8_t*>(g.c.k_pages);
        const uint8_t* vp = static_cast<const uint8_t*>(g.c.v_pages);
        // Group number (page, kv-head, group) of a tile's two groups, -1: none.
        auto groups = [&](int i, int64_t& a, int64_t& z) {
            if (dense) {
                const int32_t page = page_of(i / 4);
                a = page < 0 ? -1 : ((int64_t)page * g.s.Hkv + h) * kGroupsPerChunk + 2 * (i % 4);
                z = page < 0 ? -1 : a + 1;
            } else {
                const int32_t pa = gpage[2 * i], pz = 2 * i + 1 < ng ? gpage[2 * i + 1] : -1;
                a = pa < 0 ? -1 : ((int64_t)pa * g.s.Hkv + h) * kGroupsPerChunk + grow[2 * i] % kGroupsPerChunk;
                z = pz < 0 ? -1 : ((int64_t)pz * g.s.Hkv + h) * kGroupsPerChunk + grow[2 * i + 1] % kGroupsPerChunk;
            }
        };
        const int n_tiles = dense ? 4 * c0 : (ng + 1) / 2;
        HeldTile<D> t[2];
        int64_t a, z;
        int i = wid;
        if (i < n_tiles) {
            groups(i, a, z);
            t[0].load(kp, vp, g.c.k_scale, g.c.v_scale, a, z, lane);
        }
        while (i < n_tiles) {
            const int i1 = i + n_workers, i2 = i1 + n_workers;
            if (i1 < n_tiles) {
                groups(i1, a, z);
                t[1].load(kp, vp, g.c.k_scale, g.c.v_scale, a, z, lane);
            }
            attend_held<TIn, D, CACHE>(run, qf, t[0], lane);
            if (i1 >= n_tiles) break;
            if (i2 < n_tiles) {
                groups(i2, a, z);
                t[0].load(kp, vp, g.c.k_scale, g.c.v_scale, a, z, lane);
            }
            attend_held<TIn, D, CACHE>(run, qf, t[1], lane);
            i = i2;
        }
    }

    // Merge: the CTA's warps, then the cluster's CTAs.
    __syncthreads();                                 // the routing keys are done with
    float* om = reinterpret_cast<float*>(sm + L.merge);          // [kWarps][G][D]
    float* rm = om + kWarps * G * D;                             // [kWarps][G] references
    float* lm = rm + kWarps * G;                                 // [kWarps][G] sums
    run.store(om + warp * G * D, rm + warp * G, lm + warp * G, G, lane);
    __syncthreads();
    const int part = G * D / S;                      // outputs a CTA combines
    float* inbox = reinterpret_cast<float*>(sm + L.inbox);       // [S][part], then [S][G] references, [S][G] sums
    float* ibr = inbox + G * D;
    float* ibl = ibr + S * G;
    if (S > 1) {
        // (A cluster that did not exchange keys still waits for its first arrive.)
        cluster_wait();
    }
    for (int i = tid; i < G * D; i += kThreads) {
        const int hd = i / D;
        float M = rm[hd];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, rm[w * G + hd]);
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o = fmaf(om[w * G * D + i], exp2f(rm[w * G + hd] - M), o);
        if (S > 1)
            sm100::st_cluster_f32(peer_addr(smem_u32(inbox + rank * part + i % part), i / part), o);
        else
            inbox[i] = o;
    }
    for (int i = tid; i < G * S; i += kThreads) {
        const int hd = i % G, to = i / G;
        float M = rm[hd], l = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, rm[w * G + hd]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l = fmaf(lm[w * G + hd], exp2f(rm[w * G + hd] - M), l);
        if (S > 1) {
            sm100::st_cluster_f32(peer_addr(smem_u32(ibr + rank * G + hd), to), M);
            sm100::st_cluster_f32(peer_addr(smem_u32(ibl + rank * G + hd), to), l);
        } else {
            ibr[hd] = M;
            ibl[hd] = l;
        }
    }
    if (S > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int i = tid; i < part; i += kThreads) {
        const int e = rank * part + i, hd = e / D;
        float M = ibr[hd];
        for (int c = 1; c < S; ++c) M = fmaxf(M, ibr[c * G + hd]);
        float o = 0.f, l = 0.f;
        for (int c = 0; c < S; ++c) {
            const float f = exp2f(ibr[c * G + hd] - M);
            o = fmaf(inbox[c * part + i], f, o);
            l = fmaf(ibl[c * G + hd], f, l);
        }
        g.O[head0 * D + e] = o / l;
        if (e % D == 0) g.lse[head0 + hd] = (M + log2f(l)) * kLn2;
    }
}

template <typename TIn, int D, int CACHE>
cudaError_t launch(const Args& g, cudaStream_t st)
{
    const size_t smem = layout(g.s, !g.gidx, g.S).total;
    auto k = paged_decode_kernel<TIn, D, CACHE>;
    if (cudaError_t e = allow_smem(k, (int)smem)) return e;
    if (g.S > 8)
        if (cudaError_t e = allow_large_clusters(reinterpret_cast<const void*>(k))) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.s.B * g.s.Hkv * g.S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = g.S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g.S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, g);
}

template <typename TIn, int D>
cudaError_t by_cache(const Args& g, cudaStream_t st)
{
    return g.s.cache_dtype == HGA_INT8 ? launch<TIn, D, HGA_INT8>(g, st) : launch<TIn, D, HGA_E4M3>(g, st);
}

// CTAs per (batch, kv-head): a power of two, as many as keep the grid within
// what the GPU holds at once, and no more than there are chunks to share.
int split(const PagedShape& s, bool dense)
{
    const int most = layout(s, dense, kMaxS).total <= 64 * 1024 ? kMaxS : 8;   // 16 CTAs must fit one GPC's SMs
    const int64_t units = (int64_t)s.B * s.Hkv, room = (dense ? 8 : 4) * (int64_t)sm_count();
    int S = 1;
    while (S < most && units * S * 2 <= room && S * 4 <= s.max_chunks) S *= 2;
    return S;
}

}  // namespace

size_t paged_decode_smem(const PagedShape& s) { return layout(s, false, kMaxS).total + 2048; }

cudaError_t launch_paged_decode(const PagedShape& s, const hga_paged_cache& c, const int32_t* pos, const void* q,
                                float* O, float* lse, int32_t* cidx, int32_t* gidx, cudaStream_t st)
{
    const Args g{s, c, pos, q, O, lse, cidx, gidx, split(s, !gidx)};
    if (s.dtype == HGA_BF16) return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, st) : by_cache<__nv_bfloat16, 64>(g, st);
    return s.d == 128 ? by_cache<float, 128>(g, st) : by_cache<float, 64>(g, st);
}

HGA_CHECK_WORD_READER(check_word_paged_decode)

}  // namespace hga
