// paged_decode.cu -- one query per sequence over the paged 8-bit cache: routed
// attention.
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
// A cluster of S CTAs (of 4 warps, or 6 when S > 1) takes one (batch, kv-head).
//   * Scoring: CTA r scores the r-th part of the candidates and writes their
//     keys into every peer's shared memory; each CTA then makes the same
//     selection (paged_select.cuh).
//   * Attention: a warp takes tiles of four groups (32 keys), tile i going to
//     warp i modulo the cluster's warps, through its own ring of asynchronous
//     copies into mma.sync fragments (paged_attend.cuh).
//   * Merge: every warp has a running reference, sum and unnormalised output
//     for each head; a CTA's meet in shared memory, and each CTA
//     combines d / S elements of every head's output (distributed shared
//     memory).
//
// A step is a chain of about ten dependent steps (position, scores, exchange,
// selection, group scores, exchange, selection, tiles, merge, exchange) of
// 0.5 - 2 us each, which bounds it: 13.7 us for one sequence at 16K context
// (8 kv-heads, d 128, k_c 8, k_g 32; 2.3 MB), 41 us for 64 (103 MB, 2.5 TB/s:
// at four CTAs an SM the chains wait for memory half of their time).
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

constexpr int kMaxS = 8;                             // CTAs per (batch, kv-head); warps of one are at most as many
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

// Dynamic shared memory.  The routing's keys (and the open rows' parked
// outputs), the warps' rings and the warps' outputs follow one another in the
// same place; the page table's first
// kTable entries, the kept chunks and groups with their pages, and what peers
// write (inbox) have places of their own.
constexpr int kTable = 2048;
struct Layout {
    size_t ckeys, gkeys, scratch, parked, rings, merge, table, crow, cpage, grow, gpage, inbox, total;
};
__host__ __device__ inline size_t up16(size_t x) { return (x + 15) & ~size_t(15); }
__host__ __device__ inline size_t larger(size_t a, size_t b) { return a > b ? a : b; }
template <int D, int kWarps> __host__ __device__ inline Layout layout(const PagedShape& s, int S)
{
    Layout L;
    const size_t nc = s.max_chunks, wc = s.wc, wg = s.wg;
    L.ckeys = L.rings = L.merge = 0;
    L.gkeys = up16(L.ckeys + 8 * nc);
    L.scratch = up16(L.gkeys + 8 * 8 * wc);
    L.parked = up16(L.scratch + sizeof(SelectScratch<kWarps>));
    const size_t keys = L.parked + 4 * Running<D>::kParked * (kWarps - 1);
    const size_t rings = sizeof(Half<D>) * kHalves * kWarps, merge = 4 * (size_t)kWarps * s.G * (D + 3);
    L.table = up16(larger(keys, larger(rings, merge)));
    L.crow = L.table + 4 * (nc < kTable ? nc : kTable);
    L.cpage = L.crow + 4 * wc;
    L.grow = L.cpage + 4 * wc;
    L.gpage = L.grow + 4 * wg;
    L.inbox = up16(L.gpage + 4 * wg);
    // From each peer: d / S elements of its outputs, its G references and sums
    // (and a factor for each of them).
    L.total = up16(L.inbox + (S > 1 ? 4 * ((size_t)s.G * D + 3 * (size_t)s.G * S) : 0));
    return L;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename TIn> __device__ __forceinline__ float widen(TIn x);
template <> __device__ __forceinline__ float widen<float>(float x) { return x; }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Scores of candidates [c0, c1) as ordered keys: eight lanes take a
// candidate (four 16-byte pieces of its row each at d = 128), a warp eight
// candidates at a time, the next eight's loads issued before they are used.
// row(c) is null for one that cannot be read.
template <int D> struct Candidates {
    static constexpr int J = D / 32, kEach = 2, kStep = 4 * kEach;
    float4 x[kEach][J];
    bool have[kEach];
    template <typename Row> __device__ __forceinline__ void load(int base, int c1, Row row, int lane)
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int c = base + 4 * i + (lane >> 3);
            const float* r = c < c1 ? row(c) : nullptr;
            have[i] = r != nullptr;
#pragma unroll
            for (int j = 0; j < J; ++j)
                x[i][j] = r ? __ldg(reinterpret_cast<const float4*>(r) + (lane & 7) + 8 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void score(const double* us, int base, int c1, Key* keys, int lane) const
    {
        double a[kEach], z[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) a[i] = z[i] = 0.0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const double2 u0 = *reinterpret_cast<const double2*>(us + 4 * ((lane & 7) + 8 * j));
            const double2 u1 = *reinterpret_cast<const double2*>(us + 4 * ((lane & 7) + 8 * j) + 2);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                a[i] = fma(u0.x, (double)x[i][j].x, a[i]);
                z[i] = fma(u0.y, (double)x[i][j].y, z[i]);
                a[i] = fma(u1.x, (double)x[i][j].z, a[i]);
                z[i] = fma(u1.y, (double)x[i][j].w, z[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            a[i] += z[i];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) a[i] += __shfl_xor_sync(0xFFFFFFFFu, a[i], o);
            const int c = base + 4 * i + (lane >> 3);
            if ((lane & 7) == 0 && c < c1) keys[c] = ordered(have[i] ? a[i] : -INFINITY);
        }
    }
};
template <int D, int kWarps, typename Row>
__device__ __forceinline__ void score(const double* us, int c0, int c1, Row row, Key* keys, int warp, int lane)
{
    constexpr int kAll = Candidates<D>::kStep * kWarps;
    int base = c0 + Candidates<D>::kStep * warp;
    if (base >= c1) return;
    Candidates<D> now, next;
    now.load(base, c1, row, lane);
    for (; base + kAll < c1; base += kAll) {
        next.load(base + kAll, c1, row, lane);
        now.score(us, base, c1, keys, lane);
        now = next;
    }
    now.score(us, base, c1, keys, lane);
}

// keys[c0, c1) of this CTA into the same slots of its peers.
template <int kThreads>
__device__ __forceinline__ void push(Key* keys, int c0, int c1, int S, int rank, int tid)
{
    const int n = c1 - c0;
    for (int i = tid; i < n * S; i += kThreads) {
        const int p = i / n, c = c0 + i % n;
        if (p != rank) sm100::st_cluster_u64(peer_addr(smem_u32(keys + c), p), keys[c]);
    }
}

template <typename TIn, int D, int CACHE, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps == 4 ? 4 : 2) paged_decode_kernel(const __grid_constant__ Args g)
{
    constexpr int kThreads = 32 * kWarps;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ __align__(16) double us[D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = g.S, rank = S > 1 ? (int)cluster_rank() : 0;
    const int64_t bh = blockIdx.x / S;
    const int b = int(bh / g.s.Hkv), h = int(bh % g.s.Hkv), G = g.s.G;
    const Layout L = layout<D, kWarps>(g.s, S);
    if (S > 1) cluster_arrive();                     // waited for before the first write to a peer
    pdl_wait();
    pdl_trigger();

    const int32_t* table = g.c.table + (int64_t)b * g.s.max_chunks;
    const int64_t head0 = (int64_t)b * g.s.Hq + h * G;   // first of the kv-head's q-heads
    const TIn* q = static_cast<const TIn*>(g.q) + head0 * D;
    int32_t* tab = reinterpret_cast<int32_t*>(sm + L.table);
    int64_t p = g.pos[b];
    // The page table and the query are on their way together with the position.
    for (int c = tid; c < min(g.s.max_chunks, kTable); c += kThreads) tab[c] = __ldg(table + c);
    for (int e = tid; e < D; e += kThreads) {
        TIn x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < G ? q[i * D + e] : TIn(0.f);
        double a = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += (double)widen<TIn>(x[i]);
        us[e] = a;
    }
    if (p >= (int64_t)g.s.max_chunks * kChunk) {
        flag(kSiteLength);
        p = -1;
    }
    if (p < 0) {                                     // an empty sequence: all CTAs of the cluster alike
        if (rank == 0) {
            for (int i = tid; i < G * D; i += kThreads) g.O[head0 * D + i] = 0.f;
            for (int i = tid; i < G; i += kThreads) g.lse[head0 + i] = -INFINITY;
            for (int i = tid; i < g.s.wc; i += kThreads) g.cidx[bh * g.s.wc + i] = -1;
            for (int i = tid; i < g.s.wg; i += kThreads) g.gidx[bh * g.s.wg + i] = -1;
        }
        if (S > 1) cluster_wait();
        return;
    }
    const int c0 = int(p / kChunk), rows = int(p % kChunk) + 1;
    auto page_of = [&](int c) {
        return (int32_t)page_or_none(c < kTable ? tab[c] : __ldg(table + c), g.s.n_pages, kSitePage);
    };

    int32_t* gpage = reinterpret_cast<int32_t*>(sm + L.gpage);
    int32_t* grow = reinterpret_cast<int32_t*>(sm + L.grow);
    auto* ckeys = reinterpret_cast<Key*>(sm + L.ckeys);
    auto* gkeys = reinterpret_cast<Key*>(sm + L.gkeys);
    auto* scratch = reinterpret_cast<SelectScratch<kWarps>*>(sm + L.scratch);
    int32_t* crow = reinterpret_cast<int32_t*>(sm + L.crow);
    int32_t* cpage = reinterpret_cast<int32_t*>(sm + L.cpage);
    __syncthreads();
    const int kc = g.s.k_c > 0 ? min(g.s.k_c, c0) : c0;
    if (kc < c0) {
        const int b0 = int((int64_t)rank * c0 / S), b1 = int((int64_t)(rank + 1) * c0 / S);
        score<D, kWarps>(us, b0, b1, [&](int c) -> const float* {
            const int32_t page = page_of(c);
            return page < 0 ? nullptr : g.c.csum + ((int64_t)page * g.s.Hkv + h) * D;
        }, ckeys, warp, lane);
        __syncthreads();
        if (S > 1) {
            cluster_wait();
            push<kThreads>(ckeys, b0, b1, S, rank, tid);
            cluster_arrive();
            cluster_wait();
            cluster_arrive();                    // for the groups' push
        }
    }
    // The open rows, 16 at a time, while the first warp selects (up to 512
    // chunks are its work alone): tile i to CTA S - 1 - i mod S.
    float* parked = reinterpret_cast<float*>(sm + L.parked) + Running<D>::kParked * (warp - 1);
    const int turn = S - 1 - rank + S * (warp - 1), tiles = (rows + 15) / 16;
    const bool own_tile = turn < tiles;
    if (warp > 0 && own_tile) {
        Running<D> run;
        run.init();
        const int64_t row0 = bh * kChunk * D;
        for (int i = turn; i < tiles; i += S * (kWarps - 1))
            attend_open<TIn, D>(run, q, G, g.c.k_tail + row0, static_cast<const TIn*>(g.c.v_tail) + row0, 16 * i, rows,
                                g.s.scale * kLog2e, lane);
        run.park(parked, lane);
    }
    select<kWarps>(ckeys, c0, kc, scratch, tid, crow);
    __syncthreads();
    for (int i = tid; i < kc; i += kThreads) cpage[i] = page_of(crow[i]);
    __syncthreads();
    const int n = kc * kGroupsPerChunk;
    const int kg = g.s.k_g > 0 ? min(g.s.k_g, n) : n;
    if (kg < n) {
        const int b0 = int((int64_t)rank * n / S), b1 = int((int64_t)(rank + 1) * n / S);
        score<D, kWarps>(us, b0, b1, [&](int i) -> const float* {
            const int32_t page = cpage[i / kGroupsPerChunk];
            return page < 0 ? nullptr
                            : g.c.gsum + (((int64_t)page * g.s.Hkv + h) * kGroupsPerChunk + i % kGroupsPerChunk) * D;
        }, gkeys, warp, lane);
        __syncthreads();
        if (S > 1) {
            cluster_wait();
            push<kThreads>(gkeys, b0, b1, S, rank, tid);
            cluster_arrive();
            cluster_wait();
            cluster_arrive();                    // for the merge
        }
    }
    select<kWarps>(gkeys, n, kg, scratch, tid, grow);
    __syncthreads();
    for (int i = tid; i < kg; i += kThreads) {   // candidates to groups
        const int x = grow[i];
        grow[i] = crow[x / kGroupsPerChunk] * kGroupsPerChunk + x % kGroupsPerChunk;
        gpage[i] = cpage[x / kGroupsPerChunk];
    }
    __syncthreads();
    const int ng = kg;
    if (rank == 0) {
        for (int i = tid; i < g.s.wc; i += kThreads) g.cidx[bh * g.s.wc + i] = i < kc ? crow[i] : -1;
        for (int i = tid; i < g.s.wg; i += kThreads) g.gidx[bh * g.s.wg + i] = i < ng ? grow[i] : -1;
    }

    // Attention.
    const int wid = warp * S + rank, n_workers = S * kWarps;     // neighbouring tiles on different SMs
    Running<D> run;
    run.init();
    if (warp > 0 && own_tile) run.unpark(parked, lane);
    __syncthreads();                                 // the rings may be filled
    {
        const int n_tiles = (ng + kTileGroups - 1) / kTileGroups;
        const int mine = n_tiles > wid ? (n_tiles - wid + n_workers - 1) / n_workers : 0;
        auto group_of = [&](int i) -> int64_t {
            const int u = kTileGroups * (wid + i * n_workers) + lane / 8;
            const int32_t page = u < ng ? gpage[u] : -1;
            return page < 0 ? -1 : ((int64_t)page * g.s.Hkv + h) * kGroupsPerChunk + grow[u] % kGroupsPerChunk;
        };
        HeldTiles<TIn, D, CACHE, decltype(group_of)> held(reinterpret_cast<Half<D>*>(sm + L.rings) + kHalves * warp, g.c,
                                                          group_of, mine, lane);
        held.start();
        held.attend(run, q, G, g.s.scale * kLog2e);
    }

    // Merge: the CTA's warps, then the cluster's CTAs.  f: a warp's factor for
    // the CTA's reference, then a CTA's for the last one.
    __syncthreads();                                 // the rings are done with
    float* om = reinterpret_cast<float*>(sm + L.merge);          // [kWarps][G][D]
    float* rm = om + kWarps * G * D;                             // [kWarps][G] references
    float* lm = rm + kWarps * G;                                 // [kWarps][G] sums
    float* fm = lm + kWarps * G;                                 // [kWarps][G] factors
    run.store(om + warp * G * D, rm + warp * G, lm + warp * G, G, lane);
    __syncthreads();
    const int part = D / S, lg = __ffs(part) - 1;    // elements of a head's output that a CTA combines
    float* inbox = reinterpret_cast<float*>(sm + L.inbox);       // [S][G][part], then [S][G] references, sums, factors
    float* ibr = inbox + G * D;
    float* ibl = ibr + S * G;
    float* ibf = ibl + S * G;
    if (S > 1) cluster_wait();                       // (of the start, or of the last exchange)
    // A head's warps, then its CTAs, are eight neighbouring lanes.
    if (warp < (8 * G + 31) / 32) {
        const int hd = tid / 8, w = tid % 8;
        const bool is = hd < G && w < kWarps;
        float M = is ? rm[w * G + hd] : kFloor, l = is ? lm[w * G + hd] : 0.f;
        const float f = join_parts<8>(M, l);
        if (is) fm[w * G + hd] = S > 1 ? f : f / l;
        if (S > 1) {
            if (hd < G && w < S) {
                sm100::st_cluster_f32(peer_addr(smem_u32(ibr + rank * G + hd), w), M);
                sm100::st_cluster_f32(peer_addr(smem_u32(ibl + rank * G + hd), w), l);
            }
        } else if (is && w == 0) {
            g.lse[head0 + hd] = (M + log2f(l)) * kLn2;
        }
    }
    __syncthreads();
    for (int i = tid; i < G * D; i += kThreads) {
        const int hd = i / D, e = i % D;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o = fmaf(om[w * G * D + i], fm[w * G + hd], o);
        if (S > 1)
            sm100::st_cluster_f32(peer_addr(smem_u32(inbox + (rank * G + hd) * part + (e & (part - 1))), e >> lg), o);
        else
            g.O[head0 * D + i] = o;
    }
    if (S == 1) return;
    cluster_arrive();
    cluster_wait();
    if (warp < (8 * G + 31) / 32) {
        const int hd = tid / 8, c = tid % 8;
        const bool is = hd < G && c < S;
        float M = is ? ibr[c * G + hd] : kFloor, l = is ? ibl[c * G + hd] : 0.f;
        const float f = join_parts<8>(M, l);
        if (is) ibf[c * G + hd] = f / l;
        if (is && c == 0 && rank == 0) g.lse[head0 + hd] = (M + log2f(l)) * kLn2;
    }
    __syncthreads();
    for (int i = tid; i < G * part; i += kThreads) {
        const int hd = i >> lg;
        float o = 0.f;
        for (int c = 0; c < S; ++c) o = fmaf(inbox[c * G * part + i], ibf[c * G + hd], o);
        g.O[(head0 + hd) * D + rank * part + (i & (part - 1))] = o;
    }
}

// CTAs per (batch, kv-head), a power of two.  Measured at 16K context, k_c 8,
// k_g 32 (us a call with 1, 2, 4, 8 CTAs): 8 units 21.4, 16.2, 15.3, 14.5; 32
// units 21.7, 16.3, 15.0, 16.1; 64 units 21.8, 16.4, 17.1, 32.2; 128 units
// 25.9, 21.0, 36.7; 256 units 35.3, 42.3; 512 units 42.3, 82.1.  At 128K (k_c
// 16, k_g 64) 32 units take 98, 44, 31, 29.  So: as many as leave a CTA an SM
// to itself, two CTAs an SM for the first doubling and where there are many
// chunks to score, and no more than there are chunks to share.
int split(const PagedShape& s)
{
    const int64_t units = (int64_t)s.B * s.Hkv, sms = sm_count();
    int S = 1;
    while (S < kMaxS && S * 4 <= s.max_chunks && units * S * 2 <= (S == 1 || s.max_chunks >= 1024 ? 2 : 1) * sms) S *= 2;
    return S;
}

template <typename TIn, int D, int CACHE, int kWarps> cudaError_t launch(const Args& g, cudaStream_t st)
{
    const size_t smem = layout<D, kWarps>(g.s, g.S).total;
    auto k = paged_decode_kernel<TIn, D, CACHE, kWarps>;
    if (cudaError_t e = allow_smem(k, (int)smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.s.B * g.s.Hkv * g.S));
    cfg.blockDim = dim3(32 * kWarps);
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

template <typename TIn, int D> cudaError_t by_cache(const Args& g, cudaStream_t st)
{
    if (g.s.cache_dtype == HGA_INT8)
        return g.S > 1 ? launch<TIn, D, HGA_INT8, 6>(g, st) : launch<TIn, D, HGA_INT8, 4>(g, st);
    return g.S > 1 ? launch<TIn, D, HGA_E4M3, 6>(g, st) : launch<TIn, D, HGA_E4M3, 4>(g, st);
}

}  // namespace

size_t paged_routed_smem(const PagedShape& s) { return layout<128, 6>(s, kMaxS).total + 2048; }

cudaError_t launch_paged_routed(const PagedShape& s, const hga_paged_cache& c, const int32_t* pos, const void* q,
                                float* O, float* lse, int32_t* cidx, int32_t* gidx, cudaStream_t st)
{
    const Args g{s, c, pos, q, O, lse, cidx, gidx, split(s)};
    if (s.dtype == HGA_BF16) return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, st) : by_cache<__nv_bfloat16, 64>(g, st);
    return s.d == 128 ? by_cache<float, 128>(g, st) : by_cache<float, 64>(g, st);
}

HGA_CHECK_WORD_READER(check_word_paged_routed)

}  // namespace hga
