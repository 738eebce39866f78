// paged_decode.cu -- one query per sequence over the paged 8-bit cache: routed
// attention.
//
// The sequence's query stands at position p = pos[b] (its key and value are
// in the open rows already).  With u = the sum of the kv-head's q-heads'
// queries, chunk c < p / 64 scores u . csum[c]; the k_c highest are kept, then
// the k_g highest of their groups by u . gsum.  Scores are formed in float64:
// a score is off by at most (d + 8) 2^-53 sum |u_i| |csum_i| (u is a rounded
// sum of up to eight queries, so not every product is exact), and only
// candidates that lie closer than that can change places with the order of
// summation, which is fixed.  Every q-head attends the
// kept groups' held values and the open rows 0 .. p % 64:
//     O = softmax(scale q K^T) V,  lse = log sum exp (scale q K^T).
//
// A cluster of S CTAs (of 4, 6 or 8 warps) takes one (batch, kv-head).
//   * Scoring: CTA r scores the r-th part of the candidates and writes their
//     keys into every peer's shared memory; each CTA then makes the same
//     selection (paged_select.cuh).
//   * Attention: a warp takes tiles of four groups (32 keys), tile i going to
//     warp i modulo the cluster's warps, through its own ring of asynchronous
//     copies into mma.sync fragments (paged_attend.cuh).
//   * Merge: every warp has a reference, a sum and a mean for each head; a
//     CTA's meet in shared memory, and each CTA combines d / S elements of
//     every head's output (distributed shared memory).
//
// A step is a chain of about ten dependent steps (position, scores, exchange,
// selection, group scores, exchange, selection, tiles, merge, exchange),
// which bounds it: 13.6 us for one sequence at 16K context (8 kv-heads, d 128,
// k_c 8, k_g 32; 2.3 MB), 38.1 us for 64 (103 MB, 2.7 TB/s: all score at once,
// then all wait for each other's loads in short chains).
//
// Registers: 128 a thread with 4 or 8 warps (four and two CTAs an SM), 168 with
// 6.  At d = 128 the attention's loop wants more, and 80 - 250 bytes a thread
// go to local memory there, 24 - 44 with 6 warps; at d = 64 at most 20.
#include <algorithm>

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

// Dynamic shared memory.  The routing's keys (and the open rows, then their
// parked outputs), the warps' rings and the warps' outputs follow one another
// in the same place; the page table's first
// kTable entries, the kept chunks and groups with their pages, and what peers
// write (inbox) have places of their own.
constexpr int kTable = 2048;
struct Layout {
    uint32_t ckeys, gkeys, scratch, slots, rings, merge, table, crow, cpage, grow, gpage, query, inbox;
    int n_slots;
    size_t total;
};
inline size_t up16(size_t x) { return (x + 15) & ~size_t(15); }

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
    Layout L;
};

// Where a CTA has an SM to itself, or half of one, open rows are read when they
// are attended.  With more of them a load then takes microseconds, under the
// scoring of the others, so the copies start before the scoring (64 sequences of
// up to 16K: 41.4 us without, 37.5 with them; 32, two CTAs an SM: 25.6 and 26.0;
// one: 13.7 and 15.2).
template <int kWarps> constexpr bool kStaged = kWarps == 4;
// The slots hold open rows, then a warp's parked outputs: one for each warp but
// the first, and one for the fourth tile, as far as they leave room for four
// CTAs an SM (that many bytes each, 1 KB of the system's and 1 KB of `us`
// besides).
constexpr size_t kRoom4 = 55 * 1024;
constexpr int kOpenTiles = kChunk / 16;
template <typename TIn, int D, int kWarps> __host__ __device__ constexpr size_t slot_bytes()
{
    static_assert(OpenSlot<TIn, D>::kBytes >= 4 * Running<D>::kParked, "a warp parks its outputs in its slot");
    return kStaged<kWarps> ? OpenSlot<TIn, D>::kBytes : 4 * Running<D>::kParked;
}
template <typename TIn, int D, int kWarps> Layout layout(const PagedShape& s, int S)
{
    Layout L{};
    const size_t nc = s.max_chunks, wc = s.wc, wg = s.wg;
    const bool thin = nc > kThin || 8 * wc > kThin;
    const size_t gkeys = up16(8 * nc), scratch = up16(gkeys + 8 * 8 * wc);
    const size_t slots = up16(scratch + (thin ? sizeof(SelectScratch<kWarps>) : SelectScratch<kWarps>::kSmall));
    const size_t table = up16(4 * std::min<size_t>(nc, kTable)), crow = up16(4 * wc), grow = up16(4 * wg);
    const size_t query = kStaged<kWarps> ? up16(sizeof(TIn) * s.G * OpenSlot<TIn, D>::kQueryRow) : 0;
    constexpr size_t slot = slot_bytes<TIn, D, kWarps>();
    L.n_slots = std::min(kWarps - 1, (kOpenTiles + S - 1) / S);
    if (kStaged<kWarps>) {
        const size_t used = slots + table + 2 * crow + 2 * grow + query;
        L.n_slots = used < kRoom4 ? (int)std::clamp<size_t>((kRoom4 - used) / slot, 1, kOpenTiles) : 1;
    }
    const size_t rings = sizeof(Half<D>) * kHalves * kWarps, merge = 4 * (size_t)kWarps * s.G * (D + 3);
    size_t at = up16(std::max({slots + slot * L.n_slots, rings, merge}));
    auto take = [&](size_t n) {
        const size_t from = at;
        at += up16(n);
        return (uint32_t)from;                       // (a total that is too large is refused)
    };
    L.gkeys = (uint32_t)gkeys;
    L.scratch = (uint32_t)scratch;
    L.slots = (uint32_t)slots;
    L.table = take(table);
    L.crow = take(crow);
    L.cpage = take(crow);
    L.grow = take(grow);
    L.gpage = take(grow);
    L.query = take(query);
    // From each peer: d / S elements of its outputs, its G references and sums
    // (and a share for each of them).
    L.inbox = take(S > 1 ? 4 * ((size_t)s.G * D + 3 * (size_t)s.G * S) : 0);
    L.total = at;
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
    const Layout& L = g.L;
    if (S > 1) cluster_arrive();                     // waited for before the first write to a peer
    // The arguments come into the constant cache while the kernel before ends.
    asm volatile("" ::"r"(L.gkeys), "r"(L.inbox), "r"(L.n_slots), "r"(g.s.wg), "l"(g.c.k_pages), "l"(g.c.table), "l"(g.gidx));
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
    // The open rows, 16 at a time, go to the warps but the first (as many as have
    // slots), tile i to CTA S - 1 - i mod S.
    const int workers = min(L.n_slots, kWarps - 1);
    const int turn = S - 1 - rank + S * (warp - 1), turns = S * workers, tiles = (rows + 15) / 16;
    const bool own_tile = warp > 0 && warp <= workers && turn < tiles, spare = L.n_slots == kWarps;
    uint8_t* const slot = sm + L.slots + slot_bytes<TIn, D, kWarps>() * (warp - 1);
    auto rows_at = [&](int i) {
        const int64_t row0 = bh * kChunk * D;
        return OpenGlobal<TIn, D>{g.c.k_tail + row0, static_cast<const TIn*>(g.c.v_tail) + row0, q, 16 * i, rows};
    };
    auto slot_of = [&](int i) {
        return OpenSlot<TIn, D>{i == turn || !spare ? slot : sm + L.slots + slot_bytes<TIn, D, kWarps>() * (kWarps - 1),
                                reinterpret_cast<TIn*>(sm + L.query), rows_at(i)};
    };
    if (kStaged<kWarps> && own_tile) {
        slot_of(turn).fetch_queries(G, lane);
        for (int i = turn; i < tiles && (i == turn || spare); i += turns) slot_of(i).fetch(lane);
        fetch_commit();
    }
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
    // The open rows are attended while the first warp selects (up to 512 chunks
    // are its work alone).
    float* const parked = reinterpret_cast<float*>(slot);
    if (own_tile) {
        Running<D> run;
        run.init();
        if constexpr (kStaged<kWarps>) {
            fetch_wait_all();
#pragma unroll 1
            for (int i = turn; i < tiles; i += turns) {
                const auto open = slot_of(i);
                if (i != turn && !spare) {
                    open.fetch(lane);
                    fetch_commit();
                    fetch_wait_all();
                }
                attend_open<TIn, D>(run, G, open, rows - 16 * i, g.s.scale * kLog2e, lane);
                __syncwarp();
            }
        } else {                                     // one tile at most: the cluster has four slots or more
            attend_open<TIn, D>(run, G, rows_at(turn), rows - 16 * turn, g.s.scale * kLog2e, lane);
        }
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
    if (own_tile) run.unpark(parked, lane);
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

    // Merge: the CTA's warps, then the cluster's CTAs, by their shares of the
    // normalising sum.
    __syncthreads();                                 // the rings are done with
    float* om = reinterpret_cast<float*>(sm + L.merge);          // [kWarps][G][D]
    float* rm = om + kWarps * G * D;                             // [kWarps][G] references
    float* lm = rm + kWarps * G;                                 // [kWarps][G] sums
    float* fm = lm + kWarps * G;                                 // [kWarps][G] factors: of a mean, then times its share
    run.store(om + warp * G * D, rm + warp * G, lm + warp * G, fm + warp * G, G, lane);
    __syncthreads();
    const int part = D / S, lg = __ffs(part) - 1;    // elements of a head's output that a CTA combines
    float* inbox = reinterpret_cast<float*>(sm + L.inbox);       // [S][G][part], then [S][G] references, sums, shares
    float* ibr = inbox + G * D;
    float* ibl = ibr + S * G;
    float* ibf = ibl + S * G;
    if (S > 1) cluster_wait();                       // (of the start, or of the last exchange)
    // A head's warps, then its CTAs, are eight neighbouring lanes.
    if (warp < (8 * G + 31) / 32) {
        const int hd = tid / 8, w = tid % 8;
        const bool is = hd < G && w < kWarps;
        float M = is ? rm[w * G + hd] : kFloor, l = is ? lm[w * G + hd] : 0.f;
        const float f = join_parts<8>(M, l, S == 1);
        if (is) fm[w * G + hd] *= f;
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
        const float f = join_parts<8>(M, l, true);
        if (is) ibf[c * G + hd] = f;
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

// CTAs per (batch, kv-head), a power of two, and warps of one.  Measured when
// the rule was made, k_c 8, k_g 32, d 128, bf16, us a call ("4 x 6": four CTAs of
// 6 warps):
//   16K, units    8: 1 x 8 15.7, 8 x 6 14.1, 8 x 8 14.5
//                32: 1 x 8 16.0, 2 x 6 16.0, 4 x 6 14.2, 8 x 6 15.1
//                64: 1 x 4 20.8, 1 x 8 16.1, 2 x 6 16.1, 4 x 6 15.9
//               128: 1 x 4 22.6, 1 x 6 19.2, 1 x 8 17.7, 2 x 6 19.8
//               256: 1 x 4 29.7, 1 x 6 25.4, 1 x 8 26.1, 2 x 6 41.4
//               320: 1 x 4 34.1, 1 x 6 39.7;  512: 37.4, 46.7
//   2K,         256: 1 x 4 19.6, 1 x 6 18.8, 1 x 8 20.6
//   128K, units  32: 1 x 8 48.5, 2 x 8 33.2, 4 x 6 27.4, 4 x 8 24.6, 8 x 8 24.5
//  (k_c 16,      64: 1 x 8 63.8, 2 x 8 43.8, 4 x 6 38.0, 4 x 8 37.0
//   k_g 64)     128: 1 x 8 68.0, 2 x 6 57.8, 2 x 8 52.9;  256: 1 x 6 87.7, 1 x 8 80.3
// So: clusters as long as a CTA has an SM to itself, of 6 warps (the exchange and
// the merge grow with the warps); then 8 warps, 6 when two CTAs share an SM, and
// 4 when four do.  Where there are many chunks to score, 8 warps and clusters
// for two CTAs an SM.
struct Split {
    int S, warps;
};
Split split(const PagedShape& s)
{
    const int64_t units = (int64_t)s.B * s.Hkv, sms = sm_count();
    if (units > 2 * sms) return {1, 4};
    const bool many = s.max_chunks >= 1024;
    int S = 1;
    while (S < kMaxS && S * 4 <= s.max_chunks && units * S * 2 <= (many ? 2 * sms : sms)) S *= 2;
    return {S, many || (S == 1 && units <= sms) ? 8 : 6};
}

template <typename TIn, int D, int CACHE, int kWarps> cudaError_t launch(Args g, cudaStream_t st)
{
    g.L = layout<TIn, D, kWarps>(g.s, g.S);
    const size_t smem = g.L.total;
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

template <typename TIn, int D, int CACHE> cudaError_t by_warps(const Args& g, int warps, cudaStream_t st)
{
    return warps == 8   ? launch<TIn, D, CACHE, 8>(g, st)
           : warps == 6 ? launch<TIn, D, CACHE, 6>(g, st)
                        : launch<TIn, D, CACHE, 4>(g, st);
}

template <typename TIn, int D> cudaError_t by_cache(const Args& g, int warps, cudaStream_t st)
{
    return g.s.cache_dtype == HGA_INT8 ? by_warps<TIn, D, HGA_INT8>(g, warps, st) : by_warps<TIn, D, HGA_E4M3>(g, warps, st);
}

}  // namespace

// (bfloat16 rows take the larger slots.)
size_t paged_routed_smem(const PagedShape& s)
{
    return std::max({layout<__nv_bfloat16, 128, 4>(s, 1).total, layout<float, 128, 8>(s, 1).total,
                     layout<float, 128, 8>(s, kMaxS).total}) + 2048;
}

cudaError_t launch_paged_routed(const PagedShape& s, const hga_paged_cache& c, const int32_t* pos, const void* q,
                                float* O, float* lse, int32_t* cidx, int32_t* gidx, cudaStream_t st)
{
    const Split x = split(s);
    const Args g{s, c, pos, q, O, lse, cidx, gidx, x.S, {}};
    if (s.dtype == HGA_BF16)
        return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, x.warps, st) : by_cache<__nv_bfloat16, 64>(g, x.warps, st);
    return s.d == 128 ? by_cache<float, 128>(g, x.warps, st) : by_cache<float, 64>(g, x.warps, st);
}

HGA_CHECK_WORD_READER(check_word_paged_routed)

}  // namespace hga
