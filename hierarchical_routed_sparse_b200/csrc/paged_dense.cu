// paged_dense.cu -- one query per sequence over the whole of its paged 8-bit
// cache (no routing): O = softmax(scale q K^T) V over every complete chunk's
// held values and the open rows 0 .. pos % 64.
//
// The sequences of a batch differ in length, and one long sequence may be all
// there is, so work is cut by keys and not by sequences: the tiles (32 keys)
// of all units (batch, kv-head) stand in one row, each unit's led by kOpen that
// stand for its open rows (and for what a unit costs whatever its length), and
// every CTA takes the same number of neighbours.  A unit that one CTA holds from end to end is finished there;
// the parts of the others (mean, reference and sum of each head) go to the
// workspace, and a second kernel joins them.  Which CTA has what follows from
// the positions, which both kernels read on the device.
//
// The kernel streams every code once; what bounds it is instruction issue, at
// about 800 a tile (paged_attend.cuh; 930 with a warp's fixed part), 0.53 of a
// scheduler's slots with 12 warps an SM: 8 sequences of up to 16K, 8 kv-heads
// (156 MB) take 38 us with the join, 4.1 TB/s, and one of 50000 with 2
// kv-heads (26 MB) 14 us, most of it the two kernels' chains.  At d = 128 up to
// 120 bytes a thread of the float32 kernel's 168 registers' worth go to local
// memory, 24 of the bf16 one's.
#include "paged.cuh"
#include "paged_attend.cuh"
#include "sm100.cuh"

namespace hga {
namespace {

using namespace paged;

// 12 warps an SM, with the registers that a tile wants (16 warps of 128
// registers: 43.4 us where this takes 40.6, 8 sequences of up to 16K).
constexpr int kWarps = 6, kThreads = 32 * kWarps, kPerSm = 2;
constexpr int kLeast = 2 * kWarps;                   // tiles of a CTA, where there are few
constexpr int kOpen = kLeast;                        // tiles that a unit's open rows, start and merge count as
constexpr int kPerChunk = kGroupsPerChunk / kTileGroups;
constexpr int kSitePage = 431, kSiteLength = 432;

struct Args {
    PagedShape s;
    hga_paged_cache c;
    const int32_t* pos;
    const void* q;
    float* O;
    float* lse;
    float* parts;                                    // [grid][2][part_floats]
    int grid;                                        // CTAs of the first kernel
};

// Tiles of a sequence's units: none when it is empty (or its position is
// past the table: recorded).  The sum over all units is below 2^31 (checked
// on the host).
__device__ __forceinline__ int tiles_of(const Args& g, int b)
{
    const int32_t p = g.pos[b];
    if (p < 0) return 0;
    if (p >= (int64_t)g.s.max_chunks * kChunk) {
        flag(kSiteLength);
        return 0;
    }
    return kOpen + kPerChunk * (p / kChunk);
}

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

// The row of tiles, as every warp finds it for itself: 32 sequences at a time,
// one a lane.  CTA i's first tile is i * least + min(i, more).
struct Row {
    int total, ctas, least, more;                    // ctas: those that get tiles
    int lane_tiles;                                  // of sequence `lane`, when there are at most 32
    __device__ __forceinline__ explicit Row(const Args& g)
    {
        const int lane = threadIdx.x & 31;
        lane_tiles = 0;
        int mine = 0;
#pragma unroll 4
        for (int b = lane; b < g.s.B; b += 32) mine += lane_tiles = tiles_of(g, b);
        total = warp_sum_int(mine) * g.s.Hkv;
        ctas = max(1, min(g.grid, (total + kLeast - 1) / kLeast));
        least = total / ctas;
        more = total - least * ctas;
    }
    __device__ __forceinline__ int begin(int cta) const { return cta * least + min(cta, more); }
    __device__ __forceinline__ int cta_of(int tile) const
    {
        const int big = more * (least + 1);          // tiles of the CTAs that have one more
        return tile < big ? tile / (least + 1) : more + (tile - big) / least;
    }
};

// Sequence that holds the tile, and its first unit's first tile.
__device__ __forceinline__ void find(const Args& g, const Row& row, int tile, int& b, int& first)
{
    const int lane = threadIdx.x & 31;
    first = 0;
    for (int b0 = 0; b0 < g.s.B; b0 += 32) {
        const int n = (g.s.B <= 32 ? row.lane_tiles : b0 + lane < g.s.B ? tiles_of(g, b0 + lane) : 0) * g.s.Hkv;
        int upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, tile < first + upto);
        if (hit) {
            const int at = __ffs(hit) - 1;
            b = b0 + at;
            first += __shfl_sync(0xFFFFFFFFu, upto - n, at);
            return;
        }
        first += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    b = g.s.B;
}

// Where a border between two CTAs goes that would be `o` tiles into a unit of
// n: not among the open rows' tiles, which are one piece, nor a few tiles
// before the unit's end.
__device__ __forceinline__ int border(int o, int n)
{
    if (n < kOpen + kWarps) return 2 * o < n ? 0 : n;            // a short unit stays whole
    if (o < kOpen) return 2 * o < kOpen ? 0 : kOpen;
    return n - o < kWarps ? n : o;
}

// As find, for the border nearest to the tile; moves the tile there.
__device__ __forceinline__ void find_border(const Args& g, const Row& row, int& tile, int& b, int& first)
{
    if (tile >= row.total) return;
    find(g, row, tile, b, first);
    const int n = tiles_of(g, b), o = (tile - first) % n;
    tile += border(o, n) - o;
}

// (A multiple of 4 floats, as a part's rows are read.)
__host__ __device__ inline size_t part_floats(const PagedShape& s) { return ((size_t)s.G * s.d + 2 * (size_t)s.G + 3) & ~size_t(3); }

template <int D> constexpr size_t rings_bytes() { return sizeof(Half<D>) * kHalves * kWarps; }
template <int D> inline size_t dense_smem(const PagedShape& s)
{
    const size_t merge = 4 * (size_t)kWarps * s.G * (D + 3);
    return rings_bytes<D>() > merge ? rings_bytes<D>() : merge;
}

template <typename TIn, int D, int CACHE>
__global__ void __launch_bounds__(kThreads, kPerSm) paged_dense_kernel(const __grid_constant__ Args g)
{
    extern __shared__ __align__(16) uint8_t sm[];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = g.s.G;
    const Row row(g);
    if ((int)blockIdx.x >= row.ctas || row.total == 0) return;
    int at = row.begin(blockIdx.x), end = row.begin(blockIdx.x + 1);
    int b = 0, first = 0;                            // first: of the sequence's first unit
    find_border(g, row, end, b, first);
    find_border(g, row, at, b, first);

    while (at < end) {
        const int n = tiles_of(g, b);
        if (n == 0 || at >= first + n * g.s.Hkv) {   // to the next sequence
            first += n * g.s.Hkv;
            ++b;
            continue;
        }
        const int h = (at - first) / n;
        const int unit0 = first + n * h;             // the unit's tiles: unit0 .. unit0 + n - 1
        const int from = at - unit0, to = end - unit0 < n ? end - unit0 : n;
        const int64_t bh = (int64_t)b * g.s.Hkv + h, head0 = (int64_t)b * g.s.Hq + h * G;
        const TIn* q = static_cast<const TIn*>(g.q) + head0 * D;
        const int32_t* table = g.c.table + (int64_t)b * g.s.max_chunks;

        // Tile kOpen + j is half j % 2 of chunk j / 2.  A CTA's last warp begins,
        // since the first ones have open rows.
        const int j0 = max(from - kOpen, 0) + (kWarps - 1 - warp), j1 = to - kOpen;
        const int mine = j1 > j0 ? (j1 - j0 + kWarps - 1) / kWarps : 0;
        int32_t pages = 0;                           // pages of 32 of the warp's tiles, one a lane
        static_assert(kWarps % kPerChunk == 0, "a warp's tiles are the same part of their chunks");
        const int chunk0 = j0 / kPerChunk;
        const int in_page = h * kGroupsPerChunk + kTileGroups * (j0 % kPerChunk) + lane / 8;
        const int page_groups = g.s.Hkv * kGroupsPerChunk;
        auto group_of = [&](int i) -> int64_t {
            if (i % 32 == 0)
                pages = i + lane < mine ? (int32_t)page_or_none(__ldg(table + chunk0 + (i + lane) * (kWarps / kPerChunk)),
                                                                g.s.n_pages, kSitePage)
                                        : -1;
            const int32_t page = __shfl_sync(0xFFFFFFFFu, pages, i % 32);
            return page < 0 ? -1 : (int64_t)page * page_groups + in_page;
        };
        HeldTiles<TIn, D, CACHE, decltype(group_of)> held(reinterpret_cast<Half<D>*>(sm) + kHalves * warp, g.c, group_of, mine,
                                                          lane);
        held.start();
        Running<D> run;
        run.init();
        if (from == 0) {                             // the open rows
            const int rows = int(g.pos[b] % kChunk) + 1;
            const int64_t r0 = bh * kChunk * D;
            if (16 * warp < rows)
                attend_open<TIn, D>(run, G,
                                    OpenGlobal<TIn, D>{g.c.k_tail + r0, static_cast<const TIn*>(g.c.v_tail) + r0, q,
                                                       16 * warp, rows},
                                    rows - 16 * warp, g.s.scale * kLog2e, lane);
        }
        held.attend(run, q, G, g.s.scale * kLog2e);

        // The warps' parts meet, each times its factor for a mean and its share of the sum.
        __syncthreads();
        float* om = reinterpret_cast<float*>(sm);    // [kWarps][G][D]
        float* rm = om + kWarps * G * D;             // [kWarps][G] references, then sums, then factors
        float* lm = rm + kWarps * G;
        float* fm = lm + kWarps * G;
        run.store(om + warp * G * D, rm + warp * G, lm + warp * G, fm + warp * G, G, lane);
        __syncthreads();
        const bool whole = from == 0 && to == n;
        float* part = g.parts + (2 * (int64_t)blockIdx.x + (from == 0)) * part_floats(g.s);
        if (warp < (8 * G + 31) / 32) {              // a head's warps are eight neighbouring lanes
            const int hd = tid / 8, w = tid % 8;
            const bool is = hd < G && w < kWarps;
            float M = is ? rm[w * G + hd] : kFloor, l = is ? lm[w * G + hd] : 0.f;
            const float f = join_parts<8>(M, l, whole);
            if (is) fm[w * G + hd] *= f;
            if (is && w == 0) {
                if (whole) {
                    g.lse[head0 + hd] = (M + log2f(l)) * kLn2;
                } else {
                    part[G * D + hd] = M;
                    part[G * D + G + hd] = l;
                }
            }
        }
        __syncthreads();
        float* out = whole ? g.O + head0 * D : part;
        for (int i = tid; i < G * D; i += kThreads) {
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) o = fmaf(om[w * G * D + i], fm[w * G + i / D], o);
            out[i] = o;
        }
        __syncthreads();                             // the rings may be filled again
        at = unit0 + to;
    }
}

// One unit and head a CTA: joins the parts of a unit that several CTAs hold,
// and writes the outputs of empty sequences.  A part is read by D/4 threads,
// four elements each, kLots parts at a time.  Until pdl_wait only the caller's
// inputs are read: the first kernel's CTAs let this one start after their own
// wait, when whatever wrote the inputs is done.
// Many threads where there are few units, which have many parts each.
template <int D, int kJoinThreads> __global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ Args g)
{
    constexpr int kLots = kJoinThreads / (D / 4), kJoinWarps = kJoinThreads / 32;
    constexpr int kParts = kJoinThreads / 2;         // parts whose factors are formed at once
    __shared__ float4 s_o[kLots][D / 4];
    __shared__ float s_f[kParts], s_red[2][kJoinWarps];
    const int tid = threadIdx.x, e = tid % (D / 4), lot = tid / (D / 4), lane = tid & 31, G = g.s.G;
    const int64_t bh = blockIdx.x / G;
    const int hd = blockIdx.x % G, b = int(bh / g.s.Hkv), h = int(bh % g.s.Hkv);
    const int64_t out = (int64_t)b * g.s.Hq + h * G + hd;
    const Row row(g);
    int before = 0;
#pragma unroll 4
    for (int i = lane; i < b; i += 32) before += tiles_of(g, i);
    const int n = tiles_of(g, b), unit0 = warp_sum_int(before) * g.s.Hkv + n * h;
    int c0 = 0, c1 = 0;                              // the unit's first and last CTA
    if (n > 0) {
        c0 = row.cta_of(unit0);
        c1 = row.cta_of(unit0 + n - 1);
        while (c0 + 1 < row.ctas && row.begin(c0 + 1) < unit0 + n && border(row.begin(c0 + 1) - unit0, n) == 0) ++c0;
        while (row.begin(c1) > unit0 && border(row.begin(c1) - unit0, n) == n) --c1;
    }
    pdl_wait();
    pdl_trigger();
    if (n == 0) {
        if (lot == 0) reinterpret_cast<float4*>(g.O + out * D)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tid == 0) g.lse[out] = -INFINITY;
        return;
    }
    if (c0 == c1) return;                            // one CTA had all of it
    // CTA c0 holds the unit's first tiles, in its second part; the others begin
    // inside the unit, in their first.
    const size_t stride = part_floats(g.s);
    auto part_of = [&](int c) { return g.parts + (2 * (int64_t)c + (c == c0)) * stride; };
    float M = kFloor, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = c0; p0 <= c1; p0 += kParts) {      // (a second turn only with more than kParts CTAs on a unit)
        const int m = min(kParts, c1 - p0 + 1);
        float r = kFloor, s = 0.f;
        if (tid < m) {
            const float* mine = part_of(p0 + tid) + G * D + hd;
            r = mine[0];
            s = mine[G];
        }
        float top = r;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        if (lane == 0) s_red[0][tid / 32] = top;
        __syncthreads();
        top = M;
#pragma unroll
        for (int w = 0; w < kParts / 32; ++w) top = fmaxf(top, s_red[0][w]);
        const float before = l * ex2(M - top);
        M = top;
        float sum = s * ex2(r - top);
        if (tid < m) s_f[tid] = sum;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        if (lane == 0) s_red[1][tid / 32] = sum;
        __syncthreads();
        l = before;
#pragma unroll
        for (int w = 0; w < kParts / 32; ++w) l += s_red[1][w];
        const float inv = l == 0.f ? 0.f : 1.f / l, back = before * inv;
        o.x *= back; o.y *= back; o.z *= back; o.w *= back;
#pragma unroll 8
        for (int c = lot; c < m; c += kLots) {
            const float4 v = reinterpret_cast<const float4*>(part_of(p0 + c) + hd * D)[e];
            const float x = s_f[c] * inv;
            o.x = fmaf(v.x, x, o.x);
            o.y = fmaf(v.y, x, o.y);
            o.z = fmaf(v.z, x, o.z);
            o.w = fmaf(v.w, x, o.w);
        }
        __syncthreads();                             // s_f may be written again
    }
    s_o[lot][e] = o;
    __syncthreads();
    if (tid >= D) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kLots; ++i) sum += reinterpret_cast<const float*>(s_o[i])[tid];
    g.O[out * D + tid] = l == 0.f ? NAN : sum;       // (all scores below float32)
    if (tid == 0) g.lse[out] = (M + log2f(l)) * kLn2;
}

template <typename TIn, int D, int CACHE> cudaError_t launch(const Args& g, cudaStream_t st)
{
    auto k = paged_dense_kernel<TIn, D, CACHE>;
    const size_t smem = dense_smem<D>(g.s);
    if (cudaError_t e = allow_smem(k, (int)smem)) return e;
    if (cudaError_t e = launch_pdl(k, dim3((unsigned)g.grid), dim3(kThreads), smem, st, g)) return e;
    const dim3 grid((unsigned)(g.s.B * g.s.Hq));
    return g.s.B * g.s.Hkv < 64 ? launch_pdl(paged_join_kernel<D, 512>, grid, dim3(512), 0, st, g)
                                : launch_pdl(paged_join_kernel<D, 128>, grid, dim3(128), 0, st, g);
}

template <typename TIn, int D> cudaError_t by_cache(const Args& g, cudaStream_t st)
{
    return g.s.cache_dtype == HGA_INT8 ? launch<TIn, D, HGA_INT8>(g, st) : launch<TIn, D, HGA_E4M3>(g, st);
}

}  // namespace

// The tiles of all units are counted in 32 bits.
bool paged_dense_fits(const PagedShape& s)
{
    return (int64_t)s.B * s.Hkv * (kOpen + kPerChunk * (int64_t)s.max_chunks) <= INT32_MAX - kLeast;
}

size_t paged_dense_workspace(const PagedShape& s) { return sizeof(float) * part_floats(s) * 2 * kPerSm * (size_t)sm_count(); }

cudaError_t launch_paged_dense(const PagedShape& s, const hga_paged_cache& c, const int32_t* pos, const void* q, float* O,
                               float* lse, void* workspace, cudaStream_t st)
{
    const Args g{s, c, pos, q, O, lse, static_cast<float*>(workspace), kPerSm * sm_count()};
    if (s.dtype == HGA_BF16) return s.d == 128 ? by_cache<__nv_bfloat16, 128>(g, st) : by_cache<__nv_bfloat16, 64>(g, st);
    return s.d == 128 ? by_cache<float, 128>(g, st) : by_cache<float, 64>(g, st);
}

HGA_CHECK_WORD_READER(check_word_paged_dense)

}  // namespace hga
