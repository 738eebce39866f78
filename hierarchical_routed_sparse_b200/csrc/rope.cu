// rope.cu -- the position rotation between the projections' layout and the
// attention's, and its gradient.
//
// forward   y [B][H][T][d]  = R(pos0 + t) x [B][T][H][d]   (x by strides)
// backward  dx [B][T][H][d] = R(pos0 + t)^T dy [B][H][T][d]
// One kernel does both: a strided row is read, turned and written to another
// strided row, with the transpose of the layout and the change of type on
// the way, so each element crosses memory once in each direction.
//
// The kernel is bound by those bytes: four segments of 4096 tokens, 32 heads,
// d 128, float32 to bf16 (405 MB) take 60.2 us, 6.7 TB/s.  A thread owns one 16-element unit
// (rope.cuh) of one token, loads the unit's cosines and sines once and then
// runs kHeads heads on them, all their loads issued before the first is used.
#include "rope.cuh"

namespace hga {
namespace {

using namespace rope;

constexpr int kThreads = 256;
// Heads a thread runs on one set of angles: more of them load the angles less
// often, fewer make more CTAs (2048 tokens, 32 heads, float32 to bf16: 9.8, 9.6,
// 11.1 and 11.6 us with 1, 2, 4 and 8; four segments of 4096: 60.1 to 61.8).
constexpr int kHeads = 2;

struct RowStrides {
    int64_t batch, token, head;
};

template <typename TIn, typename TOut, int D, bool BACK>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const TIn* __restrict__ src, RowStrides si, TOut* __restrict__ dst, RowStrides so,
            const float* __restrict__ table, int64_t T, int H, int64_t pos0, int rot, bool interleaved,
            int64_t tiles)
{
    constexpr int kUnits = D / 16, kTokens = kThreads / kUnits;
    pdl_wait();
    pdl_trigger();
    const int u = threadIdx.x % kUnits;
    const int64_t b = blockIdx.x / tiles;
    const int64_t t = (blockIdx.x % tiles) * kTokens + threadIdx.x / kUnits;
    if (t >= T) return;
    const int h0 = blockIdx.y * kHeads;
    const Unit un = unit_of(u, rot, interleaved);
    const TIn* in = src + b * si.batch + t * si.token;
    Raw8<TIn> ra[kHeads], rb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (h0 + i < H) {
            const TIn* p = in + (h0 + i) * si.head;
            ra[i].load(p + un.a);
            rb[i].load(p + un.b);
        }
    }
    Angles ang;
    if (un.turned) ang.load(table + (pos0 + t) * rot, u, rot);
    TOut* out = dst + b * so.batch + t * so.token;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        if (h0 + i < H) {
            float x[16];
            ra[i].widen(x);
            rb[i].widen(x + 8);
            if (un.turned) turn<BACK>(x, ang, interleaved);
            TOut* p = out + (h0 + i) * so.head;
            store8(p + un.a, x);
            store8(p + un.b, x + 8);
        }
    }
}

template <typename TIn, typename TOut, int D>
cudaError_t launch(const RopeShape& s, bool back, const void* src, const float* table, void* dst, cudaStream_t st)
{
    constexpr int kTokens = kThreads / (D / 16);
    const int64_t tiles = (s.T + kTokens - 1) / kTokens;
    const dim3 grid((unsigned)(s.B * tiles), (unsigned)((s.H + kHeads - 1) / kHeads));
    const RowStrides x{s.x_batch, s.x_token, s.x_head}, y{(int64_t)s.H * s.T * D, D, s.T * D};
    auto* in = static_cast<const TIn*>(src);
    auto* out = static_cast<TOut*>(dst);
    if (back)
        return launch_pdl(rope_kernel<TIn, TOut, D, true>, grid, dim3(kThreads), 0, st, in, y, out, x, table, s.T,
                          s.H, s.pos0, s.rot, s.interleaved, tiles);
    return launch_pdl(rope_kernel<TIn, TOut, D, false>, grid, dim3(kThreads), 0, st, in, x, out, y, table, s.T, s.H,
                      s.pos0, s.rot, s.interleaved, tiles);
}

template <typename TIn, typename TOut>
cudaError_t by_dim(const RopeShape& s, bool back, const void* src, const float* table, void* dst, cudaStream_t st)
{
    return s.d == 128 ? launch<TIn, TOut, 128>(s, back, src, table, dst, st)
                      : launch<TIn, TOut, 64>(s, back, src, table, dst, st);
}

}  // namespace

bool rope_grid_fits(const RopeShape& s)
{
    const int64_t tokens = kThreads / (s.d / 16);
    return s.B * ((s.T + tokens - 1) / tokens) <= INT32_MAX && (s.H + kHeads - 1) / kHeads <= 65535;
}

cudaError_t launch_rope(const RopeShape& s, bool back, const void* src, const float* table, void* dst,
                        cudaStream_t st)
{
    const int in = back ? s.y_dtype : s.x_dtype, out = back ? s.x_dtype : s.y_dtype;
    if (in == HGA_BF16)
        return out == HGA_BF16 ? by_dim<__nv_bfloat16, __nv_bfloat16>(s, back, src, table, dst, st)
                               : by_dim<__nv_bfloat16, float>(s, back, src, table, dst, st);
    return out == HGA_BF16 ? by_dim<float, __nv_bfloat16>(s, back, src, table, dst, st)
                           : by_dim<float, float>(s, back, src, table, dst, st);
}

}  // namespace hga
