// forge_embedding.cu -- the embedding lookup with scaling, its gradient summed
// by tokens, and that gradient fused with the AdamW step.
//
//   Y[t] = s W[id_t];   dW[r] = s sum_{t : id_t = r} dY[t]
// The gradient of a row is the sum over its tokens in token order, so results
// do not depend on scheduling.  A negative id is padding: its output row is
// zero and its gradient row is left out.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "forge.h"
#include "forge_device.h"
#include "forge_kernel.cuh"

namespace forge {
namespace embedding {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p, int64_t i)
{
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ void store1(float* p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, int64_t i, float x)
{
    p[i] = __float2bfloat16_rn(x);
}

// The row of token t: -1 for padding.  An id past the vocabulary is recorded
// in the status word and taken as padding.
__device__ __forceinline__ int64_t id_of(const void* ids, bool wide, int64_t t, int64_t V,
                                         int* status)
{
    const int64_t r = wide ? static_cast<const int64_t*>(ids)[t]
                           : static_cast<const int32_t*>(ids)[t];
    if (r < 0) return -1;
    if (r >= V) {
        *reinterpret_cast<volatile int*>(status) = kDevInvalidArg;
        return -1;
    }
    return r;
}

// ------------------------------------------------------------------ lookup

__device__ __forceinline__ void to_float(const uint4& u, float (&x)[4])
{
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void to_float(const uint4& u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4)
        __stcs(reinterpret_cast<float4*>(p + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[N])
{
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (N == 8)
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
}

// One warp per (token, span of columns), four 16-byte loads (VEC: rows of
// whole vectors) or eight single ones in flight per lane, so that even a
// decode step's few tokens spread over the SMs.  Bound by HBM; W's rows keep
// their place in L2 (frequent tokens), Y streams past it.
template <typename W, bool VEC>
struct Span {
    static constexpr int vec = VEC ? 16 / static_cast<int>(sizeof(W)) : 1;
    static constexpr int flight = VEC ? 4 : 8;
    static constexpr int columns = 32 * vec * flight;
};

template <typename W, typename Y, bool VEC>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_kernel(const void* ids, bool wide, const W* __restrict__ w, Y* __restrict__ y,
                           int64_t T, int64_t V, int64_t D, float scale, int* status)
{
    using S = Span<W, VEC>;
    const int lane = threadIdx.x & 31;
    const int64_t spans = (D + S::columns - 1) / S::columns;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
         u < T * spans; u += warps) {
        const int64_t t = u / spans, c0 = (u - t * spans) * S::columns + lane * S::vec;
        const int64_t r = id_of(ids, wide, t, V, status);
        const W* src = w + r * D;
        Y* dst = y + t * D;
        if constexpr (VEC) {
            uint4 v[S::flight];
#pragma unroll
            for (int i = 0; i < S::flight; ++i) {
                const int64_t c = c0 + i * 32 * S::vec;
                v[i] = r >= 0 && c < D ? __ldg(reinterpret_cast<const uint4*>(src + c))
                                       : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < S::flight; ++i) {
                const int64_t c = c0 + i * 32 * S::vec;
                float x[S::vec];
                to_float(v[i], x);
#pragma unroll
                for (int k = 0; k < S::vec; ++k) x[k] *= scale;
                if (c < D) store_vec<S::vec>(dst + c, x);
            }
        } else {
            float x[S::flight];
#pragma unroll
            for (int i = 0; i < S::flight; ++i) {
                const int64_t c = c0 + i * 32;
                x[i] = r >= 0 && c < D ? load1(src, c) * scale : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < S::flight; ++i)
                if (c0 + i * 32 < D) store1(dst, c0 + i * 32, x[i]);
        }
    }
}

// ------------------------------------------------------------------ order of the tokens

// The tokens are ordered by vocabulary row, in token order within a row, by
// one launch without atomics.  Row r belongs to block r mod kClasses (the
// frequent tokens of a vocabulary sorted by frequency spread over the
// blocks).  Each block reads all ids twice: the first time to count its own
// tokens and those of the blocks before it, which gives its place in the
// order, the second time to collect its own; a warp reads a contiguous range,
// so ranks within a ballot keep the token order.  Then the block sorts its
// list by local row r / kClasses, five bits at a time: every warp counts its
// part of the list into its own 32 counters (equal digits of a warp
// instruction are found by a match, their lowest lane adds), a scan over the
// 32 x 32 counters gives the places, and the items are moved in order.
// Reading all ids in every block costs T x kClasses reads from L2, a few
// percent of the T x D gradient elements that follow.
constexpr int kClassBits = 7;
constexpr int kClasses = 1 << kClassBits;
constexpr int kOrderThreads = 1024;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int kDigitBits = 5;
constexpr int kOrderShared = 4096;  // items of a list that is sorted in shared memory
constexpr int kOrderSmem = 2 * kOrderShared * static_cast<int>(sizeof(int2));

// Token order: order[i] the token at place i, seg[r] the places [x, y) of row
// r, *total the number of tokens that are not padding.  listA, listB: room for
// T items where a block's list exceeds shared memory.
struct Order {
    int32_t* order;
    int2* seg;
    int32_t* total;
    int2* listA;
    int2* listB;
};

__global__ void __launch_bounds__(kOrderThreads, 1)
    forge_token_order_kernel(const void* ids, bool wide, int64_t T, int64_t V, Order o, int* status)
{
    extern __shared__ int2 s_list[];
    __shared__ uint32_t s_count[kOrderThreads];  // digit-major: [digit][warp]
    __shared__ uint32_t s_own[kOrderWarps], s_less[kOrderWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u;
    const int32_t cls = blockIdx.x;

    // rows without a token
    const int64_t local_rows = (V + kClasses - 1) / kClasses;
    for (int64_t k = threadIdx.x; k < local_rows; k += kOrderThreads)
        if (k * kClasses + cls < V) o.seg[k * kClasses + cls] = make_int2(0, 0);

    // count
    const int64_t chunk = (T + kOrderThreads - 1) / kOrderThreads * 32;
    const int64_t lo = warp * chunk, hi = lo + chunk < T ? lo + chunk : T;
    uint32_t own = 0, less = 0;
#pragma unroll 8
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int64_t r = id_of(ids, wide, i, V, status);
        const int32_t c = static_cast<int32_t>(r) & (kClasses - 1);
        own += r >= 0 && c == cls;
        less += r >= 0 && c < cls;
    }
    own = __reduce_add_sync(0xffffffffu, own);
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) {
        s_own[warp] = own;
        s_less[warp] = less;
    }
    __syncthreads();
    int32_t base = 0, n = 0, at = 0;
    for (int w = 0; w < kOrderWarps; ++w) {
        base += s_less[w];
        if (w == warp) at = n;
        n += s_own[w];
    }
    if (cls == kClasses - 1 && threadIdx.x == 0) *o.total = base + n;

    // collect
    const bool shared = n <= kOrderShared;
    int2* src = shared ? s_list : o.listA + base;
    int2* dst = shared ? s_list + kOrderShared : o.listB + base;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * 8) {
        int32_t r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            r[u] = i < hi ? static_cast<int32_t>(id_of(ids, wide, i, V, status)) : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool mine = r[u] >= 0 && (r[u] & (kClasses - 1)) == cls;
            const uint32_t all = __ballot_sync(0xffffffffu, mine);
            if (mine)
                src[at + __popc(all & before)] =
                    make_int2(r[u] >> kClassBits, static_cast<int32_t>(i0 + 32 * u + lane));
            at += __popc(all);
        }
    }
    __syncthreads();

    // sort by local row
    const int32_t part = (n + kOrderThreads - 1) / kOrderThreads * 32;
    const int32_t p0 = warp * part < n ? warp * part : n;
    const int32_t p1 = p0 + part < n ? p0 + part : n;
    for (int shift = 0; (local_rows - 1) >> shift; shift += kDigitBits) {
        s_count[threadIdx.x] = 0;
        __syncthreads();
        for (int32_t i0 = p0; i0 < p1; i0 += 32) {
            const bool in = i0 + lane < p1;
            const uint32_t d =
                in ? (static_cast<uint32_t>(src[i0 + lane].x) >> shift) & 31u : 32u;
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            if (in && (same & before) == 0) s_count[d * 32 + warp] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // exclusive scan over (digit, warp)
        const uint32_t v = s_count[threadIdx.x];
        uint32_t inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += up;
        }
        if (lane == 31) s_own[warp] = inc;
        __syncthreads();
        uint32_t ahead = 0;
        for (int w = 0; w < warp; ++w) ahead += s_own[w];
        s_count[threadIdx.x] = ahead + inc - v;
        __syncthreads();
        for (int32_t i0 = p0; i0 < p1; i0 += 32) {
            const bool in = i0 + lane < p1;
            const int2 item = in ? src[i0 + lane] : make_int2(0, 0);
            const uint32_t d = in ? (static_cast<uint32_t>(item.x) >> shift) & 31u : 32u;
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            if (in) dst[s_count[d * 32 + warp] + __popc(same & before)] = item;
            __syncwarp();
            if (in && (same & before) == 0) s_count[d * 32 + warp] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        int2* t = src;
        src = dst;
        dst = t;
    }

    for (int32_t i = threadIdx.x; i < n; i += kOrderThreads) {
        const int2 item = src[i];
        o.order[base + i] = item.y;
        int2* s = &o.seg[static_cast<int64_t>(item.x) * kClasses + cls];
        if (i == 0 || src[i - 1].x != item.x) s->x = base + i;
        if (i == n - 1 || src[i + 1].x != item.x) s->y = base + i + 1;
    }
}

// ------------------------------------------------------------------ sums

// A warp sums 256 columns of a row: lane l holds columns 4 l .. 4 l + 3 and
// 128 + 4 l .. of the slice, so that loads and stores are whole vectors
// (VEC: D a multiple of 4, every base aligned to four elements), or columns
// l + 32 k one by one.
constexpr int kSlice = 256;
constexpr int kPer = kSlice / 32;

template <bool VEC>
__device__ __forceinline__ int64_t column(int64_t slice, int lane, int k)
{
    return slice * kSlice + (VEC ? (k >> 2) * 128 + 4 * lane + (k & 3) : 32 * k + lane);
}

__device__ __forceinline__ void load4(const float* p, float* o)
{
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    o[0] = v.x;
    o[1] = v.y;
    o[2] = v.z;
    o[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* o)
{
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    o[0] = __uint_as_float(u.x << 16);
    o[1] = __uint_as_float(u.x & 0xFFFF0000u);
    o[2] = __uint_as_float(u.y << 16);
    o[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

template <bool VEC, typename G>
__device__ __forceinline__ void load_slice(const G* row, int64_t slice, int64_t D, int lane,
                                           float (&x)[kPer])
{
    if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = column<true>(slice, lane, 4 * h);
            if (c < D)
                load4(row + c, x + 4 * h);
            else
                x[4 * h] = x[4 * h + 1] = x[4 * h + 2] = x[4 * h + 3] = 0.0f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t c = column<false>(slice, lane, k);
            x[k] = c < D ? load1(row, c) : 0.0f;
        }
    }
}

// acc += the slices of n rows of a [*, D] array, the i-th being row of(i), in
// that order, kFlight rows in flight.
constexpr int kFlight = 4;
template <bool VEC, typename G, typename F>
__device__ __forceinline__ void add_rows(const G* base, int32_t n, F of, int64_t slice, int64_t D,
                                         int lane, float (&acc)[kPer])
{
    for (int32_t i0 = 0; i0 < n; i0 += 32) {
        const int32_t m = n - i0 < 32 ? n - i0 : 32;
        const int64_t mine = lane < m ? of(i0 + lane) : 0;
        for (int32_t j0 = 0; j0 < m; j0 += kFlight) {
            float x[kFlight][kPer];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const int64_t r = __shfl_sync(0xffffffffu, mine, (j0 + u) & 31);
                if (j0 + u < m)
                    load_slice<VEC>(base + r * D, slice, D, lane, x[u]);
                else
#pragma unroll
                    for (int k = 0; k < kPer; ++k) x[u][k] = 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] += x[u][k];
        }
    }
}

// A row with more than P = 2^piece_bits tokens (a frequent token, or one that
// fills the batch) is summed in pieces: its places are cut at the multiples
// of P, and a block of this kernel adds one piece's tokens, eight warps a
// part each, into a row of `partial`.  Within the P places b P .. there are at
// most two such pieces: one of a row that goes on from the places before
// (slot 2 b) and one of a row that starts here (slot 2 b + 1).
template <bool VEC, typename G>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_pieces_kernel(const G* dY, const void* ids, bool wide, int64_t D, Order o,
                                  int32_t piece_bits, float* partial)
{
    __shared__ float sh[kThreads / 32][kSlice];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t slices = static_cast<int32_t>((D + kSlice - 1) / kSlice);
    const int64_t slice = blockIdx.x % slices;
    const int32_t b = blockIdx.x / slices, P = 1 << piece_bits;
    const int32_t total = *o.total;
    const int32_t p0 = b << piece_bits;
    if (p0 >= total) return;
    const int32_t p1 = total - p0 < P ? total : p0 + P;
    int64_t row = -1;
    for (int which = 0; which < 2; ++which) {
        const int32_t t = o.order[which ? p1 - 1 : p0];
        const int64_t r = wide ? static_cast<const int64_t*>(ids)[t]
                               : static_cast<const int32_t*>(ids)[t];
        if (r == row) break;
        row = r;
        const int2 s = o.seg[r];
        if (s.y - s.x <= P) continue;
        const int32_t a = s.x > p0 ? s.x : p0, e = s.y < p1 ? s.y : p1;
        const int32_t per = (e - a + kThreads / 32 - 1) / (kThreads / 32);
        const int32_t wa = a + warp * per < e ? a + warp * per : e;
        const int32_t we = wa + per < e ? wa + per : e;
        float acc[kPer] = {};
        add_rows<VEC>(dY, we - wa, [&](int32_t i) { return o.order[wa + i]; }, slice, D, lane, acc);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kPer; ++k) sh[warp][column<VEC>(0, lane, k)] = acc[k];
        __syncthreads();
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) x += sh[w][threadIdx.x];
        const int64_t c = slice * kSlice + threadIdx.x;
        const int64_t slot = 2 * static_cast<int64_t>(b) + (s.x >= p0 ? 1 : 0);
        if (c < D) partial[slot * D + c] = x;
    }
}

enum { SUM_STORE = 0, SUM_ADD = 1, SUM_ADAMW = 2 };

// One warp per (row, slice), the slices of a row side by side: the sum of the
// row's tokens (or of its pieces), then the store, the addition to dW or the
// AdamW step.  Bound by HBM: dW written, or W, m, v read and written, once.
template <typename G, int MODE, int ST, bool VEC>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_grad_kernel(const G* dY, int64_t V, int64_t D, float scale, float* dW, Order o,
                                int32_t piece_bits, const float* partial, const Params p)
{
    const int lane = threadIdx.x & 31;
    const int64_t slices = (D + kSlice - 1) / kSlice;
    const int64_t units = V * slices;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    const int32_t P = 1 << piece_bits;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
         u < units; u += warps) {
        const int64_t row = u / slices, slice = u - row * slices;
        const int2 s = o.seg ? o.seg[row] : make_int2(0, 0);
        const int32_t n = s.y - s.x;
        if (MODE == SUM_ADD && n == 0) continue;
        float g[kPer] = {};
        if (n > P) {
            const int32_t b0 = s.x >> piece_bits, b1 = (s.y - 1) >> piece_bits;
            add_rows<VEC>(
                partial, b1 - b0 + 1,
                [&](int32_t i) { return 2 * static_cast<int64_t>(b0 + i) + (i == 0 ? 1 : 0); },
                slice, D, lane, g);
        } else if (n > 0) {
            add_rows<VEC>(dY, n, [&](int32_t i) { return o.order[s.x + i]; }, slice, D, lane, g);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) g[k] *= scale;
#pragma unroll
        for (int h = 0; h < (VEC ? 2 : kPer); ++h) {
            const int64_t c = column<VEC>(slice, lane, VEC ? 4 * h : h);
            if (c >= D) continue;
            const int64_t at = row * D + c;
            if constexpr (VEC) {
                float* gh = g + 4 * h;
                if constexpr (MODE == SUM_ADAMW) {
                    float w[4], a[4], b[4];
                    StateIO<ST_F32>::ld4(p.W, at, w);
                    StateIO<ST>::ld4(p.s1, at, a);
                    StateIO<ST>::ld4(p.s2, at, b);
                    step4<OP_ADAMW>(p, gh, w, a, b);
                    StateIO<ST_F32>::st4(p.W, at, w);
                    StateIO<ST>::st4(p.s1, at, a);
                    StateIO<ST>::st4(p.s2, at, b);
                } else {
                    if constexpr (MODE == SUM_ADD) {
                        float d[4];
                        StateIO<ST_F32>::ld4(dW, at, d);
#pragma unroll
                        for (int i = 0; i < 4; ++i) gh[i] += d[i];
                    }
                    StateIO<ST_F32>::st4(dW, at, gh);
                }
            } else if constexpr (MODE == SUM_ADAMW) {
                float gs[4] = {g[h], g[h], g[h], g[h]}, w[4], a[4], b[4];
                w[0] = w[1] = w[2] = w[3] = StateIO<ST_F32>::ld(p.W, at);
                a[0] = a[1] = a[2] = a[3] = StateIO<ST>::ld(p.s1, at);
                b[0] = b[1] = b[2] = b[3] = StateIO<ST>::ld(p.s2, at);
                step4<OP_ADAMW>(p, gs, w, a, b);
                StateIO<ST_F32>::st(p.W, at, w[0]);
                StateIO<ST>::st(p.s1, at, a[0]);
                StateIO<ST>::st(p.s2, at, b[0]);
            } else {
                dW[at] = MODE == SUM_ADD ? dW[at] + g[h] : g[h];
            }
        }
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : (t == FORGE_I64 ? 8 : 4); }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }
bool is_id(forge_dtype t) { return t == FORGE_I32 || t == FORGE_I64; }

forge_status check_sizes(int64_t T, int64_t V, int64_t D, float scale)
{
    if (T < 0 || V < 1 || D < 1 || T > INT32_MAX || V > INT32_MAX || D > INT32_MAX)
        return FORGE_ERR_INVALID_ARG;
    return std::isfinite(scale) ? FORGE_OK : FORGE_ERR_INVALID_ARG;
}

forge_status check_grad(const void* dY, forge_dtype dy_dtype, const void* ids,
                        forge_dtype id_dtype, int64_t T)
{
    if (T > 0 && (!dY || !ids)) return FORGE_ERR_INVALID_ARG;
    if (!is_float(dy_dtype) || !is_id(id_dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    return FORGE_OK;
}

// Tokens of a row summed by one warp; longer rows in pieces of as many.  A
// warp adds P rows one after the other, and T / P partial sums where one
// token fills the batch, so P grows with the square root of T.
int32_t piece_bits_of(int64_t T)
{
    int32_t bits = 6;
    while ((int64_t{4} << (2 * bits)) < T) ++bits;
    return bits;
}

// The order kernel's shared memory, allowed once per device.
cudaError_t allow_order_smem()
{
    static unsigned long long done = 0;  // one bit per device ordinal < 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(forge_token_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kOrderSmem);
    if (e == cudaSuccess) __atomic_fetch_or(&done, bit, __ATOMIC_ACQ_REL);
    return e;
}

template <typename G, int MODE, int ST, bool VEC>
cudaError_t launch_grad(const G* dY, const void* ids, bool wide, int64_t T, int64_t V, int64_t D,
                        float scale, float* dW, const Params& p, int sms, cudaStream_t s)
{
    const int64_t slices = (D + kSlice - 1) / kSlice;
    const int32_t bits = piece_bits_of(T);
    const int64_t pieces = (T + (int64_t{1} << bits) - 1) >> bits;
    Order o{};
    float* partial = nullptr;
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
        const int64_t order_b = up(T * 4), list_b = up(T * 8), seg_b = up(V * 8);
        const int64_t partial_b = up(2 * pieces * D * 4);
        e = scratch_alloc(&scratch, 256 + order_b + 2 * list_b + seg_b + partial_b, s);
        if (e != cudaSuccess) return e;
        uint8_t* at = static_cast<uint8_t*>(scratch);
        o.total = reinterpret_cast<int32_t*>(at);
        o.order = reinterpret_cast<int32_t*>(at += 256);
        o.listA = reinterpret_cast<int2*>(at += order_b);
        o.listB = reinterpret_cast<int2*>(at += list_b);
        o.seg = reinterpret_cast<int2*>(at += list_b);
        partial = reinterpret_cast<float*>(at += seg_b);
        e = allow_order_smem();
        if (e == cudaSuccess) {
            forge_token_order_kernel<<<kClasses, kOrderThreads, kOrderSmem, s>>>(ids, wide, T, V, o,
                                                                               p.status);
            forge_embedding_pieces_kernel<VEC>
                <<<static_cast<unsigned>(slices * pieces), kThreads, 0, s>>>(dY, ids, wide, D, o,
                                                                           bits, partial);
        }
    }
    if (e == cudaSuccess) {
        const int64_t want = (V * slices + kThreads / 32 - 1) / (kThreads / 32);
        const int blocks = static_cast<int>(want < 8LL * sms ? want : 8LL * sms);
        forge_embedding_grad_kernel<G, MODE, ST, VEC>
            <<<blocks, kThreads, 0, s>>>(dY, V, D, scale, dW, o, bits, partial, p);
        e = cudaGetLastError();
    }
    if (scratch) {
        const cudaError_t fe = scratch_free(scratch, s);
        if (e == cudaSuccess) e = fe;
    }
    return e;
}

template <int MODE, int ST>
cudaError_t grad(const void* dY, forge_dtype dy_dtype, const void* ids, forge_dtype id_dtype,
                 int64_t T, int64_t V, int64_t D, float scale, float* dW, const Params& p, int sms,
                 cudaStream_t s)
{
    const bool wide = id_dtype == FORGE_I64;
    const uintptr_t sa = ST == ST_BF16 ? 8 : 16;
    const bool vec = D % 4 == 0 && aligned(dY, 4 * size_of(dy_dtype)) &&
                     (MODE == SUM_ADAMW ? aligned(p.W, 16) && aligned(p.s1, sa) && aligned(p.s2, sa)
                                        : aligned(dW, 16));
    auto go = [&](auto* d) {
        using G = std::remove_cv_t<std::remove_pointer_t<decltype(d)>>;
        return vec ? launch_grad<G, MODE, ST, true>(d, ids, wide, T, V, D, scale, dW, p, sms, s)
                   : launch_grad<G, MODE, ST, false>(d, ids, wide, T, V, D, scale, dW, p, sms, s);
    };
    return dy_dtype == FORGE_F32 ? go(static_cast<const float*>(dY))
                                 : go(static_cast<const __nv_bfloat16*>(dY));
}

}  // namespace embedding
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_embedding(const void* ids, forge_dtype id_dtype, int64_t T,
                                        const void* W, forge_dtype w_dtype, int64_t V, int64_t D,
                                        float scale, void* Y, forge_dtype y_dtype,
                                        forge_stream_t stream)
{
    using namespace embedding;
    if (!W || (T > 0 && (!ids || !Y))) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(T, V, D, scale);
    if (st != FORGE_OK) return st;
    if (!is_id(id_dtype) || !is_float(w_dtype) || !is_float(y_dtype))
        return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(ids, size_of(id_dtype)) || !aligned(W, size_of(w_dtype)) ||
        !aligned(Y, size_of(y_dtype)))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (T == 0) return FORGE_OK;
    const void* ptrs[] = {ids, W, Y};
    if ((st = device_resident(ptrs, 3)) != FORGE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* status = device_status_word();
    auto go = [&](auto* w, auto* y) {
        using A = std::remove_cv_t<std::remove_pointer_t<decltype(w)>>;
        using B = std::remove_pointer_t<decltype(y)>;
        constexpr int64_t per = Span<A, true>::vec;
        const bool vec = D % per == 0 && aligned(w, 16) && aligned(y, sizeof(B) * per < 16 ? 8 : 16);
        const int64_t columns = vec ? Span<A, true>::columns : Span<A, false>::columns;
        const int64_t units = T * ((D + columns - 1) / columns);
        const int64_t want = (units + kThreads / 32 - 1) / (kThreads / 32);
        const int blocks = static_cast<int>(want < 8LL * sms ? want : 8LL * sms);
        if (vec)
            forge_embedding_kernel<A, B, true><<<blocks, kThreads, 0, s>>>(
                ids, id_dtype == FORGE_I64, w, y, T, V, D, scale, status);
        else
            forge_embedding_kernel<A, B, false><<<blocks, kThreads, 0, s>>>(
                ids, id_dtype == FORGE_I64, w, y, T, V, D, scale, status);
    };
    auto out = [&](auto* w) {
        if (y_dtype == FORGE_F32)
            go(w, static_cast<float*>(Y));
        else
            go(w, static_cast<__nv_bfloat16*>(Y));
    };
    if (w_dtype == FORGE_F32)
        out(static_cast<const float*>(W));
    else
        out(static_cast<const __nv_bfloat16*>(W));
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_embedding_grad(const void* dY, forge_dtype dy_dtype, const void* ids,
                                             forge_dtype id_dtype, int64_t T, int64_t V, int64_t D,
                                             float scale, float* dW, int32_t accumulate,
                                             forge_stream_t stream)
{
    using namespace embedding;
    if (!dW) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(T, V, D, scale);
    if (st != FORGE_OK || (st = check_grad(dY, dy_dtype, ids, id_dtype, T)) != FORGE_OK) return st;
    if (!aligned(dY, size_of(dy_dtype)) || !aligned(ids, size_of(id_dtype)) || !aligned(dW, 4))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* ptrs[] = {T > 0 ? dY : nullptr, T > 0 ? ids : nullptr, dW};
    if ((st = device_resident(ptrs, 3)) != FORGE_OK) return st;
    Params p{};
    p.status = device_status_word();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        accumulate ? grad<SUM_ADD, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, dW, p, sms, s)
                   : grad<SUM_STORE, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, dW, p, sms, s);
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_embedding_adamw(const void* dY, forge_dtype dy_dtype,
                                              const void* ids, forge_dtype id_dtype, int64_t T,
                                              int64_t V, int64_t D, float scale, float* W, void* m,
                                              void* v, forge_dtype state_dtype, float lr,
                                              float beta1, float beta2, float eps, float wd,
                                              int64_t step, forge_stream_t stream)
{
    using namespace embedding;
    if (!W || !m || !v) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(T, V, D, scale);
    if (st != FORGE_OK || (st = check_grad(dY, dy_dtype, ids, id_dtype, T)) != FORGE_OK) return st;
    if (!is_float(state_dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    Params p{};
    if ((st = adamw_params(&p, lr, beta1, beta2, eps, wd, step)) != FORGE_OK) return st;
    if (!aligned(dY, size_of(dy_dtype)) || !aligned(ids, size_of(id_dtype)) || !aligned(W, 4) ||
        !aligned(m, size_of(state_dtype)) || !aligned(v, size_of(state_dtype)))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* ptrs[] = {T > 0 ? dY : nullptr, T > 0 ? ids : nullptr, W, m, v};
    if ((st = device_resident(ptrs, 5)) != FORGE_OK) return st;
    p.W = W;
    p.s1 = m;
    p.s2 = v;
    p.status = device_status_word();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        state_dtype == FORGE_F32
            ? grad<SUM_ADAMW, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, nullptr, p, sms, s)
            : grad<SUM_ADAMW, ST_BF16>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, nullptr, p, sms, s);
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
