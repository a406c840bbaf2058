// forge_embedding.cu -- the embedding lookup with scaling, its gradient summed
// by tokens, and that gradient fused with the AdamW step.
//
//   Y[t] = s W[id_t];   dW[r] = s sum_{t : id_t = r} dY[t]
// The gradient of a row is the sum over its tokens in an order that the ids
// alone determine, so results do not depend on scheduling.  A negative id is
// padding: its output row is zero and its gradient row is left out.
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

// Division of numbers from 0 below 2^63: with r = floor((2^64 - 1) / by) the high
// half of q r is the quotient or one less.  Where every thread divides, a 64-bit
// division is a large part of its instructions (lookup of 44352 tokens of 557
// bf16 columns: 27.8 us with it, 22.8 with this).
struct Divide {
    uint64_t reciprocal;
    int64_t by;
    explicit Divide(int64_t d) : reciprocal(UINT64_MAX / static_cast<uint64_t>(d)), by(d) {}
    __device__ __forceinline__ int64_t operator()(int64_t q, int64_t& rest) const
    {
        int64_t n = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(q), reciprocal));
        rest = q - n * by;
        if (rest >= by) {
            rest -= by;
            ++n;
        }
        return n;
    }
};

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

// A negative id is padding.  An id past the vocabulary is recorded in the
// status word and taken as padding.  (The loads stand apart from the check, so
// that a batch of them is in flight at once.)
__device__ __forceinline__ void bad_id(int* status)
{
    *reinterpret_cast<volatile int*>(status) = kDevInvalidArg;
}

// ------------------------------------------------------------------ lookup

// N elements as they lie in memory.
template <typename T, int N>
struct Group;
template <>
struct Group<float, 4> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[4]) const
    {
        x[0] = u.x;
        x[1] = u.y;
        x[2] = u.z;
        x[3] = u.w;
    }
};
template <int N>
struct Group<__nv_bfloat16, N> {
    uint32_t u[N / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        if constexpr (N == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            u[0] = v.x;
            u[1] = v.y;
            u[2] = v.z;
            u[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            u[0] = v.x;
            u[1] = v.y;
        }
    }
    __device__ __forceinline__ void get(float (&x)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
};
template <typename T>
struct Single {
    T u;
    __device__ __forceinline__ void load(const T* p) { u = __ldg(p); }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = static_cast<float>(u); }
};
template <>
struct Group<float, 1> : Single<float> {};
template <>
struct Group<__nv_bfloat16, 1> : Single<__nv_bfloat16> {};
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

// One warp per (token, span of columns), so that even a decode step's few
// tokens spread over the SMs, with the next token's id on its way; narrow rows
// by TOKENS at a time, as a warp's time is that of one load after the other
// (89598 tokens of 79 fp32 columns: 18.6 us by one, 12.1 by four).  VEC: rows
// of whole vectors, 16 bytes of the wider type, FLIGHT of them in flight per
// lane and token; otherwise single elements, 32 apart.  Bound by HBM; W's rows
// keep their place in L2 (frequent tokens), Y streams past it.  65536 Zipf tokens of
// 131072 x 4096, fp32 to bf16: 149 us, 5.7 TB/s of what has to move (each row
// once); uniform tokens 230 us, 6.0 TB/s.
template <typename W, typename Y>
constexpr int kLookupVec = 16 / (sizeof(W) > sizeof(Y) ? sizeof(W) : sizeof(Y));

template <typename W, typename Y, bool VEC, int FLIGHT, int TOKENS>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_kernel(const void* ids, bool wide, const W* __restrict__ w, Y* __restrict__ y,
                           int64_t T, int64_t V, int64_t D, float scale, Divide spans,
                           int64_t step_tokens, int64_t step_spans, int* status)
{
    constexpr int N = VEC ? kLookupVec<W, Y> : 1;
    constexpr int kColumns = 32 * N * FLIGHT;
    const int lane = threadIdx.x & 31;
    int64_t span;
    int64_t t = spans(static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), span);
    auto id_at = [&](int64_t i) -> int64_t {
        if (i >= T) return -1;
        return wide ? __ldg(static_cast<const int64_t*>(ids) + i)
                    : __ldg(static_cast<const int32_t*>(ids) + i);
    };
    int64_t next[TOKENS];
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) next[j] = id_at(t + j * step_tokens);
    while (t < T) {
        const int64_t c0 = span * kColumns + lane * N;
        const int left = static_cast<int>(D - c0 < kColumns ? D - c0 : kColumns);
        const W* src[TOKENS];
        int there[TOKENS];  // columns to load
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            int64_t r = next[j];
            if (r >= V) {
                bad_id(status);
                r = -1;
            }
            there[j] = r >= 0 ? left : 0;
            src[j] = w + r * D + c0;
        }
        Y* const dst = y + t * D + c0;
        const int64_t now = t;
        t += TOKENS * step_tokens;
        if constexpr (TOKENS == 1) {
            span += step_spans;
            if (span >= spans.by) {
                span -= spans.by;
                ++t;
            }
        }
#pragma unroll
        for (int j = 0; j < TOKENS; ++j)  // on their way while these rows are moved
            next[j] = id_at(t + j * step_tokens);
        Group<W, N> v[TOKENS][FLIGHT];
#pragma unroll
        for (int j = 0; j < TOKENS; ++j)
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i)
                if (i * 32 * N < there[j]) v[j][i].load(src[j] + i * 32 * N);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            if (j > 0 && now + j * step_tokens >= T) break;
            Y* const out = dst + j * step_tokens * D;
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i) {
                float x[N];
                v[j][i].get(x);
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = there[j] > 0 ? x[k] * scale : 0.0f;
                if (i * 32 * N >= left) continue;
                if constexpr (VEC)
                    store_vec<N>(out + i * 32 * N, x);
                else
                    store1(out, i * 32, x[0]);
            }
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
// Reading all ids twice in every block costs 2 T kClasses reads from L2, 1 KB a
// token of 32-bit ids: an eighth of a row of 4096 bf16 gradients, eight times one
// of 64.  Bound by the latency of its steps up to some 8192 tokens, by these reads
// beyond: 6-7 us for 2048 tokens, 7-9 for 8192, 10-12 for 16384, 16 for 32768, 28
// for 65536, on 128 blocks at any number; 65536 tokens of 131072 x 64 bf16 take 46
// us in all, with 32768 x 512 66.
constexpr int kClassBits = 7;
constexpr int kClasses = 1 << kClassBits;
constexpr int kOrderThreads = 1024;
constexpr int kOrderWarps = kOrderThreads / 32;
constexpr int kDigitBits = 5;
constexpr int kFewItems = 128;      // items of a list that is sorted by counting
constexpr int kOrderShared = 4096;  // items of a list that is sorted in shared memory
constexpr int kOrderSmem = 2 * kOrderShared * static_cast<int>(sizeof(int2));

// The kernels that follow the order are launched while it runs, so that their
// blocks stand ready when it ends; they wait here for its end (and the one
// before) before they read anything.  What the kernel before wrote (order, at,
// seg, partial) is read by plain loads only: __ldg asks for data that nothing
// writes while the reading kernel lives, and this one lives by then.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Token order: order[i] the token at place i; at[i] = {its row, and the number
// of the row's places if this is the first of them, else 0} ({-1, 0} past the
// tokens that are not padding); seg[r] the places [x, y) of row r.  listA,
// listB: room for T items where a block's list exceeds shared memory.
struct Order {
    int32_t* order;
    int2* at;
    int2* seg;
    int2* listA;
    int2* listB;
    int32_t later;  // rows of `partial` in front of those of pieces that go on
};

constexpr int kIdFlight = 4;  // loads of ids in flight per lane (16 made 2048 to 18000 tokens 2-3 us slower)

template <typename ID>
__global__ void __launch_bounds__(kOrderThreads, 1)
    forge_token_order_kernel(const ID* __restrict__ ids, int64_t T, int64_t V, Order o, int* status)
{
    let_next_start();
    extern __shared__ int2 s_list[];
    __shared__ uint32_t s_count[kOrderThreads];  // digit-major: [digit][warp]
    __shared__ uint32_t s_own[kOrderWarps], s_less[kOrderWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u;
    const uint32_t cls = blockIdx.x;

    // count, this warp's ids [lo, hi).  An id is held in 32 bits without its
    // sign: padding and ids past the vocabulary are those not below V.
    const int64_t chunk = (T + kOrderThreads - 1) / kOrderThreads * 32;
    const int64_t lo = warp * chunk, hi = lo + chunk < T ? lo + chunk : T;
    const uint32_t rows = static_cast<uint32_t>(V);
    auto fetch = [&](int64_t i0, uint32_t (&r)[kIdFlight]) {
        ID id[kIdFlight];
        if (hi - i0 >= 32 * kIdFlight) {
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u) id[u] = __ldg(ids + i0 + 32 * u + lane);
        } else {
            const int32_t left = static_cast<int32_t>(hi - i0) - lane;
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u)
                id[u] = 32 * u < left ? __ldg(ids + i0 + 32 * u + lane) : static_cast<ID>(-1);
        }
#pragma unroll
        for (int u = 0; u < kIdFlight; ++u) {
            if constexpr (sizeof(ID) == 4)
                r[u] = static_cast<uint32_t>(id[u]);
            else
                r[u] = static_cast<uint64_t>(id[u]) >> 32 ? 0xFFFFFFFFu : static_cast<uint32_t>(id[u]);
        }
        if (cls == 0) {
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u)
                if (id[u] >= V) bad_id(status);
        }
    };
    uint32_t own = 0, less = 0;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kIdFlight) {
        uint32_t r[kIdFlight];
        fetch(i0, r);
#pragma unroll
        for (int u = 0; u < kIdFlight; ++u) {
            const uint32_t c = r[u] & (kClasses - 1);
            if (r[u] < rows && c == cls) ++own;
            if (r[u] < rows && c < cls) ++less;
        }
    }
    own = __reduce_add_sync(0xffffffffu, own);
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) {
        s_own[warp] = own;
        s_less[warp] = less;
    }

    // rows without a token
    const int64_t local_rows = (V + kClasses - 1) / kClasses;
    for (int64_t k = threadIdx.x; k < local_rows; k += kOrderThreads)
        if (k * kClasses + cls < V) o.seg[k * kClasses + cls] = make_int2(0, 0);
    __syncthreads();
    own = s_own[lane];
    less = __reduce_add_sync(0xffffffffu, s_less[lane]);
    const int32_t base = less;
    const int32_t n = __reduce_add_sync(0xffffffffu, own);
    int32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? own : 0u);
    if (cls == kClasses - 1)
        for (int64_t i = base + n + threadIdx.x; i < T; i += kOrderThreads)
            o.at[i] = make_int2(-1, 0);

    // collect
    const bool shared = n <= kOrderShared;
    int2* src = shared ? s_list : o.listA + base;
    int2* dst = shared ? s_list + kOrderShared : o.listB + base;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kIdFlight) {
        uint32_t r[kIdFlight];
        fetch(i0, r);
#pragma unroll
        for (int u = 0; u < kIdFlight; ++u) {
            const bool mine = r[u] < rows && (r[u] & (kClasses - 1)) == cls;
            const uint32_t all = __ballot_sync(0xffffffffu, mine);
            if (all == 0) continue;
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
    if (n <= kFewItems) {  // an item's place is the number of those before it
        if (threadIdx.x < n) {
            const int2 item = src[threadIdx.x];
            int32_t place = 0;
#pragma unroll 4
            for (int32_t j = 0; j < n; ++j) {
                const int32_t key = src[j].x;
                place += key < item.x || (key == item.x && j < static_cast<int32_t>(threadIdx.x));
            }
            dst[place] = item;
        }
        __syncthreads();
        int2* t = src;
        src = dst;
        dst = t;
    }
    for (int shift = 0; n > kFewItems && (local_rows - 1) >> shift; shift += kDigitBits) {
        s_count[threadIdx.x] = 0;
        __syncthreads();
        for (int32_t i0 = p0; i0 < p1; i0 += 32 * kIdFlight) {
            uint32_t d[kIdFlight];
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u) {
                const int32_t i = i0 + 32 * u + lane;
                d[u] = i < p1 ? (static_cast<uint32_t>(src[i].x) >> shift) & 31u : 32u;
            }
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u) {
                if (i0 + 32 * u >= p1) break;
                const uint32_t same = __match_any_sync(0xffffffffu, d[u]);
                if (d[u] < 32u && (same & before) == 0) s_count[d[u] * 32 + warp] += __popc(same);
                __syncwarp();
            }
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
        const uint32_t ahead = __reduce_add_sync(0xffffffffu, lane < warp ? s_own[lane] : 0u);
        s_count[threadIdx.x] = ahead + inc - v;
        __syncthreads();
        for (int32_t i0 = p0; i0 < p1; i0 += 32 * kIdFlight) {
            int2 item[kIdFlight];
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u) {
                const int32_t i = i0 + 32 * u + lane;
                item[u] = i < p1 ? src[i] : make_int2(0, 0);
            }
#pragma unroll
            for (int u = 0; u < kIdFlight; ++u) {
                if (i0 + 32 * u >= p1) break;
                const bool in = i0 + 32 * u + lane < p1;
                const uint32_t d = in ? (static_cast<uint32_t>(item[u].x) >> shift) & 31u : 32u;
                const uint32_t same = __match_any_sync(0xffffffffu, d);
                if (in) dst[s_count[d * 32 + warp] + __popc(same & before)] = item[u];
                __syncwarp();
                if (in && (same & before) == 0) s_count[d * 32 + warp] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        int2* t = src;
        src = dst;
        dst = t;
    }

    for (int32_t i = threadIdx.x; i < n; i += kOrderThreads) {
        const int2 item = src[i];
        const int32_t r = (item.x << kClassBits) + cls;
        o.order[base + i] = item.y;
        int2* s = &o.seg[r];
        if (i == 0 || src[i - 1].x != item.x) s->x = base + i;
        if (i == n - 1 || src[i + 1].x != item.x) s->y = base + i + 1;
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kOrderThreads) {
        const int32_t r = (src[i].x << kClassBits) + cls;
        const bool first = i == 0 || src[i - 1].x != src[i].x;
        o.at[base + i] = make_int2(r, first ? o.seg[r].y - o.seg[r].x : 0);
    }
}

// ------------------------------------------------------------------ sums

// Columns come in vectors of four (VEC: D a multiple of 4, every base aligned
// to four elements) or one by one.
template <typename G, int N>
struct Raw;
template <>
struct Raw<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void add_to(float (&g)[4]) const
    {
        g[0] += v.x;
        g[1] += v.y;
        g[2] += v.z;
        g[3] += v.w;
    }
};
template <>
struct Raw<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void add_to(float (&g)[4]) const
    {
        g[0] += __uint_as_float(v.x << 16);
        g[1] += __uint_as_float(v.x & 0xFFFF0000u);
        g[2] += __uint_as_float(v.y << 16);
        g[3] += __uint_as_float(v.y & 0xFFFF0000u);
    }
};
template <typename G>
struct Raw<G, 1> {
    G v;
    __device__ __forceinline__ void load(const G* p) { v = *p; }
    __device__ __forceinline__ void add_to(float (&g)[1]) const { g[0] += static_cast<float>(v); }
};

// g += the entries at `column` of n rows of a [*, D] array, the i-th being row
// of(i), in that order, F (a power of two) rows in flight.
template <int F, int N, typename G, typename ROW>
__device__ __forceinline__ void add_batch(const G* column, int32_t i, ROW of, int64_t D, float (&g)[N])
{
    int32_t at[F];
#pragma unroll
    for (int u = 0; u < F; ++u) at[u] = of(i + u);
    Raw<G, N> x[F];
#pragma unroll
    for (int u = 0; u < F; ++u) x[u].load(column + static_cast<int64_t>(at[u]) * D);
#pragma unroll
    for (int u = 0; u < F; ++u) x[u].add_to(g);
}
template <int F, int N, typename G, typename ROW>
__device__ __forceinline__ void add_rows(const G* column, int32_t n, ROW of, int64_t D, float (&g)[N])
{
    int32_t i = 0;
    for (; i + F <= n; i += F) add_batch<F>(column, i, of, D, g);
    if constexpr (F > 4)
        if (n - i >= 4) {
            add_batch<4>(column, i, of, D, g);
            i += 4;
        }
    if constexpr (F > 2)
        if (n - i >= 2) {
            add_batch<2>(column, i, of, D, g);
            i += 2;
        }
    if (n - i >= 1) add_batch<1>(column, i, of, D, g);
}

// How a row's tokens are added, by their number n:
//   n <= kShort   one thread a column (four), one token after the other (up to
//                 128 tokens that way, the rows of a vocabulary's front held up
//                 their blocks: 32768 Zipf tokens took 471 instead of 355 us);
//   n <= medium   (a vocabulary's frequent tokens) one block for 256 columns,
//                 its warps a part of the tokens each;
//   else          in pieces: the row's places are cut at the multiples of
//                 kPiece, and a warp adds 256 columns of a piece into a row of
//                 `partial`: row a / kHuge for the piece with which a row starts
//                 at place a (the next such start is more than kHuge places
//                 away), row later + a / kPiece for one that goes on at a.  A
//                 last kernel joins the pieces.
// Batches of up to kFew tokens do without pieces and that kernel: medium is
// kFew there, kHuge otherwise (33322 Zipf tokens of 123650 x 222 bf16 take 55 us,
// with blocks for rows of up to 2048 tokens 86; 65536 of 32768 x 512: 66, 86).
constexpr int kShort = 16;
constexpr int kFew = 2048;
constexpr int kHuge = 512;
constexpr int kPiece = 64;
constexpr int kSlice = 256;

// What becomes of a row's sum: dW written, dW added to, or the AdamW step.
enum Sum { SUM_STORE = 0, SUM_ADD = 1, SUM_ADAMW = 2 };

// How the columns lie: vectors of four in every array; in dW, W, m, v as flat
// arrays only; or anyhow.
enum Lie { LIE_VECTORS = 2, LIE_FLAT = 1, LIE_ANY = 0 };

// A warp's part of a row: H vectors of N columns a lane, 32 N columns apart,
// `width` columns from c0 on; the columns past D are left out.
template <bool VEC, int WIDTH>
struct Part {
    static constexpr int N = VEC ? 4 : 1;
    static constexpr int H = WIDTH / (32 * N);
    int64_t c0, D;
    int lane;
    __device__ __forceinline__ int column(int h) const { return (32 * h + lane) * N; }
    __device__ __forceinline__ bool has(int h) const { return c0 + column(h) < D; }
    // g += n rows of a [*, D] array, the i-th being row of(i), in that order, K in flight
    template <int K, typename G, typename ROW>
    __device__ __forceinline__ void add_rows(const G* base, int32_t n, ROW of, float (&g)[H][N]) const
    {
        for (int32_t i0 = 0; i0 < n; i0 += K) {
            Raw<G, N> x[K][H];
#pragma unroll
            for (int u = 0; u < K; ++u) {
                const G* src = base + c0 + static_cast<int64_t>(of(i0 + u)) * D;
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (i0 + u < n && has(h)) x[u][h].load(src + column(h));
            }
#pragma unroll
            for (int u = 0; u < K; ++u)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    if (i0 + u < n && has(h)) x[u][h].add_to(g[h]);
        }
    }
};
template <typename T, int N>
__device__ __forceinline__ void load_state(const T* p, float (&x)[N])
{
    if constexpr (N == 4)
        StateIO<sizeof(T) == 4 ? ST_F32 : ST_BF16>::ld4(p, 0, x);
    else
        x[0] = StateIO<sizeof(T) == 4 ? ST_F32 : ST_BF16>::ld(p, 0);
}
template <int N>
__device__ __forceinline__ void store_sum(float* p, const float (&x)[N])
{
    if constexpr (N == 4)
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *p = x[0];
}

// One warp per (kPiece places, slice): the pieces of huge rows that start among
// these places; there are two at most.
template <typename G, bool VEC>
__device__ __forceinline__ void sum_pieces(const G* dY, int64_t unit, int64_t T, int64_t D,
                                           int64_t slices, const Order& o, float* partial)
{
    static_assert(kPiece < kHuge && kHuge % kPiece == 0);
    using P = Part<VEC, kSlice>;
    constexpr int kTokens = 4;  // in flight; eight spill registers of the kernel's other parts
    const int lane = threadIdx.x & 31;
    const int64_t slice = unit % slices;
    const int32_t p0 = static_cast<int32_t>(unit / slices * kPiece);
    const P part{slice * kSlice, D, lane};
    if (p0 >= T) return;
    int32_t at = -1, n = 0;  // a huge row that starts here
#pragma unroll
    for (int i = 0; i < kPiece / 32; ++i) {
        const int32_t place = p0 + 32 * i + lane;
        const int32_t here = place < T ? o.at[place].y : 0;
        const uint32_t found = __ballot_sync(0xffffffffu, here > kHuge);
        if (found != 0) {
            at = p0 + 32 * i + __ffs(found) - 1;
            n = __shfl_sync(0xffffffffu, here, __ffs(found) - 1);
        }
    }
    auto piece = [&](int32_t a, int32_t e, int32_t slot) {
        float g[P::H][P::N] = {};
        for (int32_t i0 = a; i0 < e; i0 += 32) {
            const int32_t token = i0 + lane < e ? o.order[i0 + lane] : 0;
            part.template add_rows<kTokens>(
                dY, e - i0 < 32 ? e - i0 : 32,
                [&](int32_t i) { return __shfl_sync(0xffffffffu, token, i & 31); }, g);
        }
#pragma unroll
        for (int h = 0; h < P::H; ++h)
            if (part.has(h)) store_sum(partial + static_cast<int64_t>(slot) * D + part.c0 + part.column(h), g[h]);
    };
    const int64_t p1 = static_cast<int64_t>(p0) + kPiece;
    const int2 first = o.at[p0];
    if (first.x >= 0 && first.y == 0) {
        const int2 s = o.seg[first.x];
        if (s.y - s.x > kHuge)
            piece(p0, static_cast<int32_t>(s.y < p1 ? s.y : p1), o.later + p0 / kPiece);
    }
    if (at >= 0) piece(at, static_cast<int32_t>(at + n < p1 ? at + n : p1), at / kHuge);
}

// One column's step from the sum of its row's tokens; holds what the column had.
template <int MODE, int ST>
struct Column {
    float w, a, b;
    __device__ __forceinline__ void load(const float* dW, const Params& p, int64_t at)
    {
        if constexpr (MODE == SUM_ADAMW) {
            w = StateIO<ST_F32>::ld(p.W, at);
            a = StateIO<ST>::ld(p.s1, at);
            b = StateIO<ST>::ld(p.s2, at);
        } else if constexpr (MODE == SUM_ADD) {
            w = dW[at];
        }
    }
    __device__ __forceinline__ void finish(float* dW, const Params& p, int64_t at, float sum, float scale)
    {
        const float x = sum * scale;
        if constexpr (MODE == SUM_ADAMW) {
            float gs[4] = {x, x, x, x}, ws[4] = {w, w, w, w}, as[4] = {a, a, a, a}, bs[4] = {b, b, b, b};
            step4<OP_ADAMW>(p, gs, ws, as, bs);
            StateIO<ST_F32>::st(p.W, at, ws[0]);
            StateIO<ST>::st(p.s1, at, as[0]);
            StateIO<ST>::st(p.s2, at, bs[0]);
        } else {
            dW[at] = MODE == SUM_ADD ? fmaf(scale, sum, w) : x;
        }
    }
};

// One block per (kMediumPlaces places, slice): the medium rows that start
// there, one after the other.
constexpr int kMediumPlaces = 64;
template <typename G, int MODE, int ST, bool VEC>
__device__ __forceinline__ void medium_rows(const G* dY, int64_t block, int64_t T, int64_t D,
                                            int64_t slices, float scale, float* dW, const Order& o, const Params& p)
{
    using P = Part<VEC, kSlice>;
    constexpr int kWarps = kThreads / 32;
    constexpr int kMost = kMediumPlaces / (kShort + 1) + 1;
    constexpr int kTokens = 4;  // in flight
    __shared__ int2 s_start[2][kMost];  // place and tokens, by the warp that found them
    __shared__ int32_t s_row[2][kMost], s_count[2];
    __shared__ float sh[kWarps][kSlice];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t slice = block % slices;
    const int32_t p0 = static_cast<int32_t>(block / slices * kMediumPlaces);
    const P part{slice * kSlice, D, lane};
    static_assert(kMediumPlaces == 64);
    if (warp < 2) {
        const int32_t place = p0 + static_cast<int32_t>(threadIdx.x);
        const int2 here = place < T ? o.at[place] : make_int2(-1, 0);
        const bool start = here.y > kShort && here.y <= (T > kFew ? kHuge : kFew);
        const uint32_t found = __ballot_sync(0xffffffffu, start);
        if (start) {
            const int i = __popc(found & ((1u << lane) - 1u));
            s_start[warp][i] = make_int2(place, here.y);
            s_row[warp][i] = here.x;
        }
        if (lane == 0) s_count[warp] = __popc(found);
    }
    __syncthreads();
    const int first = s_count[0], rows = first + s_count[1];
    for (int r = 0; r < rows; ++r) {
        const int2 s = r < first ? s_start[0][r] : s_start[1][r - first];
        const int64_t c = part.c0 + threadIdx.x;
        const int64_t at = (r < first ? s_row[0][r] : s_row[1][r - first]) * D + c;
        Column<MODE, ST> state;
        if (c < D) state.load(dW, p, at);
        // tokens warp, warp + 8, ...
        float g[P::H][P::N] = {};
        for (int32_t j = warp; j < s.y; j += 32 * kWarps) {
            const int32_t mine = j + lane * kWarps;
            const int32_t token = mine < s.y ? o.order[s.x + mine] : 0;
            const int32_t n = (s.y - j + kWarps - 1) / kWarps;
            part.template add_rows<kTokens>(
                dY, n < 32 ? n : 32, [&](int32_t i) { return __shfl_sync(0xffffffffu, token, i & 31); }, g);
        }
        __syncthreads();  // the row before has been read
#pragma unroll
        for (int h = 0; h < P::H; ++h)
#pragma unroll
            for (int k = 0; k < P::N; ++k) sh[warp][part.column(h) + k] = g[h][k];
        __syncthreads();
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += sh[w][threadIdx.x];
        if (c < D) state.finish(dW, p, at, sum, scale);
    }
}

// dW or the AdamW step over all V D elements, flat, so that no width leaves
// lanes idle: a block takes `turns` tiles of U vectors a thread, one after the
// other, and a thread carries row and column along instead of dividing.  Two
// vectors (VEC; four single elements otherwise) are in hand at once, with the
// places of the next ones already on their way: most rows of a large
// vocabulary have no token, and their zeros (or their decay) must not wait for
// a table.  Rows of more than kShort tokens are left out.
template <bool VEC>
constexpr int kUnits = VEC ? 2 : 4;

template <typename G, int MODE, int ST, bool VEC>
__device__ __forceinline__ void dense_rows(const G* dY, int64_t block, uint32_t V, int32_t D,
                                           Divide vectors, float scale, float* dW, const Order& o, int32_t turns,
                                           const Params& p)
{
    constexpr int N = VEC ? 4 : 1;
    constexpr int U = kUnits<VEC>;
    constexpr int F = MODE == SUM_ADAMW ? 2 : 4;
    const uint32_t width = static_cast<uint32_t>(vectors.by);  // vectors of a row
    int64_t step_columns;
    const uint32_t step_rows = static_cast<uint32_t>(vectors(kThreads * U, step_columns));
    auto places = [&](uint32_t r) {
        return r < V && o.seg ? o.seg[r] : make_int2(0, 0);
    };
    uint32_t row[U], column[U];
    int2 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int64_t rest;
        row[u] = static_cast<uint32_t>(
            vectors(block * turns * (kThreads * U) + u * kThreads + threadIdx.x, rest));
        column[u] = static_cast<uint32_t>(rest);
        s[u] = places(row[u]);
    }
    for (int32_t turn = 0; turn < turns && row[0] < V; ++turn) {
        float g[U * N], w[U * N], a[U * N], b[U * N];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            live[u] = row[u] < V && s[u].y - s[u].x <= kShort;
            if constexpr (MODE == SUM_ADAMW) {
                const int64_t at = static_cast<int64_t>(row[u]) * D + column[u] * N;
                if (!live[u]) continue;
                if constexpr (VEC) {
                    StateIO<ST_F32>::ld4(p.W, at, w + 4 * u);
                    StateIO<ST>::ld4(p.s1, at, a + 4 * u);
                    StateIO<ST>::ld4(p.s2, at, b + 4 * u);
                } else {
                    w[u] = StateIO<ST_F32>::ld(p.W, at);
                    a[u] = StateIO<ST>::ld(p.s1, at);
                    b[u] = StateIO<ST>::ld(p.s2, at);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[N] = {};
            if (live[u] && s[u].y > s[u].x)
                add_rows<F>(dY + column[u] * N, s[u].y - s[u].x,
                            [&](int32_t i) { return o.order[s[u].x + i]; }, D, x);
#pragma unroll
            for (int k = 0; k < N; ++k) g[u * N + k] = x[k] * scale;
        }
        if constexpr (MODE == SUM_ADAMW) {
#pragma unroll
            for (int h = 0; h < U * N / 4; ++h)
                step4<OP_ADAMW>(p, g + 4 * h, w + 4 * h, a + 4 * h, b + 4 * h);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = static_cast<int64_t>(row[u]) * D + column[u] * N;
            if (live[u]) {
                if constexpr (MODE == SUM_ADAMW && VEC) {
                    StateIO<ST_F32>::st4(p.W, at, w + 4 * u);
                    StateIO<ST>::st4(p.s1, at, a + 4 * u);
                    StateIO<ST>::st4(p.s2, at, b + 4 * u);
                } else if constexpr (MODE == SUM_ADAMW) {
                    StateIO<ST_F32>::st(p.W, at, w[u]);
                    StateIO<ST>::st(p.s1, at, a[u]);
                    StateIO<ST>::st(p.s2, at, b[u]);
                } else if constexpr (VEC) {
                    StateIO<ST_F32>::st4(dW, at, g + 4 * u);
                } else {
                    StateIO<ST_F32>::st(dW, at, g[u]);
                }
            }
            row[u] += step_rows;
            column[u] += static_cast<uint32_t>(step_columns);
            if (column[u] >= width) {
                column[u] -= width;
                ++row[u];
            }
            s[u] = places(row[u]);
        }
    }
}

// The same for a width that is no multiple of four, while dW, W, m, v are
// aligned: vectors of four elements of the flat arrays, which may belong to two
// rows; dY is read element by element.
template <typename G, int MODE, int ST>
__device__ __forceinline__ void dense_ragged(const G* dY, int64_t block, uint32_t V, int32_t D,
                                             Divide width, float scale, float* dW, const Order& o, int32_t turns,
                                             const Params& p)
{
    constexpr uint32_t step = kThreads * 4;
    const int64_t total = static_cast<int64_t>(V) * D;
    int64_t rest;
    const uint32_t step_rows = static_cast<uint32_t>(width(step, rest));
    const int32_t step_columns = static_cast<int32_t>(rest);
    auto places = [&](uint32_t r) {
        return r < V && o.seg ? o.seg[r] : make_int2(0, 0);
    };
    int64_t at = (block * turns * kThreads + threadIdx.x) * 4;
    uint32_t row = static_cast<uint32_t>(width(at, rest));
    int32_t column = static_cast<int32_t>(rest);
    int2 s = places(row), s2 = column + 3 >= D ? places(row + 1) : make_int2(0, 0);
    for (int32_t turn = 0; turn < turns && at < total; ++turn) {
        const bool whole = at + 4 <= total;
        const int m = D - column < 4 ? D - column : 4;  // of the first row
        const bool short1 = s.y - s.x <= kShort, short2 = s2.y - s2.x <= kShort;
        float g[4] = {}, w[4], a[4], b[4];
        if (MODE == SUM_ADAMW && whole) {
            StateIO<ST_F32>::ld4(p.W, at, w);
            StateIO<ST>::ld4(p.s1, at, a);
            StateIO<ST>::ld4(p.s2, at, b);
        }
        auto add = [&](int2 part, int k0, int k1, int32_t c) {  // elements k0 .. k1 from column c on
            for (int32_t i = part.x; i < part.y; i += 4) {
                float x[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool there = i + u < part.y;
                    const G* row = dY + static_cast<int64_t>(o.order[there ? i + u : i]) * D + c;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[u][k] = there && k >= k0 && k < k1 ? load1(row, k) : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) g[k] += x[u][k];
            }
        };
        if (s.y > s.x && short1) add(s, 0, m, column);
        if (s2.y > s2.x && short2) add(s2, m, 4, -m);
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] *= scale;
        if (whole && short1 && short2) {
            if constexpr (MODE == SUM_ADAMW) {
                step4<OP_ADAMW>(p, g, w, a, b);
                StateIO<ST_F32>::st4(p.W, at, w);
                StateIO<ST>::st4(p.s1, at, a);
                StateIO<ST>::st4(p.s2, at, b);
            } else {
                StateIO<ST_F32>::st4(dW, at, g);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (at + k >= total || !(k < m ? short1 : short2)) continue;
                if constexpr (MODE == SUM_ADAMW) {
                    float gs[4] = {g[k], g[k], g[k], g[k]}, ws[4], as[4], bs[4];
                    ws[0] = ws[1] = ws[2] = ws[3] = StateIO<ST_F32>::ld(p.W, at + k);
                    as[0] = as[1] = as[2] = as[3] = StateIO<ST>::ld(p.s1, at + k);
                    bs[0] = bs[1] = bs[2] = bs[3] = StateIO<ST>::ld(p.s2, at + k);
                    step4<OP_ADAMW>(p, gs, ws, as, bs);
                    StateIO<ST_F32>::st(p.W, at + k, ws[0]);
                    StateIO<ST>::st(p.s1, at + k, as[0]);
                    StateIO<ST>::st(p.s2, at + k, bs[0]);
                } else {
                    StateIO<ST_F32>::st(dW, at + k, g[k]);
                }
            }
        }
        at += step;
        row += step_rows;
        column += step_columns;
        if (column >= D) {
            column -= D;
            ++row;
        }
        s = places(row);
        s2 = column + 3 >= D ? places(row + 1) : make_int2(0, 0);
    }
}

// dW += the sums, over the rows that have a token only.  One warp per (four
// places, 512 columns; 256 single ones) takes the rows of at most kShort tokens
// that start there: two loads bring the places and all their tokens.
constexpr int kTouchPlaces = 4;
template <bool VEC>
constexpr int kTouchColumns = VEC ? 512 : 256;
template <typename G, bool VEC>
__device__ __forceinline__ void touched_rows(const G* dY, int64_t unit, int64_t T, int64_t D,
                                             int64_t slices, float scale, float* dW, const Order& o)
{
    static_assert(kTouchPlaces + kShort <= 32);
    using P = Part<VEC, kTouchColumns<VEC>>;
    const int lane = threadIdx.x & 31;
    const int64_t slice = unit % slices;
    const int64_t p0 = unit / slices * kTouchPlaces, c0 = slice * kTouchColumns<VEC>;
    if (p0 >= T) return;
    const int64_t place = p0 + lane;
    const int2 here = lane < kTouchPlaces && place < T ? o.at[place] : make_int2(-1, 0);
    const int32_t token = lane < kTouchPlaces + kShort && place < T ? o.order[place] : 0;
    const P part{c0, D, lane};
    for (uint32_t left = __ballot_sync(0xffffffffu, here.y > 0 && here.y <= kShort); left != 0;
         left &= left - 1) {
        const int a = __ffs(left) - 1;
        const int32_t n = __shfl_sync(0xffffffffu, here.y, a);
        float* dst = dW + static_cast<int64_t>(__shfl_sync(0xffffffffu, here.x, a)) * D + c0;
        float d[P::H][P::N], g[P::H][P::N] = {};
#pragma unroll
        for (int h = 0; h < P::H; ++h)
            if (part.has(h)) load_state(dst + part.column(h), d[h]);
        part.template add_rows<VEC && sizeof(G) == 4 ? 1 : 2>(
            dY, n, [&](int32_t i) { return __shfl_sync(0xffffffffu, token, (a + i) & 31); }, g);
#pragma unroll
        for (int h = 0; h < P::H; ++h) {
#pragma unroll
            for (int k = 0; k < P::N; ++k) d[h][k] = fmaf(scale, g[h][k], d[h][k]);
            if (part.has(h)) store_sum(dst + part.column(h), d[h]);
        }
    }
}

// While the order is made, its memory pipes are idle: the first blocks, which
// wait for it anyway, bring the gradients (where they are few) and the state of
// the first rows into L2.  7628 x 4313 fp32 AdamW with 6 tokens: 121 us against
// 124; 33322 tokens of 123650 x 222 bf16: 55 against 59.
__device__ __forceinline__ void fetch_ahead(const void* base, int64_t from, int64_t to)
{
    for (int64_t i = from + 128 * static_cast<int32_t>(threadIdx.x); i < to; i += 128 * kThreads)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(base) + i));
}

// All rows in one launch: the blocks for the pieces of huge rows and for medium
// rows come first, as they take longest, then those for the others.  Bound by
// HBM: dW written, or W, m, v read and written, once, and dY read once.  32768
// Zipf tokens, 131072 x 4096: 377 us for dW from bf16 dY (6.4 TB/s), 1956 us
// fused with AdamW on fp32 state (6.7 TB/s), the order before included.  Sums stored from bf16
// vectors: five blocks an SM (48 registers) against four, uniform tokens 399
// against 434 us; the other forms would spill (13321 x 220 fp32: 40 us with
// five, 33 with four).
template <typename G, int MODE, int ST, int LIE>
__global__ void __launch_bounds__(kThreads, MODE == SUM_STORE && LIE == LIE_VECTORS && sizeof(G) == 2 ? 5 : 4)
    forge_embedding_grad_kernel(const G* dY, int64_t T, int32_t V, int32_t D, int64_t slices,
                                Divide parts, float scale, float* dW, Order o, float* partial, uint32_t piece_blocks,
                                uint32_t medium_blocks, int32_t turns, uint32_t ahead_blocks,
                                int64_t ahead_bytes, const Params p)
{
    constexpr int kWarps = kThreads / 32;
    constexpr bool VEC = LIE == LIE_VECTORS;
    const int warp = threadIdx.x >> 5;
    uint32_t block = blockIdx.x;
    if (block < ahead_blocks) {
        const int64_t bytes = T * D * static_cast<int64_t>(sizeof(G)), at = block * ahead_bytes;
        fetch_ahead(dY, at, at + ahead_bytes < bytes ? at + ahead_bytes : bytes);
        if constexpr (MODE == SUM_ADAMW) {
            constexpr int S = ST == ST_BF16 ? 2 : 4;
            const int64_t n = static_cast<int64_t>(turns) * kThreads * (VEC ? 8 : 4);
            const int64_t from = block * n, end = static_cast<int64_t>(V) * D;
            const int64_t to = from + n < end ? from + n : end;
            fetch_ahead(p.W, from * 4, to * 4);
            fetch_ahead(p.s1, from * S, to * S);
            fetch_ahead(p.s2, from * S, to * S);
        }
    }
    await_previous();
    if (block < piece_blocks) {
        sum_pieces<G, VEC>(dY, static_cast<int64_t>(block) * kWarps + warp, T, D, slices, o, partial);
        return;
    }
    block -= piece_blocks;
    if (block < medium_blocks) {
        medium_rows<G, MODE, ST, VEC>(dY, block, T, D, slices, scale, dW, o, p);
        return;
    }
    block -= medium_blocks;
    if constexpr (MODE == SUM_ADD)
        touched_rows<G, VEC>(dY, static_cast<int64_t>(block) * kWarps + warp, T, D, parts.by, scale, dW, o);
    else if constexpr (LIE == LIE_FLAT)
        dense_ragged<G, MODE, ST>(dY, block, V, D, parts, scale, dW, o, turns, p);
    else
        dense_rows<G, MODE, ST, VEC>(dY, block, V, D, parts, scale, dW, o, turns, p);
}

// One block per (kHuge places, slice): at most one huge row starts there; its
// warps add a part of the pieces each.
template <int MODE, int ST>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_huge_rows_kernel(int64_t T, int64_t D, float scale, float* dW, Order o,
                                     const float* partial, const Params p)
{
    using P = Part<false, kSlice>;
    constexpr int kWarps = kThreads / 32;
    __shared__ int32_t s_first, s_n, s_row;
    __shared__ float sh[kWarps][kSlice];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t slices = (D + kSlice - 1) / kSlice;
    const int32_t p0 = static_cast<int32_t>(blockIdx.x / slices * kHuge);
    const P part{static_cast<int64_t>(blockIdx.x % slices) * kSlice, D, lane};
    if (threadIdx.x == 0) s_n = 0;
    await_previous();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHuge / kThreads; ++i) {
        const int32_t place = p0 + i * kThreads + static_cast<int32_t>(threadIdx.x);
        const int2 here = place < T ? o.at[place] : make_int2(-1, 0);
        if (here.y > kHuge) {
            s_first = place;
            s_n = here.y;
            s_row = here.x;
        }
    }
    __syncthreads();
    if (s_n == 0) return;
    const int32_t first = s_first, b0 = first / kPiece, n = (first + s_n - 1) / kPiece - b0 + 1;
    float g[P::H][1] = {};
    part.template add_rows<4>(
        partial, (n - warp + kWarps - 1) / kWarps,
        [&](int32_t j) {
            const int32_t i = warp + j * kWarps;
            return i == 0 ? first / kHuge : o.later + b0 + (i < n ? i : 1);
        },
        g);
#pragma unroll
    for (int h = 0; h < P::H; ++h) sh[warp][part.column(h)] = g[h][0];
    __syncthreads();
    const int64_t c = part.c0 + threadIdx.x, at = s_row * D + c;
    if (c >= D) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh[w][threadIdx.x];
    Column<MODE, ST> state;
    state.load(dW, p, at);
    state.finish(dW, p, at, sum, scale);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : (t == FORGE_I64 ? 8 : 4); }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }
bool is_id(forge_dtype t) { return t == FORGE_I32 || t == FORGE_I64; }

forge_status check_sizes(int64_t T, int64_t V, int64_t D, float scale)
{
    if (T < 0 || V < 1 || D < 1 || T > (1 << 30) || V > INT32_MAX || D > INT32_MAX)
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

// The order kernel's shared memory, allowed once per device.
template <typename ID>
cudaError_t allow_order_smem()
{
    static unsigned long long done = 0;  // one bit per device ordinal < 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(forge_token_order_kernel<ID>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kOrderSmem);
    if (e == cudaSuccess) __atomic_fetch_or(&done, bit, __ATOMIC_ACQ_REL);
    return e;
}

template <typename ID>
cudaError_t order_tokens(const void* ids, int64_t T, int64_t V, const Order& o, int* status,
                         cudaStream_t s)
{
    const cudaError_t e = allow_order_smem<ID>();
    if (e != cudaSuccess) return e;
    forge_token_order_kernel<ID><<<kClasses, kOrderThreads, kOrderSmem, s>>>(
        static_cast<const ID*>(ids), T, V, o, status);
    return cudaGetLastError();
}

template <typename G, int MODE, int ST, int LIE>
cudaError_t launch_sums(const G* dY, int64_t T, int64_t V, int64_t D, float scale, float* dW,
                        const Order& o, float* partial, const Params& p, int sms, cudaStream_t s)
{
    const int64_t slices = (D + kSlice - 1) / kSlice;
    const int64_t units = T > kFew ? (T + kPiece - 1) / kPiece * slices : 0;
    const int64_t piece_blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t medium_blocks = T > kShort ? (T + kMediumPlaces - 1) / kMediumPlaces * slices : 0;
    int64_t turns = 1, blocks, parts;  // of a row: slices, vectors or elements
    if (MODE == SUM_ADD) {
        constexpr int columns = kTouchColumns<LIE == LIE_VECTORS>;
        parts = (D + columns - 1) / columns;
        const int64_t touch_units = (T + kTouchPlaces - 1) / kTouchPlaces * parts;
        blocks = (touch_units + kThreads / 32 - 1) / (kThreads / 32);
    } else {
        // as many turns, up to eight, as leave each SM 32 blocks
        parts = LIE == LIE_VECTORS ? D / 4 : D;
        const int64_t elements = V * D, tile = kThreads * (LIE == LIE_VECTORS ? 8 : 4);
        const int64_t tiles = (elements + tile - 1) / tile;
        turns = tiles / (32LL * sms);
        turns = turns < 1 ? 1 : (turns > 8 ? 8 : turns);
        while ((tiles + turns - 1) / turns > INT32_MAX / 2) turns *= 2;
        blocks = (tiles + turns - 1) / turns;
    }
    const int64_t all = piece_blocks + medium_blocks + blocks;
    if (all > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(all));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = early;
    cfg.numAttrs = T > 0 ? 1 : 0;  // without tokens there is no kernel before
    const int64_t ahead = 2 * sms, bytes = T * D * static_cast<int64_t>(sizeof(G));
    const int64_t ahead_bytes = bytes <= ahead << 16 ? (bytes / ahead + 127) / 128 * 128 + 128 : 0;
    cudaError_t e = cudaLaunchKernelEx(
        &cfg, forge_embedding_grad_kernel<G, MODE, ST, LIE>, dY, T, static_cast<int32_t>(V),
        static_cast<int32_t>(D), slices, Divide(parts), scale, dW, o, partial,
        static_cast<uint32_t>(piece_blocks),
        static_cast<uint32_t>(medium_blocks), static_cast<int32_t>(turns),
        static_cast<uint32_t>(T > 0 ? ahead : 0), ahead_bytes, p);
    if (e == cudaSuccess && T > kFew) {
        cfg.gridDim = dim3(static_cast<unsigned>((T + kHuge - 1) / kHuge * slices));
        e = cudaLaunchKernelEx(&cfg, forge_embedding_huge_rows_kernel<MODE, ST>, T, D, scale, dW, o,
                               static_cast<const float*>(partial), p);
    }
    return e;
}

template <typename G, int LIE>
cudaError_t launch_grad(Sum what, bool state_bf16, const G* dY, const void* ids, bool wide,
                        int64_t T, int64_t V, int64_t D, float scale, float* dW, const Params& p,
                        int sms, cudaStream_t s)
{
    if (what == SUM_ADD && T == 0) return cudaSuccess;
    Order o{};
    float* partial = nullptr;
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
        const int64_t order_b = up(T * 4), list_b = up(T * 8), seg_b = up(V * 8);
        o.later = static_cast<int32_t>((T + kHuge - 1) / kHuge);
        const int64_t slots = T > kFew ? o.later + (T + kPiece - 1) / kPiece : 0;
        e = scratch_alloc(&scratch, order_b + 3 * list_b + seg_b + slots * D * 4, s);
        if (e != cudaSuccess) return e;
        uint8_t* at = static_cast<uint8_t*>(scratch);
        o.order = reinterpret_cast<int32_t*>(at);
        o.at = reinterpret_cast<int2*>(at += order_b);
        o.listA = reinterpret_cast<int2*>(at += list_b);
        o.listB = reinterpret_cast<int2*>(at += list_b);
        o.seg = reinterpret_cast<int2*>(at += list_b);
        partial = reinterpret_cast<float*>(at += seg_b);
        e = wide ? order_tokens<int64_t>(ids, T, V, o, p.status, s)
                 : order_tokens<int32_t>(ids, T, V, o, p.status, s);
    }
    if (e == cudaSuccess) {
        if (what == SUM_STORE)
            e = launch_sums<G, SUM_STORE, ST_F32, LIE>(dY, T, V, D, scale, dW, o, partial, p, sms, s);
        else if (what == SUM_ADD)
            e = launch_sums<G, SUM_ADD, ST_F32, LIE == LIE_VECTORS ? LIE : LIE_ANY>(
                dY, T, V, D, scale, dW, o, partial, p, sms, s);
        else if (state_bf16)
            e = launch_sums<G, SUM_ADAMW, ST_BF16, LIE>(dY, T, V, D, scale, dW, o, partial, p, sms, s);
        else
            e = launch_sums<G, SUM_ADAMW, ST_F32, LIE>(dY, T, V, D, scale, dW, o, partial, p, sms, s);
    }
    if (scratch) {
        const cudaError_t fe = scratch_free(scratch, s);
        if (e == cudaSuccess) e = fe;
    }
    return e;
}

// A refused allocation or launch is this call's to report: the runtime's record of
// it is cleared, so that the next call's check of its own launch does not find it.
forge_status reported(cudaError_t e)
{
    if (e == cudaSuccess) return FORGE_OK;
    cudaGetLastError();
    return FORGE_ERR_CUDA;
}

cudaError_t grad(Sum what, bool state_bf16, const void* dY, forge_dtype dy_dtype, const void* ids,
                 forge_dtype id_dtype, int64_t T, int64_t V, int64_t D, float scale, float* dW,
                 const Params& p, int sms, cudaStream_t s)
{
    const bool wide = id_dtype == FORGE_I64;
    const uintptr_t sa = state_bf16 ? 8 : 16;
    const bool flat = aligned(dW, 16) && aligned(p.W, 16) && aligned(p.s1, sa) && aligned(p.s2, sa);
    const bool vec = flat && D % 4 == 0 && aligned(dY, 4 * size_of(dy_dtype));
    auto go = [&](auto* d) {
        using G = std::remove_cv_t<std::remove_pointer_t<decltype(d)>>;
        if (vec)
            return launch_grad<G, LIE_VECTORS>(what, state_bf16, d, ids, wide, T, V, D, scale, dW, p, sms, s);
        if (flat && D >= 4)
            return launch_grad<G, LIE_FLAT>(what, state_bf16, d, ids, wide, T, V, D, scale, dW, p, sms, s);
        return launch_grad<G, LIE_ANY>(what, state_bf16, d, ids, wide, T, V, D, scale, dW, p, sms, s);
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
        constexpr int64_t per = kLookupVec<A, B>;
        constexpr int flight = per * sizeof(A) < 16 ? 8 : 4;
        auto launch = [&](auto kernel, int64_t columns, int tokens = 1) {
            if (T < 32LL * sms) tokens = 1;  // a warp each
            const int64_t units = (T + tokens - 1) / tokens * ((D + columns - 1) / columns);
            const int64_t want = (units + kThreads / 32 - 1) / (kThreads / 32);
            // 64 blocks an SM: a few spans a warp, and blocks that end are replaced
            // (65536 x 4096 fp32 to bf16, Zipf tokens: 153 us; eight resident ones 157)
            const int blocks = static_cast<int>(want < 64LL * sms ? want : 64LL * sms);
            const int64_t spans = (D + columns - 1) / columns, warps = blocks * (kThreads / 32);
            kernel<<<blocks, kThreads, 0, s>>>(ids, id_dtype == FORGE_I64, w, y, T, V, D, scale,
                                               Divide(spans), warps / spans, warps % spans, status);
        };
        if (D % per == 0 && aligned(w, per * sizeof(A)) && aligned(y, per * sizeof(B))) {
            if (D <= 32 * per)
                launch(forge_embedding_kernel<A, B, true, 1, 4>, 32 * per, 4);
            else if (D <= 64 * per)
                launch(forge_embedding_kernel<A, B, true, 2, 2>, 64 * per, 2);
            else
                launch(forge_embedding_kernel<A, B, true, flight, 1>, 32 * per * flight);
        } else if (D <= 128) {
            launch(forge_embedding_kernel<A, B, false, 4, 4>, 128, 4);
        } else if (D <= 256) {
            launch(forge_embedding_kernel<A, B, false, 8, 2>, 256, 2);
        } else {
            launch(forge_embedding_kernel<A, B, false, 16, 1>, 512);
        }
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
    return reported(grad(accumulate ? SUM_ADD : SUM_STORE, false, dY, dy_dtype, ids, id_dtype,
                         T, V, D, scale, dW, p, sms, s));
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
    return reported(grad(SUM_ADAMW, state_dtype == FORGE_BF16, dY, dy_dtype, ids, id_dtype, T,
                         V, D, scale, nullptr, p, sms, s));
}
