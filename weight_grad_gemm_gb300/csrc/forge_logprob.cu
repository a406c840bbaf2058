// forge_logprob.cu -- log-probabilities of given tokens under rows of logits,
// with entropy and the top alternatives, and their gradient.
//
// A row x [V] of logits and a scale s (the inverse temperature) give
//   z_j = s x_j,  lse = ln sum_j exp z_j,  p_j = exp(z_j - lse),
//   logprob = z_t - lse,  H = -sum_j p_j ln p_j,
// and, for weights a of logprob and b of H,
//   d(a logprob + b H) / dx_j = s (a (1[j = t] - p_j) - b p_j (ln p_j + H)).
// Rows whose target is negative are padding: nothing of them counts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "forge.h"
#include "forge_device.h"

namespace forge {
namespace logprob {

constexpr int kMaxTop = 32;
constexpr int kWarps = 8;       // of a block
constexpr int kGroups = 64;     // most maxima that bound the top entries from below
constexpr int kRoom = 128;      // entries a warp holds before it keeps its best
constexpr float kFloor = -1000.0f;  // 2^kFloor is 0, and 0 * kFloor is not a NaN
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float nan_max(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two fp32 operations an instruction.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair(float a, float b)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ void split(Pair p, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// All blocks of the cluster have come here, and see what the others wrote.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared variable of the cluster's block q.
template <typename X>
__device__ __forceinline__ const X* remote(const X* p, int q)
{
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(p)), "r"(q));
    return reinterpret_cast<const X*>(a);
}

// Vectors of a thread in hand at once (a tile): short rows four, with the next
// four on their way, longer ones eight, other warps' loads covering the work on
// them: what a tile costs beside its elements then counts half.
template <int WARPS>
constexpr int kTile = WARPS == 1 ? 4 : 8;

// 16 bytes of a row: four fp32 or eight bf16 logits.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kNone = 0xFF800000u;  // -inf
    static __device__ __forceinline__ Pair two(const uint4& u, int i)
    {
        return i == 0 ? pair(__uint_as_float(u.x), __uint_as_float(u.y))
                      : pair(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        return __float_as_uint(nan_max(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float top(uint32_t a) { return __uint_as_float(a); }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;
    static __device__ __forceinline__ Pair two(const uint4& u, int i)
    {
        const uint32_t w = i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t y;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    static __device__ __forceinline__ float top(uint32_t a)
    {
        return nan_max(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    }
};
// The largest logit of a vector, still packed; a NaN wins.
template <typename T>
__device__ __forceinline__ uint32_t packed_max(const uint4& u)
{
    using X = Vec<T>;
    return X::max2(X::max2(u.x, u.y), X::max2(u.z, u.w));
}

// A row as whole aligned vectors of N elements and those before and after them.
struct Split {
    int64_t head;  // elements before the first aligned vector
    int64_t nvec;
    int64_t tail;  // elements after the last
};
template <int N, typename T>
__device__ __forceinline__ Split split_row(const T* x, int64_t V)
{
    const int64_t off =
        static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) & (N * sizeof(T) - 1)) / sizeof(T);
    int64_t head = off == 0 ? 0 : N - off;
    if (head > V) head = V;
    const int64_t nvec = (V - head) / N;
    return {head, nvec, V - head - nvec * N};
}

// The target of row r: -1 for padding.  A target past the vocabulary is
// recorded in the status word and its row taken as padding.
__device__ __forceinline__ int64_t target_of(const void* targets, bool wide, int64_t r, int64_t V,
                                             int* status)
{
    const int64_t t = wide ? static_cast<const int64_t*>(targets)[r]
                           : static_cast<const int32_t*>(targets)[r];
    if (t < 0) return -1;
    if (t >= V) {
        *reinterpret_cast<volatile int*>(status) = FORGE_ERR_INVALID_ARG;
        return -1;
    }
    return t;
}

// A logit and its column as one number: larger for the larger logit, then for
// the lower column.  NaN is the largest, and -0 equals 0.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v != v ? 0xFFFFFFFFu : b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kLowest = 0x00800000u;  // of the lowest finite number
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t rank_of(float v, int64_t column)
{
    return static_cast<uint64_t>(key_of(v)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(column));
}

// The online softmax of what a thread has seen: the largest logit m (raw), s =
// sum 2^d and w = sum 2^d d over d = (x - m) scale log2 e, and whether there was
// a NaN.
struct Stats {
    float m, s, w;
    bool nan;
};

struct Args {
    int64_t R, V, ld;
    const void* targets;
    int32_t wide;
    float scale;
    float* logprob;
    float* lse;
    float* entropy;
    int32_t top_k;
    int32_t* top_index;
    float* top_logprob;
    int* status;
};

// Entries a warp holds as candidates for the top ones.
struct Tops {
    uint64_t room[kRoom];
};
// The vectors whose maximum reached the bound when they passed, with their
// numbers: room for what the doublings of the row seen leave as a rule (with
// 64 + 4 k, 8192 x 131072 bf16 on one warp a row and five alternatives run over
// and take 512 instead of 324 us).
__host__ __device__ constexpr int list_of(int k) { return k > 0 ? 160 + 2 * k : 0; }

// The warp's n entries cut to the best k, in order; returns their number.
__device__ __forceinline__ int keep_best(uint64_t* room, int n, int k, int lane)
{
    uint64_t mine[kRoom / 32];
    int rank[kRoom / 32] = {};
#pragma unroll
    for (int i = 0; i < kRoom / 32; ++i) mine[i] = lane + 32 * i < n ? room[lane + 32 * i] : 0;
    for (int j = 0; j < n; ++j) {
        const uint64_t other = room[j];
#pragma unroll
        for (int i = 0; i < kRoom / 32; ++i) rank[i] += other > mine[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRoom / 32; ++i)
        if (lane + 32 * i < n && rank[i] < k) room[rank[i]] = mine[i];
    __syncwarp();
    return n < k ? n : k;
}

// The entries a warp holds, and the rank that the next one has to reach.
struct Held {
    uint64_t bound;
    int n;
};

__device__ __forceinline__ Held cut(Tops& w, Held h, int k, int lane)
{
    h.n = keep_best(w.room, h.n, k, lane);
    if (h.n == k && w.room[k - 1] > h.bound) h.bound = w.room[k - 1];
    return h;
}

// Adds one entry of each lane to the warp's room where it reaches the bound.
__device__ __forceinline__ Held offer(Tops& w, Held h, float v, int64_t column, bool live, int k,
                                      int lane)
{
    const uint64_t rank = rank_of(v, column);
    const bool pass = live && rank >= h.bound;
    const uint32_t all = __ballot_sync(0xffffffffu, pass);
    if (all == 0) return h;
    if (pass) w.room[h.n + __popc(all & ((1u << lane) - 1u))] = rank;
    h.n += __popc(all);
    __syncwarp();
    return h.n > kRoom - 32 ? cut(w, h, k, lane) : h;
}

// Keeps the entries of the noted vectors that reach the bound of now, a lane a
// vector; or, where a warp had more to note than its list takes, reads all its
// vectors again, first + lane + stride i, and offers their entries.
template <typename T>
__device__ __noinline__ Held look_into(Tops& w, const uint4* list, const int32_t* number, int noted,
                                       bool over, Held h, const uint4* xv, int64_t col0, int k,
                                       int lane, int32_t first, int32_t stride, int32_t nv)
{
    constexpr int N = Vec<T>::N;
    __syncwarp();
    for (int32_t i0 = 0; i0 < noted && !over; i0 += 32) {
        const int32_t i = i0 + lane;
        const bool live = i < noted;
        const uint4 u = live ? list[i] : make_uint4(0, 0, 0, 0);
        const int64_t column = col0 + static_cast<int64_t>(live ? number[i] : 0) * N;
        const float least = value_of(static_cast<uint32_t>(h.bound >> 32));
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            float x, y;
            split(Vec<T>::two(u, j), x, y);
            mask |= (!(x < least) ? 1u : 0u) << (2 * j) | (!(y < least) ? 2u : 0u) << (2 * j);
        }
        if (!live) mask = 0;
        if (!__any_sync(0xffffffffu, mask != 0)) continue;
        const int own = __popc(mask);
        int upto = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += up;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        const T* x = reinterpret_cast<const T*>(list + (live ? i : 0));
        if (h.n + all <= kRoom) {
            for (int at = h.n + upto - own; mask != 0; mask &= mask - 1) {
                const int j = __ffs(mask) - 1;
                w.room[at++] = rank_of(load1(x, j), column + j);
            }
            h.n += all;
            __syncwarp();
            if (h.n > kRoom - 32) h = cut(w, h, k, lane);
        } else {
#pragma unroll 1
            for (int j = 0; j < N; ++j) h = offer(w, h, load1(x, j), column + j, live, k, lane);
        }
    }
    constexpr int kLoads = 2;  // in flight
    const uint32_t end = static_cast<uint32_t>(col0) + static_cast<uint32_t>(nv) * N;
    for (int32_t v0 = first; v0 < nv && over; v0 += kLoads * stride) {
        uint4 u[kLoads];
#pragma unroll
        for (int f = 0; f < kLoads; ++f) {
            const int32_t v = v0 + f * stride + lane;
            u[f] = v < nv ? __ldg(xv + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int f = 0; f < kLoads; ++f) {
            const int32_t v = v0 + f * stride + lane;
            const bool live = v < nv;
            // a bound that is the rank of a vector's entry, found already in a lower column, has
            // to be exceeded; the row's end was offered before and lies past all vectors, as does
            // the column of a bound that is no entry
            const float least = value_of(static_cast<uint32_t>(h.bound >> 32)), top = Vec<T>::top(packed_max<T>(u[f]));
            const bool found = ~static_cast<uint32_t>(h.bound) < end;
            if (!__any_sync(0xffffffffu, live && !(found ? top <= least : top < least))) continue;
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                float a, b;
                split(Vec<T>::two(u[f], j), a, b);
                h = offer(w, h, a, col0 + static_cast<int64_t>(v) * N + 2 * j, live, k, lane);
                h = offer(w, h, b, col0 + static_cast<int64_t>(v) * N + 2 * j + 1, live, k, lane);
            }
        }
    }
    __syncwarp();
    return h;
}

// The joined statistics of a group of WIDTH lanes, in every lane of it: the
// maximum first, so that a lane rescales its sums once.
template <int WIDTH>
__device__ __forceinline__ void join_lanes(Stats& st, float c)
{
    if constexpr (WIDTH == 1) return;
    float m = st.m;
    int nan = st.nan ? 1 : 0;
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        nan |= __shfl_xor_sync(0xffffffffu, nan, o);
    }
    // a part without entries has s = w = 0 and m = -inf
    const float d = st.m == -INFINITY ? 0.0f : fmaxf((st.m - m) * c, kFloor);
    const float f = exp2_approx(d);
    float w = f * fmaf(d, st.s, st.w), s = f * st.s;
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    st = Stats{m, s, w, nan != 0};
}

// A row is the work of WARPS warps of a block (eight, or fewer where rows are
// short and a block takes several), or of a cluster of whole blocks where the
// rows are too few to fill the SMs.  Each element is read from memory once.
//
// The maximum of a thread's tile moves its reference only where it grows, so an
// element costs one exponential (of fp32, as are all sums), one addition to s
// and one to w, two elements an instruction.  A tile's sums start at zero and are
// added to the thread's (in one run over its part of the row, equal logits, whose
// roundings go one way, put lse off by up to 8e-5 in rows of 400000); the parts
// are joined by lanes, warps and blocks.  The entropy follows from the same sums:
// H = ln s - ln 2 w / s, both terms not negative.  Bound by HBM: 8192 x 131072
// bf16, no row padding, takes 297 us, 7.2 TB/s.
//
// Top entries: the threads' maxima so far, by groups of lanes, are distinct
// entries of the row, and what k of them reach bounds the k-th largest entry
// from below.  The bound is set after tiles 0, 1, 3, 7 ... and after the last.
// In the loop a tile costs one comparison of its maximum with the bound; its
// vectors that reach it, some five times k in all, are kept aside and looked
// into after the last bound, which leaves a few entries more than k.  What this
// costs is instructions: the same rows with five alternatives take 334 us, 6.4
// TB/s, with 32 396 us; looking at every vector's entries as they passed took
// 1149 and 3642 us.  Entries of -inf are never among them: where fewer than k
// others are, the first columns of -inf are added at the end (2048 x 131072 rows
// masked to three entries: 96 us, 400 with -inf in the lists).  More vectors
// than the list takes (masks of a finite value, equal logits) means that the
// warp reads its part again: 218-231 us.
template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(32 * kWarps, 4)
    forge_token_logprob_kernel(const T* logits, const Args p, int split)
{
    constexpr int N = Vec<T>::N;
    constexpr int kThreads = 32 * WARPS;       // of a row
    constexpr int kRows = kWarps / WARPS;      // of a block
    constexpr int kGroupLanes = kThreads > kGroups ? kThreads / kGroups : 1;
    constexpr int kUsed = kThreads / kGroupLanes;  // groups of a row: 32 or 64
    constexpr int F = kTile<WARPS>;
    extern __shared__ uint4 s_lists[];  // each warp's noted vectors, then all their numbers
    __shared__ Tops s_tops[TOP ? kWarps : 1];
    __shared__ float s_group[kRows][kUsed];
    __shared__ int s_held[kWarps];
    __shared__ Stats s_stats[kWarps];
    __shared__ Stats s_row[kRows];
    __shared__ uint64_t s_best[TOP ? kRows : 1][kMaxTop];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mine = warp / WARPS;             // the row's place in the block
    const int tid = threadIdx.x - mine * kThreads;
    const int rwarp = warp - mine * WARPS;
    auto sync = [&] {
        if constexpr (WARPS == 1)
            __syncwarp();
        else if constexpr (WARPS == kWarps)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "n"(kThreads) : "memory");
    };

    const int64_t block = blockIdx.x / split;
    const int part = static_cast<int>(blockIdx.x - block * split);
    const int64_t r = block * kRows + mine;
    if (r >= p.R) return;
    const T* x = logits + r * p.ld;
    const int k = p.top_k;
    const float c = p.scale * kLog2e;
    const Split sp = split_row<N>(x, p.V);
    const int64_t per = (sp.nvec + split - 1) / split;
    const int64_t v0 = part * per < sp.nvec ? part * per : sp.nvec;
    const int32_t nv = static_cast<int32_t>(v0 + per < sp.nvec ? per : sp.nvec - v0);
    const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head) + v0;
    const int64_t col0 = sp.head + v0 * N;

    // whole tiles are read without a check; the last one may end early
    const uint4 none = make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
    const int32_t whole = nv / (F * kThreads);
    const int32_t tiles = (nv + F * kThreads - 1) / (F * kThreads);
    const uint4* at = xv + tid;
    auto fetch = [&](int32_t tile, uint4 (&u)[F]) {
        if (tile < whole) {
#pragma unroll
            for (int f = 0; f < F; ++f) u[f] = __ldcs(at + f * kThreads);
        } else {
            const int32_t left = nv - tile * F * kThreads - tid;
#pragma unroll
            for (int f = 0; f < F; ++f) u[f] = f * kThreads < left ? __ldcs(at + f * kThreads) : none;
        }
        at += F * kThreads;
    };
    constexpr bool kAhead = F <= 4;
    uint4 next[kAhead ? F : 1];
    if constexpr (kAhead)  // on its way while the target comes
        if (tiles > 0) fetch(0, next);
    int64_t t = 0;
    if (p.targets) t = target_of(p.targets, p.wide, r, p.V, p.status);
    if (t < 0) {  // padding: all the row's warps leave
        if (part == 0) {
            if (tid == 0) {
                if (p.logprob) p.logprob[r] = 0.0f;
                if (p.lse) p.lse[r] = 0.0f;
                if (p.entropy) p.entropy[r] = 0.0f;
            }
            if constexpr (TOP)
                for (int i = tid; i < k; i += kThreads) {
                    p.top_index[r * k + i] = -1;
                    p.top_logprob[r * k + i] = 0.0f;
                }
        }
        return;
    }

    const float x_t = tid == 0 && p.logprob ? load1(x, t) : 0.0f;

    Stats st{-INFINITY, 0.0f, 0.0f, false};
    Tops& tops = s_tops[TOP ? warp : 0];
    const int room = list_of(k);
    uint4* const list = s_lists + warp * room;
    int32_t* const number = reinterpret_cast<int32_t*>(s_lists + kWarps * room) + warp * room;
    if constexpr (TOP)
        if (rwarp == 0) s_best[mine][lane] = 0;  // no entry
    // the warp's entries; -inf is never among them
    Held held{static_cast<uint64_t>(kLowest) << 32, 0};
    float bound_v = value_of(kLowest);  // the value that the loop's vectors have to reach
    int noted = 0;                 // the warp's vectors
    bool over = false;             // there were more than the list takes

    auto raise = [&](float m) {  // m moves the reference of the thread's sums
        if (m > st.m) {
            if (st.m != -INFINITY) {
                const float d = fmaxf((st.m - m) * c, kFloor);
                const float f = exp2_approx(d);
                st.w = f * fmaf(d, st.s, st.w);
                st.s *= f;
            }
            st.m = m;
        }
    };
    // A bound from the groups' maxima: the largest value found in some halvings
    // that at least k of them reach.  Only where `wait` is set are the
    // other warps' maxima those of now; an older one (a word is read whole, and
    // maxima only grow) leaves the bound lower, which changes what is looked
    // into but not what is found.
    auto tighten = [&](bool wait, int steps) {
        float g = st.m;
#pragma unroll
        for (int o = 1; o < kGroupLanes; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        volatile float* groups = s_group[mine];
        if constexpr (WARPS > 1) {
            if (tid % kGroupLanes == 0) groups[tid / kGroupLanes] = g;
            if (wait)
                sync();
            else
                __syncwarp();
        }
        const float a = WARPS > 1 ? groups[lane] : g;
        const float b = kUsed > 32 ? groups[lane + kUsed - 32] : -INFINITY;
        auto reach = [&](float v) {
            return __popc(__ballot_sync(0xffffffffu, a >= v)) +
                   (kUsed > 32 ? __popc(__ballot_sync(0xffffffffu, b >= v)) : 0);
        };
        // what all groups reach that have an entry, if they are k
        const uint32_t ka = key_of(a), kb = kUsed > 32 ? key_of(b) : 0;
        uint32_t least = ka >= kLowest ? ka : 0xFFFFFFFFu;
        if (kUsed > 32 && kb >= kLowest && kb < least) least = kb;
        float low = value_of(__reduce_min_sync(0xffffffffu, least));
        if (reach(value_of(kLowest)) < k) return;
        low = fmaxf(low, bound_v);
        float high = value_of(__reduce_max_sync(0xffffffffu, ka > kb ? ka : kb));
        // only what lies within 2^256 in probability of the largest entry is halved: below
        // that stand masks, and all groups' bound serves
        const float down = high - __fdividef(256.0f, c);
        if (low < down && reach(down) >= k) low = down;
        if (low >= down)
            for (int i = 0; i < steps; ++i) {
                const float middle = 0.5f * (low + high);
                if (reach(middle) >= k)
                    low = middle;
                else
                    high = middle;
            }
        bound_v = fmaxf(bound_v, low);
    };

    // the elements outside whole vectors: the first warp of the row
    if (part == 0 && rwarp == 0 && sp.head + sp.tail > 0) {
        const bool live = lane < 8 ? lane < sp.head : lane - 8 < sp.tail;
        const int64_t column = lane < 8 ? lane : p.V - sp.tail + (lane - 8);
        const float v = live ? load1(x, column) : -INFINITY;
        st.nan = v != v;
        raise(v);
        if (v > -INFINITY) {
            const float d = fmaxf((v - st.m) * c, kFloor);
            const float e = exp2_approx(d);
            st.s += e;
            st.w = fmaf(e, d, st.w);
        }
        if constexpr (TOP) held = offer(tops, held, v, column, live, k, lane);
    }

    uint32_t seen = Vec<T>::kNone;  // the packed maximum of everything: keeps a NaN
    for (int32_t tile = 0; tile < tiles; ++tile) {
        uint4 u[F];
        if constexpr (kAhead) {
#pragma unroll
            for (int f = 0; f < F; ++f) u[f] = next[f];
            if (tile + 1 < tiles) fetch(tile + 1, next);
        } else {
            fetch(tile, u);
        }
        uint32_t pm = packed_max<T>(u[0]);
#pragma unroll
        for (int f = 1; f < F; ++f) pm = Vec<T>::max2(pm, packed_max<T>(u[f]));
        seen = Vec<T>::max2(seen, pm);
        const float tm = Vec<T>::top(pm);
        raise(tm);
        if constexpr (TOP) {  // before the sums: the tile's registers end with them
            if (tile == 0 || ((tile & (tile + 1)) == 0 && tile + 1 < tiles)) tighten(tile == 0, 5);
            if (__any_sync(0xffffffffu, !(tm < bound_v))) {
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const int32_t v = (tile * F + f) * kThreads + tid;
                    const bool pass = !(Vec<T>::top(packed_max<T>(u[f])) < bound_v) && v < nv;
                    const uint32_t all = __ballot_sync(0xffffffffu, pass);
                    if (all == 0) continue;
                    if (noted <= room - 32) {
                        const int i = noted + __popc(all & ((1u << lane) - 1u));
                        if (pass) {
                            list[i] = u[f];
                            number[i] = v;
                        }
                        noted += __popc(all);
                    } else {
                        over = true;
                    }
                }
            }
        }
        const float mr = st.m == -INFINITY ? 0.0f : st.m;
        const Pair mm = pair(-mr, -mr), cc = pair(c, c);
        Pair s2 = pair(0.0f, 0.0f), w2 = s2;
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                float d0, d1;
                ::forge::logprob::split(mul2(add2(Vec<T>::two(u[f], i), mm), cc), d0, d1);
                d0 = fmaxf(d0, kFloor);
                d1 = fmaxf(d1, kFloor);
                const Pair e = pair(exp2_approx(d0), exp2_approx(d1));
                s2 = add2(s2, e);
                w2 = fma2(e, pair(d0, d1), w2);
            }
        float a, b;
        ::forge::logprob::split(s2, a, b);
        st.s += a + b;
        ::forge::logprob::split(w2, a, b);
        st.w += a + b;
    }
    if constexpr (TOP) {
        if (tiles > 1) tighten(false, 8);
        held.bound = static_cast<uint64_t>(key_of(bound_v)) << 32;
        held = look_into<T>(tops, list, number, noted, over, held, xv, col0, k, lane, tid - lane,
                            kThreads, nv);
    }
    const float top = Vec<T>::top(seen);
    st.nan = st.nan || top != top;

    // lanes, then warps
    join_lanes<32>(st, c);
    if (lane == 0) {
        s_stats[warp] = st;
        s_held[warp] = held.n;
    }
    sync();
    if (rwarp == 0) {
        st = s_stats[warp + lane % WARPS];
        join_lanes<WARPS>(st, c);
        if (lane == 0) s_row[mine] = st;
    }
    if constexpr (TOP) {
        // the best of the row's warps: an entry's place is the number of better ones
        for (int e = lane; e < held.n; e += 32) {
            const uint64_t own = tops.room[e];
            int rank = 0;
            for (int w = 0; w < WARPS; ++w) {
                const uint64_t* room = s_tops[mine * WARPS + w].room;
                const int nw = s_held[mine * WARPS + w];
                for (int j = 0; j < nw; ++j) rank += room[j] > own;
            }
            if (rank < k) s_best[mine][rank] = own;
        }
    }
    sync();

    // blocks of the row: the first one joins what the others left in shared memory
    if constexpr (WARPS == kWarps)
        if (split > 1) {
            cluster_barrier();
            if (part == 0) {
                if (warp == 0) {  // a lane for each block
                    const Stats* o = remote(&s_row[0], lane % split);
                    st = *o;
                    if (lane >= split) st = Stats{-INFINITY, 0.0f, 0.0f, false};
                    join_lanes<8>(st, c);
                    if (lane == 0) s_stats[0] = st;
                }
                if constexpr (TOP) {
                    // a warp for each block's best, which are in order: an entry's place
                    // is its own plus those of the better ones in the other lists
                    if (warp < split) tops.room[lane] = remote(&s_best[0][0], warp)[lane];
                    __syncthreads();
                    if (warp < split) {
                        const uint64_t own = tops.room[lane];
                        int rank = lane;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            if (w == warp || w >= split) continue;
                            int better = 0;
#pragma unroll
                            for (int b = kMaxTop / 2; b > 0; b >>= 1)
                                if (s_tops[w].room[better + b - 1] > own) better += b;
                            if (s_tops[w].room[better] > own) ++better;
                            rank += better;
                        }
                        if (own != 0 && rank < k) s_best[0][rank] = own;
                    }
                }
                __syncthreads();
            }
            cluster_barrier();  // no block leaves while its shared memory is read
            if (part != 0) return;
        }

    const Stats all = split > 1 ? s_stats[0] : s_row[mine];
    const bool bad = all.nan || all.m == INFINITY;
    const bool empty = !bad && all.m == -INFINITY;
    // relative to the largest logit, so that near entries keep their digits
    const float ln_s = logf(all.s);
    auto logprob_of = [&](float v) {
        if (bad) return NAN;
        if (empty || v == -INFINITY) return -INFINITY;
        return fmaf(p.scale, v - all.m, -ln_s);
    };
    if (tid == 0) {
        if (p.logprob) p.logprob[r] = logprob_of(x_t);
        if (p.lse) p.lse[r] = bad ? NAN : (empty ? -INFINITY : fmaf(p.scale, all.m, ln_s));
        if (p.entropy) p.entropy[r] = bad ? NAN : (empty ? 0.0f : ln_s - kLn2 * all.w / all.s);
    }
    if constexpr (TOP)
        if (rwarp == 0) {
            // fewer than k entries above -inf: the first columns of -inf follow, and as
            // fewer than k columns are not -inf they are among the first k
            const int have = __popc(__ballot_sync(0xffffffffu, lane < k && s_best[mine][lane] != 0));
            if (have < k) {
                const bool masked = lane < k && load1(x, lane) == -INFINITY;
                const uint32_t all = __ballot_sync(0xffffffffu, masked);
                const int at = have + __popc(all & ((1u << lane) - 1u));
                if (masked && at < k) s_best[mine][at] = rank_of(-INFINITY, lane);
                __syncwarp();
            }
        }
    if constexpr (TOP)
        for (int i = tid; i < k; i += kThreads) {
            const uint64_t e = s_best[mine][i];
            p.top_index[r * k + i] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(e));
            p.top_logprob[r * k + i] = logprob_of(value_of(static_cast<uint32_t>(e >> 32)));
        }
}

struct GradArgs {
    int64_t R, V, ld, ld_out;
    const void* targets;
    int32_t wide;
    float scale;
    const float* lse;
    const float* grad_logprob;
    const float* entropy;
    const float* grad_entropy;
    int* status;
};

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

// dx_j = s (a (1[j = t] - p_j) - b p_j (ln p_j + H)) = [j = t] s a - p_j (A + B d_j) with
// d = log2 p, A = s (a + b H), B = s b ln 2: one exponential an element, no
// reduction.  A block takes 4 vectors a thread of one row, of as many elements
// as make 16 bytes of the wider type: a warp then stores whole sectors.  Rows
// whose vectors do not meet the output's alignment go element by element.
// Bound by HBM (8192 x 131072 bf16 to bf16: 650 us, 6.5 TB/s; fp32 to fp32
// 1118 x 100525: 129 us, 6.9 TB/s).
constexpr int kGradThreads = 256;
constexpr int kFlight = 4;
template <typename T, typename O>
constexpr int kGradVec = 16 / (sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));
template <typename T, typename O, int WARPS>
constexpr int kGradSpan = 32 * WARPS * kFlight * kGradVec<T, O>;

// N logits as they lie in memory.
template <typename T, int N>
struct Group;
template <>
struct Group<__nv_bfloat16, 8> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ Pair two(int i) const { return Vec<__nv_bfloat16>::two(u, i); }
};
template <>
struct Group<__nv_bfloat16, 4> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ Pair two(int i) const
    {
        return Vec<__nv_bfloat16>::two(make_uint4(u.x, u.y, 0, 0), i);
    }
};
template <>
struct Group<float, 4> {
    uint4 u;
    __device__ __forceinline__ void load(const float* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ Pair two(int i) const { return Vec<float>::two(u, i); }
};

template <typename T, typename O, int WARPS>
__global__ void __launch_bounds__(kGradThreads)
    forge_token_logprob_grad_kernel(const T* logits, O* dlogits, const GradArgs p, uint32_t spans)
{
    constexpr int N = kGradVec<T, O>;
    constexpr int kThreads = 32 * WARPS;  // of a row
    constexpr int kSpan = kGradSpan<T, O, WARPS>;
    const int tid = threadIdx.x % kThreads;
    const uint32_t block = WARPS == kWarps ? blockIdx.x / spans : blockIdx.x;
    const int64_t span = WARPS == kWarps ? blockIdx.x - block * spans : 0;
    const int64_t r = static_cast<int64_t>(block) * (kWarps / WARPS) + threadIdx.x / kThreads;
    if (r >= p.R) return;
    const T* x = logits + r * p.ld;
    O* dx = dlogits + r * p.ld_out;
    const int64_t t = target_of(p.targets, p.wide, r, p.V, p.status);
    const float lse = p.lse[r];
    const bool dead = t < 0 || lse == -INFINITY;
    const float a = p.grad_logprob[r];
    const float b = p.grad_entropy ? p.grad_entropy[r] : 0.0f;
    const float h = p.grad_entropy ? p.entropy[r] : 0.0f;
    // a NaN among the logits has come as a NaN lse
    const float A = lse != lse ? lse : p.scale * fmaf(b, h, a), B = p.scale * b * kLn2;
    const float at_t = p.scale * a;
    auto one = [&](float v, int64_t j) {
        const float d = fmaxf(fmaf(v, p.scale, -lse) * kLog2e, kFloor);
        const float g = -exp2_approx(d) * fmaf(B, d, A);
        return j == t ? g + at_t : g;
    };

    const Split sp = split_row<N>(x, p.V);
    constexpr uintptr_t oa = N * sizeof(O) < 16 ? 8 : 16;
    const bool vec = (reinterpret_cast<uintptr_t>(dx + sp.head) & (oa - 1)) == 0;
    if (!vec) {
        const int64_t end = (span + 1) * kSpan < p.V ? (span + 1) * kSpan : p.V;
#pragma unroll 8
        for (int64_t j = span * kSpan + tid; j < end; j += kThreads)
            store1(dx, j, dead ? 0.0f : one(load1(x, j), j));
        return;
    }
    if (span == 0 && tid < 16) {
        const int i = tid & 7;
        if (i < (tid < 8 ? sp.head : sp.tail)) {
            const int64_t j = tid < 8 ? i : p.V - sp.tail + i;
            store1(dx, j, dead ? 0.0f : one(load1(x, j), j));
        }
    }
    const T* xv = x + sp.head;
    const int64_t v0 = span * kFlight * kThreads + tid;
    Group<T, N> u[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
        if (!dead && v0 + f * kThreads < sp.nvec) u[f].load(xv + (v0 + f * kThreads) * N);
    const Pair ss = pair(p.scale, p.scale), ll = pair(-lse, -lse), ee = pair(kLog2e, kLog2e);
    const Pair AA = pair(-A, -A), BB = pair(-B, -B);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
        const int64_t v = v0 + f * kThreads;
        if (v >= sp.nvec) continue;
        float g[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float d0, d1;
            ::forge::logprob::split(mul2(fma2(u[f].two(i), ss, ll), ee), d0, d1);
            d0 = fmaxf(d0, kFloor);
            d1 = fmaxf(d1, kFloor);
            const Pair e = pair(exp2_approx(d0), exp2_approx(d1));
            ::forge::logprob::split(mul2(e, fma2(BB, pair(d0, d1), AA)), g[2 * i], g[2 * i + 1]);
        }
        const int64_t j0 = sp.head + v * N;
        if (dead) {
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = 0.0f;
        } else if (t >= j0 && t < j0 + N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (j0 + i == t) g[i] += at_t;
        }
        store_vec<N>(dx + j0, g);
    }
}

template <typename T, int WARPS>
cudaError_t launch_forward(const T* x, const Args& p, int split, cudaStream_t s)
{
    constexpr int rows = kWarps / WARPS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.R + rows - 1) / rows * split));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = static_cast<size_t>(list_of(p.top_k)) * kWarps * (16 + 4);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return p.top_k > 0 ? cudaLaunchKernelEx(&cfg, forge_token_logprob_kernel<T, WARPS, true>, x, p, split)
                       : cudaLaunchKernelEx(&cfg, forge_token_logprob_kernel<T, WARPS, false>, x, p, split);
}

// Few warps a row, so that the joins at a row's end are few and other rows'
// loads cover them, but enough to bound many alternatives well.  us by one, two,
// four warps a row, 8192 rows of bf16 (vectors a row):
//   alternatives   none           5              20             32
//   1000           27  29  33     39  47  59     47  53  66     140 59  70
//   2000           47  48  49     60  70  88     98  80  96     212 88  103  (nine: 66 74 90)
//   4096           89  87  85     100 111 127    224 128 144    324 140 156
//   6250           133 133 133    142 157 181    324 181 205    429 196 220
//   8192           171 162 155    176 184 197    405 211 225    509 230 242
//   12288          252 239 228    250 260 266    577 289 301    680 325 322
//   16384          330 313 298    324 335 335    746 367 375    849 453 400
// Other numbers of rows end elsewhere in a wave, which costs one warp on a long
// row most.  Five alternatives, 6250 vectors: 1900 rows 50, 49, 53; 3600: 68, 81,
// 86; 5200: 108, 109, 121.  8192: 1900 rows 61, 57, 58; 3600: 83, 95, 94; 5200:
// 133, 127, 132.  12288: 2500 rows 114, 108, 99; 5200: 192, 180, 179.  16384: 2500
// rows 146, 138, 124; 6000: 273, 254, 251; with twenty 2500: 150 by two, 133 by
// four; 7000: 312, 324.
// More warps while the rows' warps do not fill the SMs and fewer would take the
// row in several tiles (bf16, five alternatives, 250 vectors, 1500 rows 6.9, 8.2;
// 400: 9.2, 8.2; 512 vectors, 600 rows 7.7, 5.9, 7.2; 700: 9.7, 7.7, 6.9; with
// twenty 137 vectors, 300 rows 7.4, 6.4, 6.9), then clusters of up to eight
// blocks, a join of which costs 1-2 us (114 x 10338 bf16, five: one block 7.2, two
// 8.7, four 11.7; 16 x 50001 fp32: 12.0, 11.0, 9.5, eight 9.0).
template <typename T>
cudaError_t forward(const T* x, const Args& p, int sms, cudaStream_t s)
{
    const int64_t nvec = p.V / Vec<T>::N;
    const int64_t one = p.top_k == 0 ? 4096 : (p.top_k <= 8 ? 7168 : (p.top_k <= 20 ? 1536 : 0));
    int warps = nvec <= one ? 1 : (nvec <= 12288 ? 2 : 4);
    auto enough = [&](int w) { return nvec > (w > 2 ? 128 * w : (p.top_k <= 8 ? 320 : 128)); };
    while (warps < kWarps && p.R * warps < 12 * sms && enough(2 * warps)) warps *= 2;
    if (warps == 1) return launch_forward<T, 1>(x, p, 1, s);
    if (warps == 2) return launch_forward<T, 2>(x, p, 1, s);
    if (warps == 4) return launch_forward<T, 4>(x, p, 1, s);
    int split = 1;
    while (split < 8 && p.R * split < 2 * sms && nvec / split >= 10 * 256) split *= 2;
    return launch_forward<T, 8>(x, p, split, s);
}

template <typename T, typename O, int WARPS>
cudaError_t launch_backward(const T* x, O* dx, const GradArgs& p, cudaStream_t s)
{
    constexpr int rows = kWarps / WARPS;
    const int64_t spans = (p.V + kGradSpan<T, O, WARPS> - 1) / kGradSpan<T, O, WARPS>;
    const int64_t rows_at_once = INT32_MAX / spans;
    for (int64_t r = 0; r < p.R; r += rows_at_once) {
        GradArgs q = p;
        q.R = p.R - r < rows_at_once ? p.R - r : rows_at_once;
        q.targets = static_cast<const uint8_t*>(p.targets) + r * (p.wide ? 8 : 4);
        q.lse += r;
        q.grad_logprob += r;
        if (q.grad_entropy) {
            q.entropy += r;
            q.grad_entropy += r;
        }
        forge_token_logprob_grad_kernel<T, O, WARPS>
            <<<static_cast<unsigned>((q.R + rows - 1) / rows * spans), kGradThreads, 0, s>>>(
                x + r * p.ld, dx + r * p.ld_out, q, static_cast<uint32_t>(spans));
    }
    return cudaGetLastError();
}

// As few warps a row as take it at once, so that short rows fill their blocks
// (10813 x 1155 bf16: 10.7 us, a block a row 24.5).
template <typename T, typename O>
cudaError_t backward(const T* x, O* dx, const GradArgs& p, cudaStream_t s)
{
    if (p.V <= kGradSpan<T, O, 1>) return launch_backward<T, O, 1>(x, dx, p, s);
    if (p.V <= kGradSpan<T, O, 2>) return launch_backward<T, O, 2>(x, dx, p, s);
    if (p.V <= kGradSpan<T, O, 4>) return launch_backward<T, O, 4>(x, dx, p, s);
    return launch_backward<T, O, 8>(x, dx, p, s);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : (t == FORGE_I64 ? 8 : 4); }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }
bool is_id(forge_dtype t) { return t == FORGE_I32 || t == FORGE_I64; }

forge_status check_rows(int64_t R, int64_t V, int64_t ld, float scale)
{
    if (R < 0 || V < 1 || ld < V || R > INT32_MAX || V > INT32_MAX) return FORGE_ERR_INVALID_ARG;
    // (scale log2 e stays finite)
    if (!(scale > 0.0f && scale <= 2e38f)) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

}  // namespace logprob
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_token_logprob(const void* logits, forge_dtype dtype, int64_t R,
                                            int64_t V, int64_t ld, const void* targets,
                                            forge_dtype id_dtype, float scale, float* logprob,
                                            float* lse, float* entropy, int32_t top_k,
                                            int32_t* top_index, float* top_logprob,
                                            forge_stream_t stream)
{
    using namespace logprob;
    if (R > 0 && (!logits || (logprob && !targets) ||
                  (top_k > 0 && (!top_index || !top_logprob))))
        return FORGE_ERR_INVALID_ARG;
    forge_status st = check_rows(R, V, ld, scale);
    if (st != FORGE_OK) return st;
    if (top_k < 0 || top_k > kMaxTop || top_k > V) return FORGE_ERR_INVALID_ARG;
    if (!is_float(dtype) || (targets && !is_id(id_dtype))) return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(logits, size_of(dtype)) || (targets && !aligned(targets, size_of(id_dtype))) ||
        !aligned(logprob, 4) || !aligned(lse, 4) || !aligned(entropy, 4) ||
        !aligned(top_index, 4) || !aligned(top_logprob, 4))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (R == 0) return FORGE_OK;
    const void* ptrs[] = {logits, targets, logprob, lse, entropy, top_k > 0 ? top_index : nullptr,
                          top_k > 0 ? top_logprob : nullptr};
    if ((st = device_resident(ptrs, 7)) != FORGE_OK) return st;
    const Args p{R,   V,       ld,    targets,   id_dtype == FORGE_I64, scale, logprob,
                 lse, entropy, top_k, top_index, top_logprob,           device_status_word()};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == FORGE_F32 ? forward(static_cast<const float*>(logits), p, sms, s)
                           : forward(static_cast<const __nv_bfloat16*>(logits), p, sms, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_token_logprob_grad(
    const void* logits, forge_dtype dtype, int64_t R, int64_t V, int64_t ld, const void* targets,
    forge_dtype id_dtype, float scale, const float* lse, const float* grad_logprob,
    const float* entropy, const float* grad_entropy, void* dlogits, forge_dtype out_dtype,
    int64_t ld_out, forge_stream_t stream)
{
    using namespace logprob;
    if (R > 0 && (!logits || !targets || !lse || !grad_logprob || !dlogits ||
                  (grad_entropy && !entropy)))
        return FORGE_ERR_INVALID_ARG;
    forge_status st = check_rows(R, V, ld, scale);
    if (st != FORGE_OK) return st;
    if (ld_out < V) return FORGE_ERR_INVALID_ARG;
    if (!is_float(dtype) || !is_float(out_dtype) || !is_id(id_dtype))
        return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(logits, size_of(dtype)) || !aligned(targets, size_of(id_dtype)) ||
        !aligned(lse, 4) || !aligned(grad_logprob, 4) || !aligned(entropy, 4) ||
        !aligned(grad_entropy, 4) || !aligned(dlogits, size_of(out_dtype)))
        return FORGE_ERR_MISALIGNED;
    const int64_t es = size_of(dtype), eo = size_of(out_dtype);
    const bool in_place = logits == dlogits && es == eo && (ld == ld_out || R == 1);
    if (R > 0 && !in_place &&
        rows_overlap(reinterpret_cast<uintptr_t>(logits), V * es, ld * es,
                     reinterpret_cast<uintptr_t>(dlogits), V * eo, ld_out * eo, R))
        return FORGE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (R == 0) return FORGE_OK;
    const void* ptrs[] = {logits, targets, lse, grad_logprob, entropy, grad_entropy, dlogits};
    if ((st = device_resident(ptrs, 7)) != FORGE_OK) return st;
    const GradArgs p{R,   V,            ld,      ld_out,       targets, id_dtype == FORGE_I64, scale,
                     lse, grad_logprob, entropy, grad_entropy, device_status_word()};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto in = [&](auto* x) {
        return out_dtype == FORGE_F32 ? backward(x, static_cast<float*>(dlogits), p, s)
                                      : backward(x, static_cast<__nv_bfloat16*>(dlogits), p, s);
    };
    const cudaError_t e = dtype == FORGE_F32 ? in(static_cast<const float*>(logits))
                                             : in(static_cast<const __nv_bfloat16*>(logits));
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
