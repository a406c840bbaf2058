// forge_route.cu -- a router's choice of k experts for each token, with the
// choices' places in a buffer packed by expert, per-expert counts, offsets
// and the balance loss, and the gradient by the router's logits.
//
// For token t with logits z [E]:  p = softmax(z), the k largest z (equal ones by
// the lower expert), weights p of the chosen (over their sum when normalised).
// A token without a finite logit is padding: it chooses nothing and counts
// nowhere.  With n the tokens that count, c_e the tokens that chose e and
// P_e = (1/n) sum_t p_te,
//   loss = E / (k n) sum_e c_e P_e.
// Gradient, the counts being constants:  q_te = gl E c_e / (k n^2) + (a_te),
//   dz = p (q - sum_e p q),   a_te = gw_tj where e is choice j, or normalised
//   (gw_tj - sum_i gw_ti w_ti) / S_t with S_t the sum of the chosen p.
//
// Three launches.  Tokens: a group of lanes a token (each lane up to eight,
// sixteen or thirty-two neighbouring experts in registers), k rounds of the
// group's maximum; per block of tokens the counts and the sums of p.  Scan: a
// warp an expert over the blocks.  Place: a choice's slot is its expert's
// offset, plus the earlier blocks' count, plus the earlier tokens of its own
// block, which 32-bit masks (one bit a token, a token chooses an expert at
// most once) count with popc.  No atomics: slots are in token order and sums in
// a fixed one, so that results are bitwise the same from run to run.  Batches
// of one block's tokens take one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "forge.h"
#include "forge_device.h"
#include "forge_rows.cuh"

namespace forge {
namespace route {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kMostChoices = 2048;   // tokens of a block x k
constexpr int kMostMasks = 4096;     // words of 32 tokens of a block x E
constexpr int kMostWords = 8;

struct Args {
    int64_t T, ld;
    int32_t E, k, words;  // words: a block's tokens / 32
    bool normalize;
    int32_t* experts;
    float* weights;
    int32_t *counts, *offsets, *slots, *rows, *live;
    float* loss;
    // scratch: [E + 1][blocks] counts (the last row: tokens that count), [E][blocks]
    // sums of p, then the totals of both
    int32_t blocks;
    int32_t* part;
    float* psum;
    int32_t* total;
    float* ptotal;
};

// Logits as integers of the same order: equal values are equal (-0 as 0), NaN
// is above all.
__device__ __forceinline__ int32_t key_of(float v)
{
    const int32_t b = __float_as_int(v + 0.0f);
    return v != v ? INT_MAX : (b < 0 ? b ^ 0x7FFFFFFF : b);
}
__device__ __forceinline__ float value_of(int32_t key)
{
    return __int_as_float(key < 0 ? key ^ 0x7FFFFFFF : key);
}
constexpr int32_t kNone = static_cast<int32_t>(0x807FFFFF);  // key_of(-inf)

template <int LANES>
__device__ __forceinline__ int32_t lanes_max(int32_t v)
{
    if constexpr (LANES == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}

template <typename X>
__device__ __forceinline__ float load1(const X* p)
{
    return entry(load_packed<X, 1>(p), 0);
}

// The masks of a block's choices: bit i of mask[w][e] is set where token 32 w + i
// chose e.  A warp takes a word; `choice(token, j)` gives a choice or -1.
template <typename F>
__device__ __forceinline__ void make_masks(uint32_t* mask, const Args& p, F choice)
{
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < p.words * p.E; i += kThreads) mask[i] = 0;
    __syncthreads();
    for (int w = threadIdx.x >> 5; w < p.words; w += kWarps) {
        for (int j = 0; j < p.k; ++j) {
            const int e = choice(32 * w + lane, j);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && (same & ((1u << lane) - 1)) == 0) mask[w * p.E + e] |= same;
            __syncwarp();
        }
    }
    __syncthreads();
}

// offsets [E + 1] (shared memory) of counts that `count(e)` gives; all threads.
template <typename F>
__device__ __forceinline__ void make_offsets(int32_t* offs, int E, F count)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int32_t sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int32_t n = e0 + lane < E ? count(e0 + lane) : 0;
            int32_t up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += v;
            }
            if (e0 + lane < E) offs[e0 + lane] = sum + up - n;
            sum += __shfl_sync(0xffffffffu, up, 31);
        }
        if (lane == 0) offs[E] = sum;
    }
    __syncthreads();
}

// What one block writes for the whole call: counts, offsets, live and the loss.
template <typename C, typename S>
__device__ __forceinline__ void write_totals(const Args& p, const int32_t* offs, int32_t live,
                                             C count, S mass)
{
    for (int e = threadIdx.x; e <= p.E; e += kThreads) {
        p.offsets[e] = offs[e];
        if (e < p.E) p.counts[e] = count(e);
    }
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int e = threadIdx.x; e < p.E; e += 32) s += static_cast<double>(count(e)) * mass(e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            const double n = live > 0 ? live : 1;
            if (p.loss) *p.loss = static_cast<float>(s * p.E / (n * n * p.k));
            if (p.live) *p.live = live;
        }
    }
}

// Slots and packed rows of a block's choices; base[e]: the first slot of the
// block's choices of e.  `first`: the block's first token.
template <typename F>
__device__ __forceinline__ void place(const Args& p, int64_t first, const uint32_t* mask,
                                      int32_t* base, F choice)
{
    // base[w][e]: the earlier words' choices added
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        int32_t at = base[e];
        for (int w = 0; w < p.words; ++w) {
            base[w * p.E + e] = at;
            at += __popc(mask[w * p.E + e]);
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int w = threadIdx.x >> 5; w < p.words; w += kWarps) {
        const int64_t t = first + 32 * w + lane;
        if (t >= p.T) continue;
        for (int j = 0; j < p.k; ++j) {
            const int e = choice(32 * w + lane, j);
            int32_t slot = -1;
            if (e >= 0)
                slot = base[w * p.E + e] + __popc(mask[w * p.E + e] & ((1u << lane) - 1));
            if (p.slots) p.slots[t * p.k + j] = slot;
            if (p.rows && slot >= 0) p.rows[slot] = static_cast<int32_t>(t);
        }
    }
}

// LPR lanes a token, EPL experts a lane.  ONE: the call's only block.
template <typename X, int LPR, int EPL, bool ONE>
__global__ void __launch_bounds__(kThreads)
    forge_route_tokens_kernel(const X* __restrict__ logits, const Args p)
{
    extern __shared__ uint8_t smem[];
    const int C = 32 * p.words;
    int32_t* chosen = reinterpret_cast<int32_t*>(smem);                 // [C][k]
    float* weight = reinterpret_cast<float*>(chosen + C * p.k);         // [C][k], before division
    float* inverse = weight + C * p.k;                                  // [C]
    uint32_t* mask = reinterpret_cast<uint32_t*>(inverse + C);          // [words][E]
    float* mass = reinterpret_cast<float*>(mask + p.words * p.E);       // [warps][E]
    int32_t* base = reinterpret_cast<int32_t*>(mass + kWarps * p.E);    // ONE: [words][E]
    int32_t* offs = base + p.words * p.E;                               // ONE: [E + 1]
    __shared__ int32_t lives[kWarps];

    constexpr int G = kThreads / LPR;  // tokens at once
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const uint32_t group = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (lane / LPR * LPR);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * C;
    float sums[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) sums[i] = 0.0f;
    int32_t live_count = 0;
    for (int r0 = 0; r0 < C; r0 += G) {
        const int r = r0 + g;
        const bool in = r < C && first + r < p.T;
        const X* row = logits + (in ? (first + r) * p.ld : 0);
        int32_t key[EPL];
        float e[EPL];
        int32_t best = kNone;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int x = l * EPL + i;
            key[i] = in && x < p.E ? key_of(load1(row + x)) : kNone;
            best = max(best, key[i]);
        }
        const int32_t top = lanes_max<LPR>(best);
        const bool live = top > kNone;
        live_count += live && l == 0;
        const float m = live ? value_of(top) : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            e[i] = __expf(value_of(key[i]) - m);
            s += e[i];
        }
        s = lanes_sum<LPR>(s);
        const float inv = live ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sums[i] = live ? fmaf(e[i], inv, sums[i]) : sums[i];
        float sum = 0.0f;  // of the chosen
        for (int j = 0; j < p.k; ++j) {
            const int32_t t = lanes_max<LPR>(best);
            const uint32_t who = __ballot_sync(0xffffffffu, best == t) & group;
            const bool mine = lane == __ffs(who) - 1;
            const float w = t > kNone ? __expf(value_of(t) - m) : 0.0f;
            sum += w;
            if (mine) {
                int at = -1;
                best = kNone;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const bool it = at < 0 && key[i] == t;
                    at = it ? i : at;
                    key[i] = it ? kNone : key[i];
                    best = max(best, key[i]);
                }
                if (r < C) {
                    chosen[r * p.k + j] = t > kNone ? l * EPL + at : -1;
                    weight[r * p.k + j] = w;
                }
            }
        }
        if (l == 0 && r < C) inverse[r] = !live ? 0.0f : (p.normalize ? 1.0f / sum : inv);
    }
    __syncthreads();
    const int64_t left = p.T - first;
    const int tokens = left < C ? static_cast<int>(left) : C;
    for (int i = threadIdx.x; i < tokens * p.k; i += kThreads) {
        p.experts[first * p.k + i] = chosen[i];
        p.weights[first * p.k + i] = weight[i] * inverse[i / p.k];
    }
    auto choice = [&](int t, int j) { return chosen[t * p.k + j]; };
    make_masks(mask, p, choice);
    // sums of p: lanes with the same experts, then the warps in order
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
        if (lane < LPR && l * EPL + i < p.E) mass[warp * p.E + l * EPL + i] = sums[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) live_count += __shfl_xor_sync(0xffffffffu, live_count, o);
    if (lane == 0) lives[warp] = live_count;
    __syncthreads();
    int32_t lives_here = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lives_here += lives[w];
    auto count_of = [&](int x) {
        int32_t n = 0;
        for (int w = 0; w < p.words; ++w) n += __popc(mask[w * p.E + x]);
        return n;
    };
    auto mass_of = [&](int x) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += mass[w * p.E + x];
        return s;
    };
    if constexpr (ONE) {
        make_offsets(offs, p.E, count_of);
        write_totals(p, offs, lives_here, count_of, mass_of);
        for (int x = threadIdx.x; x < p.E; x += kThreads) base[x] = offs[x];
        __syncthreads();
        place(p, first, mask, base, choice);
        if (p.rows)
            for (int64_t i = offs[p.E] + threadIdx.x; i < p.T * p.k; i += kThreads) p.rows[i] = -1;
    } else {
        for (int x = threadIdx.x; x < p.E; x += kThreads) {
            p.part[static_cast<int64_t>(x) * p.blocks + blockIdx.x] = count_of(x);
            p.psum[static_cast<int64_t>(x) * p.blocks + blockIdx.x] = mass_of(x);
        }
        if (threadIdx.x == 0)
            p.part[static_cast<int64_t>(p.E) * p.blocks + blockIdx.x] = lives_here;
        let_dependents_start();
    }
}

// A warp a row of part: its exclusive sums over the blocks in place, and the totals.
__global__ void __launch_bounds__(kThreads) forge_route_scan_kernel(const Args p)
{
    await_prerequisites();
    const int e = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e <= p.E) {
        int32_t* part = p.part + static_cast<int64_t>(e) * p.blocks;
        const float* psum = p.psum + static_cast<int64_t>(e) * p.blocks;
        int32_t sum = 0;
        float mass = 0.0f;
        for (int b0 = 0; b0 < p.blocks; b0 += 32) {
            const int b = b0 + lane;
            const int32_t n = b < p.blocks ? part[b] : 0;
            if (e < p.E && b < p.blocks) mass += psum[b];
            int32_t up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += v;
            }
            if (b < p.blocks) part[b] = sum + up - n;
            sum += __shfl_sync(0xffffffffu, up, 31);
        }
        mass = lanes_sum<32>(mass);
        if (lane == 0) {
            p.total[e] = sum;
            if (e < p.E) p.ptotal[e] = mass;
        }
    }
    let_dependents_start();
}

__global__ void __launch_bounds__(kThreads) forge_route_place_kernel(const Args p)
{
    extern __shared__ uint8_t smem[];
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem);                  // [words][E]
    int32_t* base = reinterpret_cast<int32_t*>(mask + p.words * p.E);    // [words][E]
    int32_t* offs = base + p.words * p.E;                                // [E + 1]
    await_prerequisites();
    make_offsets(offs, p.E, [&](int e) { return p.total[e]; });
    if (blockIdx.x == 0)
        write_totals(
            p, offs, p.total[p.E], [&](int e) { return p.total[e]; },
            [&](int e) { return p.ptotal[e]; });
    if (!p.slots && !p.rows) return;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * 32 * p.words;
    auto choice = [&](int t, int j) {
        return first + t < p.T ? p.experts[(first + t) * p.k + j] : -1;
    };
    for (int e = threadIdx.x; e < p.E; e += kThreads)
        base[e] = offs[e] + p.part[static_cast<int64_t>(e) * p.blocks + blockIdx.x];
    make_masks(mask, p, choice);
    place(p, first, mask, base, choice);
    if (p.rows) {
        const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
        for (int64_t i = offs[p.E] + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
             i < p.T * p.k; i += step)
            p.rows[i] = -1;
    }
}

struct GradArgs {
    int64_t T, ld, ld_out;
    int32_t E, k;
    bool normalize;
    const int32_t *experts, *counts, *live;
    const float *grad_weights, *grad_loss;
    void* dlogits;
    bool f32;
};

template <typename X, int LPR, int EPL>
__global__ void __launch_bounds__(kThreads)
    forge_route_grad_kernel(const X* __restrict__ logits, const GradArgs p)
{
    constexpr int G = kThreads / LPR;
    const int l = threadIdx.x % LPR;
    float c[EPL];  // the loss's q
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = 0.0f;
    if (p.grad_loss) {
        const float n = fmaxf(1.0f, static_cast<float>(*p.live));
        const float f = *p.grad_loss * static_cast<float>(p.E) / (static_cast<float>(p.k) * n);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (l * EPL + i < p.E) c[i] = f * (static_cast<float>(p.counts[l * EPL + i]) / n);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * G; t0 < p.T; t0 += step) {
        const int64_t t = t0 + threadIdx.x / LPR;
        const bool in = t < p.T;
        const X* row = logits + (in ? t * p.ld : 0);
        float v[EPL];
        float m = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = in && l * EPL + i < p.E ? load1(row + l * EPL + i) : -INFINITY;
            nan |= v[i] != v[i];
            m = fmaxf(m, v[i]);
        }
        m = nan ? INFINITY : m;  // (every p of a row with a NaN is NaN, as with +inf)
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.0f : m;
        float gw[EPL];
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) gw[i] = 0.0f;
        if (p.grad_weights && in) {
            for (int j = 0; j < p.k; ++j) {
                const int e = p.experts[t * p.k + j];
                const float w = p.grad_weights[t * p.k + j];
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e == l * EPL + i) {
                        gw[i] = w;
                        hit |= 1u << i;
                    }
            }
        }
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // exp, exp c, chosen exp, chosen exp gw
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = __expf(v[i] - ref);
            s[0] += v[i];
            s[1] = fmaf(v[i], c[i], s[1]);
            s[2] += hit >> i & 1 ? v[i] : 0.0f;
            s[3] = fmaf(v[i], gw[i], s[3]);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < 4; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
        const float inv = s[0] != 0.0f ? 1.0f / s[0] : 0.0f;
        // normalised weights: (gw - sum gw w) / S; else gw as it is.  Then
        // sum p q = (exp c + exp by) / sum exp, the second sum 0 when normalised.
        const bool norm = p.normalize && s[2] > 0.0f;
        const float mean = norm ? s[3] / s[2] : 0.0f;
        const float over = norm ? s[0] / s[2] : 1.0f;
        const float pq = (s[1] + (p.normalize ? 0.0f : s[3])) * inv;
        float out[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float by = hit >> i & 1 ? (gw[i] - mean) * over : 0.0f;
            out[i] = v[i] * inv * (c[i] + by - pq);
        }
        if (in) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float one[1] = {out[i]};
                if (l * EPL + i < p.E) store_as(p.dlogits, p.f32, t * p.ld_out + l * EPL + i, one);
            }
        }
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : 4; }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }

// f(lanes a token, experts a lane) as compile-time values: up to eight experts a
// lane, more only where 32 lanes are not enough.
template <int LPR, int EPL>
struct Shape {
    static constexpr int lpr = LPR, epl = EPL;
};
template <typename F>
cudaError_t by_experts(int E, F f)
{
    if (E <= 8) return f(Shape<1, 8>());
    if (E <= 16) return f(Shape<2, 8>());
    if (E <= 32) return f(Shape<4, 8>());
    if (E <= 64) return f(Shape<8, 8>());
    if (E <= 128) return f(Shape<16, 8>());
    if (E <= 256) return f(Shape<32, 8>());
    if (E <= 512) return f(Shape<32, 16>());
    return f(Shape<32, 32>());
}

cudaError_t after(void (*kernel)(const Args), int grid, size_t smem, const Args& p, cudaStream_t s)
{
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename X>
cudaError_t forward(const X* logits, Args p, int sms, cudaStream_t s)
{
    // a block's words: as many as leave every SM four blocks, within the room
    int most = kMostChoices / (32 * p.k);
    if (most > kMostMasks / p.E) most = kMostMasks / p.E;
    if (most > kMostWords) most = kMostWords;
    if (most < 1) most = 1;
    const int64_t all = (p.T + 31) / 32;
    int64_t words = all <= most ? all : all / (4LL * sms);
    p.words = static_cast<int>(words < 1 ? 1 : (words > most ? most : words));
    const int64_t blocks = (all + p.words - 1) / p.words;
    if (blocks > INT32_MAX / 2) return cudaErrorInvalidValue;
    p.blocks = static_cast<int32_t>(blocks < 1 ? 1 : blocks);
    const bool one = p.blocks == 1;
    const size_t C = 32 * p.words;
    const size_t tokens_smem =
        4 * (2 * C * p.k + C + static_cast<size_t>(p.words) * p.E + static_cast<size_t>(kWarps) * p.E +
             (one ? static_cast<size_t>(p.words) * p.E + p.E + 1 : 0));
    const size_t place_smem = 4 * (2 * static_cast<size_t>(p.words) * p.E + p.E + 1);
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (!one) {
        const int64_t rows = p.E + 1, cells = rows * p.blocks;
        e = scratch_alloc(&scratch, 4 * (2 * cells + 2 * rows), s);
        if (e != cudaSuccess) return e;
        p.part = static_cast<int32_t*>(scratch);
        p.psum = reinterpret_cast<float*>(p.part + cells);
        p.total = reinterpret_cast<int32_t*>(p.psum + cells);
        p.ptotal = reinterpret_cast<float*>(p.total + rows);
    }
    e = by_experts(p.E, [&](auto shape) {
        auto kernel = one ? forge_route_tokens_kernel<X, shape.lpr, shape.epl, true>
                          : forge_route_tokens_kernel<X, shape.lpr, shape.epl, false>;
        if (tokens_smem > 48 * 1024) {
            const cudaError_t f = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
            if (f != cudaSuccess) return f;
        }
        kernel<<<p.blocks, kThreads, tokens_smem, s>>>(logits, p);
        return cudaGetLastError();
    });
    if (e == cudaSuccess && !one) {
        e = after(forge_route_scan_kernel, (p.E + kWarps) / kWarps, 0, p, s);
        if (e == cudaSuccess)
            e = after(forge_route_place_kernel, p.slots || p.rows ? p.blocks : 1, place_smem, p, s);
    }
    if (scratch) {
        const cudaError_t fe = scratch_free(scratch, s);
        if (e == cudaSuccess) e = fe;
    }
    return e;
}

forge_status check_sizes(int64_t T, int32_t E, int64_t ld, int32_t k)
{
    if (T < 0 || E < 1 || E > kMaxExperts || ld < E || k < 1 || k > kMaxTop || k > E ||
        T > INT32_MAX / k)
        return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

}  // namespace route
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_moe_route(const void* logits, forge_dtype dtype, int64_t T, int32_t E,
                                        int64_t ld, int32_t k, int32_t normalize, int32_t* experts,
                                        float* weights, int32_t* counts, int32_t* offsets,
                                        int32_t* slots, int32_t* rows, int32_t* live, float* loss,
                                        forge_stream_t stream)
{
    using namespace route;
    if (!counts || !offsets || (T > 0 && (!logits || !experts || !weights)))
        return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(T, E, ld, k);
    if (st != FORGE_OK) return st;
    if (!is_float(dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(logits, size_of(dtype)) || !aligned(experts, 4) || !aligned(weights, 4) ||
        !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(slots, 4) || !aligned(rows, 4) ||
        !aligned(live, 4) || !aligned(loss, 4))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const bool any = T > 0;
    const void* ptrs[] = {any ? logits : nullptr,  any ? experts : nullptr,
                          any ? weights : nullptr, any ? slots : nullptr,
                          any ? rows : nullptr,    counts,
                          offsets,                 live,
                          loss};
    if ((st = device_resident(ptrs, 9)) != FORGE_OK) return st;
    Args p{};
    p.T = T;
    p.ld = ld;
    p.E = E;
    p.k = k;
    p.normalize = normalize != 0;
    p.experts = experts;
    p.weights = weights;
    p.counts = counts;
    p.offsets = offsets;
    p.slots = slots;
    p.rows = rows;
    p.live = live;
    p.loss = loss;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == FORGE_F32 ? forward(static_cast<const float*>(logits), p, sms, s)
                           : forward(static_cast<const __nv_bfloat16*>(logits), p, sms, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_moe_route_grad(const void* logits, forge_dtype dtype, int64_t T,
                                             int32_t E, int64_t ld, int32_t k, int32_t normalize,
                                             const int32_t* experts, const int32_t* counts,
                                             const int32_t* live, const float* grad_weights,
                                             const float* grad_loss, void* dlogits,
                                             forge_dtype out_dtype, int64_t ld_out,
                                             forge_stream_t stream)
{
    using namespace route;
    if ((grad_loss && (!counts || !live)) ||
        (T > 0 && (!logits || !dlogits || (grad_weights && !experts))))
        return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(T, E, ld, k);
    if (st != FORGE_OK) return st;
    if (ld_out < E) return FORGE_ERR_INVALID_ARG;
    if (!is_float(dtype) || !is_float(out_dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(out_dtype)) ||
        !aligned(experts, 4) || !aligned(counts, 4) || !aligned(live, 4) ||
        !aligned(grad_weights, 4) || !aligned(grad_loss, 4))
        return FORGE_ERR_MISALIGNED;
    const int64_t es = size_of(dtype), eo = size_of(out_dtype);
    const bool in_place = logits == dlogits && es == eo && (ld == ld_out || T == 1);
    if (T > 0 && !in_place &&
        rows_overlap(reinterpret_cast<uintptr_t>(logits), E * es, ld * es,
                     reinterpret_cast<uintptr_t>(dlogits), E * eo, ld_out * eo, T))
        return FORGE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (T == 0) return FORGE_OK;
    const void* ptrs[] = {logits, experts, counts, live, grad_weights, grad_loss, dlogits};
    if ((st = device_resident(ptrs, 7)) != FORGE_OK) return st;
    const GradArgs p{T,      ld,   ld_out,       E,         k,       normalize != 0,
                     experts, counts, live, grad_weights, grad_loss, dlogits, out_dtype == FORGE_F32};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto* x) {
        return by_experts(E, [&](auto shape) {
            const int64_t want = (T * shape.lpr + kThreads - 1) / kThreads, most = 8LL * sms;
            using X = std::remove_cv_t<std::remove_pointer_t<decltype(x)>>;
            forge_route_grad_kernel<X, shape.lpr, shape.epl>
                <<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, s>>>(x, p);
            return cudaGetLastError();
        });
    };
    const cudaError_t e = dtype == FORGE_F32 ? go(static_cast<const float*>(logits))
                                             : go(static_cast<const __nv_bfloat16*>(logits));
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
