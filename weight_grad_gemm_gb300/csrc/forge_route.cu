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
// Tokens: a group of lanes a token (each lane up to eight, sixteen or thirty-two
// neighbouring experts in registers), the k largest, and per block of tokens the
// counts, the sums of p and each choice's place among the block's choices of its
// expert: 32-bit masks (one bit a token, a token chooses an expert at most once) are
// counted with popc.  Scan: prefix sums over the blocks.  Place: a choice's slot is its
// expert's offset, the earlier blocks' count and its place in its own.  Few blocks
// scan in the place kernel; batches of one block's tokens take one launch.  No
// atomics: slots are in token order and sums in a fixed one, so that results are
// bitwise the same from run to run.
//
// Measured: 65536 x 256 fp32 to 8 and back 86 us, of it the tokens kernel 47 (bound by
// instructions: 74% of the issue slots beside 1.4 TB/s), scan 6 and place 12 (latency), the
// gradient 28 (4.7 TB/s over both ways, a third of it in L2; 65% of the issue slots).
// 16384 x 8 bf16 to 2 and back: 17 to 22 us for three launches; 16 x 8, one launch: 6.4.
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
// 65536 x 256 logits (the whole call): by rounds of the maximum 46 us at k = 1, 51 at 4, 56
// at 6, 60 at 8 and 71 at 12; by comparing all lanes 52, 54, 56, 59 and 64
constexpr int kMostRounds = 6;
// blocks x E that every place block scans by itself, which spares a launch: 1000 x 16 (2,016)
// in 10.4 us, with the scan kernel 10.5; 4096 x 64 (8,192) 26.6 and 13.5
constexpr int kFewCounts = 2048;

struct Args {
    int64_t T, ld;
    int32_t E, k, tokens, words;  // a block's tokens, and its masks' words of 32
    bool normalize, vec;  // vec: rows of logits in 16-byte loads
    int32_t* experts;
    float* weights;
    int32_t *counts, *offsets, *slots, *rows, *live;
    float* loss;
    // scratch: [blocks][E + 1] counts (the last column: tokens that count), [blocks][E]
    // sums of p, the totals of both, and the choices' places in their blocks
    int32_t blocks;
    int32_t* part;
    float* psum;
    int32_t* total;
    float* ptotal;
    uint16_t* place;
};

// Logits as integers of the same order: equal values are equal (-0 as 0), a NaN without
// its sign above all.  (One with its sign is below all: rows with a NaN sum take
// any_key_of.)
__device__ __forceinline__ int32_t key_of(float v)
{
    const int32_t b = __float_as_int(v + 0.0f);
    return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ int32_t any_key_of(float v) { return v != v ? INT_MAX : key_of(v); }
__device__ __forceinline__ float value_of(int32_t key)
{
    return __int_as_float(key < 0 ? key ^ 0x7FFFFFFF : key);
}
constexpr int32_t kNone = static_cast<int32_t>(0x807FFFFF);  // key_of(-inf)

// exp(v - m), m the row's largest logit.  The subtraction comes first: it is exact to half
// a step whatever the row's size, and 0 at the largest.  (As fma(v, log2 e, -m log2 e) the
// second product's rounding stays in the exponent, a factor that all of a row's terms have
// but that from |m| of some 1e9 on leaves fp32's range; 65536 x 256 to 8 and back takes 86 us
// either way.)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_from(float v, float m)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((v - m) * kLog2e));
    return y;
}

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

// EPL neighbouring logits of a row from x on, -inf past E (or everywhere: !in).
template <typename X, int EPL>
__device__ __forceinline__ void load_logits(float (&v)[EPL], const X* row, int x, int E, bool in,
                                            bool vec)
{
    constexpr int V = 16 / sizeof(X);
    if (vec && in && x + EPL <= E) {
#pragma unroll
        for (int i = 0; i < EPL; i += V) {
            const Packed<X, V> q = load_plain<X, V>(row + x + i);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i + j] = entry(q, j);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            v[i] = in && x + i < E ? entry(load_plain<X, 1>(row + x + i), 0) : -INFINITY;
    }
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

// offsets [E + 1] (shared memory) of counts that `count(e)` gives; all threads.  A lane of
// the first warp has a run of experts.
template <typename F>
__device__ __forceinline__ void make_offsets(int32_t* offs, int E, F count)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int run = (E + 31) / 32, lo = min(lane * run, E), hi = min(lo + run, E);
        int32_t sum = 0;
        for (int e = lo; e < hi; ++e) sum += count(e);
        int32_t up = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += v;
        }
        if (lane == 31) offs[E] = up;
        up -= sum;
        for (int e = lo; e < hi; ++e) {
            offs[e] = up;
            up += count(e);
        }
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
        const float n = live > 0 ? static_cast<float>(live) : 1.0f;
        float s = 0.0f;
        for (int e = threadIdx.x; e < p.E; e += 32)
            s = fmaf(static_cast<float>(count(e)) / n, mass(e), s);
        s = lanes_sum<32>(s);
        if (threadIdx.x == 0) {
            if (p.loss) *p.loss = s * (static_cast<float>(p.E) / (static_cast<float>(p.k) * n));
            if (p.live) *p.live = live;
        }
    }
}

// The k largest of a row of E > 128 logits, a warp a row, each lane EPL of them as keys:
// calls take(rank, key, expert) in one lane for each.  The k-th largest of the
// lanes' maxima bounds them from below; the few keys that reach it are gathered, one
// a lane, and ranked by comparing each with each.  Rows with more than 32 such keys
// (equal ones) take k rounds of the maximum.
template <int EPL, typename F>
__device__ __forceinline__ void top_of_warp(int32_t (&key)[EPL], int k, int32_t* list, F take)
{
    const int lane = threadIdx.x & 31;
    int32_t best = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
    int32_t bound = kNone;
    if (k > kMostRounds) {
        // (the lanes' maxima that fewer than k others exceed)
        list[lane] = best;
        __syncwarp();
        int above = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const int4 q = *reinterpret_cast<const int4*>(list + j);
            above += (q.x > best) + (q.y > best) + (q.z > best) + (q.w > best);
        }
        bound = __reduce_min_sync(0xffffffffu, above < k ? best : INT_MAX);
        __syncwarp();
    } else {
        int32_t left = best;
        for (int n = 0; n < k;) {
            bound = __reduce_max_sync(0xffffffffu, left);
            if (bound == kNone) break;
            const bool is = left == bound;
            n += __popc(__ballot_sync(0xffffffffu, is));
            left = is ? kNone : left;
        }
    }
    bound = max(bound, kNone + 1);
    int here = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) here += key[i] >= bound;
    int at = here;  // the lanes' before this one's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
    }
    const int found = __shfl_sync(0xffffffffu, at, 31);
    at -= here;
    if (here > 0 && found <= 32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] >= bound) {
                list[at] = key[i];
                list[32 + at++] = lane * EPL + i;
            }
    }
    __syncwarp();
    if (found <= 32) {
        // (the list is in the experts' order: of equal keys the earlier goes first.
        // What lies behind its end is below every key: -inf is not gathered)
        if (lane >= found) list[lane] = kNone;
        __syncwarp();
        const int32_t mine = list[lane], from = mine - 1;
        int rank = 0;
        for (int j = 0; j < found; j += 4) {
            const int4 q = *reinterpret_cast<const int4*>(list + j);
            rank += q.x > (j < lane ? from : mine);
            rank += q.y > (j + 1 < lane ? from : mine);
            rank += q.z > (j + 2 < lane ? from : mine);
            rank += q.w > (j + 3 < lane ? from : mine);
        }
        if (lane < found && rank < k) take(rank, mine, list[32 + lane]);
        if (lane >= found && lane < k) take(lane, kNone, -1);
    } else {
        for (int j = 0; j < k; ++j) {
            const int32_t t = __reduce_max_sync(0xffffffffu, best);
            const uint32_t who = __ballot_sync(0xffffffffu, best == t);
            if (lane == __ffs(who) - 1) {
                int at = -1;
                best = kNone;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const bool it = at < 0 && key[i] == t;
                    at = it ? i : at;
                    key[i] = it ? kNone : key[i];
                    best = max(best, key[i]);
                }
                take(j, t, t > kNone ? lane * EPL + at : -1);
            }
            __syncwarp();
        }
    }
    __syncwarp();
}

// LPR lanes a token, EPL experts a lane.  ONE: the call's only block.
template <typename X, int LPR, int EPL, bool ONE>
__global__ void __launch_bounds__(kThreads)
    forge_route_tokens_kernel(const X* __restrict__ logits, const Args p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int C = p.tokens;
    int32_t* lists = reinterpret_cast<int32_t*>(smem);  // [warps][2][32]: keys, experts
    int32_t* chosen = lists + kWarps * 64;              // [C][k]
    float* weight = reinterpret_cast<float*>(chosen + C * p.k);         // [C][k], before division
    float* inverse = weight + C * p.k;                                  // [C]
    uint32_t* mask = reinterpret_cast<uint32_t*>(inverse + C);          // [words][E]
    float* mass = reinterpret_cast<float*>(mask + p.words * p.E);       // [warps][E]
    int32_t* lives = reinterpret_cast<int32_t*>(mass + kWarps * p.E);   // [warps]
    int32_t* offs = lives + kWarps;                                     // ONE: [E + 1]

    constexpr int G = kThreads / LPR;  // tokens at once
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const uint32_t group = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (lane / LPR * LPR);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * C;
    float sums[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) sums[i] = 0.0f;
    int32_t live_count = 0;
    float ahead[EPL];
    auto load = [&](int r) {
        const bool in = r < C && first + r < p.T;
        load_logits(ahead, logits + (in ? (first + r) * p.ld : 0), l * EPL, p.E, in, p.vec);
    };
    load(g);
    for (int r0 = 0; r0 < C; r0 += G) {
        const int r = r0 + g;
        float e[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) e[i] = ahead[i];
        if (r0 + G < C) load(r + G);
        int32_t key[EPL];
        int32_t best, top;
        auto keys = [&](auto of) {
            best = kNone;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                key[i] = of(e[i]);
                best = max(best, key[i]);
            }
            top = lanes_max<LPR>(best);
        };
        keys(key_of);
        const float m = top > kNone ? value_of(top) : 0.0f;
        float s = 0.0f, exps[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            exps[i] = exp_from(e[i], m);
            s += exps[i];
        }
        s = lanes_sum<LPR>(s);
        if (__any_sync(0xffffffffu, s != s)) keys(any_key_of);  // a NaN, or +inf
        const bool live = top > kNone;
        live_count += live && l == 0;
        const float inv = live ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) sums[i] = fmaf(exps[i], inv, sums[i]);
        float sum = 0.0f;  // of the chosen
        if constexpr (LPR == 32) {
            if (r < C) {  // (the same for the whole warp)
                float mine = 0.0f;
                top_of_warp(key, p.k, lists + warp * 64, [&](int j, int32_t t, int x) {
                    const float w = t > kNone ? exp_from(value_of(t), m) : 0.0f;
                    mine += w;
                    chosen[r * p.k + j] = x;
                    weight[r * p.k + j] = w;
                });
                sum = lanes_sum<32>(mine);
            }
        } else {
            for (int j = 0; j < p.k; ++j) {
                const int32_t t = lanes_max<LPR>(best);
                const uint32_t who = __ballot_sync(0xffffffffu, best == t) & group;
                const float w = t > kNone ? exp_from(value_of(t), m) : 0.0f;
                sum += w;
                if (lane == __ffs(who) - 1) {
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
    make_masks(mask, p, [&](int t, int j) { return t < C ? chosen[t * p.k + j] : -1; });
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
    // a choice's place among the block's choices of its expert
    auto place_of = [&](int i, int x) {
        const int t = i / p.k;
        int32_t n = __popc(mask[(t >> 5) * p.E + x] & ((1u << (t & 31)) - 1));
        for (int w = 0; w < t >> 5; ++w) n += __popc(mask[w * p.E + x]);
        return n;
    };
    if constexpr (ONE) {
        make_offsets(offs, p.E, count_of);
        write_totals(p, offs, lives_here, count_of, mass_of);
        for (int i = threadIdx.x; i < tokens * p.k; i += kThreads) {
            const int x = chosen[i];
            const int32_t slot = x >= 0 ? offs[x] + place_of(i, x) : -1;
            if (p.slots) p.slots[i] = slot;
            if (p.rows && slot >= 0) p.rows[slot] = i / p.k;
        }
        if (p.rows)
            for (int64_t i = offs[p.E] + threadIdx.x; i < p.T * p.k; i += kThreads) p.rows[i] = -1;
    } else {
        if (p.place)
            for (int i = threadIdx.x; i < tokens * p.k; i += kThreads) {
                const int x = chosen[i];
                p.place[first * p.k + i] = static_cast<uint16_t>(x >= 0 ? place_of(i, x) : 0);
            }
        int32_t* part = p.part + static_cast<int64_t>(blockIdx.x) * (p.E + 1);
        for (int x = threadIdx.x; x < p.E; x += kThreads) {
            part[x] = count_of(x);
            p.psum[static_cast<int64_t>(blockIdx.x) * p.E + x] = mass_of(x);
        }
        if (threadIdx.x == 0) part[p.E] = lives_here;
        let_dependents_start();
    }
}

// Eight columns of part and psum a block, 128 threads a column, each a run of blocks:
// exclusive sums over the blocks in place, and the totals.
constexpr int kScanColumns = 8, kScanRuns = 128, kScanAhead = 8;
__global__ void __launch_bounds__(kScanColumns * kScanRuns) forge_route_scan_kernel(const Args p)
{
    constexpr int kWarpsHere = kScanColumns * kScanRuns / 32;
    static_assert(kWarpsHere == 32 && 32 % kScanColumns == 0, "a lane for each warp's sums");
    __shared__ int32_t runs[kWarpsHere][kScanColumns + 1];
    __shared__ float masses[kWarpsHere][kScanColumns + 1];
    await_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = threadIdx.x % kScanColumns, run = threadIdx.x / kScanColumns;
    const int e = blockIdx.x * kScanColumns + col;
    const int per = (p.blocks + kScanRuns - 1) / kScanRuns;
    const int lo = run * per, hi = min(lo + per, p.blocks);
    int32_t n[kScanAhead];  // a run's first counts: the whole of it, but for very many blocks
    int32_t sum = 0;
    float mass = 0.0f;
    for (int b0 = lo; b0 < hi; b0 += kScanAhead) {
        float m[kScanAhead];
#pragma unroll
        for (int i = 0; i < kScanAhead; ++i) {
            const int64_t b = b0 + i;
            n[i] = b < hi && e <= p.E ? p.part[b * (p.E + 1) + e] : 0;
            m[i] = b < hi && e < p.E ? p.psum[b * p.E + e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kScanAhead; ++i) {
            sum += n[i];
            mass += m[i];
        }
    }
    // within the warp (four runs of each column), then over the warps: warp c has column c
    int32_t up = sum;
#pragma unroll
    for (int o = kScanColumns; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
        mass += __shfl_xor_sync(0xffffffffu, mass, o);
    }
    if (lane >= 32 - kScanColumns) {
        runs[warp][col] = up;
        masses[warp][col] = mass;
    }
    __syncthreads();
    if (warp < kScanColumns) {
        const int32_t own = runs[lane][warp];
        int32_t all = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, all, o);
            if (lane >= o) all += v;
        }
        const float m = lanes_sum<32>(masses[lane][warp]);
        runs[lane][warp] = all - own;
        const int c = blockIdx.x * kScanColumns + warp;
        if (lane == 31 && c <= p.E) p.total[c] = all;
        if (lane == 31 && c < p.E) p.ptotal[c] = m;
    }
    __syncthreads();
    int32_t at = runs[warp][col] + up - sum;
    for (int b0 = lo; e <= p.E && b0 < hi; b0 += kScanAhead) {
#pragma unroll
        for (int i = 0; i < kScanAhead; ++i) {
            const int64_t b = b0 + i;
            if (b >= hi) continue;
            int32_t* cell = p.part + b * (p.E + 1) + e;
            const int32_t here = per <= kScanAhead ? n[i] : *cell;
            *cell = at;
            at += here;
        }
    }
    let_dependents_start();
}

// SCAN: from the blocks' own counts, else from their exclusive sums.
template <bool SCAN>
__global__ void __launch_bounds__(kThreads) forge_route_place_kernel(const Args p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    int32_t* offs = reinterpret_cast<int32_t*>(smem);  // [E + 1]
    int32_t* base = offs + p.E + 1;                    // [E + 1]: the earlier blocks' choices
    int32_t* total = base + p.E + 1;                   // [E + 1]
    float* mass = reinterpret_cast<float*>(total + p.E + 1);  // SCAN, first block: [E]
    await_prerequisites();
    const int E1 = p.E + 1, b = blockIdx.x;
    if constexpr (SCAN) {
        // `ways` threads an expert, every ways-th block each
        __shared__ int32_t befores[kThreads], alls[kThreads];
        __shared__ float masses[kThreads];
        const int ways = E1 < kThreads ? kThreads / E1 : 1;
        for (int e0 = 0; e0 <= p.E; e0 += kThreads) {
            const int e = e0 + (ways > 1 ? threadIdx.x % E1 : threadIdx.x), way = ways > 1 ? threadIdx.x / E1 : 0;
            int32_t before = 0, all = 0;
            float s = 0.0f;
            if (e <= p.E && way < ways) {
#pragma unroll 4
                for (int i = way; i < p.blocks; i += ways) {
                    const int32_t n = p.part[i * E1 + e];
                    all += n;
                    before += i < b ? n : 0;
                    if (b == 0 && e < p.E) s += p.psum[i * p.E + e];
                }
            }
            befores[threadIdx.x] = before;
            alls[threadIdx.x] = all;
            masses[threadIdx.x] = s;
            __syncthreads();
            if (e <= p.E && way == 0) {
                for (int k = 1; k < ways; ++k) {
                    before += befores[threadIdx.x + k * E1];
                    all += alls[threadIdx.x + k * E1];
                    s += masses[threadIdx.x + k * E1];
                }
                base[e] = before;
                total[e] = all;
                if (e < p.E) mass[e] = s;
            }
            __syncthreads();
        }
    } else {
        for (int e = threadIdx.x; e <= p.E; e += kThreads) {
            base[e] = p.part[static_cast<int64_t>(b) * E1 + e];
            total[e] = p.total[e];
        }
    }
    __syncthreads();
    auto count = [&](int e) { return total[e]; };
    make_offsets(offs, p.E, count);
    if (b == 0)
        write_totals(p, offs, count(p.E), count,
                     [&](int e) { return SCAN ? mass[e] : p.ptotal[e]; });
    if (!p.place) return;
    const int64_t first = static_cast<int64_t>(b) * p.tokens;
    const int64_t left = p.T - first;
    const int tokens = left < p.tokens ? static_cast<int>(left) : p.tokens;
    for (int i = threadIdx.x; i < tokens * p.k; i += kThreads) {
        const int64_t at = first * p.k + i;
        const int e = p.experts[at];
        const int32_t slot = e >= 0 ? offs[e] + base[e] + p.place[at] : -1;
        if (p.slots) p.slots[at] = slot;
        if (p.rows && slot >= 0) p.rows[slot] = static_cast<int32_t>(first + i / p.k);
    }
    if (p.rows) {
        const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
        for (int64_t i = offs[p.E] + static_cast<int64_t>(b) * kThreads + threadIdx.x;
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
    bool f32, vec;  // vec: rows of logits and dlogits in vectors
};

__device__ __forceinline__ float nan_max(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Four sums over a token's lanes, in all of them: each half of the lanes takes two of them
// on, each quarter one.
template <int LPR>
__device__ __forceinline__ void sum_four(float (&s)[4])
{
    if constexpr (LPR < 8) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < 4; ++n) s[n] += __shfl_xor_sync(0xffffffffu, s[n], o);
    } else {
        constexpr int H = LPR / 2, Q = LPR / 4;
        const int lane = threadIdx.x & 31;
        const bool h = lane & H, q = lane & Q;
        const float a = (h ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, h ? s[0] : s[2], H);
        const float b = (h ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, h ? s[1] : s[3], H);
        float v = (q ? b : a) + __shfl_xor_sync(0xffffffffu, q ? a : b, Q);
#pragma unroll
        for (int o = Q / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            s[n] = __shfl_sync(0xffffffffu, v, (n >> 1) * H + (n & 1) * Q, LPR);
    }
}

// A token's row is written without its weights' part, p (c - sum p q); the lanes that
// take its choices (each loads its expert's logit for itself) then write theirs over it.
template <typename X, int LPR, int EPL>
__global__ void __launch_bounds__(kThreads, EPL == 8 && LPR >= 8 ? 4 : 1)
    forge_route_grad_kernel(const X* logits, const GradArgs p)
{
    constexpr int G = kThreads / LPR;
    constexpr int kMost = LPR * EPL < kMaxTop ? LPR * EPL : kMaxTop;  // k <= E <= LPR EPL
    constexpr int kPer = (kMost + LPR - 1) / LPR;                      // choices of a lane
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
    float f = 0.0f;  // of a count in the loss's q
    if (p.grad_loss) {
        const float n = fmaxf(1.0f, static_cast<float>(*p.live));
        f = *p.grad_loss * static_cast<float>(p.E) / (static_cast<float>(p.k) * n) / n;
    }
    float c[EPL];  // the loss's q
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        c[i] = p.grad_loss && l * EPL + i < p.E ? f * static_cast<float>(p.counts[l * EPL + i]) : 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    // a token's row and its choices l, l + LPR, .. in this lane, the next token's on their
    // way while this one's are computed
    float ahead[EPL], gws_ahead[kPer];
    int xs_ahead[kPer];
    auto load = [&](int64_t t) {
        const bool in = t < p.T;
        load_logits(ahead, logits + (in ? t * p.ld : 0), l * EPL, p.E, in, p.vec);
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            const int j = l + n * LPR;
            const bool is = p.grad_weights && in && j < p.k;
            xs_ahead[n] = is ? p.experts[t * p.k + j] : -1;
            gws_ahead[n] = is ? p.grad_weights[t * p.k + j] : 0.0f;
        }
    };
    load(static_cast<int64_t>(blockIdx.x) * G + g);
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * G; t0 < p.T; t0 += step) {
        const int64_t t = t0 + g;
        const bool in = t < p.T;
        const X* row = logits + (in ? t * p.ld : 0);
        float v[EPL], gws[kPer], es[kPer];
        int xs[kPer];
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = ahead[i];
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            xs[n] = xs_ahead[n] < p.E ? xs_ahead[n] : -1;
            gws[n] = gws_ahead[n];
            es[n] = xs[n] >= 0 ? entry(load_plain<X, 1>(row + xs[n]), 0) : 0.0f;
        }
        load(t + step);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = nan_max(m, v[i]);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.0f : m;  // (a NaN makes all p NaN)
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // exp, exp c, chosen exp, chosen exp gw
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            if (xs[n] < 0) continue;
            es[n] = exp_from(es[n], ref);
            s[2] += es[n];
            s[3] = fmaf(es[n], gws[n], s[3]);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = exp_from(v[i], ref);
            s[0] += v[i];
            s[1] = fmaf(v[i], c[i], s[1]);
        }
        sum_four<LPR>(s);
        const float inv = s[0] != 0.0f ? 1.0f / s[0] : 0.0f;
        // normalised weights: (gw - sum gw w) / S; else gw as it is.  Then
        // sum p q = (exp c + exp by) / sum exp, the second sum 0 when normalised.
        const bool norm = p.normalize && s[2] > 0.0f;
        const float mean = norm ? s[3] / s[2] : 0.0f;
        const float over = norm ? s[0] / s[2] : 1.0f;
        const float pq = (s[1] + (p.normalize ? 0.0f : s[3])) * inv;
        const int64_t at = t * p.ld_out;
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = v[i] * inv * (c[i] - pq);
        __syncwarp();  // (in place: every lane has read the row)
        if (in) {
            if (p.vec && l * EPL + EPL <= p.E) {
                store_as(p.dlogits, p.f32, at + l * EPL, v);
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const float one[1] = {v[i]};
                    if (l * EPL + i < p.E) store_as(p.dlogits, p.f32, at + l * EPL + i, one);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int n = 0; n < kPer; ++n) {
            if (xs[n] < 0) continue;
            const float q = p.grad_loss ? f * static_cast<float>(p.counts[xs[n]]) : 0.0f;
            const float one[1] = {es[n] * inv * (q + (gws[n] - mean) * over - pq)};
            store_as(p.dlogits, p.f32, at + xs[n], one);
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

cudaError_t after(void (*kernel)(const Args), int grid, int threads, size_t smem, const Args& p,
                  cudaStream_t s)
{
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename X>
cudaError_t forward(const X* logits, Args p, int sms, cudaStream_t s)
{
    // a block's tokens: whole turns of its groups, as many as give every SM four blocks
    // (which run at once: a fifth would run alone), 8 at least (1024 x 256: 16.7 us, with 32
    // 19.9), within the room
    int most = kMostChoices / (32 * p.k);
    if (most > kMostMasks / p.E) most = kMostMasks / p.E;
    if (most > kMostWords) most = kMostWords;
    if (most < 1) most = 1;
    int lanes = 1;  // a token
    while (lanes < 32 && 8 * lanes < p.E) lanes *= 2;
    const int64_t at_once = kThreads / lanes;
    int64_t tokens = (p.T + 4LL * sms - 1) / (4LL * sms);
    tokens = ((tokens < 8 ? 8 : tokens) + at_once - 1) / at_once * at_once;
    // one block for up to two turns of its groups: there a second launch costs more than it
    // saves (256 x 16: 8.3 us, in two launches 10.4; four turns, 128 x 64 and 32 x 256: 15.8
    // and 16.6, in two or three 12.4 and 13.3)
    if (p.T <= 32 * most && p.T <= 2 * at_once) tokens = p.T;
    if (tokens > 32 * most) tokens = 32 * most;
    p.tokens = static_cast<int>(tokens < 1 ? 1 : tokens);
    p.words = (p.tokens + 31) / 32;
    const int64_t blocks = (p.T + p.tokens - 1) / p.tokens;
    if (blocks > INT32_MAX / 2) return cudaErrorInvalidValue;
    p.blocks = static_cast<int32_t>(blocks < 1 ? 1 : blocks);
    const bool one = p.blocks == 1, place = p.slots || p.rows;
    const size_t C = p.tokens, E = p.E;
    // (all of the tokens kernel's shared memory: static arrays would count in the 48 KB too)
    const size_t tokens_smem = 8 * kWarps * 32 + 4 * (2 * C * p.k + C + p.words * E + kWarps * E +
                                                      kWarps + (one ? E + 1 : 0));
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (!one) {
        const int64_t counts = (E + 1) * p.blocks, masses = E * p.blocks;
        const int64_t choices = place ? p.T * p.k : 0;
        e = scratch_alloc(&scratch, 4 * (counts + masses + 2 * (E + 1)) + 2 * choices, s);
        if (e != cudaSuccess) return e;
        p.part = static_cast<int32_t*>(scratch);
        p.psum = reinterpret_cast<float*>(p.part + counts);
        p.total = reinterpret_cast<int32_t*>(p.psum + masses);
        p.ptotal = reinterpret_cast<float*>(p.total + E + 1);
        if (place) p.place = reinterpret_cast<uint16_t*>(p.ptotal + E + 1);
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
        const int grid = place ? p.blocks : 1;
        const size_t smem = 4 * 4 * (E + 1);
        if (p.blocks * (E + 1) <= kFewCounts) {
            e = after(forge_route_place_kernel<true>, grid, kThreads, smem, p, s);
        } else {
            e = after(forge_route_scan_kernel, static_cast<int>((E + kScanColumns) / kScanColumns),
                      kScanColumns * kScanRuns, 0, p, s);
            if (e == cudaSuccess)
                e = after(forge_route_place_kernel<false>, grid, kThreads, smem, p, s);
        }
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
    p.vec = aligned(logits, 16) && ld * size_of(dtype) % 16 == 0;
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
                     experts, counts, live, grad_weights, grad_loss, dlogits, out_dtype == FORGE_F32,
                     aligned(logits, 16) && ld * es % 16 == 0 && aligned(dlogits, 16) &&
                         ld_out * eo % 16 == 0};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto* x) {
        return by_experts(E, [&](auto shape) {
            const int64_t want = (T * shape.lpr + kThreads - 1) / kThreads, most = 4LL * sms;
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
