// forge_layer_norm.cu -- layer norm and its gradient, with the reduction of the
// weight's and the bias's gradients over the rows.
//
// A row x [D], weight w and bias b give
//   mu = mean x,  rstd = 1 / sqrt(mean (x - mu)^2 + eps),  xh = (x - mu) rstd,
//   y = xh w + b,
// and a gradient dy of y, with g = dy w,
//   dx = rstd (g - mean g - xh mean(g xh)),  dw = sum_r dy xh,  db = sum_r dy.
//
// Both are bound by memory: a row is read once into registers, by one warp
// or by a block of W warps, and everything is computed from there (mu first and
// the squares of x - mu after it, so that no digits are lost to a mean that is
// large against the deviations).  Each thread owns the same columns of every
// row its block takes, so dw and db are sums in its registers; a block writes
// them once, and a second kernel adds the blocks' in a fixed order: bitwise the
// same from run to run.
//
// Measured (the copy bandwidth is 6.68 TB/s): 16384 x 4096 bf16 forward 48 us (5.6 TB/s;
// captured, 4.6 TB/s reach DRAM, the rest of y is in L2 yet, and the two barriers of
// a row leave 57% of the issue slots), the gradient 81 (5.0 TB/s; 75 for the rows, 6 for the
// fold).  The gradient of 777 x 1023 fp32: 10.4 us, two kernels' latency.  16 x 4096 forward:
// 4.3 us; 4096 x 16384 bf16 68 (a block of 32 warps a row, weights read again for each).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "forge.h"
#include "forge_device.h"
#include "forge_ptx.cuh"
#include "forge_rows.cuh"

namespace forge {
namespace norm {

constexpr int kRowWarps = 8;      // warps of a block whose warps take a row each
// Of a block in the gradient of rows too wide for registers, two blocks an SM (4096 x 16384
// bf16, all kernels: 144 us, with one block of 1024 threads 154; 2048 x 16384 fp32: 134, 134)
constexpr int kWideThreads = 512;
constexpr int kLongThreads = 1024;  // of a block on a row too wide for registers
constexpr int kThreadsAtWork = 512;  // of an SM: 128 registers each
// Of an SM in the gradient.  fp32 rows have the fewest entries a byte, and are
// quicker with twice the threads of half the registers (8192 x 4096 fp32: 71 us, with
// 512 threads 75; 16384 x 4096 bf16: 87 and 82; 16384 x 1023 bf16, entry by entry: 38 and 32).
__host__ __device__ constexpr int grad_threads(int V, int E) { return V == 4 && E == 8 ? 1024 : 512; }
constexpr int64_t kMaxForward = 16384, kMaxBackward = 8192;  // widths that registers hold

// Threads of a block with W warps a row.
__host__ __device__ constexpr int threads_of(int W) { return 32 * (W == 1 ? kRowWarps : W); }

struct Forward {
    int64_t R, D, ldx, ldy;
    const float *weight, *bias;
    void* y;
    bool y_f32;
    float *mean, *rstd;
    float eps;
};

struct Backward {
    int64_t R, D, ldg, ldx, ldo;
    const float *weight, *mean, *rstd;
    void* dx;
    bool dx_f32;
    float* part;  // [blocks][2][D]; null: launch nothing, tell how many blocks write one
};

// A row by 32 W threads (thread t of them) in three passes, the second and third from L2.
// Rows whose squares, or whose sum, pass the largest number are taken at kSmall times
// their size, which is far from the other end of the range (one of their deviations is
// above some 1e14); rows with a NaN or an infinity end as NaN all the same.
constexpr float kSmall = 0x1p-96f;
template <bool OVER, typename X, int V, int W>
__device__ __forceinline__ void row_in_passes(const X* row, const Forward& p, int64_t r, int t,
                                              float* sh0, float* sh1)
{
    const float inv = 1.0f / static_cast<float>(p.D);
    const int64_t step = 32 * W * V;
    float s[1], q[1], mu;
    auto each = [&](auto use) {
        for (int64_t c = t * V; c < p.D; c += step) use(load_row<OVER, X, V>(row + c), c);
    };
    // mean and sum of squares of f times the row
    auto statistics = [&](float f) {
        s[0] = q[0] = 0.0f;
        each([&](const Packed<X, V>& raw, int64_t) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] = fmaf(entry(raw, j), f, s[0]);
        });
        block_sums<W>(s, sh0);
        mu = s[0] * inv;
        each([&](const Packed<X, V>& raw, int64_t) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = fmaf(entry(raw, j), f, -mu);
                q[0] = fmaf(d, d, q[0]);
            }
        });
        block_sums<W>(q, sh1);
    };
    statistics(1.0f);
    const bool far = !(q[0] <= FLT_MAX);  // (alike in all of the row's threads)
    if (far) statistics(kSmall);
    const float f = far ? kSmall : 1.0f;
    const float rstd = 1.0f / sqrtf(fmaf(q[0], inv, far ? p.eps * kSmall * kSmall : p.eps));
    if (t == 0) {
        if (p.mean) p.mean[r] = far ? mu * (1.0f / kSmall) : mu;
        if (p.rstd) p.rstd[r] = rstd * f;
    }
    each([&](const Packed<X, V>& raw, int64_t c) {
        const Packed<float, V> w = load_packed<float, V>(p.weight + c);
        const Packed<float, V> b =
            p.bias ? load_packed<float, V>(p.bias + c) : zero_packed<float, V>();
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = fmaf(fmaf(entry(raw, j), f, -mu) * rstd, entry(w, j), entry(b, j));
        store_as(p.y, p.y_f32, r * p.ldy + c, v);
    });
}

// E entries a thread in vectors of V, W warps a row, RB rows at a time; the rows after
// them are on their way while these are computed.  Few threads with many registers
// hold the weights too: read for every row, from L1, they kept the load-store unit
// busy for most of a row's time (16384 x 4096 bf16: 56 us, with them in registers and
// two rows at a time 48; 2 x the threads and half the registers 56).
template <typename X, int V, int E, int W, int RB>
__global__ void __launch_bounds__(threads_of(W), W < 32 ? kThreadsAtWork / threads_of(W) : 1)
    forge_layer_norm_kernel(const X* x, const Forward p)
{
    constexpr int NV = E / V;
    __shared__ float sh[2][W * RB];
    const int teams = W == 1 ? kRowWarps : 1;
    const int t = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const uint32_t step = gridDim.x * teams * RB;
    const float inv = 1.0f / static_cast<float>(p.D);
    uint32_t r = (blockIdx.x * teams + (W == 1 ? threadIdx.x >> 5 : 0)) * RB;
    Packed<X, V> next[RB][NV];
    auto load = [&](uint32_t r) {
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * W * 32 + t) * V;
                next[k][i] = c < p.D && r + k < p.R
                                 ? load_plain<X, V>(x + static_cast<int64_t>(r + k) * p.ldx + c)
                                 : zero_packed<X, V>();
            }
    };
    constexpr bool kHold = W < 32;  // (1024 threads have 64 registers each)
    Packed<float, V> w[NV], b[NV];
    auto load_weights = [&](int i) {
        const int c = (i * W * 32 + t) * V;
        w[i] = c < p.D ? load_packed<float, V>(p.weight + c) : zero_packed<float, V>();
        b[i] = c < p.D && p.bias ? load_packed<float, V>(p.bias + c) : zero_packed<float, V>();
    };
    load(r);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (kHold) load_weights(i);
    for (; r < p.R; r += step) {
        float d[RB][E];
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) d[k][i] = entry(next[k][i / V], i % V);
        if (r + step < p.R) load(r + step);
        float mu[RB], rstd[RB];
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            mu[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) mu[k] += d[k][i];
        }
        block_sums<W>(mu, sh[0]);
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            mu[k] *= inv;
            rstd[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if ((i * W * 32 + t) * V < p.D) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        d[k][i * V + j] -= mu[k];
                        rstd[k] = fmaf(d[k][i * V + j], d[k][i * V + j], rstd[k]);
                    }
                }
            }
        }
        block_sums<W>(rstd, sh[1]);
        // A row of the turn is not for registers (alike in all threads of the rows): the loop
        // ends before the turn's stores.  (By a vote 16384 x 4099 bf16 124 us, by the flag
        // alone 134; 32 warps with their 64 registers the flag behind the stores that
        // it skips, 2048 x 16383 bf16 70.4 and 72.3.)
        bool far = false;
#pragma unroll
        for (int k = 0; k < RB; ++k) far |= !(rstd[k] <= FLT_MAX);
        if (W < 32 && __any_sync(0xffffffffu, far)) break;
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            rstd[k] = 1.0f / sqrtf(fmaf(rstd[k], inv, p.eps));
            if (t == 0 && r + k < p.R) {
                if (p.mean) p.mean[r + k] = mu[k];
                if (p.rstd) p.rstd[r + k] = rstd[k];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * W * 32 + t) * V;
            if (c < p.D && (W < 32 || !far)) {
                if (!kHold) load_weights(i);
#pragma unroll
                for (int k = 0; k < RB; ++k) {
                    if (r + k >= p.R) break;
                    float v[V];
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        v[j] = fmaf(d[k][i * V + j] * rstd[k], entry(w[i], j), entry(b[i], j));
                    store_as(p.y, p.y_f32, static_cast<int64_t>(r + k) * p.ldy + c, v);
                }
            }
        }
        if (W == 32 && far) break;
    }
    // from the first turn with such a row on, one row after another (ordinary ones to the same
    // bits: their sums run in the same order)
    for (; r < p.R; r += step)
#pragma unroll 1
        for (int k = 0; k < RB && r + k < p.R; ++k)
            row_in_passes<true, X, V, W>(x + static_cast<int64_t>(r + k) * p.ldx, p, r + k, t,
                                         sh[0], sh[1]);
}

// Rows wider than the registers hold; OVER: y is x.  (Rows that nothing writes are read by
// read-only loads, which the compiler takes over the stores before them: 2048 x 20001 fp32
// 93 us, by plain loads 122.)
template <bool OVER, typename X, int V>
__global__ void __launch_bounds__(kLongThreads)
    forge_layer_norm_long_kernel(const X* x, const Forward p)
{
    __shared__ float sh[2][kLongThreads / 32];
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x)
        row_in_passes<OVER, X, V, kLongThreads / 32>(x + r * p.ldx, p, r, threadIdx.x, sh[0],
                                                     sh[1]);
}

// E entries a thread in vectors of V, W warps a row.  The weights lie in shared memory,
// a thread's vectors of four apart by the block, so that no two lanes meet in a bank.
// The next rows are on their way while one is computed: each thread copies its own
// vectors of the kDepth rows ahead into shared memory (cp.async: no thread reads
// another's, so no barrier), or, entry by entry, the one row ahead into registers.
// (One row ahead for vectors too: 16384 x 4096 bf16 in 88 instead of 82 us.)
constexpr int kDepth = 3;
template <int V, int E, int W, typename G, typename X>
constexpr int ring_bytes()
{
    return V == 1 ? 0 : kDepth * 32 * (W == 1 ? kRowWarps : W) * E * static_cast<int>(sizeof(G) + sizeof(X));
}
template <typename G, typename X, int V, int E, int W>
__global__ void __launch_bounds__(threads_of(W), grad_threads(V, E) / threads_of(W))
    forge_layer_norm_grad_kernel(const G* dy, const X* x,
                                 const Backward p)
{
    constexpr int NV = E / V;
    extern __shared__ __align__(16) uint8_t ring[];  // [kDepth]{[NV][threads] of dy, of x}
    __shared__ float sh[2][2 * W];
    __shared__ float4 weight[E / 4][32 * W];
    const int teams = W == 1 ? kRowWarps : 1;
    const int t = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t r = static_cast<int64_t>(blockIdx.x) * teams + (W == 1 ? threadIdx.x >> 5 : 0);
    const float inv = 1.0f / static_cast<float>(p.D);
    Packed<G, V> gnext[NV];
    Packed<X, V> xnext[NV];
    float mu = 0.0f, rstd = 0.0f;
    auto places = [&](int slot, Packed<G, V>*& g, Packed<X, V>*& x) {
        constexpr int kRow = threads_of(W) * E;
        uint8_t* at = ring + slot * (kRow * static_cast<int>(sizeof(G) + sizeof(X)));
        g = reinterpret_cast<Packed<G, V>*>(at) + threadIdx.x;
        x = reinterpret_cast<Packed<X, V>*>(at + kRow * sizeof(G)) + threadIdx.x;
    };
    // row r on its way (into `slot` of the ring); every call is one copy group
    auto fetch = [&](int64_t r, int slot) {
        if constexpr (V == 1) {
            if (r >= p.R) return;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = i * W * 32 + t;
                gnext[i] = c < p.D ? load_plain<G, V>(dy + r * p.ldg + c) : zero_packed<G, V>();
                xnext[i] = c < p.D ? load_plain<X, V>(x + r * p.ldx + c) : zero_packed<X, V>();
            }
        } else {
            Packed<G, V>* g;
            Packed<X, V>* q;
            places(slot, g, q);
            if (r < p.R) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * W * 32 + t) * V;
                    const bool in = c < p.D;  // (else zeros)
                    ptx::cp_async(g + i * threads_of(W), dy + r * p.ldg + (in ? c : 0),
                                  g->kBytes, in ? g->kBytes : 0);
                    ptx::cp_async(q + i * threads_of(W), x + r * p.ldx + (in ? c : 0), q->kBytes,
                                  in ? q->kBytes : 0);
                }
            }
            ptx::cp_async_commit();
        }
    };
    auto statistics = [&](int64_t r) {
        mu = __ldg(p.mean + r);
        rstd = __ldg(p.rstd + r);
    };
    if (V == 1) {
        fetch(r, 0);
    } else {
        for (int d = 0; d < kDepth; ++d) fetch(r + d * step, d);
    }
    if (r < p.R) statistics(r);
    if (W > 1 || threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = (i / V * W * 32 + t) * V + i % V;
            reinterpret_cast<float*>(&weight[i / 4][t])[i % 4] = c < p.D ? p.weight[c] : 0.0f;
        }
    }
    __syncthreads();
    float dw[E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
    int turn = 0, slot = 0;
    for (; r < p.R; r += step, turn ^= 1) {
        if constexpr (V > 1) {
            ptx::cp_async_wait<kDepth - 1>();  // the oldest row is here
            Packed<G, V>* g;
            Packed<X, V>* q;
            places(slot, g, q);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                gnext[i] = g[i * threads_of(W)];
                xnext[i] = q[i * threads_of(W)];
            }
        }
        float g[E], xh[E];
        float s[2] = {0.0f, 0.0f};  // of g and of g xh (columns past D have dy = 0)
        const float scale = rstd;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 w4 = weight[i / 4][t];
            const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = entry(gnext[(i + j) / V], (i + j) % V);
                xh[i + j] = (entry(xnext[(i + j) / V], (i + j) % V) - mu) * rstd;
                g[i + j] = d * w[j];
                s[0] += g[i + j];
                s[1] = fmaf(g[i + j], xh[i + j], s[1]);
                dw[i + j] = fmaf(d, xh[i + j], dw[i + j]);
                db[i + j] += d;
            }
        }
        // (its values are in registers, and used: its place may be written)
        if constexpr (V == 1) {
            fetch(r + step, 0);
        } else {
            fetch(r + kDepth * step, slot);
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }
        if (r + step < p.R) statistics(r + step);
        block_sums<W>(s, sh[turn]);
        const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * W * 32 + t) * V;
            if (c < p.D) {
                float v[V];
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = scale * (g[i * V + j] - a - xh[i * V + j] * b);
                store_as(p.dx, p.dx_f32, r * p.ldo + c, v);
            }
        }
    }
    let_dependents_start();
    float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    if constexpr (W == 1) {
        // the block's warps one after another
        __shared__ float acc[2][E * 32];
        for (int k = 0; k < kRowWarps; ++k) {
            if (static_cast<int>(threadIdx.x >> 5) == k) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int c = (i * 32 + t) * V + j;
                        acc[0][c] = (k ? acc[0][c] : 0.0f) + dw[i * V + j];
                        acc[1][c] = (k ? acc[1][c] : 0.0f) + db[i * V + j];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < p.D; c += 32 * kRowWarps) {
            part[c] = acc[0][c];
            part[p.D + c] = acc[1][c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * W * 32 + t) * V;
            if (c < p.D) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    part[c + j] = dw[i * V + j];
                    part[p.D + c + j] = db[i * V + j];
                }
            }
        }
    }
}

// dx of rows too wide for dw and db to stay in registers beside them: two passes over
// a row, the first kHeld vectors of a thread kept from the first, the rest from L2
// (4096 x 16384 bf16 with dw and db: 144 us, all from L2 162; 2048 x 16384 fp32 134, with
// eight vectors of its twice as many registers 158).
// OVER: dx is dy or x, as above (2048 x 20001 bf16 164 us, by plain loads 215).
template <bool OVER, typename G, typename X, int V>
__global__ void __launch_bounds__(kWideThreads, 1024 / kWideThreads)
    forge_layer_norm_grad_long_kernel(const G* dy, const X* x,
                                      const Backward p)
{
    constexpr int kHeld = sizeof(G) + sizeof(X) <= 4 ? 8 : 4;  // (registers)
    __shared__ float sh[2][2 * kWideThreads / 32];
    const float inv = 1.0f / static_cast<float>(p.D);
    const int64_t step = static_cast<int64_t>(kWideThreads) * V;
    const int64_t c0 = threadIdx.x * V;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x, turn ^= 1) {
        const G* grow = dy + r * p.ldg;
        const X* xrow = x + r * p.ldx;
        Packed<G, V> gheld[kHeld];
        Packed<X, V> xheld[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t c = c0 + i * step;
            gheld[i] = c < p.D ? load_row<OVER, G, V>(grow + c) : zero_packed<G, V>();
            xheld[i] = c < p.D ? load_row<OVER, X, V>(xrow + c) : zero_packed<X, V>();
        }
        const float mu = p.mean[r], rstd = p.rstd[r];
        float s[2] = {0.0f, 0.0f};
        auto add = [&](const Packed<G, V>& graw, const Packed<X, V>& xraw, int64_t c) {
            const Packed<float, V> w = load_packed<float, V>(p.weight + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float g = entry(graw, j) * entry(w, j);
                s[0] += g;
                s[1] = fmaf(g, (entry(xraw, j) - mu) * rstd, s[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (c0 + i * step < p.D) add(gheld[i], xheld[i], c0 + i * step);
        for (int64_t c = c0 + kHeld * step; c < p.D; c += step)
            add(load_row<OVER, G, V>(grow + c), load_row<OVER, X, V>(xrow + c), c);
        block_sums<kWideThreads / 32>(s, sh[turn]);
        const float a = s[0] * inv, b = s[1] * inv;
        auto store = [&](const Packed<G, V>& graw, const Packed<X, V>& xraw, int64_t c) {
            const Packed<float, V> w = load_packed<float, V>(p.weight + c);
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = rstd * (fmaf(entry(graw, j), entry(w, j), -a) -
                               (entry(xraw, j) - mu) * rstd * b);
            store_as(p.dx, p.dx_f32, r * p.ldo + c, v);
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (c0 + i * step < p.D) store(gheld[i], xheld[i], c0 + i * step);
        for (int64_t c = c0 + kHeld * step; c < p.D; c += step)
            store(load_row<OVER, G, V>(grow + c), load_row<OVER, X, V>(xrow + c), c);
    }
}

// dw and db of such rows, before dx (which may be written over dy): a block
// takes 32 x kLongWarps vectors of columns of every gridDim.y-th row (4096 x 16384 bf16,
// entry by entry: 204 us for the whole call, in vectors of four 162).
constexpr int kLongWarps = 4;
template <typename G, typename X, int V>
__global__ void __launch_bounds__(32 * kLongWarps)
    forge_layer_norm_columns_kernel(const G* dy, const X* x,
                                    const Backward p)
{
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * (32 * kLongWarps) + threadIdx.x) * V;
    if (c >= p.D) return;
    float dw[V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < p.R; r += gridDim.y) {
        const Packed<G, V> graw = load_row<false, G, V>(dy + r * p.ldg + c);
        const Packed<X, V> xraw = load_row<false, X, V>(x + r * p.ldx + c);
        const float mu = p.mean[r], rstd = p.rstd[r];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float d = entry(graw, j);
            dw[j] = fmaf(d, (entry(xraw, j) - mu) * rstd, dw[j]);
            db[j] += d;
        }
    }
    float* part = p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        part[c + j] = dw[j];
        part[p.D + c + j] = db[j];
    }
}

// The sum of the blocks' parts, 32 columns a block, its warps every 32nd part.
constexpr int kFoldWarps = 32;
__global__ void __launch_bounds__(32 * kFoldWarps)
    forge_layer_norm_fold_kernel(const float* part, int32_t parts, int64_t D, float* dweight,
                                 float* dbias, int32_t accumulate)
{
    __shared__ float sh[kFoldWarps][33];
    await_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // of [2][D]
    float s = 0.0f;
    if (c < 2 * D) {
#pragma unroll 8
        for (int k = warp; k < parts; k += kFoldWarps)
            s += part[static_cast<int64_t>(k) * 2 * D + c];
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * D) {
#pragma unroll
        for (int k = 1; k < kFoldWarps; ++k) s += sh[k][lane];
        float* out = c < D ? dweight : dbias;
        if (out) {
            const int64_t at = c < D ? c : c - D;
            out[at] = accumulate ? out[at] + s : s;
        }
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : 4; }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }

// Whether rows of `ld` elements of `es` bytes from `p` on can be taken in
// vectors of V elements (of at most 16 bytes an instruction).
bool rows_fit(const void* p, int64_t es, int64_t ld, int V)
{
    const int64_t bytes = V * es < 16 ? V * es : 16;
    return aligned(p, bytes) && ld % V == 0;
}

int blocks_for(int64_t rows, int64_t rows_a_block, int64_t most)
{
    const int64_t want = (rows + rows_a_block - 1) / rows_a_block;
    return static_cast<int>(want < most ? want : most);
}

template <typename X, int V>
void forward(const X* x, const Forward& p, int sms, cudaStream_t s)
{
    const int64_t D = p.D;
    auto go = [&](auto kernel, int W, int RB) {
        const int teams = W == 1 ? kRowWarps : 1, threads = threads_of(W);
        const int64_t at_work = W < 32 ? kThreadsAtWork / threads : 1;
        kernel<<<blocks_for(p.R, teams * RB, sms * at_work), threads, 0, s>>>(x, p);
    };
    if (D <= 256)
        go(forge_layer_norm_kernel<X, V, 8, 1, 4>, 1, 4);
    else if (D <= 512)
        // (entry by entry one row at a time: 32768 x 511 bf16 23.2 us, two 28.3; fp32 30.6, 33.4)
        go(forge_layer_norm_kernel<X, V, 16, 1, V == 1 ? 1 : 2>, 1, V == 1 ? 1 : 2);
    else if (D <= 1024)
        go(forge_layer_norm_kernel<X, V, 16, 2, 2>, 2, 2);
    else if (D <= 2048)
        go(forge_layer_norm_kernel<X, V, 16, 4, 2>, 4, 2);
    else if (D <= 4096)
        go(forge_layer_norm_kernel<X, V, 16, 8, 2>, 8, 2);
    else if (D <= 8192)
        go(forge_layer_norm_kernel<X, V, 16, 16, 2>, 16, 2);
    else if (D <= kMaxForward)
        go(forge_layer_norm_kernel<X, V, 16, 32, 1>, 32, 1);
    else if (x == p.y)
        forge_layer_norm_long_kernel<true, X, V>
            <<<blocks_for(p.R, 1, 2LL * sms), kLongThreads, 0, s>>>(x, p);
    else
        forge_layer_norm_long_kernel<false, X, V>
            <<<blocks_for(p.R, 1, 2LL * sms), kLongThreads, 0, s>>>(x, p);
}

// The rows in registers; returns the number of parts of dw and db (0 with an error): a block
// has two rows at least, so that few rows leave few parts to add.
template <typename G, typename X, int V, int E, int W>
int backward_with(const G* dy, const X* x, const Backward& p, int sms, cudaStream_t s)
{
    constexpr int teams = W == 1 ? kRowWarps : 1, threads = threads_of(W);
    constexpr int bytes = ring_bytes<V, E, W, G, X>();
    const int blocks = blocks_for(p.R, 2 * teams, static_cast<int64_t>(sms) * grad_threads(V, E) / threads);
    if (!p.part) return blocks;
    auto kernel = forge_layer_norm_grad_kernel<G, X, V, E, W>;
    if (bytes > 16 * 1024) {  // (with the weights beyond what a launch has by itself)
        static int ready[64];  // per device (and kernel)
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 0;  // (the error stays for the caller)
        if (__atomic_load_n(&ready[dev & 63], __ATOMIC_ACQUIRE) == 0) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
                cudaSuccess)
                return 0;
            __atomic_store_n(&ready[dev & 63], 1, __ATOMIC_RELEASE);
        }
    }
    kernel<<<blocks, threads, bytes, s>>>(dy, x, p);
    return blocks;
}

template <typename G, typename X, int V, int E>
int backward(const G* dy, const X* x, const Backward& p, int sms, cudaStream_t s)
{
    const int64_t D = p.D;
    if (D <= 256) return backward_with<G, X, V, 8, 1>(dy, x, p, sms, s);
    if (D <= 512) return backward_with<G, X, V, E, 16 / E>(dy, x, p, sms, s);
    if (D <= 1024) return backward_with<G, X, V, E, 32 / E>(dy, x, p, sms, s);
    if (D <= 2048) return backward_with<G, X, V, E, 64 / E>(dy, x, p, sms, s);
    if (D <= 4096) return backward_with<G, X, V, E, 128 / E>(dy, x, p, sms, s);
    return backward_with<G, X, V, 16, 16>(dy, x, p, sms, s);
}

constexpr int kColumnParts = 64;  // of the column kernel at most
template <typename G, typename X>
int backward_any(const G* dy, const X* x, const Backward& p, int V, int sms, cudaStream_t s)
{
    if (p.D <= kMaxBackward) {
        if constexpr (sizeof(G) == 2 && sizeof(X) == 2) {
            if (V == 8) return backward<G, X, 8, 16>(dy, x, p, sms, s);
        }
        return V == 4 ? backward<G, X, 4, 8>(dy, x, p, sms, s)
                      : backward<G, X, 1, 8>(dy, x, p, sms, s);
    }
    const int parts = blocks_for(p.R, 1, kColumnParts);
    if (!p.part) return parts;
    auto go = [&](auto v) {
        constexpr int N = decltype(v)::value;
        constexpr int slab = 32 * kLongWarps * N;
        const unsigned slabs = static_cast<unsigned>((p.D + slab - 1) / slab);
        forge_layer_norm_columns_kernel<G, X, N><<<dim3(slabs, parts), 32 * kLongWarps, 0, s>>>(dy, x, p);
        auto rows = p.dx == static_cast<const void*>(dy) || p.dx == static_cast<const void*>(x)
                        ? forge_layer_norm_grad_long_kernel<true, G, X, N>
                        : forge_layer_norm_grad_long_kernel<false, G, X, N>;
        rows<<<blocks_for(p.R, 1, 1024LL / kWideThreads * sms), kWideThreads, 0, s>>>(dy, x, p);
    };
    if (V == 1)
        go(std::integral_constant<int, 1>());
    else
        go(std::integral_constant<int, 4>());
    return parts;
}

forge_status check_sizes(int64_t R, int64_t D)
{
    return R < 0 || D < 1 || R > INT32_MAX || D > (1 << 30) ? FORGE_ERR_INVALID_ARG : FORGE_OK;
}

// Whether `out` is `in` itself, row by row, or shares no memory with it.
bool apart_or_same(const void* in, forge_dtype ti, int64_t ldi, const void* out, forge_dtype to,
                   int64_t ldo, int64_t R, int64_t D)
{
    const int64_t ei = size_of(ti), eo = size_of(to);
    if (in == out && ti == to && (ldi == ldo || R == 1)) return true;
    return R == 0 || !rows_overlap(reinterpret_cast<uintptr_t>(in), D * ei, ldi * ei,
                                   reinterpret_cast<uintptr_t>(out), D * eo, ldo * eo, R);
}

}  // namespace norm
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_layer_norm(const void* x, forge_dtype x_dtype, int64_t ldx,
                                         const float* weight, const float* bias, int64_t R,
                                         int64_t D, float eps, void* y, forge_dtype y_dtype,
                                         int64_t ldy, float* mean, float* rstd,
                                         forge_stream_t stream)
{
    using namespace norm;
    if (!weight || (R > 0 && (!x || !y))) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(R, D);
    if (st != FORGE_OK) return st;
    if (ldx < D || ldy < D || !(eps > 0.0f) || !std::isfinite(eps)) return FORGE_ERR_INVALID_ARG;
    if (!is_float(x_dtype) || !is_float(y_dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(x, size_of(x_dtype)) || !aligned(y, size_of(y_dtype)) || !aligned(weight, 4) ||
        !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return FORGE_ERR_MISALIGNED;
    if (!apart_or_same(x, x_dtype, ldx, y, y_dtype, ldy, R, D)) return FORGE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (R == 0) return FORGE_OK;
    const void* ptrs[] = {x, weight, bias, y, mean, rstd};
    if ((st = device_resident(ptrs, 6)) != FORGE_OK) return st;
    const Forward p{R, D, ldx, ldy, weight, bias, y, y_dtype == FORGE_F32, mean, rstd, eps};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int V = x_dtype == FORGE_BF16 ? 8 : 4;
    const bool fits = D % V == 0 && rows_fit(x, size_of(x_dtype), ldx, V) &&
                      rows_fit(y, size_of(y_dtype), ldy, V) && aligned(weight, 16) &&
                      aligned(bias, 16);
    if (x_dtype == FORGE_F32) {
        const float* f = static_cast<const float*>(x);
        fits ? forward<float, 4>(f, p, sms, s) : forward<float, 1>(f, p, sms, s);
    } else {
        const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
        fits ? forward<__nv_bfloat16, 8>(h, p, sms, s) : forward<__nv_bfloat16, 1>(h, p, sms, s);
    }
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_layer_norm_grad(const void* dy, forge_dtype dy_dtype, int64_t lddy,
                                              const void* x, forge_dtype x_dtype, int64_t ldx,
                                              const float* weight, const float* mean,
                                              const float* rstd, int64_t R, int64_t D, void* dx,
                                              forge_dtype dx_dtype, int64_t lddx, float* dweight,
                                              float* dbias, int32_t accumulate,
                                              forge_stream_t stream)
{
    using namespace norm;
    if (!weight || !dweight || (R > 0 && (!dy || !x || !mean || !rstd || !dx)))
        return FORGE_ERR_INVALID_ARG;
    forge_status st = check_sizes(R, D);
    if (st != FORGE_OK) return st;
    if (lddy < D || ldx < D || lddx < D) return FORGE_ERR_INVALID_ARG;
    if (!is_float(dy_dtype) || !is_float(x_dtype) || !is_float(dx_dtype))
        return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(dy, size_of(dy_dtype)) || !aligned(x, size_of(x_dtype)) ||
        !aligned(dx, size_of(dx_dtype)) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return FORGE_ERR_MISALIGNED;
    if (!apart_or_same(dy, dy_dtype, lddy, dx, dx_dtype, lddx, R, D) ||
        !apart_or_same(x, x_dtype, ldx, dx, dx_dtype, lddx, R, D))
        return FORGE_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* ptrs[] = {R > 0 ? dy : nullptr,   R > 0 ? x : nullptr,  weight,
                          R > 0 ? mean : nullptr, R > 0 ? rstd : nullptr, R > 0 ? dx : nullptr,
                          dweight,                dbias};
    if ((st = device_resident(ptrs, 8)) != FORGE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = dy_dtype == FORGE_BF16 && x_dtype == FORGE_BF16 && D <= kMaxBackward;
    int V = wide ? 8 : 4;
    if (D % V != 0 || !rows_fit(dy, size_of(dy_dtype), lddy, V) ||
        !rows_fit(x, size_of(x_dtype), ldx, V) || !rows_fit(dx, size_of(dx_dtype), lddx, V) ||
        !aligned(weight, 16))
        V = 1;
    Backward p{R,    D,  lddy, ldx, lddx, weight, mean,
               rstd, dx, dx_dtype == FORGE_F32, nullptr};
    auto backward_of = [&]() {
        auto by_x = [&](auto* g) {
            return x_dtype == FORGE_F32
                       ? backward_any(g, static_cast<const float*>(x), p, V, sms, s)
                       : backward_any(g, static_cast<const __nv_bfloat16*>(x), p, V, sms, s);
        };
        return dy_dtype == FORGE_F32 ? by_x(static_cast<const float*>(dy))
                                     : by_x(static_cast<const __nv_bfloat16*>(dy));
    };
    // scratch for the parts that are written, and no more: the pool keeps what it has given
    // once (16384 x 4096 bf16: 10 MB; sixteen blocks an SM, which only rows of at
    // most 512 entries have, would be 80)
    void* scratch = nullptr;
    int parts = R > 0 ? backward_of() : 0;
    if (R > 0) {
        if (scratch_alloc(&scratch, sizeof(float) * 2 * D * parts, s) != cudaSuccess) {
            cudaGetLastError();
            return FORGE_ERR_CUDA;
        }
        p.part = static_cast<float*>(scratch);
        parts = backward_of();
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        cudaLaunchAttribute early[1];
        early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>((2 * D + 31) / 32));
        cfg.blockDim = dim3(32 * kFoldWarps);
        cfg.stream = s;
        cfg.attrs = early;
        cfg.numAttrs = R > 0 && D <= kMaxBackward ? 1 : 0;
        e = cudaLaunchKernelEx(&cfg, forge_layer_norm_fold_kernel,
                               static_cast<const float*>(p.part), parts, D, dweight, dbias,
                               accumulate);
    }
    if (scratch) {
        const cudaError_t fe = scratch_free(scratch, s);
        if (e == cudaSuccess) e = fe;
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
