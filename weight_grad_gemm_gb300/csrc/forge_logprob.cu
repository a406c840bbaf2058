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

__device__ __forceinline__ float nan_max(float a, float b)
{
    return (a != a) ? a : ((b != b) ? b : fmaxf(a, b));
}

// A value and its column, ordered by value and then by the lower column; a
// NaN stands above every number.
struct Ranked {
    float v;
    int i;
};
__device__ __forceinline__ bool above(const Ranked& a, const Ranked& b)
{
    const bool an = a.v != a.v, bn = b.v != b.v;
    if (an || bn) return an && (!bn || a.i < b.i);
    return a.v > b.v || (a.v == b.v && a.i < b.i);
}

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

template <typename F>
__device__ __forceinline__ float block_fold(float x, float* sh, F f)
{
    __syncthreads();
    sh[threadIdx.x] = x;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) sh[threadIdx.x] = f(sh[threadIdx.x], sh[threadIdx.x + o]);
        __syncthreads();
    }
    return sh[0];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) forge_token_logprob_kernel(const T* logits, const Args p)
{
    __shared__ float sh[kThreads];
    __shared__ Ranked sr[kThreads];
    const int64_t r = blockIdx.x;
    const T* x = logits + r * p.ld;
    int64_t t = 0;
    if (p.targets) t = target_of(p.targets, p.wide, r, p.V, p.status);
    if (t < 0) {
        if (threadIdx.x == 0) {
            if (p.logprob) p.logprob[r] = 0.0f;
            if (p.lse) p.lse[r] = 0.0f;
            if (p.entropy) p.entropy[r] = 0.0f;
        }
        for (int k = threadIdx.x; k < p.top_k; k += kThreads) {
            p.top_index[r * p.top_k + k] = -1;
            p.top_logprob[r * p.top_k + k] = 0.0f;
        }
        return;
    }
    float m = -INFINITY;
    for (int64_t j = threadIdx.x; j < p.V; j += kThreads) m = nan_max(m, load1(x, j));
    m = block_fold(m, sh, nan_max) * p.scale;
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, w = 0.0f;
    for (int64_t j = threadIdx.x; j < p.V; j += kThreads) {
        const float d = load1(x, j) * p.scale - ref;
        const float e = expf(d);
        s += e;
        if (!(e == 0.0f)) w += e * d;
    }
    auto add = [](float a, float b) { return a + b; };
    s = block_fold(s, sh, add);
    w = block_fold(w, sh, add);
    const bool none = m == -INFINITY;
    const float lse = ref + logf(s);
    if (threadIdx.x == 0) {
        if (p.logprob) p.logprob[r] = none ? -INFINITY : load1(x, t) * p.scale - lse;
        if (p.lse) p.lse[r] = lse;
        if (p.entropy) p.entropy[r] = none ? 0.0f : logf(s) - w / s;
    }
    // the top alternatives, one pass each: the best entry below the last one
    Ranked last{0.0f, -1};
    for (int k = 0; k < p.top_k; ++k) {
        Ranked best{0.0f, -1};
        for (int64_t j = threadIdx.x; j < p.V; j += kThreads) {
            const Ranked c{load1(x, j), static_cast<int>(j)};
            if (k > 0 && !above(last, c)) continue;
            if (best.i < 0 || above(c, best)) best = c;
        }
        __syncthreads();
        sr[threadIdx.x] = best;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (threadIdx.x < o) {
                const Ranked c = sr[threadIdx.x + o];
                if (c.i >= 0 && (sr[threadIdx.x].i < 0 || above(c, sr[threadIdx.x])))
                    sr[threadIdx.x] = c;
            }
            __syncthreads();
        }
        last = sr[0];
        if (threadIdx.x == 0) {
            p.top_index[r * p.top_k + k] = last.i;
            p.top_logprob[r * p.top_k + k] = none ? -INFINITY : last.v * p.scale - lse;
        }
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

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads)
    forge_token_logprob_grad_kernel(const T* logits, O* dlogits, const GradArgs p)
{
    const int64_t r = blockIdx.x;
    const T* x = logits + r * p.ld;
    O* dx = dlogits + r * p.ld_out;
    const int64_t t = target_of(p.targets, p.wide, r, p.V, p.status);
    const float lse = p.lse[r];
    const bool dead = t < 0 || lse == -INFINITY;
    const float a = p.grad_logprob[r];
    const float b = p.grad_entropy ? p.grad_entropy[r] : 0.0f;
    const float h = p.grad_entropy ? p.entropy[r] : 0.0f;
    for (int64_t j = threadIdx.x; j < p.V; j += kThreads) {
        float g = 0.0f;
        if (!dead) {
            const float d = load1(x, j) * p.scale - lse;
            const float e = expf(d);
            g = -e * (a + b * ((e == 0.0f ? 0.0f : d) + h));
            if (j == t) g += a;
            g *= p.scale;
        }
        store1(dx, j, g);
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : (t == FORGE_I64 ? 8 : 4); }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }
bool is_id(forge_dtype t) { return t == FORGE_I32 || t == FORGE_I64; }

forge_status check_rows(int64_t R, int64_t V, int64_t ld, float scale)
{
    if (R < 0 || V < 1 || ld < V || R > INT32_MAX || V > INT32_MAX) return FORGE_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FORGE_ERR_INVALID_ARG;
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
    const int grid = static_cast<int>(R);
    if (dtype == FORGE_F32)
        forge_token_logprob_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float*>(logits), p);
    else
        forge_token_logprob_kernel<<<grid, kThreads, 0, s>>>(
            static_cast<const __nv_bfloat16*>(logits), p);
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
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
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    if (R == 0) return FORGE_OK;
    const void* ptrs[] = {logits, targets, lse, grad_logprob, entropy, grad_entropy, dlogits};
    if ((st = device_resident(ptrs, 7)) != FORGE_OK) return st;
    const GradArgs p{R,   V,            ld,      ld_out,       targets, id_dtype == FORGE_I64, scale,
                     lse, grad_logprob, entropy, grad_entropy, device_status_word()};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(R);
    auto go = [&](auto* x, auto* dx) {
        forge_token_logprob_grad_kernel<<<grid, kThreads, 0, s>>>(x, dx, p);
    };
    auto in = [&](auto* x) {
        if (out_dtype == FORGE_F32)
            go(x, static_cast<float*>(dlogits));
        else
            go(x, static_cast<__nv_bfloat16*>(dlogits));
    };
    if (dtype == FORGE_F32)
        in(static_cast<const float*>(logits));
    else
        in(static_cast<const __nv_bfloat16*>(logits));
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
