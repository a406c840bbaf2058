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

template <typename W, typename Y>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_kernel(const void* ids, bool wide, const W* w, Y* y, int64_t V, int64_t D,
                           float scale, int* status)
{
    const int64_t t = blockIdx.x;
    const int64_t r = id_of(ids, wide, t, V, status);
    for (int64_t j = threadIdx.x; j < D; j += kThreads)
        store1(y, t * D + j, r < 0 ? 0.0f : load1(w, r * D + j) * scale);
}

enum { SUM_STORE = 0, SUM_ADD = 1, SUM_ADAMW = 2 };

// One block per vocabulary row: its threads read the ids in order and add the
// rows of the tokens that match.
template <typename G, int MODE, int ST>
__global__ void __launch_bounds__(kThreads)
    forge_embedding_grad_kernel(const G* dY, const void* ids, bool wide, int64_t T, int64_t V,
                                int64_t D, float scale, float* dW, const Params p)
{
    const int64_t r = blockIdx.x;
    for (int64_t j = threadIdx.x; j < D; j += kThreads) {
        float g = 0.0f;
        for (int64_t t = 0; t < T; ++t)
            if (id_of(ids, wide, t, V, p.status) == r) g += load1(dY, t * D + j);
        g *= scale;
        const int64_t at = r * D + j;
        if constexpr (MODE == SUM_ADAMW) {
            float gs[4] = {g, g, g, g}, w[4], a[4], b[4];
            for (int i = 0; i < 4; ++i) {
                w[i] = StateIO<ST_F32>::ld(p.W, at);
                a[i] = StateIO<ST>::ld(p.s1, at);
                b[i] = StateIO<ST>::ld(p.s2, at);
            }
            step4<OP_ADAMW>(p, gs, w, a, b);
            StateIO<ST_F32>::st(p.W, at, w[0]);
            StateIO<ST>::st(p.s1, at, a[0]);
            StateIO<ST>::st(p.s2, at, b[0]);
        } else {
            dW[at] = MODE == SUM_ADD ? dW[at] + g : g;
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

template <int MODE, int ST>
cudaError_t grad(const void* dY, forge_dtype dy_dtype, const void* ids, forge_dtype id_dtype,
                 int64_t T, int64_t V, int64_t D, float scale, float* dW, const Params& p,
                 cudaStream_t s)
{
    const int grid = static_cast<int>(V);
    const bool wide = id_dtype == FORGE_I64;
    if (dy_dtype == FORGE_F32)
        forge_embedding_grad_kernel<float, MODE, ST><<<grid, kThreads, 0, s>>>(
            static_cast<const float*>(dY), ids, wide, T, V, D, scale, dW, p);
    else
        forge_embedding_grad_kernel<__nv_bfloat16, MODE, ST><<<grid, kThreads, 0, s>>>(
            static_cast<const __nv_bfloat16*>(dY), ids, wide, T, V, D, scale, dW, p);
    return cudaGetLastError();
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
        forge_embedding_kernel<<<static_cast<int>(T), kThreads, 0, s>>>(
            ids, id_dtype == FORGE_I64, w, y, V, D, scale, status);
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
        accumulate ? grad<SUM_ADD, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, dW, p, s)
                   : grad<SUM_STORE, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, dW, p, s);
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
            ? grad<SUM_ADAMW, ST_F32>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, nullptr, p, s)
            : grad<SUM_ADAMW, ST_BF16>(dY, dy_dtype, ids, id_dtype, T, V, D, scale, nullptr, p, s);
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
