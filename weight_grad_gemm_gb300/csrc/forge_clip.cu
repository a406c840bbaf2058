// forge_clip.cu -- the global norm of many gradient tensors, and their
// clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g min(1, max_norm / (norm + 1e-6))
// Exact global-norm clipping needs every gradient before it may touch one, so
// it cannot be fused with the weight gradient ("Math verified, not asserted",
// P2); it serves the paths that hold gradients in memory, in front of the
// owner's step.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "forge.h"
#include "forge_device.h"

namespace forge {
namespace clip {

constexpr int kThreads = 256;
constexpr int kBlocks = 512;

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

__device__ __forceinline__ double block_sum(double x, double* sh)
{
    sh[threadIdx.x] = x;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
        __syncthreads();
    }
    return sh[0];
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    forge_square_sum_kernel(const T* g, int64_t n, double* part)
{
    __shared__ double sh[kThreads];
    float s = 0.0f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(kBlocks) * kThreads) {
        const float x = load1(g, i);
        s = fmaf(x, x, s);
    }
    const double total = block_sum(s, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads)
    forge_norm_fold_kernel(const double* part, int64_t n, float* norm)
{
    __shared__ double sh[kThreads];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[i];
    s = block_sum(s, sh);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads)
    forge_clip_kernel(const T* g, O* out, int64_t n, const float* norm, float max_norm)
{
    const float q = max_norm / (*norm + 1e-6f);
    const float c = q > 1.0f ? 1.0f : q;  // a NaN stays
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(kBlocks) * kThreads)
        store1(out, i, load1(g, i) * c);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(forge_dtype t) { return t == FORGE_BF16 ? 2 : 4; }
bool is_float(forge_dtype t) { return t == FORGE_F32 || t == FORGE_BF16; }

forge_status check_list(const void* const* ptr, const int64_t* n, int32_t P)
{
    if (P < 0 || (P > 0 && (!ptr || !n))) return FORGE_ERR_INVALID_ARG;
    for (int32_t j = 0; j < P; ++j)
        if (n[j] < 0 || (n[j] > 0 && !ptr[j])) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

forge_status check_memory(const void* const* ptr, const int64_t* n, int32_t P, forge_dtype dt)
{
    for (int32_t j = 0; j < P; ++j) {
        if (n[j] == 0) continue;
        const forge_status st = device_resident(&ptr[j], 1);
        if (st != FORGE_OK) return st;
        if (!aligned(ptr[j], size_of(dt))) return FORGE_ERR_MISALIGNED;
    }
    return FORGE_OK;
}

}  // namespace clip
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_grad_norm(const void* const* grads, const int64_t* n, int32_t P,
                                        forge_dtype dtype, float* norm, forge_stream_t stream)
{
    using namespace clip;
    if (!norm) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_list(grads, n, P);
    if (st != FORGE_OK) return st;
    if (!is_float(dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* one[] = {norm};
    if ((st = device_resident(one, 1)) != FORGE_OK) return st;
    if ((st = check_memory(grads, n, P, dtype)) != FORGE_OK) return st;
    if (!aligned(norm, 4)) return FORGE_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t parts = static_cast<int64_t>(P) * kBlocks;
    void* scratch = nullptr;
    if (scratch_alloc(&scratch, (parts + 1) * sizeof(double), s) != cudaSuccess) {
        cudaGetLastError();
        return FORGE_ERR_CUDA;
    }
    double* part = static_cast<double*>(scratch);
    for (int32_t j = 0; j < P; ++j) {
        if (dtype == FORGE_F32)
            forge_square_sum_kernel<<<kBlocks, kThreads, 0, s>>>(
                static_cast<const float*>(grads[j]), n[j], part + static_cast<int64_t>(j) * kBlocks);
        else
            forge_square_sum_kernel<<<kBlocks, kThreads, 0, s>>>(
                static_cast<const __nv_bfloat16*>(grads[j]), n[j],
                part + static_cast<int64_t>(j) * kBlocks);
    }
    forge_norm_fold_kernel<<<1, kThreads, 0, s>>>(part, parts, norm);
    cudaError_t e = cudaGetLastError();
    const cudaError_t fe = scratch_free(scratch, s);
    if (e == cudaSuccess) e = fe;
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

extern "C" forge_status forge_clip_grads(const void* const* grads, const int64_t* n, int32_t P,
                                         forge_dtype dtype, const float* norm, float max_norm,
                                         void* const* out, forge_dtype out_dtype,
                                         forge_stream_t stream)
{
    using namespace clip;
    if (!norm || !(max_norm >= 0.0f)) return FORGE_ERR_INVALID_ARG;
    forge_status st = check_list(grads, n, P);
    if (st != FORGE_OK || (st = check_list(out, n, P)) != FORGE_OK) return st;
    if (!is_float(dtype) || !is_float(out_dtype)) return FORGE_ERR_UNSUPPORTED_DTYPE;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* one[] = {norm};
    if ((st = device_resident(one, 1)) != FORGE_OK) return st;
    if ((st = check_memory(grads, n, P, dtype)) != FORGE_OK ||
        (st = check_memory(out, n, P, out_dtype)) != FORGE_OK)
        return st;
    if (!aligned(norm, 4)) return FORGE_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int32_t j = 0; j < P; ++j) {
        if (n[j] == 0) continue;
        auto go = [&](auto* g, auto* o) {
            forge_clip_kernel<<<kBlocks, kThreads, 0, s>>>(g, o, n[j], norm, max_norm);
        };
        auto in = [&](auto* g) {
            if (out_dtype == FORGE_F32)
                go(g, static_cast<float*>(out[j]));
            else
                go(g, static_cast<__nv_bfloat16*>(out[j]));
        };
        if (dtype == FORGE_F32)
            in(static_cast<const float*>(grads[j]));
        else
            in(static_cast<const __nv_bfloat16*>(grads[j]));
    }
    return cudaGetLastError() == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
