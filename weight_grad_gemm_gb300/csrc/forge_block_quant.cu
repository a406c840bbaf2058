// forge_block_quant.cu -- e4m3 codes with one scale for each block of 128
// entries of a row, or for each square of 128 x 128: the operands of
// forge_linear_e4m3.
//
// A block with the largest magnitude amax takes s = amax / 448 (an fp32
// division; 1 where that is 0) and codes e4m3(x / s), nearest, ties to even,
// saturating: forge_quantize_e4m3's recipe, block by block.  One pass: a block
// is held in registers between its maximum and its codes, so that x is read
// once (1 + 4 / 128 or 1 + 4 / 16384 bytes written for each entry): memory
// bounds both forms.
//   rows     eight lanes a block, four blocks a warp;
//   squares  256 threads a square, 64 entries each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "forge.h"
#include "forge_device.h"
#include "forge_rows.cuh"

namespace forge {
namespace block_quant {

constexpr int kBlock = 128;
constexpr int kThreads = 256;
constexpr int kLanes = 8;  // of a block of a row

__device__ __forceinline__ float scale_of(float amax)
{
    const float s = __fdiv_rn(amax, 448.0f);
    return s > 0.0f ? s : 1.0f;
}

// Two fp32 values to e4m3 (nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename X, int V>
__device__ __forceinline__ float amax_of(const Packed<X, V>& x)
{
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, fabsf(entry(x, j)));  // leaves NaN out
    return m;
}

template <typename X, int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const Packed<X, V>& x, float s)
{
    if constexpr (V == 1) {
        *q = static_cast<uint8_t>(e4m3x2(__fdiv_rn(entry(x, 0), s), 0.0f));
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            w[i] = e4m3x2(__fdiv_rn(entry(x, 4 * i), s), __fdiv_rn(entry(x, 4 * i + 1), s)) |
                   e4m3x2(__fdiv_rn(entry(x, 4 * i + 2), s), __fdiv_rn(entry(x, 4 * i + 3), s))
                       << 16;
        if constexpr (V == 4)
            *reinterpret_cast<uint32_t*>(q) = w[0];
        else
            *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    }
}

template <typename X, int V>
__global__ void __launch_bounds__(kThreads)
    forge_quantize_rows_kernel(const X* __restrict__ x, int64_t ldx, uint32_t units, uint32_t C,
                               uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    constexpr int NV = kBlock / kLanes / V;
    const uint32_t u = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const uint32_t l = threadIdx.x % kLanes;
    const uint32_t per_row = (C + kBlock - 1) / kBlock;
    const bool live = u < units;  // (all lanes of a warp stay for the maximum)
    const uint32_t row = live ? u / per_row : 0, c0 = live ? (u - row * per_row) * kBlock : 0;
    Packed<X, V> raw[NV];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = c0 + (i * kLanes + l) * V;
        raw[i] = live && c < C ? load_packed<X, V>(x + row * ldx + c) : zero_packed<X, V>();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, amax_of(raw[i]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!live) return;
    const float s = scale_of(m);
    if (l == 0) scales[u] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t c = c0 + (i * kLanes + l) * V;
        if (c < C) store_codes(codes + static_cast<int64_t>(row) * C + c, raw[i], s);
    }
}

template <typename X, int V>
__global__ void __launch_bounds__(kThreads)
    forge_quantize_squares_kernel(const X* __restrict__ x, int64_t ldx, int64_t R, int64_t C,
                                  uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    constexpr int NV = kBlock * kBlock / kThreads / V;
    __shared__ float sh[kThreads / 32];
    const int64_t across = (C + kBlock - 1) / kBlock, down = (R + kBlock - 1) / kBlock;
    const int64_t cb = blockIdx.x % across, rest = blockIdx.x / across;
    const int64_t rb = rest % down, e = rest / down;
    const int64_t r0 = rb * kBlock, c0 = cb * kBlock;
    const X* base = x + e * R * ldx;
    Packed<X, V> raw[NV];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * kThreads + threadIdx.x) * V;
        const int64_t r = r0 + at / kBlock, c = c0 + at % kBlock;
        raw[i] = r < R && c < C ? load_packed<X, V>(base + r * ldx + c) : zero_packed<X, V>();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, amax_of(raw[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, sh[i]);
    const float s = scale_of(m);
    if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * kThreads + threadIdx.x) * V;
        const int64_t r = r0 + at / kBlock, c = c0 + at % kBlock;
        if (r < R && c < C) store_codes(codes + (e * R + r) * C + c, raw[i], s);
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename X, int V>
cudaError_t launch(const X* x, int64_t ldx, int64_t E, int64_t R, int64_t C, int block_rows,
                   uint8_t* codes, float* scales, cudaStream_t s)
{
    const int64_t across = (C + kBlock - 1) / kBlock;
    if (block_rows == 1) {
        // units of one launch stay below 2^31
        const int64_t rows = E * R, most = (int64_t{1} << 30) / across;
        for (int64_t r = 0; r < rows; r += most) {
            const int64_t n = (rows - r < most ? rows - r : most) * across;
            forge_quantize_rows_kernel<X, V>
                <<<static_cast<unsigned>((n + kThreads / kLanes - 1) / (kThreads / kLanes)),
                   kThreads, 0, s>>>(x + r * ldx, ldx, static_cast<uint32_t>(n),
                                     static_cast<uint32_t>(C), codes + r * C, scales + r * across);
        }
    } else {
        const int64_t squares = E * ((R + kBlock - 1) / kBlock) * across;
        if (squares > INT32_MAX) return cudaErrorInvalidConfiguration;
        forge_quantize_squares_kernel<X, V><<<static_cast<unsigned>(squares), kThreads, 0, s>>>(
            x, ldx, R, C, codes, scales);
    }
    return cudaGetLastError();
}

}  // namespace block_quant
}  // namespace forge

using namespace forge;

extern "C" forge_status forge_quantize_e4m3_blocks(const void* x, forge_dtype x_dtype, int64_t ldx,
                                                   int64_t E, int64_t R, int64_t C,
                                                   int32_t block_rows, uint8_t* codes,
                                                   float* scales, forge_stream_t stream)
{
    using namespace block_quant;
    if (E < 0 || R < 0 || C < 1 || ldx < C || E > INT32_MAX || R > INT32_MAX || C > (1 << 30) ||
        (block_rows != 1 && block_rows != kBlock))
        return FORGE_ERR_INVALID_ARG;
    // (below 2^40 rows, so that no product of sizes overflows)
    if (E * R > int64_t{1} << 40 || E * R * (C / 2 + 1) > int64_t{1} << 60) return FORGE_ERR_INVALID_ARG;
    if (E * R > 0 && (!x || !codes || !scales)) return FORGE_ERR_INVALID_ARG;
    if (x_dtype != FORGE_F32 && x_dtype != FORGE_BF16) return FORGE_ERR_UNSUPPORTED_DTYPE;
    const int es = x_dtype == FORGE_F32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(scales, 4)) return FORGE_ERR_MISALIGNED;
    int sms = 0;
    forge_status st = device_sms(&sms);
    if (st != FORGE_OK) return st;
    if (E * R == 0) return FORGE_OK;
    const void* ptrs[] = {x, codes, scales};
    if ((st = device_resident(ptrs, 3)) != FORGE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto fits = [&](int V) {
        return C % V == 0 && ldx % V == 0 && aligned(x, V * es) && aligned(codes, V);
    };
    cudaError_t e;
    if (x_dtype == FORGE_F32) {
        const float* f = static_cast<const float*>(x);
        e = fits(4) ? launch<float, 4>(f, ldx, E, R, C, block_rows, codes, scales, s)
                    : launch<float, 1>(f, ldx, E, R, C, block_rows, codes, scales, s);
    } else {
        const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
        e = fits(8)   ? launch<__nv_bfloat16, 8>(h, ldx, E, R, C, block_rows, codes, scales, s)
            : fits(4) ? launch<__nv_bfloat16, 4>(h, ldx, E, R, C, block_rows, codes, scales, s)
                      : launch<__nv_bfloat16, 1>(h, ldx, E, R, C, block_rows, codes, scales, s);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
