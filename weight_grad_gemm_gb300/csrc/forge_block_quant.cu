// forge_block_quant.cu -- e4m3 codes with one scale for each block of 128
// entries of a row, or for each square of 128 x 128: the operands of
// forge_linear_e4m3.
//
// A block with the largest magnitude amax takes s = amax / 448 (an fp32
// division; 1 where that is 0) and codes e4m3(x / s), nearest, ties to even,
// saturating: forge_quantize_e4m3's recipe, block by block.  One pass: a block
// is held in registers between its maximum and its codes, so that x is read
// once (1 + 4 / 128 or 1 + 4 / 16384 bytes written for each entry): memory
// bounds both forms, once the quotients do not (see Quotient).
//   rows     eight lanes a block, four blocks a warp;
//   squares  512 threads a square, 32 entries each.
//
// Measured (the copy bandwidth is 6.68 TB/s): rows, 16384 x 4096 bf16 39 us (5.3 TB/s, 73%
// of the issue slots), 8192 x 4095 48 (entry by entry: instructions); squares, 14336 x 4096
// fp32 51 us (5.8 TB/s).
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
constexpr int kSquareThreads = 512;
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

// x / s in fp32, nearest.  A division for each entry costs more than its memory
// traffic, so: with r = 1 / s, nearest, q = x r is within 1.5 fp32 steps of the
// quotient; q + r (x - q s), the remainder exact by fma, is within one; and from such a
// q the same step gives the nearest (Markstein 1990).  For scales from 2^-80 to
// 2^80 no remainder underflows that belongs to a code but 0 (x / s >= 2^-11); other
// blocks divide.
struct Quotient {
    float s, r;
    bool fast;
};
__device__ __forceinline__ Quotient quotient_by(float s)
{
    return {s, __fdiv_rn(1.0f, s), s > 0x1p-80f && s < 0x1p80f};
}

template <typename X, int V>
__device__ __forceinline__ void store_codes(uint8_t* out, const Packed<X, V>& x, const Quotient& by)
{
    float q[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        q[j] = entry(x, j) * by.r;
        // (the remainder with its sign turned: it is +0 where q s = x, and taking +0 from q
        // leaves -0 as it is, which adding it does not)
        q[j] = fmaf(-fmaf(q[j], by.s, -entry(x, j)), by.r, q[j]);
        q[j] = fmaf(-fmaf(q[j], by.s, -entry(x, j)), by.r, q[j]);
    }
    if (!by.fast) {
#pragma unroll 1
        for (int j = 0; j < V; ++j) {
            float e = entry(x, 0);
#pragma unroll
            for (int k = 1; k < V; ++k) e = j == k ? entry(x, k) : e;
            e = __fdiv_rn(e, by.s);
#pragma unroll
            for (int k = 0; k < V; ++k) q[k] = j == k ? e : q[k];
        }
    }
    if constexpr (V == 1) {
        *out = static_cast<uint8_t>(e4m3x2(q[0], 0.0f));
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            w[i] = e4m3x2(q[4 * i], q[4 * i + 1]) | e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16;
        if constexpr (V == 4)
            *reinterpret_cast<uint32_t*>(out) = w[0];
        else
            *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    }
}

// A thread has a part of two units, loaded before the first one's maximum (16384 x 4096
// bf16: 39 us, with one unit 48, with three or four 39); one where it takes entries one
// by one (8192 x 4095 bf16: 48 us, with two 62).
__host__ __device__ constexpr int turns_of(int V) { return V == 1 ? 1 : 2; }
template <typename X, int V>
__global__ void __launch_bounds__(kThreads)
    forge_quantize_rows_kernel(const X* __restrict__ x, int64_t ldx, uint32_t units, uint32_t C,
                               uint8_t* __restrict__ codes, float* __restrict__ scales)
{
    constexpr int NV = kBlock / kLanes / V, kTurns = turns_of(V);
    const uint32_t l = threadIdx.x % kLanes;
    const uint32_t per_row = (C + kBlock - 1) / kBlock;
    Packed<X, V> raw[kTurns][NV];
    uint32_t us[kTurns], rows[kTurns], cs[kTurns];
#pragma unroll
    for (int n = 0; n < kTurns; ++n) {
        us[n] = (blockIdx.x * kTurns + n) * (kThreads / kLanes) + threadIdx.x / kLanes;
        rows[n] = us[n] / per_row;
        cs[n] = (us[n] - rows[n] * per_row) * kBlock + l * V;
        const X* at = x + rows[n] * ldx + cs[n];
#pragma unroll
        for (int i = 0; i < NV; ++i)  // (all lanes of a warp stay for the maximum)
            raw[n][i] = us[n] < units && cs[n] + i * kLanes * V < C
                            ? load_packed<X, V>(at + i * kLanes * V)
                            : zero_packed<X, V>();
    }
#pragma unroll
    for (int n = 0; n < kTurns; ++n) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, amax_of(raw[n][i]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (us[n] >= units) continue;
        const float s = scale_of(m);
        if (l == 0) scales[us[n]] = s;
        const Quotient by = quotient_by(s);
        uint8_t* at = codes + static_cast<int64_t>(rows[n]) * C + cs[n];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (cs[n] + i * kLanes * V < C) store_codes(at + i * kLanes * V, raw[n][i], by);
    }
}

// Persistent, one block an SM: the next square is on its way into registers while this
// one's codes are made (14336 x 4096 fp32: 52 us; a square a block, two or three blocks
// an SM, 65).
template <typename X, int V>
__global__ void __launch_bounds__(kSquareThreads)
    forge_quantize_squares_kernel(const X* __restrict__ x, int64_t ldx, uint32_t R, uint32_t C,
                                  uint32_t squares, uint8_t* __restrict__ codes,
                                  float* __restrict__ scales)
{
    constexpr int NV = kBlock * kBlock / kSquareThreads / V;
    constexpr uint32_t kStep = kSquareThreads * V / kBlock;  // rows between a thread's vectors
    __shared__ float sh[2][kSquareThreads / 32];
    const uint32_t across = (C + kBlock - 1) / kBlock, down = (R + kBlock - 1) / kBlock;
    const uint32_t dr = threadIdx.x * V / kBlock, dc = threadIdx.x * V % kBlock;
    Packed<X, V> ahead[NV];
    // the thread's first row and column of square n, and its matrix
    auto place = [&](uint32_t n, uint32_t& e, uint32_t& r, uint32_t& c) {
        const uint32_t rest = n / across;
        c = (n - rest * across) * kBlock + dc;
        e = rest / down;
        r = (rest - e * down) * kBlock + dr;
    };
    auto load = [&](uint32_t n) {
        uint32_t e, r, c;
        place(n, e, r, c);
        const X* at = x + (static_cast<int64_t>(e) * R + r) * ldx + c;
#pragma unroll
        for (int i = 0; i < NV; ++i, at += kStep * ldx)
            ahead[i] = r + i * kStep < R && c < C ? load_packed<X, V>(at) : zero_packed<X, V>();
    };
    if (blockIdx.x < squares) load(blockIdx.x);
    int turn = 0;
    for (uint32_t n = blockIdx.x; n < squares; n += gridDim.x, turn ^= 1) {
        Packed<X, V> raw[NV];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i] = ahead[i];
            m = fmaxf(m, amax_of(raw[i]));
        }
        if (n + gridDim.x < squares) load(n + gridDim.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) sh[turn][threadIdx.x >> 5] = m;
        __syncthreads();
        m = sh[turn][threadIdx.x & (kSquareThreads / 32 - 1)];
#pragma unroll
        for (int o = kSquareThreads / 64; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = scale_of(m);
        if (threadIdx.x == 0) scales[n] = s;
        const Quotient by = quotient_by(s);
        uint32_t e, r, c;
        place(n, e, r, c);
        uint8_t* at = codes + (static_cast<int64_t>(e) * R + r) * C + c;
#pragma unroll
        for (int i = 0; i < NV; ++i, at += static_cast<int64_t>(kStep) * C)
            if (r + i * kStep < R && c < C) store_codes(at, raw[i], by);
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename X, int V>
cudaError_t launch(const X* x, int64_t ldx, int64_t E, int64_t R, int64_t C, int block_rows,
                   uint8_t* codes, float* scales, int sms, cudaStream_t s)
{
    const int64_t across = (C + kBlock - 1) / kBlock;
    if (block_rows == 1) {
        // units of one launch stay below 2^31
        constexpr int kUnits = kThreads / kLanes * turns_of(V);  // of a block
        const int64_t rows = E * R, most = (int64_t{1} << 30) / across;
        for (int64_t r = 0; r < rows; r += most) {
            const int64_t n = (rows - r < most ? rows - r : most) * across;
            forge_quantize_rows_kernel<X, V>
                <<<static_cast<unsigned>((n + kUnits - 1) / kUnits), kThreads, 0, s>>>(x + r * ldx, ldx, static_cast<uint32_t>(n),
                                     static_cast<uint32_t>(C), codes + r * C, scales + r * across);
        }
    } else {
        const int64_t squares = E * ((R + kBlock - 1) / kBlock) * across;
        if (squares > INT32_MAX) return cudaErrorInvalidConfiguration;
        forge_quantize_squares_kernel<X, V>
            <<<static_cast<unsigned>(squares < sms ? squares : sms), kSquareThreads, 0, s>>>(
                x, ldx, static_cast<uint32_t>(R), static_cast<uint32_t>(C),
                static_cast<uint32_t>(squares), codes, scales);
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
        e = fits(4) ? launch<float, 4>(f, ldx, E, R, C, block_rows, codes, scales, sms, s)
                    : launch<float, 1>(f, ldx, E, R, C, block_rows, codes, scales, sms, s);
    } else {
        const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(x);
        e = fits(8)   ? launch<__nv_bfloat16, 8>(h, ldx, E, R, C, block_rows, codes, scales, sms, s)
            : fits(4) ? launch<__nv_bfloat16, 4>(h, ldx, E, R, C, block_rows, codes, scales, sms, s)
                      : launch<__nv_bfloat16, 1>(h, ldx, E, R, C, block_rows, codes, scales, sms, s);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}
