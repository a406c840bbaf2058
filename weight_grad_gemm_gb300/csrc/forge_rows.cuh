// forge_rows.cuh -- rows of fp32 or bf16 read and written in vectors, and the
// sums of a warp or a block over them: what the row-wise kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace forge {

// V consecutive entries of T as they lie in memory, in 32-bit registers (one
// entry of bf16 takes a whole one).
template <typename T, int V>
struct alignas(V * sizeof(T) >= 16 ? 16 : (V * sizeof(T) == 8 ? 8 : 4)) Packed {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T));
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
};

// From an address aligned to the vector, at most 16 bytes an instruction.  Read-only
// loads: for what nothing writes while the kernel lives.
template <typename T, int V>
__device__ __forceinline__ Packed<T, V> load_packed(const T* p)
{
    Packed<T, V> r;
    if constexpr (r.kBytes == 2) {
        r.w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
    } else if constexpr (r.kBytes == 4) {
        r.w[0] = __ldg(reinterpret_cast<const unsigned int*>(p));
    } else if constexpr (r.kBytes == 8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        r.w[0] = u.x;
        r.w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < r.kWords / 4; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            r.w[4 * i] = u.x;
            r.w[4 * i + 1] = u.y;
            r.w[4 * i + 2] = u.z;
            r.w[4 * i + 3] = u.w;
        }
    }
    return r;
}

// The same by plain loads: for rows that the kernel itself may write over (calls in place).
template <typename T, int V>
__device__ __forceinline__ Packed<T, V> load_plain(const T* p)
{
    Packed<T, V> r;
    if constexpr (r.kBytes == 2) {
        r.w[0] = *reinterpret_cast<const unsigned short*>(p);
    } else if constexpr (r.kBytes == 4) {
        r.w[0] = *reinterpret_cast<const unsigned int*>(p);
    } else if constexpr (r.kBytes == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        r.w[0] = u.x;
        r.w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < r.kWords / 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[i];
            r.w[4 * i] = u.x;
            r.w[4 * i + 1] = u.y;
            r.w[4 * i + 2] = u.z;
            r.w[4 * i + 3] = u.w;
        }
    }
    return r;
}

// Of rows that the call writes over (OVER), or leaves alone.
template <bool OVER, typename T, int V>
__device__ __forceinline__ Packed<T, V> load_row(const T* p)
{
    if constexpr (OVER)
        return load_plain<T, V>(p);
    else
        return load_packed<T, V>(p);
}

template <typename T, int V>
__device__ __forceinline__ Packed<T, V> zero_packed()
{
    Packed<T, V> r;
#pragma unroll
    for (int i = 0; i < r.kWords; ++i) r.w[i] = 0;
    return r;
}

// Entry i of a vector as fp32.
template <int V>
__device__ __forceinline__ float entry(const Packed<float, V>& p, int i)
{
    return __uint_as_float(p.w[i]);
}
template <int V>
__device__ __forceinline__ float entry(const Packed<__nv_bfloat16, V>& p, int i)
{
    return __uint_as_float(i & 1 ? p.w[i / 2] & 0xFFFF0000u : p.w[i / 2] << 16);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// V fp32 values to an address aligned to the stored vector; bf16 rounds to
// nearest even.
template <int V>
__device__ __forceinline__ void store_vector(float* p, const float (&v)[V])
{
    if constexpr (V == 1) {
        p[0] = v[0];
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            reinterpret_cast<float4*>(p)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
template <int V>
__device__ __forceinline__ void store_vector(__nv_bfloat16* p, const float (&v)[V])
{
    if constexpr (V == 1) {
        p[0] = __float2bfloat16_rn(v[0]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t*>(p) = bf16x2(v[0], v[1]);
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 8)
            reinterpret_cast<uint4*>(p)[i / 8] =
                make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]),
                           bf16x2(v[i + 4], v[i + 5]), bf16x2(v[i + 6], v[i + 7]));
    }
}

// An output of either type, chosen at run time (a branch that all threads
// take alike costs less than twice the kernels).
template <int V>
__device__ __forceinline__ void store_as(void* base, bool f32, int64_t at, const float (&v)[V])
{
    if (f32)
        store_vector(static_cast<float*>(base) + at, v);
    else
        store_vector(static_cast<__nv_bfloat16*>(base) + at, v);
}

// The sum over LANES neighbouring lanes, in all of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sums of N values over a block of W warps, in every thread, in an order
// that does not depend on the schedule.  `sh` holds W * N floats; callers
// alternate between two such buffers, so one barrier a call is enough.
template <int W, int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* sh)
{
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = lanes_sum<32>(v[n]);
    if constexpr (W > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) sh[n * W + warp] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = lanes_sum<W>(sh[n * W + (lane & (W - 1))]);
    }
}

// Programmatic dependent launch: the next kernel of the stream may start, and
// what the previous one wrote is there.
__device__ __forceinline__ void let_dependents_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void await_prerequisites()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace forge
