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
constexpr int kBlocksPerSm = 8;
constexpr int kTable = 512;                       // tensors of one launch
constexpr int kMinChunkBits = 11, kMaxChunkBits = 15;
constexpr int kFlight = 4;                        // 16-byte loads in flight per thread

// The tensors of one launch, cut into chunks of 2^chunk_bits elements; tensor
// j's chunks are [begin[j], begin[j + 1]) of the launch's.
struct Table {
    const void* in[kTable];
    void* out[kTable];
    int64_t n[kTable];
    uint32_t begin[kTable + 1];
    int32_t count;
    int32_t chunk_bits;
};

// The tensor that chunk c belongs to: begin[j] <= c < begin[j + 1].
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t c)
{
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.begin[mid] <= c)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

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

__device__ __forceinline__ void to_float(const uint4& u, float (&x)[4])
{
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void to_float(const uint4& u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
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

__device__ __forceinline__ bool is_aligned(const void* p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

__device__ __forceinline__ double block_sum(double x, double* sh)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += sh[w];
    return s;
}

// The squares of a thread's part of a chunk, nv vectors and the elements behind
// them, in fp64.
template <typename T>
__device__ __noinline__ double wide_square_sum(const T* g, int nv, int n)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    double s = 0.0;
    auto add = [&](int i) {
        const double x = static_cast<double>(load1(g, i));
        s = fma(x, x, s);
    };
    for (int v = threadIdx.x; v < nv; v += kThreads)
        for (int k = 0; k < N; ++k) add(v * N + k);
    for (int i = nv * N + threadIdx.x; i < n; i += kThreads) add(i);
    return s;
}

// part[block] = the sum of squares over this block's chunks.  A thread adds at
// most 2^15 / 256 = 128 squares in fp32 before it goes on in fp64; where that sum
// is infinite, or so small that squares may have lost digits below 2^-149 or
// vanished, it adds them again in fp64.  The bits of all elements together tell
// zeros, which need no second look, from squares that vanished.  Bound by HBM:
// each gradient is read once.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    forge_square_sum_kernel(const __grid_constant__ Table t, double* part)
{
    __shared__ double sh[kThreads / 32];
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    double total = 0.0;
    for (uint32_t c = blockIdx.x; c < t.begin[t.count]; c += gridDim.x) {
        const int j = tensor_of(t, c);
        const int64_t first = static_cast<int64_t>(c - t.begin[j]) << t.chunk_bits;
        const T* g = static_cast<const T*>(t.in[j]) + first;
        const int64_t left = t.n[j] - first;
        const int n = static_cast<int>(left < (1 << t.chunk_bits) ? left : 1 << t.chunk_bits);
        float s[4] = {};
        uint32_t bits = 0;
        int done = 0;
        if (is_aligned(g, 16)) {
            const int nv = n / N;
            for (int v0 = threadIdx.x; v0 < nv; v0 += kFlight * kThreads) {
                uint4 u[kFlight];
#pragma unroll
                for (int f = 0; f < kFlight; ++f)
                    u[f] = v0 + f * kThreads < nv
                               ? __ldg(reinterpret_cast<const uint4*>(g) + v0 + f * kThreads)
                               : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    float x[N];
                    to_float(u[f], x);
                    bits |= (u[f].x | u[f].y) | (u[f].z | u[f].w);
#pragma unroll
                    for (int k = 0; k < N; ++k) s[k & 3] = fmaf(x[k], x[k], s[k & 3]);
                }
            }
            done = nv * N;
        }
        for (int i = done + threadIdx.x; i < n; i += kThreads) {
            const float x = load1(g, i);
            bits |= __float_as_uint(x);
            s[0] = fmaf(x, x, s[0]);
        }
        const float sum = (s[0] + s[1]) + (s[2] + s[3]);
        constexpr uint32_t kNoSigns = sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
        if ((sum < 0x1p-100f && (bits & kNoSigns) != 0) || sum == INFINITY)
            total += wide_square_sum(g, done / N, n);
        else
            total += static_cast<double>(sum);
    }
    total = block_sum(total, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads)
    forge_norm_fold_kernel(const double* part, int64_t n, float* norm)
{
    __shared__ double sh[kThreads / 32];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[i];
    s = block_sum(s, sh);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

// N elements as they lie in memory.
template <typename T, int N>
struct Group;
template <>
struct Group<float, 4> {
    uint4 u;
    __device__ __forceinline__ void load(const float* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[4]) const { to_float(u, x); }
};
template <>
struct Group<__nv_bfloat16, 8> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const { to_float(u, x); }
};
template <>
struct Group<__nv_bfloat16, 4> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void get(float (&x)[4]) const
    {
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
};

// out = in times the factor, in vectors of 16 bytes of the wider type, so that
// a warp stores whole sectors.  The chunks are walked from the last to the
// first: what the norm's pass read last is still in L2.  Bound by HBM: 973 M
// fp32 gradients into bf16, the norm's pass with it, 1430-1470 us for the 9.7 GB
// that two passes move, 6.7 TB/s.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads)
    forge_clip_kernel(const __grid_constant__ Table t, const float* norm, float max_norm)
{
    constexpr int N = 16 / (sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));
    constexpr int F = N * sizeof(T) < 16 ? 2 * kFlight : kFlight;
    const float all = *norm;
    const float q = max_norm / (all + 1e-6f);
    // without a limit nothing is clipped, an infinite norm neither; a NaN stays
    const float m = q > 1.0f || (all == INFINITY && max_norm == INFINITY) ? 1.0f : q;
    const uint32_t chunks = t.begin[t.count];
    for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
        const uint32_t c = chunks - 1 - b;
        const int j = tensor_of(t, c);
        if (m == 1.0f && t.in[j] == t.out[j]) continue;  // in place, nothing to scale
        const int64_t first = static_cast<int64_t>(c - t.begin[j]) << t.chunk_bits;
        const T* g = static_cast<const T*>(t.in[j]) + first;
        O* o = static_cast<O*>(t.out[j]) + first;
        const int64_t left = t.n[j] - first;
        const int n = static_cast<int>(left < (1 << t.chunk_bits) ? left : 1 << t.chunk_bits);
        int done = 0;
        if (is_aligned(g, N * sizeof(T)) && is_aligned(o, N * sizeof(O))) {
            const int nv = n / N;
            for (int v0 = threadIdx.x; v0 < nv; v0 += F * kThreads) {
                Group<T, N> u[F];
#pragma unroll
                for (int f = 0; f < F; ++f)
                    if (v0 + f * kThreads < nv)
                        u[f].load(g + (v0 + f * kThreads) * N);
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    if (v0 + f * kThreads >= nv) continue;
                    float x[N];
                    u[f].get(x);
#pragma unroll
                    for (int k = 0; k < N; ++k) x[k] *= m;
                    store_vec<N>(o + static_cast<int64_t>(v0 + f * kThreads) * N, x);
                }
            }
            done = nv * N;
        }
        for (int i = done + threadIdx.x; i < n; i += kThreads) store1(o, i, load1(g, i) * m);
    }
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

// No tensor shares memory with its own output but in place.
forge_status check_overlap(const void* const* in, int64_t es, void* const* out, int64_t eo,
                           const int64_t* n, int32_t P)
{
    for (int32_t j = 0; j < P; ++j) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(in[j]), y = reinterpret_cast<uintptr_t>(out[j]);
        if (n[j] == 0 || (x == y && es == eo)) continue;
        const uintptr_t size = y < x ? n[j] * eo : n[j] * es;  // of the lower one
        if ((y < x ? x - y : y - x) < size) return FORGE_ERR_INVALID_ARG;
    }
    return FORGE_OK;
}

forge_status check_memory(const void* const* ptr, const int64_t* n, int32_t P, forge_dtype dt)
{
    // runs of tensors with elements (an empty tensor's pointer means nothing)
    for (int32_t j = 0, first = 0; j <= P; ++j) {
        if (j < P && n[j] > 0) {
            if (!aligned(ptr[j], size_of(dt))) return FORGE_ERR_MISALIGNED;
            continue;
        }
        const forge_status st = device_resident(ptr + first, j - first);
        if (st != FORGE_OK) return st;
        first = j + 1;
    }
    return FORGE_OK;
}

// Cuts the tensors into tables of at most kTable and calls launch(table,
// blocks) for each that has elements.  Chunks are as long as leaves every
// block four of them, within limits.
template <typename F>
forge_status for_tables(const void* const* in, void* const* out, const int64_t* n, int32_t P,
                        int sms, F launch)
{
    const uint32_t full = static_cast<uint32_t>(kBlocksPerSm) * sms;
    int32_t j = 0;
    while (j < P) {
        Table t;
        int64_t total = 0;
        int32_t k = j;
        t.count = 0;
        for (; k < P && t.count < kTable; ++k) {
            if (n[k] == 0) continue;
            t.in[t.count] = in[k];
            t.out[t.count] = out ? out[k] : nullptr;
            t.n[t.count++] = n[k];
            total += n[k];
        }
        j = k;
        if (t.count == 0) break;
        t.chunk_bits = kMaxChunkBits;
        while (t.chunk_bits > kMinChunkBits && (total >> t.chunk_bits) < 4 * full) --t.chunk_bits;
        int64_t chunks = 0;
        for (int32_t i = 0; i < t.count; ++i) {
            t.begin[i] = static_cast<uint32_t>(chunks);
            chunks += (t.n[i] + (int64_t{1} << t.chunk_bits) - 1) >> t.chunk_bits;
            if (chunks > UINT32_MAX / 2) return FORGE_ERR_INVALID_ARG;
        }
        t.begin[t.count] = static_cast<uint32_t>(chunks);
        launch(t, static_cast<uint32_t>(chunks) < full ? static_cast<uint32_t>(chunks) : full);
        if (cudaGetLastError() != cudaSuccess) return FORGE_ERR_CUDA;
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
    const int64_t tables = (P + kTable - 1) / kTable;
    void* scratch = nullptr;
    if (scratch_alloc(&scratch, (tables * kBlocksPerSm * sms + 1) * sizeof(double), s) !=
        cudaSuccess) {
        cudaGetLastError();
        return FORGE_ERR_CUDA;
    }
    double* part = static_cast<double*>(scratch);
    int64_t parts = 0;
    st = for_tables(grads, nullptr, n, P, sms, [&](const Table& t, uint32_t blocks) {
        if (dtype == FORGE_F32)
            forge_square_sum_kernel<float><<<blocks, kThreads, 0, s>>>(t, part + parts);
        else
            forge_square_sum_kernel<__nv_bfloat16><<<blocks, kThreads, 0, s>>>(t, part + parts);
        parts += blocks;
    });
    if (st == FORGE_OK) {
        forge_norm_fold_kernel<<<1, kThreads, 0, s>>>(part, parts, norm);
        if (cudaGetLastError() != cudaSuccess) st = FORGE_ERR_CUDA;
    }
    if (scratch_free(scratch, s) != cudaSuccess && st == FORGE_OK) st = FORGE_ERR_CUDA;
    return st;
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
    if ((st = check_overlap(grads, size_of(dtype), out, size_of(out_dtype), n, P)) != FORGE_OK) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != FORGE_OK) return st;
    const void* one[] = {norm};
    if ((st = device_resident(one, 1)) != FORGE_OK) return st;
    if ((st = check_memory(grads, n, P, dtype)) != FORGE_OK) return st;
    if ((out != grads || out_dtype != dtype) && (st = check_memory(out, n, P, out_dtype)) != FORGE_OK)
        return st;
    if (!aligned(norm, 4)) return FORGE_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return for_tables(grads, out, n, P, sms, [&](const Table& t, uint32_t blocks) {
        if (dtype == FORGE_F32 && out_dtype == FORGE_F32)
            forge_clip_kernel<float, float><<<blocks, kThreads, 0, s>>>(t, norm, max_norm);
        else if (dtype == FORGE_F32)
            forge_clip_kernel<float, __nv_bfloat16><<<blocks, kThreads, 0, s>>>(t, norm, max_norm);
        else if (out_dtype == FORGE_F32)
            forge_clip_kernel<__nv_bfloat16, float><<<blocks, kThreads, 0, s>>>(t, norm, max_norm);
        else
            forge_clip_kernel<__nv_bfloat16, __nv_bfloat16>
                <<<blocks, kThreads, 0, s>>>(t, norm, max_norm);
    });
}
