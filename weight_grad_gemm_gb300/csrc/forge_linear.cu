// forge_linear.cu -- products of e4m3 codes that carry a scale for each block
// of 128: a linear layer's Y = A W, and its input gradient Y = A W^T, dense or
// by experts.
//
// With A [T, K] (a scale for each 128 entries of a row) and W (a scale for each
// 128 x 128 square),
//   Y[t][o] = sum over blocks b of 128 of K:  sA[t][b] sW[b][o / 128] P_b[t][o],
//   P_b[t][o] = sum over k in block b of A[t][k] W[k][o].
// The tensor core sums a block's products P_b in fp32 in tensor memory, and the
// epilogue warps add it, times its two scales, to the tile's sum in their
// registers (fp32): every block has its own scale, so no two blocks meet
// in one accumulator before they are scaled.  Two P_b alternate in tensor memory;
// while one is read the tensor core fills the other.
//
// The contraction runs over A's contiguous index, so A is K-major.  W [N, M]
// (d_in x d_out, row-major) is MN-major for Y = A W and K-major for A W^T: the
// same codes and scales serve both, because a square's scale does not depend
// on the direction.
//
// Two forms.  Many tokens: CTA pairs (tcgen05.mma.cta_group::2) on tiles of 256
// tokens x 256 outputs, persistent; tokens are the rows (lanes) of the accumulator.
// Few tokens: the product is turned round, 128 outputs are the rows and 16 to 128
// tokens the columns, so that the tensor core and the epilogue do no more than the
// tokens ask for while the weight streams; the CTAs of a cluster share a tile's
// contraction and add their sums through distributed shared memory, in rank order,
// so that all SMs read the weight however few its tiles are.  By experts, a tile
// lies within one expert's rows; rows of A behind the expert's end reach only rows or
// columns of the accumulator that are not stored.
//
// Measured (cuBLAS reaches 3.86 PFLOP/s with e4m3): 8192 x 14336 x 4096 400 us (2.40
// PFLOP/s; captured, the tensor core is busy 53% of the time), 8192 x 4096 x 4096 132
// (2.09), 32768 tokens by 8 experts of 14336 x 4096 1630 to 1750 from box to box (2.20 to
// 2.36).  What bounds them is the
// hand-over: a block's MMAs take 512 cycles, but from the last of them through the
// epilogue's wait, its four loads, the sums of the first two and back to the issuer takes
// some 1,100, so that with two slots a block comes every 820 to 870.  Without the
// sums it would be 308 us, with half the loads 326, without the scales' loads 361.
// Slower were: three slots of 160 columns (517 us), tiles of 128 columns, Y by TMA
// stores, scales through shared memory, packed pairs of sums, one lane's load and
// shuffles for the weight's scales (401 to 403).  Few tokens: 16 x 4096 x 14336 16.5 us
// (3.6 TB/s of the weight's 59 MB, and the start and end of two CTAs an SM; 13.1 where the
// weight is in L2), 128 x 14336 x 4096 22.8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "forge.h"
#include "forge_device.h"
#include "forge_kernel.cuh"
#include "forge_rows.cuh"

namespace forge {
namespace linear {

constexpr int kBlock = 128;       // entries under one scale, and k of a stage
constexpr int kThreads = 384;     // producer, two MMA issuers, one idle and eight epilogue warps
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kStageA = 128 * kBlock;  // 128 token rows
constexpr int kStageB = 128 * kBlock;  // 128 outputs
constexpr int kStageBytes = kStageA + kStageB;
constexpr int kSlots = 2;         // P_b in tensor memory
constexpr int kStoreBytes = 2048;  // 32 rows x 64 bytes of Y on their way out
constexpr int kMostSplit = 8;     // CTAs that share a tile's contraction
constexpr int kScaleRing = 4;     // chunks of four k-blocks' scales
constexpr int kBand = 8;          // token tiles of a band of the tile walk

// Tiles of the forms: tokens x outputs.
struct Many {
    static constexpr int rows = 256, cols = 256;
    static constexpr int stages = 6;
    static_assert(stages % kSlots == 0,
                  "a stage belongs to one issuer, which so waits for each of its rounds");
    static constexpr int warp_cols = cols / 2;
    static constexpr int tmem_cols = kSlots * cols;
    // registers a thread: 168 at launch, moved from the first warpgroup to the two
    // that hold the sums (3 x 168 = 56 + 2 x 224)
    static constexpr int few_regs = 56, many_regs = 224;
    static constexpr int bar_at = stages * kStageBytes;
    static constexpr int store_at = bar_at + 256;
    static constexpr int table_at = store_at + kEpiWarps * kStoreBytes;
    static constexpr int bytes(int E) { return table_at + (E > 0 ? 8 * (E + 1) : 0) + 1024; }
};
template <int NT>
struct Few {
    static constexpr int rows = NT, cols = 128;
    static constexpr int stages = NT <= 64 ? 4 : 6;
    static constexpr int slots = NT <= 64 ? 4 : 2;
    static constexpr int stage_bytes = kStageB + NT * kBlock;
    static constexpr int tmem_cols = slots * NT;
    static constexpr int ctas = NT <= 64 ? 2 : 1;  // an SM
    // producer, two MMA issuers, four or eight epilogue warps (`mine` tokens each), scales
    static constexpr int issuers = 2;
    static_assert(stages % issuers == 0 && slots % issuers == 0,
                  "a stage and a slot belong to one issuer, which so waits for each round");
    static constexpr int groups = NT <= 64 ? 1 : 2, mine = NT / groups;
    static constexpr int epi_warp0 = 1 + issuers;
    static constexpr int threads = 32 * (epi_warp0 + 4 * groups + 1);
    static constexpr int pitch = 132;              // floats between the tokens of a share
    static constexpr int scale_at = stages * stage_bytes;
    static constexpr int bar_at = scale_at + kScaleRing * 4 * NT * 4;
    static constexpr int table_at = bar_at + 256;
    static constexpr int bytes(int E) { return table_at + (E > 0 ? 8 * (E + 1) : 0) + 1024; }
    static_assert(NT * pitch * 4 <= scale_at, "a share fits the ring");
    static_assert(ctas * (bytes(kMaxExperts) + 1024) <= 228 * 1024, "the CTAs of an SM");
};

struct LParams {
    int64_t T, K, O;       // tokens, contraction, outputs
    const float *sA, *sW;
    int64_t sa_ld;             // between rows of A's scales
    int64_t sw_k, sw_o, sw_e;  // strides of W's scales along K, outputs, experts
    void* Y;
    int32_t f32, vec;      // Y's type; rows of Y take 16-byte stores
    int32_t sa_vec;        // rows of A's scales take 16-byte loads
    int32_t E;             // experts, 0: dense
    const int32_t* offsets;
    int32_t tiles_o, nk;
    Params w;              // timeout_ns and status for the bounded waits
};

struct Tile {
    int32_t expert, t0, t_end, o0;
};

// Tile t: dense calls walk bands of kBand token tiles, tokens fastest, so that
// the CTAs at work share both operands' blocks in L2; by experts, one expert's
// tiles after another's, each walked the same way.
template <typename F, bool GROUPED>
__device__ __forceinline__ Tile tile_of(int32_t t, const LParams& p, const int32_t* offs,
                                        const int32_t* begin)
{
    Tile r;
    int32_t lo = 0, hi = static_cast<int32_t>(p.T);
    r.expert = 0;
    if constexpr (GROUPED) {
        int a = 0, b = p.E;  // begin[a] <= t < begin[b]
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (begin[m] <= t)
                a = m;
            else
                b = m;
        }
        r.expert = a;
        t -= begin[a];
        lo = offs[a];
        hi = offs[a + 1];
    }
    const int32_t tiles_t = (hi - lo + F::rows - 1) / F::rows;
    const int32_t band = t / (kBand * p.tiles_o), in = t - band * kBand * p.tiles_o;
    const int32_t left = tiles_t - band * kBand, high = left < kBand ? left : kBand;
    r.t0 = lo + (band * kBand + in % high) * F::rows;
    r.t_end = hi;
    r.o0 = in / high * F::cols;
    return r;
}

// wait_bounded for waits that mostly fail at first: a block's hand-over between
// the tensor core and the epilogue comes every 0.4 us, and reading the global
// timer before the second try alone takes longer than that.
__device__ __forceinline__ bool wait_often(uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag, const Params& p)
{
    const uint32_t a = ptx::smem_addr(bar);
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (ptx::mbar_try_wait(a, parity)) return true;
    return wait_bounded(bar, parity, abort_flag, p);
}

// Offsets into shared memory, checked, and the first tile of each expert;
// false (and the status word set) where the offsets are not an ascending list
// within the T rows.  All threads of the CTA.
template <typename F>
__device__ bool group_table(const LParams& p, int32_t* offs, int32_t* begin)
{
    int bad = 0;
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
        const int32_t v = p.offsets[e], before = e > 0 ? p.offsets[e - 1] : 0;
        offs[e] = v;
        bad |= v < before || v > p.T;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) *reinterpret_cast<volatile int*>(p.w.status) = kDevInvalidArg;
        return false;
    }
    if (threadIdx.x < 32) {
        int32_t sum = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            int32_t n = 0;
            if (e < p.E)
                n = (offs[e + 1] - offs[e] + F::rows - 1) / F::rows * p.tiles_o;
            int32_t up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
                if (static_cast<int>(threadIdx.x) >= o) up += v;
            }
            if (e < p.E) begin[e] = sum + up - n;
            sum += __shfl_sync(0xffffffffu, up, 31);
        }
        if (threadIdx.x == 0) begin[p.E] = sum;
    }
    __syncthreads();
    return true;
}

// Loads that stay where they are written: the compiler moves an ordinary load
// down to its first use, and the wait for it with it.  Plain, not read-only ones: scales whose
// rows are copied in front are still being written when this kernel starts.
__device__ __forceinline__ float load_early(const float* p)
{
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float4 load4_early(const float* p)
{
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// N outputs of one row, in registers, from column c on.
template <int N>
__device__ __forceinline__ void store_row(const LParams& p, int64_t row, int64_t c,
                                          const float (&v)[N])
{
    const int64_t at = row * p.O + c;
    if (p.vec && c + N <= p.O) {
        store_as(p.Y, p.f32, at, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float one[1] = {v[j]};
            if (c + j < p.O) store_as(p.Y, p.f32, at + j, one);
        }
    }
}

// A warp's 32 rows x 128 outputs, a lane a row, from row r0 and column c0 on: through
// shared memory, 64 bytes of a row at a time, so that four lanes write a row's
// neighbouring 16 bytes (a lane writing its own row instead, 16 bytes an
// instruction, took 7,000 cycles a tile).  Rows of Y that no 16-byte store can address take
// a lane an output (3001 x 5003 bf16 by 2777: 84 us, a lane a row 207).
__device__ __forceinline__ void store_tile(const LParams& p, uint8_t* stage, int64_t r0,
                                           int64_t r_end, int64_t c0, const float (&acc)[128],
                                           int lane)
{
    // the 16-byte unit u of row r lies at place u ^ (r / 2 % 4): no bank conflicts
    uint4* mine = reinterpret_cast<uint4*>(stage) + 4 * lane;
    const int turn = lane >> 1 & 3;
    const int from = lane & 3, down = lane >> 2;
    auto out = [&](auto one, int64_t c) {
        using U = decltype(one);  // an output's bits
        constexpr int kUnit = 16 / sizeof(U), kRow = 64 / sizeof(U);
        U* y = static_cast<U*>(p.Y);
        __syncwarp();
        if (p.vec) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 8 * k + down;
                const uint4 v = reinterpret_cast<const uint4*>(stage)[4 * r + (from ^ (r >> 1 & 3))];
                const int64_t col = c + from * kUnit;
                if (r0 + r < r_end && col < p.O)
                    *reinterpret_cast<uint4*>(y + (r0 + r) * p.O + col) = v;
            }
        } else {
            // a lane an output, 32 / kRow rows at once
            const int in = lane % kRow;
#pragma unroll 8
            for (int r = lane / kRow; r < 32; r += 32 / kRow) {
                const U v = reinterpret_cast<const U*>(
                    stage)[(4 * r + (in / kUnit ^ (r >> 1 & 3))) * kUnit + in % kUnit];
                if (r0 + r < r_end && c + in < p.O) y[(r0 + r) * p.O + c + in] = v;
            }
        }
        __syncwarp();
    };
    if (p.f32) {
#pragma unroll
        for (int j = 0; j < 128; j += 16) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                mine[u ^ turn] = make_uint4(
                    __float_as_uint(acc[j + 4 * u]), __float_as_uint(acc[j + 4 * u + 1]),
                    __float_as_uint(acc[j + 4 * u + 2]), __float_as_uint(acc[j + 4 * u + 3]));
            out(uint32_t{}, c0 + j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 128; j += 32) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float* a = acc + j + 8 * u;
                mine[u ^ turn] = make_uint4(bf16x2(a[0], a[1]), bf16x2(a[2], a[3]),
                                            bf16x2(a[4], a[5]), bf16x2(a[6], a[7]));
            }
            out(uint16_t{}, c0 + j);
        }
    }
}

template <bool W_MN, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1)
    forge_linear_kernel(const __grid_constant__ CUtensorMap tmA,  // A [T, K]
                        const __grid_constant__ CUtensorMap tmW,  // W [E][N][M]
                        const LParams p)
{
    using F = Many;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::bar_at);
    uint64_t* empty = full + F::stages;
    uint64_t* tfull = empty + F::stages;
    uint64_t* tempty = tfull + kSlots;
    uint64_t* drain = tempty + kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + kSlots);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* offs = reinterpret_cast<int32_t*>(smem + F::table_at);
    int32_t* begin = offs + p.E + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;  // of the pair: issues its MMAs
    if constexpr (GROUPED) {
        // every CTA of a cluster reads the same offsets and leaves alike
        if (!group_table<F>(p, offs, begin)) return await_prerequisites();
    }
    int32_t total;
    if constexpr (GROUPED) {
        total = begin[p.E];
    } else {
        total = static_cast<int32_t>((p.T + F::rows - 1) / F::rows) * p.tiles_o;
    }
    const int32_t first = static_cast<int32_t>(blockIdx.x >> 1);
    const int32_t step = static_cast<int32_t>(gridDim.x >> 1);
    if (first >= total) return await_prerequisites();  // (the whole pair)

    if (threadIdx.x == 0) {
        for (int s = 0; s < F::stages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kSlots; ++b) {
            ptx::mbar_init(&drain[b], 1);
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 2 * kEpiWarps);
        }
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmW);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(tmem_slot, F::tmem_cols);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    await_prerequisites();  // rows copied in front of this launch

    if (warp < kEpiWarp0) {
        ptx::registers_down<F::few_regs>();
        if (warp == 0) {
            // ---------------------------------------------------- TMA producer
            if (lane == 0) {
                const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(&full[0]), 0);
                int s = 0;
                uint32_t ph = 0;
                uint32_t issued_mask = 0, last_parity = 0;
                bool ok = true;
                for (int32_t t = first; ok && t < total; t += step) {
                    const Tile tl = tile_of<F, GROUPED>(t, p, offs, begin);
                    const int32_t ta = tl.t0 + static_cast<int32_t>(rank) * 128;
                    const int32_t ob = tl.o0 + static_cast<int32_t>(rank) * 128;
                    for (int32_t kb = 0; kb < p.nk; ++kb) {
                        if (!wait_often(&empty[s], ph ^ 1u, abort_flag, p.w)) {
                            ok = false;
                            break;
                        }
                        uint8_t* sa = smem + s * kStageBytes;
                        const int32_t k = kb * kBlock;
                        const int32_t wx = W_MN ? ob : k, wy = W_MN ? k : ob;
                        if (leader) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                        const uint32_t bar = full0 + s * 8;
                        ptx::tma_load_2d_pair(sa, &tmA, bar, k, ta);
                        ptx::tma_load_3d_pair(sa + kStageA, &tmW, bar, wx, wy, tl.expert);
                        issued_mask |= 1u << s;
                        last_parity = (last_parity & ~(1u << s)) | (ph << s);
                        if (++s == F::stages) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (!ok && leader) {
                    // wait (bounded) for the copies still in flight
                    const uint64_t tw = ptx::globaltimer_ns();
                    for (int q = 0; q < F::stages; ++q) {
                        if (!(issued_mask & (1u << q))) continue;
                        const uint32_t a = ptx::smem_addr(&full[q]);
                        while (!ptx::mbar_try_wait(a, (last_parity >> q) & 1u)) {
                            if (static_cast<int64_t>(ptx::globaltimer_ns() - tw) > p.w.timeout_ns)
                                break;
                        }
                    }
                }
            }
        } else if (warp <= kSlots) {
            // ---------------------------------------------------- MMA issuers (lane 0)
            // Warp 1 + b fills slot b with every other k-block's products: one thread's
            // waits, instructions and commits take 1,200 cycles a k-block, more than
            // the tensor core's 512.
            if (leader && lane == 0) {
                constexpr uint32_t idesc = ptx::make_idesc(0, 0, false, W_MN, F::rows, F::cols);
                // K-major: a step of 32 k is 32 bytes inside the swizzle row, groups of eight
                // rows lie 1024 bytes apart.  MN-major: 32 rows of 128 bytes.  (In 16-byte
                // units: an address below 256 KB never carries out of its field.)
                constexpr uint64_t kStepA = 32 >> 4, kStepB = (W_MN ? 32 * 128 : 32) >> 4;
                const uint32_t ring = ptx::smem_addr(smem);
                const uint64_t a_desc = ptx::smem_desc_sw128(ring, 16, 1024);
                const uint64_t b_desc =
                    ptx::smem_desc_sw128(ring + kStageA, W_MN ? kStageB : 16, 1024);
                const int b = warp - 1;
                const uint32_t d_tmem = tmem_base + b * F::cols;
                const int64_t blocks = int64_t{p.nk} * ((total - first + step - 1) / step);
                int s = b;
                uint32_t ph = 0, turn = 1;
                bool ok = true;
                bool issued_any = false;
                for (int64_t ct = b; ct < blocks; ct += kSlots, turn ^= 1u) {
                    // (the operands are there long before the place for the sums is:
                    // nothing but the instructions themselves follows the second wait)
                    ok = wait_often(&full[s], ph, abort_flag, p.w) &&
                         wait_often(&tempty[b], turn, abort_flag, p.w);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint64_t ad = a_desc + s * (kStageBytes >> 4);
                    const uint64_t bd = b_desc + s * (kStageBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        ptx::umma_f8_pair(d_tmem, ad + ks * kStepA, bd + ks * kStepB, idesc,
                                          ks != 0 ? 1u : 0u);
                    }
                    issued_any = true;
                    ptx::umma_commit_pair(&tfull[b], 0x3);
                    ptx::umma_commit_pair(&empty[s], 0x3);
                    s += kSlots;
                    if (s >= F::stages) {
                        s -= F::stages;
                        ph ^= 1u;
                    }
                }
                if (!ok && issued_any) {
                    ptx::umma_commit_pair(&drain[b], 0x1);
                    const uint32_t a = ptx::smem_addr(&drain[b]);
                    const uint64_t tw = ptx::globaltimer_ns();
                    while (!ptx::mbar_try_wait(a, 0)) {
                        if (static_cast<int64_t>(ptx::globaltimer_ns() - tw) > p.w.timeout_ns) break;
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        ptx::registers_up<F::many_regs>();
        // Warp (q, g): TMEM lanes 32 q .. (tokens) x columns C g ..; a lane owns one
        // token row.
        constexpr int C = F::warp_cols;
        const int q = warp & 3;
        const int g = (warp - kEpiWarp0) >> 2;
        const uint32_t tempty0 = ptx::mapa_shared(ptx::smem_addr(&tempty[0]), 0);
        const int32_t my_row = static_cast<int32_t>(rank) * 128 + 32 * q + lane;
        const int32_t my_col = C * g;
        const uint32_t my_tmem = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + C * g;
        uint32_t ct = 0;
        bool ok = true;
        int64_t row, row_end, c0;
        const float *sa, *sw;
        float na[4], nw[4];
        // Scales four blocks ahead (their product is taken when they are needed, so that
        // nothing waits for the loads), a tile's first before the last one's stores.
        auto load_scales = [&](int32_t kb) {
            if (p.sa_vec) {
                const float4 v = load4_early(sa + kb);
                na[0] = v.x;
                na[1] = v.y;
                na[2] = v.z;
                na[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    na[i] = load_early(sa + min(kb + i, p.nk - 1));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                nw[i] = load_early(sw + min(kb + i, p.nk - 1) * p.sw_k);
        };
        auto begin_tile = [&](int32_t t) {
            const Tile tl = tile_of<F, GROUPED>(t, p, offs, begin);
            row = int64_t{tl.t0} + my_row;
            row_end = tl.t_end;
            c0 = int64_t{tl.o0} + my_col;
            // (scales of rows and columns outside the call are read from its first)
            sa = p.sA + (row < row_end ? row : 0) * p.sa_ld;
            sw = p.sW + tl.expert * p.sw_e + (c0 < p.O ? c0 / kBlock : 0) * p.sw_o;
            load_scales(0);
        };
        begin_tile(first);
        for (int32_t t = first; ok && t < total; t += step) {
            float acc[C];
#pragma unroll
            for (int j = 0; j < C; ++j) acc[j] = 0.0f;
            for (int32_t k0 = 0; ok && k0 < p.nk; k0 += 4) {
                float now[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = na[i] * nw[i];
                if (k0 + 4 < p.nk) load_scales(k0 + 4);
                const int n = min(4, p.nk - k0);
#pragma unroll 1
                for (int i = 0; i < n; ++i, ++ct) {
                    const float f = i < 2 ? (i == 0 ? now[0] : now[1]) : (i == 2 ? now[2] : now[3]);
                    const uint32_t b = ct % kSlots;
                    ok = wait_often(&tfull[b], ct / kSlots & 1u, abort_flag, p.w);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t tcol = my_tmem + b * F::cols;
                    uint32_t r[2][32];
                    auto load = [&](int c) {
                        ptx::tmem_ld_32x32b_x32(tcol + 32 * c, r[c & 1]);
                    };
                    auto add = [&](int c) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            acc[32 * c + j] =
                                fmaf(__uint_as_float(r[c & 1][j]), f, acc[32 * c + j]);
                    };
                    auto wait = [&]() {
                        ptx::tmem_ld_wait_for(r[0]);
                        ptx::tmem_ld_wait_for(r[1]);
                    };
                    // two loads at a time, and as little as can be before the last is in
                    // (one at a time: 450 instead of 400 us at 8192 x 14336 x 4096)
                    load(0);
                    load(1);
                    wait();
                    add(0);
                    load(2);
                    add(1);
                    load(3);
                    wait();
                    // this P_b is read: its issuer may fill the slot again
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader)
                            ptx::mbar_arrive(&tempty[b]);
                        else
                            ptx::mbar_arrive_cluster_unordered(tempty0 + 8 * b);
                    }
                    add(2);
                    add(3);
                }
            }
            if (!ok) break;
            const int64_t r0 = row - lane, r_end = row_end, c = c0;
            if (t + step < total) begin_tile(t + step);
            store_tile(p, smem + F::store_at + (warp - kEpiWarp0) * kStoreBytes, r0, r_end, c, acc,
                       lane);
        }
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();  // no CTA leaves while the other may still signal it
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, F::tmem_cols);
    }
}

// The form for few tokens: a CTA has one tile of 128 outputs x NT tokens and blocks
// k_lo to k_hi of its contraction; the CTAs of a cluster (along y) have the others.
template <int NT, bool W_MN, bool GROUPED>
__global__ void __launch_bounds__(Few<NT>::threads, Few<NT>::ctas)
    forge_linear_few_kernel(const __grid_constant__ CUtensorMap tmA,  // A [T, K], NT rows a box
                            const __grid_constant__ CUtensorMap tmW,  // W [E][N][M]
                            const LParams p)
{
    using F = Few<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::bar_at);
    uint64_t* empty = full + F::stages;
    uint64_t* tfull = empty + F::stages;
    uint64_t* tempty = tfull + F::slots;
    uint64_t* sfull = tempty + F::slots;
    uint64_t* sempty = sfull + kScaleRing;
    uint64_t* drain = sempty + kScaleRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + F::issuers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* scales = reinterpret_cast<float*>(smem + F::scale_at);  // [ring][4][NT]
    int32_t* offs = reinterpret_cast<int32_t*>(smem + F::table_at);
    int32_t* begin = offs + p.E + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const uint32_t split = gridDim.y;
    int32_t total;
    if constexpr (GROUPED) {
        // every CTA of a cluster reads the same offsets and leaves alike
        if (!group_table<F>(p, offs, begin)) return await_prerequisites();
        total = begin[p.E];
    } else {
        total = static_cast<int32_t>((p.T + F::rows - 1) / F::rows) * p.tiles_o;
    }
    if (static_cast<int32_t>(blockIdx.x) >= total)
        return await_prerequisites();  // (the whole cluster)
    const Tile tl = tile_of<F, GROUPED>(static_cast<int32_t>(blockIdx.x), p, offs, begin);
    const int32_t k_lo = static_cast<int32_t>(int64_t{p.nk} * rank / split);
    const int32_t n = static_cast<int32_t>(int64_t{p.nk} * (rank + 1) / split) - k_lo;

    auto load = [&](int32_t i) {
        const int s = i % F::stages;
        ptx::mbar_arrive_expect_tx(&full[s], F::stage_bytes);
        uint8_t* sw = smem + s * F::stage_bytes;
        const int32_t k = (k_lo + i) * kBlock;
        ptx::tma_load_3d(sw, &tmW, &full[s], W_MN ? tl.o0 : k, W_MN ? k : tl.o0, tl.expert);
        ptx::tma_load_2d(sw + kStageB, &tmA, &full[s], k, tl.t0);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::stages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < F::slots; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], 4 * F::groups);
        }
        for (int c = 0; c < kScaleRing; ++c) {
            ptx::mbar_init(&sfull[c], 1);
            ptx::mbar_init(&sempty[c], 4 * F::groups);
        }
        for (int w = 0; w < F::issuers; ++w) ptx::mbar_init(&drain[w], 1);
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
        // the first stages are on their way while the other warps set up
        await_prerequisites();  // rows copied in front of this launch
        for (int32_t i = 0; i < F::stages && i < n; ++i) load(i);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, F::tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int64_t o = int64_t{tl.o0} + 32 * (warp & 3) + lane;  // an epilogue lane's output
    constexpr int C = F::mine;  // tokens of an epilogue warp, from c0 on
    const int c0 = F::groups == 1 ? 0 : (warp - F::epi_warp0) / 4 * C;
    float acc[C];

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            bool ok = true;
            int32_t i = min(F::stages, n);
            for (; i < n; ++i) {
                const int s = i % F::stages;
                ok = wait_often(&empty[s], (i / F::stages & 1u) ^ 1u, abort_flag, p.w);
                if (!ok) break;
                load(i);
            }
            if (!ok) {
                // wait (bounded) for the copies still in flight: the last ones issued
                const uint64_t tw = ptx::globaltimer_ns();
                for (int32_t c = max(0, i - F::stages); c < i; ++c) {
                    const uint32_t a = ptx::smem_addr(&full[c % F::stages]);
                    while (!ptx::mbar_try_wait(a, c / F::stages & 1u)) {
                        if (static_cast<int64_t>(ptx::globaltimer_ns() - tw) > p.w.timeout_ns)
                            break;
                    }
                }
            }
        }
    } else if (warp <= F::issuers) {
        // ---------------------------------------------------- MMA issuers (lane 0)
        // Every other block each, as the pairs' (128 tokens of 14336 x 4096: 22.8 us, by one
        // issuer 25.0; 16 of 4096 x 14336 where L2 holds the weight 13.0 and 16.4, and 16.4 by
        // either where it comes from memory).
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::make_idesc(0, 0, W_MN, false, 128, NT);
            constexpr uint64_t kStepW = (W_MN ? 32 * 128 : 32) >> 4, kStepA = 32 >> 4;
            const uint32_t ring = ptx::smem_addr(smem);
            const uint64_t w_desc = ptx::smem_desc_sw128(ring, W_MN ? kStageB : 16, 1024);
            const uint64_t a_desc = ptx::smem_desc_sw128(ring + kStageB, 16, 1024);
            bool ok = true;
            bool issued_any = false;
            for (int32_t i = warp - 1; i < n; i += F::issuers) {
                const int s = i % F::stages, b = i % F::slots;
                ok = wait_often(&full[s], i / F::stages & 1u, abort_flag, p.w) &&
                     wait_often(&tempty[b], (i / F::slots & 1u) ^ 1u, abort_flag, p.w);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t wd = w_desc + s * (F::stage_bytes >> 4);
                const uint64_t ad = a_desc + s * (F::stage_bytes >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    ptx::umma_f8(tmem_base + b * NT, wd + ks * kStepW, ad + ks * kStepA, idesc,
                                 ks != 0 ? 1u : 0u);
                issued_any = true;
                ptx::umma_commit(&tfull[b]);
                if (i + F::stages < n) ptx::umma_commit(&empty[s]);  // (a stage that is used again)
            }
            if (!ok && issued_any) {
                ptx::umma_commit(&drain[warp - 1]);
                const uint32_t a = ptx::smem_addr(&drain[warp - 1]);
                const uint64_t tw = ptx::globaltimer_ns();
                while (!ptx::mbar_try_wait(a, 0)) {
                    if (static_cast<int64_t>(ptx::globaltimer_ns() - tw) > p.w.timeout_ns) break;
                }
            }
        }
    } else if (warp < F::epi_warp0 + 4 * F::groups) {
        // ---------------------------------------------------- epilogue
        // Warp (q, g): TMEM lanes 32 q .. (outputs) x columns C g ..; a lane owns one output's
        // C tokens.
        const uint32_t mine = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c0;
#pragma unroll
        for (int j = 0; j < C; ++j) acc[j] = 0.0f;
        bool ok = true;
#pragma unroll 1
        for (int32_t i = 0; i < n; ++i) {
            const int b = i % F::slots, c = i / 4 % kScaleRing;
            if (i % 4 == 0) ok = wait_often(&sfull[c], i / 4 / kScaleRing & 1u, abort_flag, p.w);
            ok = ok && wait_often(&tfull[b], i / F::slots & 1u, abort_flag, p.w);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const float4* f = reinterpret_cast<const float4*>(scales + (c * 4 + i % 4) * NT + c0);
            const uint32_t from = mine + b * NT;
            auto add = [&](const auto& r, int j0, int N) {
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    const float4 q = f[(j0 + j) / 4];
                    acc[j0 + j] = fmaf(__uint_as_float(r[j]), q.x, acc[j0 + j]);
                    acc[j0 + j + 1] = fmaf(__uint_as_float(r[j + 1]), q.y, acc[j0 + j + 1]);
                    acc[j0 + j + 2] = fmaf(__uint_as_float(r[j + 2]), q.z, acc[j0 + j + 2]);
                    acc[j0 + j + 3] = fmaf(__uint_as_float(r[j + 3]), q.w, acc[j0 + j + 3]);
                }
            };
            auto release = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&tempty[b]);
            };
            if constexpr (NT == 16) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(from, r);
                ptx::tmem_ld_wait_for(r);
                release();
                add(r, 0, 16);
            } else {
#pragma unroll
                for (int h = 0; h < C / 32; ++h) {
                    uint32_t r[32];
                    ptx::tmem_ld_32x32b_x32(from + 32 * h, r);
                    ptx::tmem_ld_wait_for(r);
                    if (h == C / 32 - 1) release();
                    add(r, 32 * h, 32);
                }
            }
            if (i % 4 == 3) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sempty[c]);
            }
        }
        if (split == 1) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float one[1] = {acc[j]};
                if (ok && tl.t0 + c0 + j < tl.t_end && o < p.O)
                    store_as(p.Y, p.f32, (int64_t{tl.t0} + c0 + j) * p.O + o, one);
            }
        } else {
            // this CTA's share into its ring: the last slot that it waited for was the last
            // to be filled, so every copy into the ring and every MMA on it is complete
            float* share = reinterpret_cast<float*>(smem) + 32 * (warp & 3) + lane;
            if (ok) {
#pragma unroll
                for (int j = 0; j < C; ++j)
                    if (tl.t0 + c0 + j < tl.t_end) share[(c0 + j) * F::pitch] = acc[j];
            }
        }
    } else {
        // ---------------------------------------------------- scales
        // Of four blocks at a time, for each token the product of its scale and the
        // weight's, up to four chunks ahead.
        const float* sw = p.sW + tl.expert * p.sw_e + tl.o0 / kBlock * p.sw_o;
        const int32_t last = k_lo + n - 1;
        for (int32_t c = 0; c < (n + 3) / 4; ++c) {
            const int32_t kb = k_lo + 4 * c;
            float w[4], a[(NT + 31) / 32][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(sw + min(kb + i, last) * p.sw_k);
#pragma unroll
            for (int h = 0; h < (NT + 31) / 32; ++h) {
                // (tokens outside the tile take the call's first scales)
                const int64_t row = int64_t{tl.t0} + 32 * h + lane;
                const float* at = p.sA + (row < tl.t_end ? row : 0) * p.sa_ld;
                if (p.sa_vec && kb % 4 == 0) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(at + kb));
                    a[h][0] = v.x;
                    a[h][1] = v.y;
                    a[h][2] = v.z;
                    a[h][3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[h][i] = __ldg(at + min(kb + i, last));
                }
            }
            const int r = c % kScaleRing;
            const bool ok = wait_often(&sempty[r], (c / kScaleRing & 1u) ^ 1u, abort_flag, p.w);
            if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
            for (int h = 0; h < (NT + 31) / 32; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (32 * h + lane < NT) scales[(r * 4 + i) * NT + 32 * h + lane] = a[h][i] * w[i];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sfull[r]);
        }
    }

    __syncthreads();
    if (split > 1) {
        ptx::cluster_sync();  // every share of the tile is written
        if (*abort_flag == 0) {
            const int32_t tokens = min(NT, tl.t_end - tl.t0);
            const int32_t units = tokens * (F::cols / 4);  // of four outputs
            const uint32_t ring = ptx::smem_addr(smem);
            for (int32_t u = static_cast<int32_t>(rank) * F::threads + threadIdx.x; u < units;
                 u += static_cast<int32_t>(split) * F::threads) {
                const int32_t j = u / (F::cols / 4), c = u % (F::cols / 4) * 4;
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (uint32_t k = 0; k < split; ++k) {
                    const uint32_t at = ring + (j * F::pitch + c) * 4;
                    const float4 x = ptx::ld_cluster_f4(ptx::mapa_shared(at, k));
                    v[0] += x.x;
                    v[1] += x.y;
                    v[2] += x.z;
                    v[3] += x.w;
                }
                if (tl.o0 + c < p.O) store_row(p, int64_t{tl.t0} + j, int64_t{tl.o0} + c, v);
            }
        }
    }
    ptx::tc_fence_before();
    if (split > 1)
        ptx::cluster_sync();  // no CTA leaves while another may still read its share
    else
        __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, F::tmem_cols);
    }
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Launch {
    const CUtensorMap &a, &w;
    const LParams& p;
    int split;    // few tokens: CTAs that share a tile's contraction
    bool staged;  // behind a copy of rows: may start before that ends
    cudaStream_t stream;
};

// KERN, of the form F.  Pairs: as many as can be resident at once; else a cluster of
// `split` CTAs for each tile.
template <typename F, bool GROUPED, auto KERN>
cudaError_t launch(const Launch& l)
{
    constexpr bool pairs = std::is_same<F, Many>::value;
    constexpr int threads = [] {
        if constexpr (pairs)
            return kThreads;
        else
            return F::threads;
    }();
    auto kern = KERN;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    constexpr int most = F::bytes(GROUPED ? kMaxExperts : 0);
    static_assert(most <= 227 * 1024, "ring and table within one CTA's shared memory");
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pairs ? 2 : 1;
    attr[0].val.clusterDim.y = pairs ? 1 : l.split;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static int ready[64] = {0};  // per device (and kernel): resident pairs, or 1
    int& mc = ready[dev & 63];
    if (__atomic_load_n(&mc, __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        int n = 1;
        if (pairs) {
            cfg.gridDim = dim3(2);
            cfg.dynamicSmemBytes = most;
            if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
        }
        __atomic_store_n(&mc, n, __ATOMIC_RELEASE);
    }
    // by experts the tiles are known on the device only: at most one more a
    // column of tiles for each expert than the rows alone would make
    const int64_t rows = (l.p.T + F::rows - 1) / F::rows;
    const int64_t extra = GROUPED ? (l.p.E < l.p.T ? l.p.E : l.p.T) : 0;
    const int64_t total = (rows + extra) * l.p.tiles_o;
    if (total > INT32_MAX / 16) return cudaErrorInvalidValue;
    if (pairs)
        cfg.gridDim = dim3(static_cast<unsigned>(2 * (total < mc ? total : mc)));
    else
        cfg.gridDim = dim3(static_cast<unsigned>(total), static_cast<unsigned>(l.split));
    cfg.dynamicSmemBytes = static_cast<size_t>(F::bytes(GROUPED ? l.p.E : 0));
    cfg.stream = l.stream;
    cfg.numAttrs = l.staged ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, l.a, l.w, l.p);
}

template <bool W_MN, bool GROUPED>
cudaError_t launch_form(int tokens, const Launch& l)
{
    switch (tokens) {
    case 16: return launch<Few<16>, GROUPED, forge_linear_few_kernel<16, W_MN, GROUPED>>(l);
    case 32: return launch<Few<32>, GROUPED, forge_linear_few_kernel<32, W_MN, GROUPED>>(l);
    case 64: return launch<Few<64>, GROUPED, forge_linear_few_kernel<64, W_MN, GROUPED>>(l);
    case 128: return launch<Few<128>, GROUPED, forge_linear_few_kernel<128, W_MN, GROUPED>>(l);
    default: return launch<Many, GROUPED, forge_linear_kernel<W_MN, GROUPED>>(l);
    }
}

// Clusters of `split` CTAs, one CTA an SM, that are resident at once: GPCs hold whole
// clusters (of 152 CTAs in clusters of 2 all are, in clusters of 8 120).
int resident(int dev, int split, int sms)
{
    static int known[64][kMostSplit + 1];  // per device
    int& n = known[dev & 63][split];
    int got = __atomic_load_n(&n, __ATOMIC_ACQUIRE);
    if (got > 0) return got;
    using F = Few<128>;
    auto kern = forge_linear_few_kernel<128, false, false>;
    static_assert(F::ctas == 1, "one CTA an SM");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = split;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, split);
    cfg.blockDim = dim3(F::threads);
    cfg.dynamicSmemBytes = F::bytes(kMaxExperts);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             F::bytes(kMaxExperts)) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&got, kern, &cfg) != cudaSuccess || got < 1) {
        cudaGetLastError();
        return sms / split;  // (an estimate; the launch itself reports what is wrong)
    }
    __atomic_store_n(&n, got, __ATOMIC_RELEASE);
    return got;
}

// The tokens of a tile (256: pairs), and the CTAs that share its contraction: the form and
// split that take the least time by what was measured.  Pairs: 0.46 us a block and 2.5 a
// tile, turn by turn, 5.7 once, and 2.5 where the scales' rows are copied first.  Few
// tokens, a turn of the resident clusters: 0.46 us a block (128 tokens) and 18 blocks' time
// for a CTA's start and end, 6 where two CTAs an SM overlap theirs; the joining one block and
// more with its bytes.  (128 tokens, 5776 x 6048: by two CTAs a tile 20.7 us, by three,
// not all of them resident, 30.3, by pairs 31.7; 4096 x 14336: by pairs 23.1, by one CTA
// a tile 23.0.)
struct Choice {
    int tokens, split;
};
Choice choose(const LParams& p, int sms)
{
    const char* env = std::getenv("FORGE_LINEAR_KERNEL");
    const bool pair = env && std::strcmp(env, "pair") == 0;
    const bool few = env && std::strncmp(env, "few", 3) == 0;
    if (pair) return {256, 1};
    const int64_t experts = p.E > 0 ? (p.E < p.T ? p.E : p.T) : 1;
    const int64_t each = (p.T + experts - 1) / experts;  // tokens of an expert
    Choice c{each <= 16 ? 16 : (each <= 32 ? 32 : (each <= 64 ? 64 : 128)), 1};
    if (few && env[3]) {
        c.split = std::atoi(env + 3);
        c.split = c.split < 1 ? 1 : (c.split > kMostSplit ? kMostSplit : c.split);
        if (c.split > p.nk) c.split = p.nk;
        return c;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return {256, 1};  // (the launch reports it)
    const bool two = c.tokens <= 64;  // CTAs an SM
    const int64_t tiles = (each + c.tokens - 1) / c.tokens * experts * ((p.O + 127) / 128);
    int64_t best = INT64_MAX;
    for (int s = 1; s <= kMostSplit && s <= p.nk; ++s) {
        const int64_t at_once = int64_t{resident(dev, s, sms)} * (two ? 2 : 1);
        const int64_t cost =
            (tiles + at_once - 1) / at_once * ((p.nk + s - 1) / s + (two ? 6 : 18)) +
            (s > 1 ? 1 + s * c.tokens / 512 : 0);
        if (cost < best) {
            best = cost;
            c.split = s;
        }
    }
    if (few || two) return c;
    const int64_t pairs = (each + 255) / 256 * experts * ((p.O + 255) / 256);
    const int64_t turns = (pairs + sms / 2 - 1) / (sms / 2);
    const int64_t once = p.sa_vec ? 570 : 820;
    return once + turns * (250 + 46 * int64_t{p.nk}) <= 46 * best ? Choice{256, 1} : c;
}

// Rows that TMA, or a 16-byte load, cannot address, copied to 16-byte boundaries: up to
// three arrays in one launch, behind which the product's starts early (4099 x 4100 codes,
// their scales and 4096 x 4100 codes: 102 us with the product, by a launch each 112; 16
// tokens of 4099 to 4101: 23, 39).  A thread builds four chunks of 16 bytes, from words at
// any byte; what lies behind a row's end within its last word goes into the padding.
constexpr int kStageThreads = 256, kStageChunks = 4;
struct StageJob {
    const uint8_t* src;
    uint8_t* dst;
    int64_t rows, row_bytes, pitch;  // pitch: of dst
    int64_t block0;                  // the job's first block
};
struct StageJobs {
    StageJob job[3];
    int n;
};
__global__ void __launch_bounds__(kStageThreads) forge_linear_stage_kernel(const StageJobs jobs)
{
    let_dependents_start();
    int which = 0;
    while (which + 1 < jobs.n && jobs.job[which + 1].block0 <= blockIdx.x) ++which;
    const StageJob& b = jobs.job[which];
    const uint32_t per_row = static_cast<uint32_t>((b.row_bytes + 15) / 16);
    const int64_t first = (blockIdx.x - b.block0) * (kStageThreads * kStageChunks);
    const int64_t left = b.rows * per_row - first;
    const int64_t r0 = first / per_row;
    const uint32_t c0 = static_cast<uint32_t>(first - r0 * per_row);
    uint4 v[kStageChunks];
    uint8_t* to[kStageChunks];
#pragma unroll
    for (int j = 0; j < kStageChunks; ++j) {
        const uint32_t i = threadIdx.x + kStageThreads * j;
        to[j] = nullptr;
        if (i >= left) continue;
        const uint32_t down = (c0 + i) / per_row, c = c0 + i - down * per_row;
        to[j] = b.dst + (r0 + down) * b.pitch + int64_t{16} * c;
        const uint8_t* from = b.src + (r0 + down) * b.row_bytes + int64_t{16} * c;
        const int64_t end = b.row_bytes - int64_t{16} * c;
        const int n = end < 16 ? static_cast<int>(end) : 16;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 3);
        const uint32_t* words = reinterpret_cast<const uint32_t*>(from - off);
        uint32_t w[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = 4 * k < off + n ? __ldcs(words + k) : 0u;
        v[j] = make_uint4(__funnelshift_r(w[0], w[1], 8 * off), __funnelshift_r(w[1], w[2], 8 * off),
                          __funnelshift_r(w[2], w[3], 8 * off), __funnelshift_r(w[3], w[4], 8 * off));
    }
#pragma unroll
    for (int j = 0; j < kStageChunks; ++j)
        if (to[j]) *reinterpret_cast<uint4*>(to[j]) = v[j];
}

cudaError_t stage(StageJobs& jobs, cudaStream_t s)
{
    int64_t blocks = 0;
    for (int i = 0; i < jobs.n; ++i) {
        StageJob& b = jobs.job[i];
        constexpr int64_t each = kStageThreads * kStageChunks;
        b.block0 = blocks;
        blocks += (b.rows * ((b.row_bytes + 15) / 16) + each - 1) / each;
    }
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    forge_linear_stage_kernel<<<static_cast<unsigned>(blocks), kStageThreads, 0, s>>>(jobs);
    return cudaGetLastError();
}

struct Operands {
    const uint8_t *A, *W;
    int64_t ldA, ldW;  // bytes between rows, multiples of 16
};

cudaError_t run(const Operands& o, int64_t N, int64_t M, bool transpose, LParams p,
                const Choice& c, bool staged, cudaStream_t stream)
{
    const int64_t E = p.E > 0 ? p.E : 1;
    CUtensorMap ta, tw;
    if (encode_bytes(&ta, o.A, p.K, p.T, 0, o.ldA, c.tokens < 128 ? c.tokens : 128) != cudaSuccess ||
        encode_bytes(&tw, o.W, M, N, E, o.ldW, 128) != cudaSuccess)
        return cudaErrorInvalidValue;
    const int cols = c.tokens == 256 ? 256 : 128;
    p.tiles_o = static_cast<int32_t>((p.O + cols - 1) / cols);
    const Launch l{ta, tw, p, c.split, staged, stream};
    if (p.E > 0)
        return transpose ? launch_form<false, true>(c.tokens, l) : launch_form<true, true>(c.tokens, l);
    return transpose ? launch_form<false, false>(c.tokens, l) : launch_form<true, false>(c.tokens, l);
}

forge_status linear(const uint8_t* A, const float* sA, const uint8_t* W, const float* sW, void* Y,
                    forge_dtype y_dtype, const int32_t* offsets, int32_t E, int64_t T, int64_t N,
                    int64_t M, int32_t transpose, forge_stream_t stream)
{
    if (T < 0 || N < 1 || M < 1 || T > INT32_MAX - 512 || N > INT32_MAX - 512 ||
        M > INT32_MAX - 512)
        return FORGE_ERR_INVALID_ARG;
    if (!W || !sW || (T > 0 && (!A || !sA || !Y))) return FORGE_ERR_INVALID_ARG;
    if (y_dtype != FORGE_F32 && y_dtype != FORGE_BF16) return FORGE_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(sA, 4) || !aligned(sW, 4) || !aligned(offsets, 4) ||
        !aligned(Y, y_dtype == FORGE_F32 ? 4 : 2))
        return FORGE_ERR_MISALIGNED;
    int sms = 0;
    forge_status st = device_sms(&sms);
    if (st != FORGE_OK) return st;
    if (T == 0) return FORGE_OK;
    const void* ptrs[] = {A, sA, W, sW, Y, offsets};
    if ((st = device_resident(ptrs, 6)) != FORGE_OK) return st;
    LParams p{};
    p.T = T;
    p.K = transpose ? M : N;
    p.O = transpose ? N : M;
    p.sA = sA;
    p.sW = sW;
    const int64_t across = (M + kBlock - 1) / kBlock, down = (N + kBlock - 1) / kBlock;
    p.sw_k = transpose ? 1 : across;
    p.sw_o = transpose ? across : 1;
    p.sw_e = across * down;
    p.Y = Y;
    p.f32 = y_dtype == FORGE_F32;
    p.vec = p.O % (p.f32 ? 4 : 8) == 0 && aligned(Y, 16);
    p.E = E;
    p.offsets = offsets;
    p.nk = static_cast<int32_t>((p.K + kBlock - 1) / kBlock);
    p.sa_ld = p.nk;
    p.sa_vec = p.nk % 4 == 0 && aligned(sA, 16);
    p.w.timeout_ns = wait_timeout();
    p.w.status = device_status_word();

    // Rows that TMA cannot address go through rows padded to 16 bytes, and so do, for many
    // tokens, rows of A's scales that no 16-byte load can address: a load for each
    // scale keeps the load-store unit, and with it the barriers, busy.
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Choice c = choose(p, sms);
    const int64_t rows_w = (E > 0 ? E : 1) * N;
    const int64_t pad_a = (p.K + 15) / 16 * 16, pad_w = (M + 15) / 16 * 16;
    const int64_t pad_s = (int64_t{p.nk} * 4 + 15) / 16 * 16;
    const bool stage_a = p.K % 16 != 0 || !aligned(A, 16);
    const bool stage_w = M % 16 != 0 || !aligned(W, 16);
    const bool stage_s = c.tokens == 256 && !p.sa_vec;
    Operands o{A, W, p.K, M};
    void* scratch = nullptr;
    cudaError_t e = cudaSuccess;
    if (stage_a || stage_w || stage_s) {
        auto whole = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
        const int64_t a_bytes = stage_a ? whole(pad_a * T) : 0;
        const int64_t s_bytes = stage_s ? whole(pad_s * T) : 0;
        e = scratch_alloc(&scratch, a_bytes + s_bytes + (stage_w ? pad_w * rows_w : 0), s);
        uint8_t* at = static_cast<uint8_t*>(scratch);
        StageJobs jobs{};
        auto copy = [&](const void* src, int64_t rows, int64_t row_bytes, int64_t pitch) {
            jobs.job[jobs.n++] = {static_cast<const uint8_t*>(src), at, rows, row_bytes, pitch, 0};
            uint8_t* to = at;
            at += whole(pitch * rows);
            return to;
        };
        if (e == cudaSuccess) {
            if (stage_a) {
                o.A = copy(A, T, p.K, pad_a);
                o.ldA = pad_a;
            }
            if (stage_s) {
                p.sA = reinterpret_cast<const float*>(copy(sA, T, int64_t{p.nk} * 4, pad_s));
                p.sa_ld = pad_s / 4;
                p.sa_vec = 1;
            }
            if (stage_w) {
                o.W = copy(W, rows_w, M, pad_w);
                o.ldW = pad_w;
            }
            e = stage(jobs, s);
        }
    }
    if (e == cudaSuccess) e = run(o, N, M, transpose != 0, p, c, scratch != nullptr, s);
    if (scratch) {
        const cudaError_t fe = scratch_free(scratch, s);
        if (e == cudaSuccess) e = fe;
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? FORGE_OK : FORGE_ERR_CUDA;
}

}  // namespace linear
}  // namespace forge

extern "C" forge_status forge_linear_e4m3(const uint8_t* A, const float* sA, const uint8_t* W,
                                          const float* sW, void* Y, forge_dtype y_dtype, int64_t T,
                                          int64_t N, int64_t M, int32_t transpose,
                                          forge_stream_t stream)
{
    return forge::linear::linear(A, sA, W, sW, Y, y_dtype, nullptr, 0, T, N, M, transpose, stream);
}

extern "C" forge_status forge_grouped_linear_e4m3(const uint8_t* A, const float* sA,
                                                  const uint8_t* W, const float* sW,
                                                  const int32_t* offsets, int32_t E, void* Y,
                                                  forge_dtype y_dtype, int64_t T_max, int64_t N,
                                                  int64_t M, int32_t transpose,
                                                  forge_stream_t stream)
{
    if (!offsets || E < 1 || E > forge::kMaxExperts) return FORGE_ERR_INVALID_ARG;
    return forge::linear::linear(A, sA, W, sW, Y, y_dtype, offsets, E, T_max, N, M, transpose,
                                 stream);
}
