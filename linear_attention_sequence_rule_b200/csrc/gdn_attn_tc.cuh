// gdn_attn_tc.cuh -- what the tensor-core attention kernels (bf16) share: bounded waits, tile loads,
// the MMA loops over a 128-row tile, and the exchange between TMEM rows and memory.
#pragma once

#include <cuda_bf16.h>

#include "gdn_attn.h"
#include "gdn_attn_tile.cuh"
#include "gdn_tmap.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace attn {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int BT = 128;               // rows of every tile (queries or keys)
constexpr int kSub = BT * 128;        // bytes of a 64-column sub-tile: 128 rows of 128 bytes, swizzled

// Barriers with bounded waits: a wait that runs out records it and raises the CTA's abort flag, after
// which no wait waits and every role ends with its current step.  A wait that finds its phase complete
// costs one probe: between batches of products the issuing warp's own latency leaves the tensor pipe
// idle (its queue holds a few instructions), so the flag is looked at once a step and in waits that wait.
struct Waits {
    int *abort, *error;
    __device__ __forceinline__ bool aborted() const { return *(volatile int *)abort != 0; }
    // the same for a whole warp, so that its lanes leave a loop together
    __device__ __forceinline__ bool stopped() const { return __any_sync(0xffffffffu, aborted()); }
    // (without a time of its own the probe sleeps for what the hardware sees fit, and wakes sooner)
    __device__ __forceinline__ static bool over(uint64_t *b, uint32_t parity)
    {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(b)), "r"(parity)
            : "memory");
        return ok != 0;
    }
    __device__ __forceinline__ void wait(uint64_t *b, int phase) const
    {
        if (over(b, phase & 1)) return;
        const uint64_t t0 = globaltimer_ns();
        while (!aborted()) {
            if (over(b, phase & 1)) return;
            if (globaltimer_ns() - t0 > kWaitNs) {
                atomicOr(error, 1);
                *(volatile int *)abort = 1;
            }
        }
    }
    // the same for a whole warp ahead of an instruction that its lanes must execute together (tensor memory's loads and
    // stores): lanes that found the phase over at different probes meet again here
    __device__ __forceinline__ void wait_warp(uint64_t *b, int phase) const
    {
        wait(b, phase);
        __syncwarp();
    }
};

__device__ __forceinline__ void arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}

// One arrival for a warp, behind what all its lanes have done (32 arrivals on one barrier would be
// served one after the other).
__device__ __forceinline__ void warp_arrive(uint64_t *b, int lane)
{
    __syncwarp();
    if (lane == 0) arrive(b);
}

// Pairs of fp32 in one 64-bit register: one instruction for two results.
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 128 rows of one head from token `row` on: D / 64 sub-tiles
template <int D>
__device__ __forceinline__ void load_tile(unsigned char *dst, const CUtensorMap *m, uint64_t *bar, int head, int row)
{
#pragma unroll
    for (int x = 0; x < D / 64; ++x) tma_load_3d(dst + x * kSub, m, bar, 64 * x, head, row);
}

// Zero rows n .. 127 of a tile (one warp): rows behind the sequence's end belong to a neighbour, and a
// weight of 0 times a NaN there would be NaN.
template <int D> __device__ __forceinline__ void zero_rows(unsigned char *tile, int n, int lane)
{
    for (int i = lane; i < (BT - n) * 8; i += 32)
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
            *reinterpret_cast<uint4 *>(tile + x * kSub + n * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// The products are issued by a whole warp whose leader alone executes them (elect.sync): in code that
// one lane runs by itself the descriptors cannot live in uniform registers, and moving them there
// instruction by instruction costs more than twice the time of the products (at d = 128 about
// 145 cycles an instruction of 64).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// D[128 x N] = A B^T over the head size: both tiles K-major in shared memory (b: the first of N rows)
template <int D, int N = BT> __device__ __forceinline__ void mma_nt(uint32_t d, const unsigned char *a, const unsigned char *b)
{
    constexpr uint32_t id = idesc_bf16(BT, N, 0, 0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (kk >> 2) * kSub + (kk & 3) * 32;
        mma_ss(d, sdesc_sw128(smem_u32(a) + o, 16, 1024), sdesc_sw128(smem_u32(b) + o, 16, 1024), id, kk > 0);
    }
}

// The same with A (128 rows of D, bf16: D / 2 columns) in tensor memory
template <int D, int N = BT> __device__ __forceinline__ void mma_nt_ta(uint32_t d, uint32_t a, const unsigned char *b)
{
    constexpr uint32_t id = idesc_bf16(BT, N, 0, 0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        mma_ts(d, a + 8 * kk, sdesc_sw128(smem_u32(b) + (kk >> 2) * kSub + (kk & 3) * 32, 16, 1024), id, kk > 0);
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Elements e0 .. e0 + NE - 1 of row r of a tile in shared memory to tensor memory (address t of the row's
// element 0, the warp's lanes included).  Operands that stay for a whole CTA are kept there: a product
// of two shared operands takes all of shared memory's bandwidth, and every other access (a barrier's
// probe, a row's statistics) then waits some 300 cycles.
template <int NE> __device__ __forceinline__ void row_to_tmem(uint32_t t, const unsigned char *tile, int r, int e0)
{
#pragma unroll
    for (int x = 0; x < NE / 32; ++x) {
        uint32_t v[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = e0 / 8 + 4 * x + u;  // 16-byte unit of the row
            const uint4 y = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * kSub + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            v[4 * u] = y.x, v[4 * u + 1] = y.y, v[4 * u + 2] = y.z, v[4 * u + 3] = y.w;
        }
        tmem_st16(t + (e0 + 32 * x) / 2, v);
    }
}

// D[128 x D] (+)= A B: A (128 x 128, bf16) in tensor memory, B's rows (the 128 of the sum) in shared
// memory, read MN-major; k steps k0 .. k1 - 1 of 16
template <int D>
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t a, const unsigned char *b, int k0, int k1, bool accumulate)
{
    constexpr uint32_t id = idesc_bf16(BT, D, 0, 1);
#pragma unroll
    for (int kk = k0; kk < k1; ++kk)
        mma_ts(d, a + 8 * kk, sdesc_sw128(smem_u32(b) + kk * 2048, kSub, 1024), id, accumulate || kk > k0);
}

// NC columns from column c0 on of an accumulator (tensor memory address t of column 0; thread = row of
// its warp's 32), scaled and written as bf16: through the warp's own rows of `buf` (D * 2 bytes a row,
// 16-byte units XORed with the row), then in whole row parts to g + row * ld for rows below n.
template <int D, int NC>
__device__ __forceinline__ void store_rows(uint32_t t, float f, unsigned char *buf, int warp, int lane, int c0,
                                           __nv_bfloat16 *g, int64_t ld, int n)
{
    constexpr int UN = NC / 8;  // 16-byte units a row
    const int r = 32 * warp + lane, u0 = c0 / 8;
#pragma unroll 1  // (code that a CTA runs once comes from memory, line by line)
    for (int x = 0; x < NC / 32; ++x) {
        float o[32];
        tmem_ld32(t + c0 + 32 * x, o);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint4 w;
            w.x = pack_bf16x2(o[8 * u] * f, o[8 * u + 1] * f);
            w.y = pack_bf16x2(o[8 * u + 2] * f, o[8 * u + 3] * f);
            w.z = pack_bf16x2(o[8 * u + 4] * f, o[8 * u + 5] * f);
            w.w = pack_bf16x2(o[8 * u + 6] * f, o[8 * u + 7] * f);
            *reinterpret_cast<uint4 *>(buf + r * (2 * D) + (((u0 + 4 * x + u) ^ (r & 7)) << 4)) = w;
        }
    }
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < 32 * UN; i += 32) {
        const int rr = 32 * warp + i / UN, u = u0 + i % UN;
        if (rr < n)
            *reinterpret_cast<uint4 *>(g + (int64_t)rr * ld + 8 * u) =
                *reinterpret_cast<const uint4 *>(buf + rr * (2 * D) + ((u ^ (rr & 7)) << 4));
    }
}

// 3-D view [tokens][heads][d] of a bf16 tensor; box = 64 features x 1 head x 128 tokens, 128-byte swizzle
inline bool make_map(CUtensorMap *m, const void *base, int64_t tokens, int heads, int d)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    const cuuint32_t box[3] = {64, 1, BT};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace gdn
