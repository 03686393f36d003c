// gdn_attn_simt.cu -- causal softmax attention over whole prompts and its gradients on CUDA cores,
// fp32 throughout.
//
// Forward, per (sequence, query head, block of BM query rows): one pass over the key blocks of 64
// with the running maximum m and sum l of a softmax,
//     s = scale q k^T,  m' = max(m, max_j s),  p = exp(s - m'),
//     l' = l exp(m - m') + sum_j p,  o' = o exp(m - m') + p v,     out = o / l,  lse = m + log l.
// Backward: two launches after D_i = dout_i . out_i.  The query side forms dq per query block over
// its key blocks; the key side forms dk, dv per key block and query head over the head's query blocks, and
// a last launch adds up the heads that share a key head, in order: every gradient is summed in one
// order.  (One CTA for all heads that share a key block would need no last launch, but has few and long
// CTAs: 1024 tokens, 4 heads on 1, d 64: 760 us against 283; 2 x 4096, 12 on 4: 6.18 ms against 5.53.)
//
// Tiles sit in shared memory in fp32 (rows of D + 4 floats: a quarter warp's float4 reads of 8
// rows hit 8 different bank groups).  256 threads as 16 x 16; a thread holds RPT rows (ty RPT + i)
// and, in products over the head size, columns tx + 16 j; in products with D columns, the float4
// groups tx + 16 g.
#include <math.h>

#include "gdn_attn.h"
#include "gdn_attn_tile.cuh"
#include "sm100_ptx.cuh"

namespace gdn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int BN = 64;       // keys per block
constexpr int LDP = BN + 4;  // row stride of a score tile
constexpr int NT = 256;

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }

// ROWS rows of one head, from row r0 on, into shared memory; rows past `len` are zero.  `g` is the
// head's row 0 of the sequence, `ld` the elements between tokens.
template <int ROWS, int D>
__device__ __forceinline__ void load_tile(float *s, const float *g, int64_t ld, int r0, int len)
{
    constexpr int C = D / 4;
#pragma unroll 4
    for (int i = threadIdx.x; i < ROWS * C; i += NT) {
        const int r = i / C, c = i % C;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < len) x = load4(g + (int64_t)(r0 + r) * ld + 4 * c);
        *reinterpret_cast<float4 *>(s + r * (D + 4) + 4 * c) = x;
    }
}

// The same by cp.async; the caller commits and waits.
template <int ROWS, int D>
__device__ __forceinline__ void load_tile_async(float *s, const float *g, int64_t ld, int r0, int len)
{
    constexpr int C = D / 4;
#pragma unroll
    for (int i = threadIdx.x; i < ROWS * C; i += NT) {
        const int r = i / C, c = i % C;
        const bool on = r0 + r < len;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(s + r * (D + 4) + 4 * c)),
                     "l"(g + (int64_t)(on ? r0 + r : 0) * ld + 4 * c), "r"(on ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float dot4(float4 a, float4 b, float c)
{
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// acc[i][j] += A row (ra + i) . B row (tx + 16 j), both rows of D + 4 floats
template <int RPT, int D>
__device__ __forceinline__ void mul_nt(float (&acc)[RPT][4], const float *A, const float *Bs, int ra, int tx)
{
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[RPT], b[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (ra + i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(Bs + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = dot4(a[i], b[j], acc[i][j]);
    }
}

// acc[i][g] += sum_k P[ra + i][k] B[k][4 (tx + 16 g) ..], k over the 64 columns of P
template <int RPT, int D>
__device__ __forceinline__ void mul_nn(float4 (&acc)[RPT][D / 64], const float *P, const float *Bs, int ra, int tx)
{
#pragma unroll 2
    for (int k = 0; k < BN; k += 4) {
        float4 a[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) a[i] = *reinterpret_cast<const float4 *>(P + (ra + i) * LDP + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int g = 0; g < D / 64; ++g) {
                const float4 b = *reinterpret_cast<const float4 *>(Bs + (k + e) * (D + 4) + 4 * (tx + 16 * g));
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float x = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
                    acc[i][g].x = fmaf(x, b.x, acc[i][g].x);
                    acc[i][g].y = fmaf(x, b.y, acc[i][g].y);
                    acc[i][g].z = fmaf(x, b.z, acc[i][g].z);
                    acc[i][g].w = fmaf(x, b.w, acc[i][g].w);
                }
            }
    }
}

// acc[i][g] += sum_k P[k][ra + i] B[k][4 (tx + 16 g) ..], k over the 64 rows of P; RPT = 4
template <int D>
__device__ __forceinline__ void mul_tn(float4 (&acc)[4][D / 64], const float *P, const float *Bs, int ra, int tx)
{
#pragma unroll 4
    for (int k = 0; k < BN; ++k) {
        const float4 a = *reinterpret_cast<const float4 *>(P + k * LDP + ra);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
            const float4 b = *reinterpret_cast<const float4 *>(Bs + k * (D + 4) + 4 * (tx + 16 * g));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][g].x = fmaf(av[i], b.x, acc[i][g].x);
                acc[i][g].y = fmaf(av[i], b.y, acc[i][g].y);
                acc[i][g].z = fmaf(av[i], b.z, acc[i][g].z);
                acc[i][g].w = fmaf(av[i], b.w, acc[i][g].w);
            }
        }
    }
}

__device__ __forceinline__ float row_max16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---- forward -------------------------------------------------------------------------------------

// BM = 16 RPT query rows.
template <int D, int RPT> constexpr int fwd_smem()
{
    return ((16 * RPT + 4 * BN) * (D + 4) + 16 * RPT * LDP) * 4;
}

template <int D, int RPT>
__global__ void __launch_bounds__(NT) attn_fwd_simt(const float *__restrict__ q, const float *__restrict__ k,
                                                    const float *__restrict__ v, float *__restrict__ out,
                                                    float *__restrict__ lse, const int32_t *__restrict__ cu, FastDiv B,
                                                    int Tn, int Hq, int Hk, float scale2)
{
    constexpr int BM = 16 * RPT;
    extern __shared__ float sm[];
    constexpr int TS = BN * (D + 4);
    float *Qs = sm, *KV = Qs + BM * (D + 4), *Ps = KV + 4 * TS;  // K, V of this block and of the next
    const AttnTile t = attn_tile(cu, B, Tn, BM, blockIdx.x);
    if (t.seq < 0) return;
    const int h = blockIdx.y, hk = h / (Hq / Hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ra = ty * RPT;
    const int q0 = t.block * BM;
    const int64_t ldq = (int64_t)Hq * D, ldk = (int64_t)Hk * D;
    const float *kg = k + t.t0 * ldk + (int64_t)hk * D, *vg = v + t.t0 * ldk + (int64_t)hk * D;
    load_tile<BM, D>(Qs, q + t.t0 * ldq + (int64_t)h * D, ldq, q0, t.len);
    float m[RPT], l[RPT];
    float4 o[RPT][D / 64];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) o[i][g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int kend = min(q0 + BM, t.len);
    load_tile_async<BN, D>(KV, kg, ldk, 0, t.len);
    load_tile_async<BN, D>(KV + TS, vg, ldk, 0, t.len);
    async_commit();
    for (int k0 = 0, b = 0; k0 < kend; k0 += BN, b ^= 1) {
        const float *Ks = KV + 2 * b * TS, *Vs = Ks + TS;
        if (k0 + BN < kend) {
            float *next = KV + 2 * (b ^ 1) * TS;
            load_tile_async<BN, D>(next, kg, ldk, k0 + BN, t.len);
            load_tile_async<BN, D>(next + TS, vg, ldk, k0 + BN, t.len);
        }
        async_commit();
        async_wait<1>();
        __syncthreads();
        float s[RPT][4] = {};
        mul_nt<RPT, D>(s, Qs, Ks, ra, tx);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = k0 + tx + 16 * j <= q0 + ra + i ? s[i][j] * scale2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = row_max16(mx);
            // key 0 is visible to every row and comes first, so mx is -inf only where scores are
            const float ms = mx == -INFINITY ? 0.f : mx;
            const float f = exp2f(m[i] - ms);
            m[i] = mx;
            l[i] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ms);
                l[i] += p;
                Ps[(ra + i) * LDP + tx + 16 * j] = p;
            }
#pragma unroll
            for (int g = 0; g < D / 64; ++g) {
                o[i][g].x *= f;
                o[i][g].y *= f;
                o[i][g].z *= f;
                o[i][g].w *= f;
            }
        }
        __syncwarp();  // a row's 16 threads lie in one warp
        mul_nn<RPT, D>(o, Ps, Vs, ra, tx);
        __syncthreads();  // this block's tiles have been read
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = q0 + ra + i;
        const float ls = row_sum16(l[i]);
        if (row >= t.len) continue;
        const float inv = 1.f / ls;
        float *og = out + (t.t0 + row) * ldq + (int64_t)h * D;
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            store4(og + 4 * (tx + 16 * g),
                   make_float4(o[i][g].x * inv, o[i][g].y * inv, o[i][g].z * inv, o[i][g].w * inv));
        if (lse && tx == 0) lse[(t.t0 + row) * Hq + h] = (m[i] + log2f(ls)) * kLn2;
    }
}

// ---- backward ------------------------------------------------------------------------------------

// D_i = dout_i . out_i, one warp per (token, head)
template <int D>
__global__ void __launch_bounds__(NT) attn_bwd_dot(const float *__restrict__ out, const float *__restrict__ dout,
                                                   float *__restrict__ dot, int64_t rows,
                                                   const int32_t *__restrict__ cu, int B, int Hq)
{
    const int64_t n = cu ? min(rows, (int64_t)max(cu[B], 0) * Hq) : rows;
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    if (r >= n) return;
    float x = 0.f;
    if (lane * 4 < D) x = dot4(load4(out + r * D + 4 * lane), load4(dout + r * D + 4 * lane), 0.f);
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) dot[r] = x;
}

template <int D> constexpr int bwd_smem() { return (4 * 64 * (D + 4) + 2 * 64 * LDP + 128) * 4; }

// p and ds of a 64 x 64 tile (rows: queries q0.., columns: keys k0..) from the tiles in shared memory
template <int D>
__device__ __forceinline__ void tile_p_ds(float (&p)[4][4], float (&ds)[4][4], const float *Qs, const float *Os,
                                          const float *Ks, const float *Vs, const float *ls, const float *dt, int q0,
                                          int k0, int len, float scale2, int ra, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[i][j] = ds[i][j] = 0.f;
    mul_nt<4, D>(p, Qs, Ks, ra, tx);
    mul_nt<4, D>(ds, Os, Vs, ra, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = k0 + tx + 16 * j <= q0 + ra + i && q0 + ra + i < len;
            p[i][j] = on ? exp2f(p[i][j] * scale2 - ls[ra + i]) : 0.f;
            ds[i][j] = on ? p[i][j] * (ds[i][j] - dt[ra + i]) : 0.f;
        }
}

__device__ __forceinline__ void load_rowstats(float *ls, float *dt, const float *lse, const float *dot, int64_t t0,
                                              int Hq, int h, int q0, int len)
{
    if (threadIdx.x < 64) {
        const int r = q0 + threadIdx.x;
        ls[threadIdx.x] = r < len ? lse[(t0 + r) * Hq + h] * kLog2e : 0.f;
        dt[threadIdx.x] = r < len ? dot[(t0 + r) * Hq + h] : 0.f;
    }
}

template <int D>
__global__ void __launch_bounds__(NT) attn_bwd_dq_simt(const float *__restrict__ q, const float *__restrict__ k,
                                                       const float *__restrict__ v, const float *__restrict__ dout,
                                                       const float *__restrict__ lse, const float *__restrict__ dot,
                                                       float *__restrict__ dq, const int32_t *__restrict__ cu, FastDiv B,
                                                       int Tn, int Hq, int Hk, float scale)
{
    extern __shared__ float sm[];
    constexpr int TS = 64 * (D + 4);
    float *Qs = sm, *Os = Qs + TS, *Ks = Os + TS, *Vs = Ks + TS, *Ds = Vs + TS, *ls = Ds + 2 * 64 * LDP, *dt = ls + 64;
    const AttnTile t = attn_tile(cu, B, Tn, 64, blockIdx.x);
    if (t.seq < 0) return;
    const int h = blockIdx.y, hk = h / (Hq / Hk);
    const int tx = threadIdx.x & 15, ra = (threadIdx.x >> 4) * 4;
    const int q0 = t.block * 64;
    const int64_t ldq = (int64_t)Hq * D, ldk = (int64_t)Hk * D;
    load_tile<64, D>(Qs, q + t.t0 * ldq + (int64_t)h * D, ldq, q0, t.len);
    load_tile<64, D>(Os, dout + t.t0 * ldq + (int64_t)h * D, ldq, q0, t.len);
    load_rowstats(ls, dt, lse, dot, t.t0, Hq, h, q0, t.len);
    float4 acc[4][D / 64] = {};
    for (int k0 = 0; k0 <= q0; k0 += BN) {
        __syncthreads();
        load_tile<BN, D>(Ks, k + t.t0 * ldk + (int64_t)hk * D, ldk, k0, t.len);
        load_tile<BN, D>(Vs, v + t.t0 * ldk + (int64_t)hk * D, ldk, k0, t.len);
        __syncthreads();
        float p[4][4], ds[4][4];
        tile_p_ds<D>(p, ds, Qs, Os, Ks, Vs, ls, dt, q0, k0, t.len, scale * kLog2e, ra, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) Ds[(ra + i) * LDP + tx + 16 * j] = ds[i][j];
        __syncwarp();
        mul_nn<4, D>(acc, Ds, Ks, ra, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (q0 + ra + i >= t.len) continue;
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            store4(dq + (t.t0 + q0 + ra + i) * ldq + (int64_t)h * D + 4 * (tx + 16 * g),
                   make_float4(acc[i][g].x * scale, acc[i][g].y * scale, acc[i][g].z * scale, acc[i][g].w * scale));
    }
}

// dk and dv of one query head's (blockIdx.y) queries, laid out as [tokens, Hq, D].
template <int D>
__global__ void __launch_bounds__(NT) attn_bwd_dkv_simt(const float *__restrict__ q, const float *__restrict__ k,
                                                        const float *__restrict__ v, const float *__restrict__ dout,
                                                        const float *__restrict__ lse, const float *__restrict__ dot,
                                                        float *__restrict__ dk, float *__restrict__ dv,
                                                        const int32_t *__restrict__ cu, FastDiv B, int Tn, int Hq, int Hk,
                                                        float scale)
{
    extern __shared__ float sm[];
    constexpr int TS = 64 * (D + 4);
    float *Ks = sm, *Vs = Ks + TS, *Qs = Vs + TS, *Os = Qs + TS, *Ps = Os + TS, *Ds = Ps + 64 * LDP, *ls = Ds + 64 * LDP,
          *dt = ls + 64;
    const AttnTile t = attn_tile(cu, B, Tn, 64, blockIdx.x);
    if (t.seq < 0) return;
    const int h = blockIdx.y, hk = h / (Hq / Hk);
    const int tx = threadIdx.x & 15, ra = (threadIdx.x >> 4) * 4;
    // the tiles come last block first, the fewest queries: take them the other way round
    const int k0 = ((t.len + 63) / 64 - 1 - t.block) * 64;
    const int64_t ldq = (int64_t)Hq * D, ldk = (int64_t)Hk * D;
    load_tile<64, D>(Ks, k + t.t0 * ldk + (int64_t)hk * D, ldk, k0, t.len);
    load_tile<64, D>(Vs, v + t.t0 * ldk + (int64_t)hk * D, ldk, k0, t.len);
    float4 ak[4][D / 64] = {}, av[4][D / 64] = {};
    for (int q0 = k0; q0 < t.len; q0 += 64) {
        __syncthreads();
        load_tile<64, D>(Qs, q + t.t0 * ldq + (int64_t)h * D, ldq, q0, t.len);
        load_tile<64, D>(Os, dout + t.t0 * ldq + (int64_t)h * D, ldq, q0, t.len);
        load_rowstats(ls, dt, lse, dot, t.t0, Hq, h, q0, t.len);
        __syncthreads();
        float p[4][4], ds[4][4];
        tile_p_ds<D>(p, ds, Qs, Os, Ks, Vs, ls, dt, q0, k0, t.len, scale * kLog2e, ra, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Ps[(ra + i) * LDP + tx + 16 * j] = p[i][j];
                Ds[(ra + i) * LDP + tx + 16 * j] = ds[i][j];
            }
        __syncthreads();
        mul_tn<D>(av, Ps, Os, ra, tx);
        mul_tn<D>(ak, Ds, Qs, ra, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (k0 + ra + i >= t.len) continue;
        const int64_t at = ((t.t0 + k0 + ra + i) * Hq + h) * D;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
            store4(dk + at + 4 * (tx + 16 * g),
                   make_float4(ak[i][g].x * scale, ak[i][g].y * scale, ak[i][g].z * scale, ak[i][g].w * scale));
            store4(dv + at + 4 * (tx + 16 * g), av[i][g]);
        }
    }
}

// dk and dv [tokens, Hk, D] from the G parts of each key head, added in order; a thread has 4 elements
__global__ void __launch_bounds__(NT) attn_bwd_add_heads(const float *__restrict__ pk, const float *__restrict__ pv,
                                                         float *__restrict__ dk, float *__restrict__ dv, int64_t n4, int G,
                                                         int d4, const int32_t *__restrict__ cu, int B, int Hk)
{
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= (cu ? min(n4, (int64_t)max(cu[B], 0) * Hk * d4) : n4)) return;
    const float4 *p = reinterpret_cast<const float4 *>(blockIdx.y ? pv : pk) + i / d4 * G * d4 + i % d4;
    float4 x = p[0];
    for (int g = 1; g < G; ++g) {
        const float4 y = p[(int64_t)g * d4];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    reinterpret_cast<float4 *>(blockIdx.y ? dv : dk)[i] = x;
}

template <int D, int RPT> cudaError_t run_fwd(const AttnArgs &a, cudaStream_t st)
{
    auto kern = attn_fwd_simt<D, RPT>;
    constexpr int smem = fwd_smem<D, RPT>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)attn_tiles(a.cu, a.B, a.T, 16 * RPT), a.Hq);
    kern<<<grid, NT, smem, st>>>((const float *)a.q, (const float *)a.k, (const float *)a.v, (float *)a.out, a.lse, a.cu,
                                 FastDiv(a.B), a.T, a.Hq, a.Hk, a.scale * kLog2e);
    return cudaGetLastError();
}

template <int D> cudaError_t run_bwd(const AttnArgs &a, cudaStream_t st)
{
    constexpr int smem = bwd_smem<D>();
    cudaError_t e = cudaFuncSetAttribute(attn_bwd_dq_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_bwd_dkv_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t rows = (a.cu ? (int64_t)a.T : (int64_t)a.B * a.T) * a.Hq;
    float *dot = static_cast<float *>(a.workspace);
    attn_bwd_dot<D><<<(unsigned)((rows + NT / 32 - 1) / (NT / 32)), NT, 0, st>>>((const float *)a.out, (const float *)a.dout,
                                                                                 dot, rows, a.cu, a.B, a.Hq);
    const unsigned tiles = (unsigned)attn_tiles(a.cu, a.B, a.T, 64);
    attn_bwd_dq_simt<D><<<dim3(tiles, a.Hq), NT, smem, st>>>((const float *)a.q, (const float *)a.k, (const float *)a.v,
                                                                (const float *)a.dout, a.lse, dot, (float *)a.dq, a.cu,
                                                                FastDiv(a.B), a.T, a.Hq, a.Hk, a.scale);
    const bool shared = a.Hq > a.Hk;
    float *pk = dot + (rows + 63) / 64 * 64, *pv = pk + rows * D;  // behind D, if heads are shared
    attn_bwd_dkv_simt<D><<<dim3(tiles, a.Hq), NT, smem, st>>>(
        (const float *)a.q, (const float *)a.k, (const float *)a.v, (const float *)a.dout, a.lse, dot,
        shared ? pk : (float *)a.dk, shared ? pv : (float *)a.dv, a.cu, FastDiv(a.B), a.T, a.Hq, a.Hk, a.scale);
    if (shared) {
        const int64_t n4 = rows / a.Hq * a.Hk * (D / 4);
        attn_bwd_add_heads<<<dim3((unsigned)((n4 + NT - 1) / NT), 2), NT, 0, st>>>(
            pk, pv, (float *)a.dk, (float *)a.dv, n4, a.Hq / a.Hk, D / 4, a.cu, a.B, a.Hk);
    }
    return cudaGetLastError();
}

}  // namespace

size_t attn_bwd_simt_workspace(int B, int T, int Hq, int Hk, int d, int varlen)
{
    const size_t rows = (varlen ? (size_t)T : (size_t)B * T) * Hq, parts = Hq > Hk ? 2 * rows * d : 0;
    return ((rows + 63) / 64 * 64 + parts) * sizeof(float);
}

cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t st)
{
    // Query rows a CTA: 64, but 32 or 16 where blocks of 64 would leave most SMs without one (256 tokens, 2
    // heads, d 64: 22.8 us with 64, 16.7 with 32, 13.8 with 16; 512 tokens, 8 heads, d 128: 68, 52 and
    // 74 us; 2 x 1024 tokens, 8 heads, d 64: 127, 139 and 196 us).
    const long n = attn_tiles(a.cu, a.B, a.T, 64) * a.Hq;
    if (n < 48) return a.d == 128 ? run_fwd<128, 1>(a, st) : run_fwd<64, 1>(a, st);
    if (n < 148) return a.d == 128 ? run_fwd<128, 2>(a, st) : run_fwd<64, 2>(a, st);
    return a.d == 128 ? run_fwd<128, 4>(a, st) : run_fwd<64, 4>(a, st);
}

cudaError_t launch_attn_bwd_simt(const AttnArgs &a, cudaStream_t st)
{
    return a.d == 128 ? run_bwd<128>(a, st) : run_bwd<64>(a, st);
}

}  // namespace gdn
