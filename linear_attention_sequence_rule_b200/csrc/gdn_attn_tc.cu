// gdn_attn_tc.cu -- causal softmax attention over whole prompts on the tcgen05 tensor cores (bf16).
//
// Per (sequence, query head, 256 query rows): S = Q K^T, running maximum m and sum l of a softmax over
// blocks of 128 keys, P = exp2(scale log2e S - m), O = O exp2(m_old - m) + P V, out = O / l,
// lse = (m + log2 l) ln 2.
//
// One CTA holds two query tiles of 128 rows, which share every K and V tile that TMA brings (half the
// L2 traffic of one tile).  They work in steps of 64 keys: a tile's O (D columns) and two (d = 128) or
// three (d = 64) S tiles of 64 columns fill the 512 columns of tensor memory, and P (bf16) is written
// over the S it came from.  So the scores of the next steps are formed while a step's softmax runs; with
// one S tile of 128 keys a query tile had only one of the two under way, and a step of 128 keys took
// 4500 cycles for 2048 of products or exponentials.
// 16384 tokens, 16 heads on 4: 0.84-0.87 ms at d = 128 (1310-1260 TFLOP/s, 78-75 % of what a large plain product
// reaches; 1.01 ms in a long run under the power cap) and 0.73-0.76 ms at d = 64, where the exponentials, 16 a
// cycle and SM, take 0.47 ms at full clocks and the products less.
// P is rounded to bf16 for its product: both operands of a product have one type, and V is bf16 (P as a sum of two would
// double the product).  l sums the weights unrounded, in fp32.  The result is off by 2.0e-3 (relative, root mean square),
// 1.7e-3 of it from its own rounding.
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread holds a row
//   warps 8, 9       issue the MMAs of tile 0, 1
//   warp 10          loads; zeroes V rows behind the sequence's end
// The maximum is moved only when a row's new one passes it by 2^8 (weights up to 2^8 are as exact in
// bf16), so that O is rarely rescaled.
#include <math.h>

#include "gdn_attn_tc.cuh"
#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {

__device__ int g_attn_fwd_error = 0;

namespace {

using namespace attn;

constexpr int NTH = 384;

constexpr int HT = 64;           // keys a step
constexpr int kHalf = HT * 128;  // bytes from a tile's first half to its second (in each sub-tile)

template <int D> struct FwdCfg {
    static constexpr int NB = D == 64 ? 3 : 2;  // S tiles
    static constexpr int NS = D == 64 ? 4 : 2;  // K and V stages
    static constexpr int TILE = BT * D * 2;
    static constexpr int Q = 0, K = 2 * TILE, V = K + NS * TILE, BAR = V + NS * TILE;
    // barriers
    static constexpr int q_full = 0;                // [2]
    static constexpr int k_full = 2;                // [NS]
    static constexpr int k_empty = k_full + NS;     // [NS] both tiles' S products have read it
    static constexpr int v_full = k_empty + NS;     // [NS]
    static constexpr int v_empty = v_full + NS;     // [NS]
    static constexpr int v_zeroed = v_empty + NS;   // [1]
    static constexpr int s_full = v_zeroed + 1;     // [2][NB] S of a step is there
    static constexpr int p_full = s_full + 2 * NB;  // [2][NB] P of a step is there (one barrier a tile would not
                                                    // do: a warp may be a step ahead of another)
    static constexpr int pv_done = p_full + 2 * NB; // [2][2] by the step's parity: O holds the step
    static constexpr int all_done = pv_done + 4;    // [2]
    static constexpr int drain = all_done + 2;      // [2]
    static constexpr int NBAR = drain + 2;
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int TOTAL = 1024 + MISC + 16;
    __host__ __device__ static constexpr uint32_t tS(int t) { return NB * HT * t; }
    __host__ __device__ static constexpr uint32_t tO(int t) { return 2 * NB * HT + D * t; }
    static_assert(2 * NB * HT + 2 * D <= 512, "tensor memory budget");
};

template <int D>
__global__ void __launch_bounds__(NTH, 1)
    attn_fwd_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse,
                const int32_t *__restrict__ cu, FastDiv B, int T, FastDiv heads, FastDiv group,
                float scale2)
{
    using C = FwdCfg<D>;
    constexpr int NS = C::NS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    int *abort_flag = reinterpret_cast<int *>(sm + C::MISC + 4);
    const Waits w{abort_flag, &g_attn_fwd_error};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int Hq = (int)heads.d, index = heads.div(blockIdx.x);
    const AttnTile at = attn_tile(cu, B, T, 2 * BT, index);
    if (at.seq < 0) return;
    const int h = blockIdx.x - index * Hq, hk = group.div(h);
    const int q0 = at.block * 2 * BT, rows = at.len - q0;  // rows of this CTA's queries that exist
    // steps of the two tiles (the keys their rows see), and key tiles of 128
    const int n0 = (min(at.len, q0 + BT) + HT - 1) / HT, n1 = rows > BT ? (min(at.len, q0 + 2 * BT) + HT - 1) / HT : 0;
    const int tiles = (max(n0, n1) + 1) / 2;

    auto load_k = [&](int j) {
        const int s = j % NS;
        mbar_arrive_expect_tx(&bar[C::k_full + s], C::TILE);
        load_tile<D>(sm + C::K + s * C::TILE, &tmK, &bar[C::k_full + s], hk, (int)at.t0 + j * BT);
    };
    auto load_v = [&](int j) {
        const int s = j % NS;
        mbar_arrive_expect_tx(&bar[C::v_full + s], C::TILE);
        load_tile<D>(sm + C::V + s * C::TILE, &tmV, &bar[C::v_full + s], hk, (int)at.t0 + j * BT);
    };
    if (warp == 10) {  // the first loads are under way before the rest is set up
        for (int i = lane; i < C::NBAR; i += 32) {
            int n = 1;
            if ((i >= C::k_empty && i < C::v_full) || (i >= C::v_empty && i < C::v_zeroed)) n = n1 ? 2 : 1;
            if (i >= C::p_full && i < C::pv_done) n = BT / 32;  // one a warp
            mbar_init(&bar[i], n);
        }
        fence_mbar_init();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            *abort_flag = 0;
            for (int t = 0; t < (n1 ? 2 : 1); ++t) {
                mbar_arrive_expect_tx(&bar[C::q_full + t], C::TILE);
                load_tile<D>(sm + C::Q + t * C::TILE, &tmQ, &bar[C::q_full + t], h, (int)at.t0 + q0 + t * BT);
                if (t == 0) load_k(0);
            }
            load_v(0);
        }
        __syncwarp();
    }
    if (warp == 11) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // registers: 384 x 168 = 64512 at launch; 128 x 48 + 256 x 224 = 63488 after the two roles' changes
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 10) {
        // ---- loads ----
        if (lane == 0) {
            for (int j = 1; j < tiles && !w.aborted(); ++j) {
                const int s = j % NS;
                if (j >= NS) w.wait(&bar[C::k_empty + s], j / NS - 1);
                if (w.aborted()) break;
                load_k(j);
                if (j >= NS) w.wait(&bar[C::v_empty + s], j / NS - 1);
                if (w.aborted()) break;
                load_v(j);
            }
        }
        __syncwarp();
        const int last = at.len - (tiles - 1) * BT;
        if (last < BT) {
            const int s = (tiles - 1) % NS;
            w.wait(&bar[C::v_full + s], (tiles - 1) / NS);
            if (!w.stopped()) zero_rows<D>(sm + C::V + s * C::TILE, last, lane);
            if (lane == 0) arrive(&bar[C::v_zeroed]);
        }
    } else if (warp < 10) {
        // ---- products of tile t ----
        const int t = warp - 8, n = t ? n1 : n0;
        if (n > 0) {
            const unsigned char *qt = sm + C::Q + t * C::TILE;
            auto scores = [&](int j) {
                const int k = j >> 1, s = k % NS, b = j % C::NB;
                w.wait(&bar[C::k_full + s], k / NS);
                tc_fence_after();
                mma_nt<D, HT>(tmem + C::tS(t) + HT * b, qt, sm + C::K + s * C::TILE + (j & 1) * kHalf);
                commit(&bar[C::s_full + C::NB * t + b]);
                if ((j & 1) || j == n - 1) commit(&bar[C::k_empty + s]);
            };
            w.wait(&bar[C::q_full + t], 0);
            for (int j = 0; j < C::NB && j < n; ++j) scores(j);
            for (int j = 0; j < n && !w.stopped(); ++j) {
                const int k = j >> 1, s = k % NS;
                w.wait(&bar[C::v_full + s], k / NS);
                if (k == tiles - 1 && at.len < tiles * BT) w.wait(&bar[C::v_zeroed], 0);
                w.wait(&bar[C::p_full + C::NB * t + j % C::NB], j / C::NB);
                tc_fence_after();
                mma_tn<D>(tmem + C::tO(t), tmem + C::tS(t) + HT * (j % C::NB), sm + C::V + s * C::TILE + (j & 1) * kHalf, 0,
                          HT / 16, j > 0);
                commit(&bar[C::pv_done + 2 * t + (j & 1)]);
                if ((j & 1) || j == n - 1) commit(&bar[C::v_empty + s]);
                if (j + C::NB < n) {  // over P
                    w.wait(&bar[C::pv_done + 2 * t + (j & 1)], j >> 1);
                    scores(j + C::NB);
                }
            }
            commit(&bar[C::all_done + t]);
            for (int k = (n + 1) / 2; k < tiles; ++k) {  // key tiles that this query tile has no part in
                const int s = k % NS;
                w.wait(&bar[C::k_full + s], k / NS);
                if (lane == 0) arrive(&bar[C::k_empty + s]);
                w.wait(&bar[C::v_full + s], k / NS);
                if (lane == 0) arrive(&bar[C::v_empty + s]);
            }
            if (w.stopped()) {  // products issued already end before the tensor memory is freed
                commit(&bar[C::drain + t]);
                mbar_wait_bounded(&bar[C::drain + t], 0, 100000000ull);
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ---- softmax of tile t; thread = row ----
        const int t = warp >> 2, n = t ? n1 : n0, wq = warp & 3, r = tid & (BT - 1);
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t tS = tmem + lanes + C::tS(t), tO = tmem + lanes + C::tO(t);
        const int jd = 2 * (2 * at.block + t);  // first step of the diagonal block
        float m = -INFINITY, l = 0.f;           // m in units of S
        auto fetch = [&](int j, float (&x)[2][32]) {
            w.wait_warp(&bar[C::s_full + C::NB * t + j % C::NB], j / C::NB);
            tc_fence_after();
            tmem_ld32(tS + HT * (j % C::NB), x[0]);
            tmem_ld32(tS + HT * (j % C::NB) + 32, x[1]);
        };
        // step j, whose scores are s; those of the next step are fetched into `next`
        auto step = [&](int j, float (&s)[2][32], float (&next)[2][32]) {
            tmem_wait_ld();
            if (j >= jd) {
                const int c0 = HT * (j - jd);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c0 + 32 * x + i > r) s[x][i] = -INFINITY;
            }
            float mx[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                mx[x] = fmaxf(s[x][0], s[x][1]);
#pragma unroll
                for (int i = 2; i < 32; i += 2) mx[x] = max3(mx[x], s[x][i], s[x][i + 1]);
            }
            const float top = fmaxf(mx[0], mx[1]);
            const bool move = (top - m) * scale2 > 8.f;  // also from -inf
            if (__any_sync(0xffffffffu, move)) {
                const float to = move ? top : m;
                const float f = move ? ex2_approx((m - to) * scale2) : 1.f;
                m = to;
                l *= f;
                if (j > 0) {  // once O is at rest
                    w.wait_warp(&bar[C::pv_done + 2 * t + ((j - 1) & 1)], (j - 1) >> 1);
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        float o[32];
                        tmem_ld32(tO + 32 * x, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= f;
                        tmem_st32(tO + 32 * x, o);
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.f : m * scale2;
            const uint64_t sc2 = pack2(scale2, scale2), ms2 = pack2(-ms, -ms);
            uint64_t sum[2] = {0, 0};
            float p[32];  // 64 weights, two bf16 each
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float a, b;
                unpack2(fma2(pack2(s[i >> 4][2 * (i & 15)], s[i >> 4][2 * (i & 15) + 1]), sc2, ms2), a, b);
                a = ex2_approx(a);
                b = ex2_approx(b);
                sum[i & 1] = add2(sum[i & 1], pack2(a, b));
                p[i] = __uint_as_float(pack_bf16x2(a, b));
            }
            tmem_st32(tS + HT * (j % C::NB), p);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar[C::p_full + C::NB * t + j % C::NB], lane);
            float a, b;
            unpack2(add2(sum[0], sum[1]), a, b);
            l += a + b;
            if (j + 1 < n) fetch(j + 1, next);
        };
        if (n > 0) {
            float x[2][32], y[2][32];
            fetch(0, x);
            for (int j = 0; j < n && !w.stopped(); j += 2) {
                step(j, x, y);
                if (j + 1 < n) step(j + 1, y, x);
            }
            w.wait_warp(&bar[C::all_done + t], 0);
            tc_fence_after();
            if (!w.stopped()) {
                const int64_t row0 = at.t0 + q0 + t * BT;
                store_rows<D, D>(tO, 1.f / l, sm + C::Q + t * C::TILE, wq, lane, 0, out + (row0 * Hq + h) * D,
                                 (int64_t)Hq * D, rows - t * BT);
                if (lse && r < rows - t * BT) lse[(row0 + r) * Hq + h] = fmaf(m, scale2, log2f(l)) * kLn2;
            }
        }
    }
    if (w.aborted() && warp == 10 && lane == 0)  // copies in flight end before the CTA does
        for (int i = C::q_full; i < C::v_zeroed; ++i)
            if (i < C::k_empty || (i >= C::v_full && i < C::v_empty)) {
                mbar_wait_bounded(&bar[i], 0, 1000000ull);
                mbar_wait_bounded(&bar[i], 1, 1000000ull);
            }
    tc_fence_before();
    __syncthreads();
    if (warp == 11) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t run_fwd(const AttnArgs &a, cudaStream_t st)
{
    using C = FwdCfg<D>;
    const int64_t tokens = a.cu ? (int64_t)a.T : (int64_t)a.B * a.T;
    cudaError_t e = cudaFuncSetAttribute(attn_fwd_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::TOTAL);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, a.q, tokens, a.Hq, D) || !make_map(&mk, a.k, tokens, a.Hk, D) || !make_map(&mv, a.v, tokens, a.Hk, D))
        return cudaErrorInvalidValue;
    const long tiles = attn_tiles(a.cu, a.B, a.T, 2 * BT);
    attn_fwd_tc<D><<<(unsigned)(tiles * a.Hq), NTH, C::TOTAL, st>>>(mq, mk, mv, static_cast<__nv_bfloat16 *>(a.out), a.lse,
                                                                   a.cu, FastDiv(a.B), a.T, FastDiv(a.Hq), FastDiv(a.Hq / a.Hk),
                                                                   a.scale * kLog2e);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t st)
{
    return a.d == 128 ? run_fwd<128>(a, st) : run_fwd<64>(a, st);
}

int read_and_clear_attn_fwd_error()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_fwd_error, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_attn_fwd_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
