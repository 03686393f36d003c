// gdn_attn_tc_bwd.cu -- gradients of causal softmax attention on the tcgen05 tensor cores (bf16).
//
//   P = exp(scale Q K^T - lse),  dP = dO V^T,  dS = P (dP - D),  D_i = dO_i . O_i
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two launches.  The query side holds a block of 128 query rows and passes over its key blocks (S, dP
// and dQ: three products a step); the key side holds a block of 128 keys and passes over the query
// heads that share them and their query blocks (S^T, dP^T, dV, dK: four products a step).  S and dP
// are formed twice (seven products where one kernel would need five), and in return every gradient is
// summed in tensor memory by one CTA in one order: no atomics, no partial sums in HBM, a call repeats
// bit for bit.
//
// D from the rounded result is off by up to 2^-8 sum |dO| |O|, which counts where dS is small beside D: a row of few keys, or
// of values that lie near one another.  The first kExactBlocks query blocks of a sequence, where rows have few keys,
// therefore form D as sum_j P_ij dP_ij in a pass of their own (for every block that would be a pass of two products more
// than the three of the query side); behind them D is taken from out as it was rounded.  The query side writes D and
// -lse log2 e for the key side, head by head ([Hq][tokens] each), into the workspace.
// P and dS are rounded to bf16 for their products: both operands of a product have one type, and Q, K and dO are bf16.
// Gradients are off by 2.3e-3 (relative, root mean square), 1.7e-3 of it from their own rounding.
//
// Both kernels work in steps of 64 keys (query side) or 64 queries (key side): 128 x 64 tiles of S and
// dP in tensor memory beside the gradients, two of each at d = 128 (2 x 64 + 2 x 64 + 256 columns) and three at
// d = 64, so that the products of the next steps run while a step's elements are worked on.  What bounds them is
// the chain of waits between products and elements: at d = 64 (16384 tokens, 16 heads) the query side, when it took
// 0.88 ms (0.82 now), took 0.80 without its exponentials, 0.75 without any product, and still 0.53 without both and
// the rest of the element-wise work.  Steps of 128 with one dP (or, on the key side, one S) tile spend half their time on it, and
// half again as many element-wise warps change nothing.
// A product 64 wide of two shared operands takes 48 cycles for 32 cycles' work, so the query side moves Q and dO
// to tensor memory.  The key side leaves K and V in shared memory: at d = 64 a third tile of S and dP gives more
// (8 x 4096 tokens, 12 heads on 4: 412 us, with K and V in their place 455), at d = 128 there is no room (with K
// there and one dP tile a step takes 1920 cycles, with two dP tiles 1640).
// A CTA's start and end cost some 5 us (setting up, the first loads, a chain of products and elements with nothing
// beside it, the results), a quarter of its time at 4096 tokens; CTAs that take one tile after another
// instead of being launched anew were no faster.
// 16384 tokens, 16 heads on 4: query side 1.17 ms at d = 128 and 0.82 at d = 64, key side 1.64 and 1.00 ms.
//   warps 0-7, 8-15  element by element, the even and the odd steps: a thread has a row, 32 columns
//   warps 16-18      issue the products (key side: 16-19; one product a warp, since its waits and commits
//                    take longer than the product)
//   warp 19 (20)     loads; zeroes rows behind the sequence's end
// P and dS (bf16) are written over the first half of the very S or dP columns they came from, which
// their own thread has read.
#include <math.h>

#include "gdn_attn_tc.cuh"
#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {

__device__ int g_attn_bwd_error = 0;

namespace {

using namespace attn;

constexpr int NTH = 640, NTH_KEY = 768;
constexpr int NEL = 512;         // threads of the element-wise warps
constexpr int HT = 64;           // rows of the other side a step
constexpr int kHalf = HT * 128;  // bytes from a tile's first half to its second (in each sub-tile)
constexpr int kExactBlocks = 2;

// N tiles in tensor memory that the steps take in turn, step i tile i % N.  Even and odd steps belong to
// different warps, and a warp that passes over phases of a barrier cannot tell them by parity: so each barrier
// belongs to steps of one parity, and with three tiles there are six.
template <int N> struct Turns {
    static constexpr int TILES = N, BARS = N % 2 ? 2 * N : N;
    __device__ __forceinline__ static int tile(int i) { return i % N; }
    __device__ __forceinline__ static int bar(int i) { return i % BARS; }
    __device__ __forceinline__ static int phase(int i) { return i / BARS; }
    // the same for the steps of one parity, counted up
    int b, ph = 0;
    __device__ __forceinline__ explicit Turns(int first) : b(first) {}
    __device__ __forceinline__ int tile() const { return N == 2 ? b : b >= N ? b - N : b; }
    __device__ __forceinline__ void next()
    {
        if (N == 2) {
            ++ph;
        } else if ((b += 2) >= BARS) {
            b -= BARS;
            ++ph;
        }
    }
};

// D[128 x D] (+)= A B over a step's 64 rows of B: A (bf16) in two chunks of 32 columns (16 of tensor
// memory) that lie 32 apart
template <int D>
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, const unsigned char *b, bool accumulate)
{
    constexpr uint32_t id = idesc_bf16(BT, D, 0, 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        mma_ts(d, a + 32 * (kk >> 1) + 8 * (kk & 1), sdesc_sw128(smem_u32(b) + kk * 2048, kSub, 1024), id,
               accumulate || kk > 0);
}

__device__ __forceinline__ void named_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// After a wait ran out: copies in flight end before the CTA does.
__device__ __forceinline__ void drain_loads(uint64_t *bar, int first, int count)
{
    for (int i = first; i < first + count; ++i) {
        mbar_wait_bounded(&bar[i], 0, 1000000ull);
        mbar_wait_bounded(&bar[i], 1, 1000000ull);
    }
}

// ---- query side ------------------------------------------------------------------------------------

// A K stage is held from the scores to dQ, a V stage only for dP: with two K stages of d = 128 every
// load would be waited for.
template <int D> struct DqCfg {
    static constexpr int NK = D == 64 ? 4 : 3, NV = D == 64 ? 4 : 2;
    using TS = Turns<D == 64 ? 3 : 2>;  // tiles of S
    using TP = Turns<D == 64 ? 3 : 2>;  // tiles of dP
    static constexpr bool BOTH = TS::TILES == 3;  // both tiles of a step are there when it begins
    static constexpr int TILE = BT * D * 2;
    static constexpr int Q = 0, O = TILE, K = 2 * TILE, V = K + NK * TILE, RED = V + NV * TILE, BAR = RED + 2 * BT * 4;
    static constexpr int q_full = 0;               // Q and dO
    static constexpr int k_full = 1;               // [NK]
    static constexpr int v_full = k_full + NK;     // [NV]
    static constexpr int k_empty = v_full + NV;    // [NK]
    static constexpr int v_empty = k_empty + NK;   // [NV]
    static constexpr int k_zeroed = v_empty + NV;  // [NK] the stage has no row behind the end (ragged ends only)
    static constexpr int v_zeroed = k_zeroed + NK; // [NV]
    static constexpr int s_full = v_zeroed + NV;        // [TS] one a turn: S (BOTH: S and dP)
    static constexpr int dp_full = s_full + TS::BARS;   // [TP] dP
    static constexpr int s_free = dp_full + TP::BARS;   // [TS] S has been read
    static constexpr int ds_full = s_free + TS::BARS;   // [TP] dS is there (first pass: dP has been read)
    static constexpr int dq_done = ds_full + TP::BARS;  // [TP] dS has been used
    static constexpr int a_full = dq_done + TP::BARS;   // Q and dO are in tensor memory
    static constexpr int all_done = a_full + 1;    // dQ is there (a barrier of one phase: a warp that
                                                   // passes over phases cannot tell them by parity)
    static constexpr int drain = all_done + 1;     // [3]
    static constexpr int NBAR = drain + 3;
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int TOTAL = 1024 + MISC + 16;
    static constexpr uint32_t tS = 0, tP = HT * TS::TILES, tG = tP + HT * TP::TILES, tQ = tG + D, tO = tQ + D / 2;
    static_assert(tO + D / 2 <= 512, "tensor memory budget");
    static_assert(TOTAL <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(NTH, 1)
    attn_bwd_dq_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                   const __nv_bfloat16 *__restrict__ out, const float *__restrict__ lse, __nv_bfloat16 *__restrict__ dq,
                   float *__restrict__ nlse, float *__restrict__ ndot, const int32_t *__restrict__ cu, FastDiv B, int T,
                   FastDiv heads, FastDiv group, float scale, int64_t tokens)
{
    using C = DqCfg<D>;
    using TS = typename C::TS;
    using TP = typename C::TP;
    constexpr int NK = C::NK, NV = C::NV;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    int *abort_flag = reinterpret_cast<int *>(sm + C::MISC + 4);
    float *red = reinterpret_cast<float *>(sm + C::RED);
    const Waits w{abort_flag, &g_attn_bwd_error};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int Hq = (int)heads.d, index = heads.div(blockIdx.x);
    const AttnTile at = attn_tile(cu, B, T, BT, index);
    if (at.seq < 0) return;
    const int h = blockIdx.x - index * Hq, hk = group.div(h);
    const int rows = at.len - at.block * BT;       // that exist
    const int n = (min(at.len, (at.block + 1) * BT) + HT - 1) / HT;  // steps of a pass
    const int nt = (n + 1) / 2;                    // key tiles of a pass
    const bool exact = at.block < kExactBlocks;
    const int passes = exact ? 2 : 1, steps = passes * n;  // the first of two passes forms D
    const int64_t row0 = at.t0 + at.block * BT;

    auto load_k = [&](int i, int j) {
        const int s = i % NK;
        mbar_arrive_expect_tx(&bar[C::k_full + s], C::TILE);
        load_tile<D>(sm + C::K + s * C::TILE, &tmK, &bar[C::k_full + s], hk, (int)at.t0 + j * BT);
    };
    auto load_v = [&](int i, int j) {
        const int s = i % NV;
        mbar_arrive_expect_tx(&bar[C::v_full + s], C::TILE);
        load_tile<D>(sm + C::V + s * C::TILE, &tmV, &bar[C::v_full + s], hk, (int)at.t0 + j * BT);
    };
    if (warp == 19) {  // the first loads are under way before the rest is set up
        for (int i = lane; i < C::NBAR; i += 32)
            mbar_init(&bar[i], i == C::a_full ? NEL / 32 : i >= C::s_free && i < C::dq_done ? NEL / 64  // one a warp
                               : C::BOTH && i >= C::s_full && i < C::dp_full ? 2 : 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            *abort_flag = 0;
            mbar_arrive_expect_tx(&bar[C::q_full], 2 * C::TILE);
            load_tile<D>(sm + C::Q, &tmQ, &bar[C::q_full], h, (int)row0);
            load_tile<D>(sm + C::O, &tmO, &bar[C::q_full], h, (int)row0);
            load_k(0, 0);
            load_v(0, 0);
        }
        __syncwarp();
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // registers: 640 x 96 = 61440 at launch; 128 x 56 + 512 x 104 = 60416 after the two roles' changes
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 19) {
            for (int i = 0; i < passes * nt; ++i) {
                const int sk = i % NK, sv = i % NV, j = i % nt;
                if (lane == 0 && i > 0) {
                    if (i >= NK) w.wait(&bar[C::k_empty + sk], i / NK - 1);
                    if (!w.aborted()) load_k(i, j);
                    if (i >= NV) w.wait(&bar[C::v_empty + sv], i / NV - 1);
                    if (!w.aborted()) load_v(i, j);
                }
                __syncwarp();
                if (w.stopped()) break;
                if (rows < BT) {
                    if (j == nt - 1) {
                        w.wait(&bar[C::k_full + sk], i / NK);
                        w.wait(&bar[C::v_full + sv], i / NV);
                        if (w.stopped()) break;
                        zero_rows<D>(sm + C::K + sk * C::TILE, rows, lane);
                        zero_rows<D>(sm + C::V + sv * C::TILE, rows, lane);
                    }
                    if (lane == 0) {
                        arrive(&bar[C::k_zeroed + sk]);
                        arrive(&bar[C::v_zeroed + sv]);
                    }
                }
            }
        } else if (warp == 16) {  // S
            w.wait(&bar[C::a_full], 0);
            for (int p = 0, i = 0; p < passes; ++p)
                for (int s = 0; s < n && !w.stopped(); ++s, ++i) {
                    const int j = p * nt + (s >> 1);
                    if (!(s & 1)) {
                        w.wait(&bar[C::k_full + j % NK], j / NK);
                        if (rows < BT) w.wait(&bar[C::k_zeroed + j % NK], j / NK);
                    }
                    if (i >= TS::TILES) w.wait(&bar[(C::BOTH ? C::ds_full : C::s_free) + TS::bar(i - TS::TILES)], TS::phase(i - TS::TILES));
                    tc_fence_after();
                    mma_nt_ta<D, HT>(tmem + C::tS + HT * TS::tile(i), tmem + C::tQ, sm + C::K + (j % NK) * C::TILE + (s & 1) * kHalf);
                    commit(&bar[C::s_full + TS::bar(i)]);
                }
        } else if (warp == 17) {  // dP
            w.wait(&bar[C::a_full], 0);
            for (int p = 0, i = 0; p < passes; ++p)
                for (int s = 0; s < n && !w.stopped(); ++s, ++i) {
                    const int j = p * nt + (s >> 1);
                    if (!(s & 1)) {
                        w.wait(&bar[C::v_full + j % NV], j / NV);
                        if (rows < BT) w.wait(&bar[C::v_zeroed + j % NV], j / NV);
                    }
                    if (i >= TP::TILES) w.wait(&bar[C::dq_done + TP::bar(i - TP::TILES)], TP::phase(i - TP::TILES));
                    tc_fence_after();
                    mma_nt_ta<D, HT>(tmem + C::tP + HT * TP::tile(i), tmem + C::tO, sm + C::V + (j % NV) * C::TILE + (s & 1) * kHalf);
                    commit(&bar[(C::BOTH ? C::s_full : C::dp_full) + TP::bar(i)]);
                    if ((s & 1) || s == n - 1) commit(&bar[C::v_empty + j % NV]);
                }
        } else {  // dQ
            for (int p = 0, i = 0; p < passes; ++p)
                for (int s = 0; s < n && !w.stopped(); ++s, ++i) {
                    const int j = p * nt + (s >> 1);
                    w.wait(&bar[C::ds_full + TP::bar(i)], TP::phase(i));
                    tc_fence_after();
                    if (p == passes - 1)
                        mma_step<D>(tmem + C::tG, tmem + C::tP + HT * TP::tile(i),
                                    sm + C::K + (j % NK) * C::TILE + (s & 1) * kHalf, s > 0);
                    commit(&bar[C::dq_done + TP::bar(i)]);
                    if ((s & 1) || s == n - 1) commit(&bar[C::k_empty + j % NK]);
                }
            commit(&bar[C::all_done]);
        }
        if (warp < 19 && w.stopped()) {  // products issued already end before the tensor memory is freed
            commit(&bar[C::drain + warp - 16]);
            mbar_wait_bounded(&bar[C::drain + warp - 16], 0, 100000000ull);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int g = warp >> 2, wq = warp & 3, r = tid & (BT - 1);
        const int set = g >> 1, c0 = 32 * (g & 1);  // steps of this parity, these columns
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const bool live = r < rows;
        const float nl = live ? -lse[(row0 + r) * Hq + h] * kLog2e : 0.f;
        float nd = 0.f;
        // D from out: a warp has 8 rows, D / 8 lanes a row
        constexpr int LR = D / 8;
        uint4 ov[D / 32];
        const int ro = 8 * warp + lane / LR, un = lane % LR;
        if (!exact) {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
                const int x = ro + u * (32 / LR);
                if (x < rows) ov[u] = *(reinterpret_cast<const uint4 *>(out + ((row0 + x) * Hq + h) * D) + un);
            }
        }
        w.wait_warp(&bar[C::q_full], 0);  // groups 0, 1: halves of Q's rows, 2, 3: of dO's
        row_to_tmem<D / 2>(tmem + lanes + (g < 2 ? C::tQ : C::tO), sm + (g < 2 ? C::Q : C::O), r, (g & 1) * (D / 2));
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bar[C::a_full], lane);
        auto known = [&]() {  // for the key side too
            if (g == 0 && live) {
                nlse[(int64_t)h * tokens + row0 + r] = nl;
                ndot[(int64_t)h * tokens + row0 + r] = nd;
            }
        };
        if (!exact) {
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
                const int x = ro + u * (32 / LR);
                float acc = 0.f;
                if (x < rows) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(sm + C::O + (un >> 3) * kSub + x * 128 + (((un & 7) ^ (x & 7)) << 4));
                    const uint32_t av[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc = fmaf(__uint_as_float(av[e] << 16), -__uint_as_float(bv[e] << 16), acc);
                        acc = fmaf(__uint_as_float(av[e] & 0xffff0000u), -__uint_as_float(bv[e] & 0xffff0000u), acc);
                    }
                }
#pragma unroll
                for (int o = LR / 2; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
                if (un == 0) red[x] = acc;
            }
            named_bar(1, NEL);
            nd = red[r];
            known();
        }
        auto join = [&]() {  // the four parts of D from the first pass
            if (g >= 2) red[(g - 2) * BT + r] = nd;
            named_bar(1, NEL);
            if (g < 2) red[g * BT + r] += nd;
            named_bar(1, NEL);
            nd = red[r] + red[BT + r];
            known();
        };
        bool joined = !exact;
        const uint64_t sc2 = pack2(scale * kLog2e, scale * kLog2e), nl2 = pack2(nl, nl);
        TS ts(set);
        TP tp(set);
        for (int i = set; i < steps; i += 2, ts.next(), tp.next()) {
            if (!joined && i >= n) {
                join();
                joined = true;
            }
            const uint64_t nd2 = pack2(nd, nd);
            const int key0 = (i < n ? i : i - n) * HT + c0 - at.block * BT;  // of this thread's columns, as r counts
            const uint32_t tS = tmem + lanes + C::tS + HT * ts.tile() + c0, tP = tmem + lanes + C::tP + HT * tp.tile() + c0;
            float s[32], dp[32];
            w.wait_warp(&bar[C::s_full + ts.b], ts.ph);
            tc_fence_after();
            tmem_ld32(tS, s);
            if (C::BOTH) tmem_ld32(tP, dp);
            tmem_wait_ld();
            if (!C::BOTH) {
                tc_fence_before();
                warp_arrive(&bar[C::s_free + ts.b], lane);
            }
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                unpack2(fma2(pack2(s[x], s[x + 1]), sc2, nl2), s[x], s[x + 1]);
                s[x] = ex2_approx(s[x]);
                s[x + 1] = ex2_approx(s[x + 1]);
            }
            if (key0 >= 0) {  // the diagonal block
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (key0 + x > r) s[x] = 0.f;
            }
            if (!C::BOTH) {
                w.wait_warp(&bar[C::dp_full + tp.b], tp.ph);
                tc_fence_after();
                tmem_ld32(tP, dp);
                tmem_wait_ld();
            }
            if (exact && i < n) {
                uint64_t acc = 0;
#pragma unroll
                for (int x = 0; x < 32; x += 2) acc = fma2(pack2(s[x], s[x + 1]), pack2(dp[x], dp[x + 1]), acc);
                float a, b;
                unpack2(acc, a, b);
                nd -= a + b;
            } else {
                uint32_t ds[16];
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    float a, b;
                    unpack2(mul2(pack2(s[x], s[x + 1]), add2(pack2(dp[x], dp[x + 1]), nd2)), a, b);
                    ds[x >> 1] = pack_bf16x2(a, b);
                }
                tmem_st16(tP, ds);
                tmem_wait_st();
            }
            tc_fence_before();
            warp_arrive(&bar[C::ds_full + tp.b], lane);
        }
        if (!joined) join();  // no step in the second pass, or left early: the other warps still come by
        if (!w.stopped()) {
            w.wait_warp(&bar[C::all_done], 0);
            tc_fence_after();
            if (!w.stopped() && g < 2)
                store_rows<D, D / 2>(tmem + lanes + C::tG, scale, sm + C::Q, wq, lane, g * (D / 2),
                                     dq + (row0 * Hq + h) * D, (int64_t)Hq * D, rows);
        }
    }
    if (w.aborted() && warp == 19 && lane == 0) drain_loads(bar, C::q_full, 1 + NK + NV);
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- key side ----------------------------------------------------------------------------------------

template <int D> struct DkvCfg {
    static constexpr int NS = D == 64 ? 4 : 2;
    using TS = Turns<D == 64 ? 3 : 2>;  // tiles of S^T
    using TP = Turns<D == 64 ? 3 : 2>;  // tiles of dP^T
    static constexpr int TILE = BT * D * 2;
    static constexpr int K = 0, V = TILE, Q = 2 * TILE, O = Q + NS * TILE, ST = O + NS * TILE, BAR = ST + NS * 2 * BT * 4;
    static constexpr int kv_full = 0;
    static constexpr int q_full = 1;               // [NS] Q, and -lse log2 e and -D of its rows
    static constexpr int o_full = q_full + NS;     // [NS] dO
    static constexpr int empty = o_full + NS;      // [NS] dV and dK have used the stage
    static constexpr int zeroed = empty + NS;      // [NS] the stage has no row behind the end (ragged ends only)
    static constexpr int s_full = zeroed + NS;          // [TS] one a turn:
    static constexpr int dp_full = s_full + TS::BARS;   // [TP]
    static constexpr int p_full = dp_full + TP::BARS;   // [TS] P^T is there
    static constexpr int ds_full = p_full + TS::BARS;   // [TP] dS^T is there
    static constexpr int dv_done = ds_full + TP::BARS;  // [TS] P^T has been used
    static constexpr int dk_done = dv_done + TS::BARS;  // [TP] dS^T has been used
    static constexpr int all_done = dk_done + TP::BARS; // dV and dK are there
    static constexpr int drain = all_done + 1;     // [4]
    static constexpr int NBAR = drain + 4;
    static constexpr int MISC = BAR + NBAR * 8;
    static constexpr int TOTAL = 1024 + MISC + 16;
    static constexpr uint32_t tS = 0, tP = HT * TS::TILES, tGV = tP + HT * TP::TILES, tGK = tGV + D;
    static_assert(tGK + D <= 512, "tensor memory budget");
    static_assert(TOTAL <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(NTH_KEY, 1)
    attn_bwd_dkv_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                    const float *__restrict__ nlse, const float *__restrict__ ndot, __nv_bfloat16 *__restrict__ dk,
                    __nv_bfloat16 *__restrict__ dv, const int32_t *__restrict__ cu, FastDiv B, int T, FastDiv heads, int G,
                    float scale, int64_t tokens)
{
    using C = DkvCfg<D>;
    using TS = typename C::TS;
    using TP = typename C::TP;
    constexpr int NS = C::NS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::MISC);
    int *abort_flag = reinterpret_cast<int *>(sm + C::MISC + 4);
    const Waits w{abort_flag, &g_attn_bwd_error};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int Hk = (int)heads.d, index = heads.div(blockIdx.x);
    const AttnTile at = attn_tile(cu, B, T, BT, index);
    if (at.seq < 0) return;
    const int hk = blockIdx.x - index * Hk;
    const int blocks = (at.len + BT - 1) / BT;
    const int kb = blocks - 1 - at.block;          // the first key blocks see the most queries
    const int n = (at.len - kb * BT + HT - 1) / HT;  // steps per head
    const int nt = blocks - kb;                    // query tiles per head
    const int steps = G * n;
    const int rows = at.len - kb * BT;             // keys that exist
    const int tail = at.len - (blocks - 1) * BT;   // queries of the last block
    const int64_t row0 = at.t0 + kb * BT;

    if (warp == 20) {  // the first loads are under way before the rest is set up
        for (int i = lane; i < C::NBAR; i += 32) {
            int c = 1;
            if (i >= C::q_full && i < C::o_full) c = 1 + 32;
            if (i >= C::p_full && i < C::dv_done) c = NEL / 64;  // one a warp
            if ((i >= C::empty && i < C::zeroed) || i == C::all_done) c = 2;  // dV and dK
            mbar_init(&bar[i], c);
        }
        fence_mbar_init();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            *abort_flag = 0;
            mbar_arrive_expect_tx(&bar[C::kv_full], 2 * C::TILE);
            load_tile<D>(sm + C::K, &tmK, &bar[C::kv_full], hk, (int)row0);
            load_tile<D>(sm + C::V, &tmV, &bar[C::kv_full], hk, (int)row0);
            mbar_arrive_expect_tx(&bar[C::q_full], C::TILE);
            load_tile<D>(sm + C::Q, &tmQ, &bar[C::q_full], hk * G, (int)row0);
            mbar_arrive_expect_tx(&bar[C::o_full], C::TILE);
            load_tile<D>(sm + C::O, &tmO, &bar[C::o_full], hk * G, (int)row0);
        }
        __syncwarp();
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // registers: 768 x 80 = 61440 at launch; 512 x 96 + 256 x 48 = 61440 after the roles' changes (warps
    // 21-23 are there because registers are dealt out by four warps)
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 20) {
            for (int i = 0; i < G * nt; ++i) {
                const int s = i % NS, h = hk * G + i / nt, qb = kb + i % nt;
                if (i >= NS) w.wait(&bar[C::empty + s], i / NS - 1);
                if (w.stopped()) break;
                const int64_t q0 = at.t0 + qb * BT;
                if (lane == 0 && i > 0) {
                    mbar_arrive_expect_tx(&bar[C::q_full + s], C::TILE);
                    load_tile<D>(sm + C::Q + s * C::TILE, &tmQ, &bar[C::q_full + s], h, (int)q0);
                    mbar_arrive_expect_tx(&bar[C::o_full + s], C::TILE);
                    load_tile<D>(sm + C::O + s * C::TILE, &tmO, &bar[C::o_full + s], h, (int)q0);
                }
                // rows behind the end get 0, 0: a weight of 1 on a row of zeros
                float *st = reinterpret_cast<float *>(sm + C::ST) + s * 2 * BT;
                const int live = qb == blocks - 1 ? tail : BT;
#pragma unroll
                for (int x = lane; x < BT; x += 32) {
                    const int64_t o = (int64_t)h * tokens + q0 + min(x, live - 1);
                    cp_async_4(st + x, nlse + o, x < live ? 4u : 0u);
                    cp_async_4(st + BT + x, ndot + o, x < live ? 4u : 0u);
                }
                cp_async_mbar_arrive(&bar[C::q_full + s]);
                if (qb == blocks - 1 && tail < BT) {
                    w.wait(&bar[C::q_full + s], i / NS);
                    w.wait(&bar[C::o_full + s], i / NS);
                    if (w.stopped()) break;
                    zero_rows<D>(sm + C::Q + s * C::TILE, tail, lane);
                    zero_rows<D>(sm + C::O + s * C::TILE, tail, lane);
                }
                if (tail < BT && lane == 0) arrive(&bar[C::zeroed + s]);
                __syncwarp();
            }
        } else if (warp == 16) {  // S^T
            w.wait(&bar[C::kv_full], 0);
            for (int g = 0, i = 0; g < G; ++g)
                for (int x = 0; x < n && !w.stopped(); ++x, ++i) {
                    const int j = g * nt + (x >> 1), s = j % NS;
                    if (i >= TS::TILES) w.wait(&bar[C::dv_done + TS::bar(i - TS::TILES)], TS::phase(i - TS::TILES));
                    if (!(x & 1)) {
                        w.wait(&bar[C::q_full + s], j / NS);
                        if (tail < BT) w.wait(&bar[C::zeroed + s], j / NS);
                    }
                    tc_fence_after();
                    mma_nt<D, HT>(tmem + C::tS + HT * TS::tile(i), sm + C::K, sm + C::Q + s * C::TILE + (x & 1) * kHalf);
                    commit(&bar[C::s_full + TS::bar(i)]);
                }
        } else if (warp == 17) {  // dP^T
            w.wait(&bar[C::kv_full], 0);
            for (int g = 0, i = 0; g < G; ++g)
                for (int x = 0; x < n && !w.stopped(); ++x, ++i) {
                    const int j = g * nt + (x >> 1), s = j % NS;
                    if (i >= TP::TILES) w.wait(&bar[C::dk_done + TP::bar(i - TP::TILES)], TP::phase(i - TP::TILES));
                    if (!(x & 1)) {
                        w.wait(&bar[C::o_full + s], j / NS);
                        if (tail < BT) w.wait(&bar[C::zeroed + s], j / NS);
                    }
                    tc_fence_after();
                    mma_nt<D, HT>(tmem + C::tP + HT * TP::tile(i), sm + C::V, sm + C::O + s * C::TILE + (x & 1) * kHalf);
                    commit(&bar[C::dp_full + TP::bar(i)]);
                }
        } else if (warp == 18) {  // dV
            for (int g = 0, i = 0; g < G; ++g)
                for (int x = 0; x < n && !w.stopped(); ++x, ++i) {
                    const int j = g * nt + (x >> 1), s = j % NS;
                    if (!(x & 1)) {
                        w.wait(&bar[C::o_full + s], j / NS);
                        if (tail < BT) w.wait(&bar[C::zeroed + s], j / NS);
                    }
                    w.wait(&bar[C::p_full + TS::bar(i)], TS::phase(i));
                    tc_fence_after();
                    mma_step<D>(tmem + C::tGV, tmem + C::tS + HT * TS::tile(i), sm + C::O + s * C::TILE + (x & 1) * kHalf, i > 0);
                    commit(&bar[C::dv_done + TS::bar(i)]);
                    if ((x & 1) || x == n - 1) commit(&bar[C::empty + s]);
                }
            commit(&bar[C::all_done]);
        } else if (warp == 19) {  // dK
            for (int g = 0, i = 0; g < G; ++g)
                for (int x = 0; x < n && !w.stopped(); ++x, ++i) {
                    const int s = (g * nt + (x >> 1)) % NS;
                    w.wait(&bar[C::ds_full + TP::bar(i)], TP::phase(i));
                    tc_fence_after();
                    mma_step<D>(tmem + C::tGK, tmem + C::tP + HT * TP::tile(i), sm + C::Q + s * C::TILE + (x & 1) * kHalf, i > 0);
                    commit(&bar[C::dk_done + TP::bar(i)]);
                    if ((x & 1) || x == n - 1) commit(&bar[C::empty + s]);
                }
            commit(&bar[C::all_done]);
        }
        if (warp < 20 && w.stopped()) {  // products issued already end before the tensor memory is freed
            commit(&bar[C::drain + warp - 16]);
            mbar_wait_bounded(&bar[C::drain + warp - 16], 0, 100000000ull);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        const int g = warp >> 2, wq = warp & 3, r = tid & (BT - 1);  // r: key row
        const int set = g >> 1, c0 = 32 * (g & 1);  // steps of this parity, these columns
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint64_t sc2 = pack2(scale * kLog2e, scale * kLog2e);
        TS ts(set);
        TP tp(set);
        int x0 = set, j0 = 0;  // step of a head's, and the head's first tile
        for (int i = set; i < steps; i += 2, x0 += 2, ts.next(), tp.next()) {
            for (; x0 >= n; x0 -= n) j0 += nt;
            const int j = j0 + (x0 >> 1), s = j % NS;
            const float *st = reinterpret_cast<const float *>(sm + C::ST) + s * 2 * BT + (x0 & 1) * HT + c0;
            const uint32_t tS = tmem + lanes + C::tS + HT * ts.tile() + c0, tP = tmem + lanes + C::tP + HT * tp.tile() + c0;
            float p[32], dp[32];
            w.wait(&bar[C::s_full + ts.b], ts.ph);
            w.wait_warp(&bar[C::q_full + s], j / NS);  // over by now: for the rows' -lse and -D
            tc_fence_after();
            tmem_ld32(tS, p);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                const float4 nl = *reinterpret_cast<const float4 *>(st + x);
                unpack2(fma2(pack2(p[x], p[x + 1]), sc2, pack2(nl.x, nl.y)), p[x], p[x + 1]);
                unpack2(fma2(pack2(p[x + 2], p[x + 3]), sc2, pack2(nl.z, nl.w)), p[x + 2], p[x + 3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) p[x + e] = ex2_approx(p[x + e]);
            }
            if (x0 < 2) {  // the diagonal block: queries before the key
                const int q0 = x0 * HT + c0;
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (q0 + x < r) p[x] = 0.f;
            }
            {
                uint32_t pk[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) pk[x] = pack_bf16x2(p[2 * x], p[2 * x + 1]);
                tmem_st16(tS, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar[C::p_full + ts.b], lane);
            w.wait_warp(&bar[C::dp_full + tp.b], tp.ph);
            tc_fence_after();
            tmem_ld32(tP, dp);
            tmem_wait_ld();
            uint32_t ds[16];
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                const float4 nd = *reinterpret_cast<const float4 *>(st + BT + x);
                float a, b;
                unpack2(mul2(pack2(p[x], p[x + 1]), add2(pack2(dp[x], dp[x + 1]), pack2(nd.x, nd.y))), a, b);
                ds[x >> 1] = pack_bf16x2(a, b);
                unpack2(mul2(pack2(p[x + 2], p[x + 3]), add2(pack2(dp[x + 2], dp[x + 3]), pack2(nd.z, nd.w))), a, b);
                ds[(x >> 1) + 1] = pack_bf16x2(a, b);
            }
            tmem_st16(tP, ds);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bar[C::ds_full + tp.b], lane);
        }
        if (!w.stopped()) {
            w.wait_warp(&bar[C::all_done], 0);
            tc_fence_after();
            if (!w.stopped()) {  // groups 0 and 1 store dV, 2 and 3 dK
                __nv_bfloat16 *to = (g >= 2 ? dk : dv) + (row0 * Hk + hk) * D;
                store_rows<D, D / 2>(tmem + lanes + (g >= 2 ? C::tGK : C::tGV), g >= 2 ? scale : 1.f,
                                     sm + (g >= 2 ? C::K : C::V), wq, lane, (g & 1) * (D / 2), to, (int64_t)Hk * D, rows);
            }
        }
    }
    if (w.aborted() && warp == 20) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0) drain_loads(bar, C::kv_full, 1 + 2 * NS);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D> cudaError_t run_bwd(const AttnArgs &a, cudaStream_t st)
{
    using A = DqCfg<D>;
    using Bc = DkvCfg<D>;
    const int64_t tokens = a.cu ? (int64_t)a.T : (int64_t)a.B * a.T;
    cudaError_t e = cudaFuncSetAttribute(attn_bwd_dq_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, A::TOTAL);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_bwd_dkv_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Bc::TOTAL);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv, mo;
    if (!make_map(&mq, a.q, tokens, a.Hq, D) || !make_map(&mk, a.k, tokens, a.Hk, D) ||
        !make_map(&mv, a.v, tokens, a.Hk, D) || !make_map(&mo, a.dout, tokens, a.Hq, D))
        return cudaErrorInvalidValue;
    float *nlse = static_cast<float *>(a.workspace), *ndot = nlse + tokens * a.Hq;
    const long tiles = attn_tiles(a.cu, a.B, a.T, BT);
    const int G = a.Hq / a.Hk;
    attn_bwd_dq_tc<D><<<(unsigned)(tiles * a.Hq), NTH, A::TOTAL, st>>>(
        mq, mk, mv, mo, static_cast<const __nv_bfloat16 *>(a.out), a.lse, static_cast<__nv_bfloat16 *>(a.dq), nlse, ndot,
        a.cu, FastDiv(a.B), a.T, FastDiv(a.Hq), FastDiv(G), a.scale, tokens);
    attn_bwd_dkv_tc<D><<<(unsigned)(tiles * a.Hk), NTH_KEY, Bc::TOTAL, st>>>(
        mq, mk, mv, mo, nlse, ndot, static_cast<__nv_bfloat16 *>(a.dk), static_cast<__nv_bfloat16 *>(a.dv), a.cu, FastDiv(a.B),
        a.T, FastDiv(a.Hk), G, a.scale, tokens);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_tc(const AttnArgs &a, cudaStream_t st)
{
    return a.d == 128 ? run_bwd<128>(a, st) : run_bwd<64>(a, st);
}

int read_and_clear_attn_bwd_error()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_bwd_error, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_attn_bwd_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
