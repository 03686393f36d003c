// gdn_attn_decode.cu -- one-token softmax attention over a paged e4m3 cache with one scale per
// (page, head).
//
// Per (request, key head): s_j = scale q . (ks_j K8_j), out = sum_j softmax_j(s) vs_j V8_j over the
// request's cached tokens, for the G query heads that share the key head.  HBM bounds it: 2 d bytes
// per token and key head against 4 G d flops.  The cache is therefore read once for up to 16 query
// heads by warp-level MMAs (m16n8k16, fp16 operands, fp32 accumulators): the cached bytes, converted to fp16
// (exact) in registers, are their A operands (16 tokens of K; 16 elements of V, transposed), and 8 heads their N
// columns, so that few heads leave little idle: conversions are made once for all heads, and with up to 8 of them
// half the MMAs and exponentials of a layout with heads as rows do (256 contexts of up to 8192 tokens, 4 heads on
// one: 301 us, with heads as rows 334).  The 128-row tcgen05 shape, which would pad G rows to 128 and need the bytes converted through shared
// memory, has nothing to give here.
//
// Each warp runs alone: it takes every fourth 32-token tile of its CTA's range through its own ring
// of TMA loads (K and V tiles of 32 rows, swizzled), keeps its own running maximum, sum and output
// (online softmax), and the four warps join at the end.  A long context is split over CTAs whose
// partial results a second kernel joins.
//
// The weights' frame: p_j = 2^15 exp2(s_j + log2 vs_j - M), M the least whole number at or above every
// s_j + log2 vs_j, so that p_j V8_j needs no further scale; the softmax sum takes p_j / vs_j.  p_j is rounded to fp16
// for the product (a half step of 2^-11 against bf16's 2^-8, and V8 must be fp16 beside it), and in an fp32 call to
// the sum of two fp16 (2^-22).  2^15 uses all of fp16's range: the largest weight lies in (2^14, 2^15], and what
// falls below fp16's normal numbers is off by 2^-39 of it at most; with the largest at 1 that floor was 2^-25, and
// 8192 tokens behind one that has 2^26 times the weight of each and a value of 0 came out 6e-2 off (now 4.8e-6 in fp32
// calls, 1.7e-3 in bf16 calls).
// M is whole so that moving it (powers of two) and taking 15 from it are exact.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "gdn_attn.h"
#include "gdn_tmap.h"
#include "sm100_ptx.cuh"
#include "../../include/gdn.h"

namespace gdn {

using namespace sm100;

__device__ int g_attn_decode_error = 0;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TT = 32;    // tokens per tile
constexpr int NW = 4;     // warps per CTA
constexpr int NSTG = 2;   // ring stages per warp
constexpr int OCC = 3;    // CTAs per SM: while one starts (a chain of dependent loads) the others stream (256 ragged
                          // contexts: 301 us; with two CTAs of three stages 319)
constexpr int JW = 16;    // warps of the join
constexpr float kFrame = 15.f;  // log2 of the largest weight in its frame (above)
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 in the low half -> two fp16
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w)
{
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// (page, head)-contiguous cache [pages][Hk][page][d] bytes: rows y.. of head z of page w
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int y, int z, int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// Tiles of a context (its length may be close to 2^31)
__device__ __forceinline__ int context_tiles(int len) { return len > 0 ? (len - 1) / TT + 1 : 0; }

// Tiles per split of a context of `len` tokens over at most `n` splits; those past its end are empty.
__device__ __forceinline__ int split_tiles(int len, int n)
{
    return max(1, (context_tiles(len) + n - 1) / n);
}

__device__ __forceinline__ int context_len(const int32_t *lens, int n, int max_blocks, int page)
{
    return (int)max(0LL, min((long long)lens[n], (long long)max_blocks * page));
}

// Requests in order of their lengths, the longest first, so that a launch of more CTAs than there are places does
// not end with a long context alone: the request of a rank, found by every CTA for itself from all lengths
// (at most kOrdered), in classes a quarter of a power of two wide and by number within a class.  It costs a
// CTA about a microsecond, so contexts that cannot be long stay in order of number (8 key heads, d 128: 256 contexts of
// 128 to 8192 tokens 301 us by length, 324 by number; 64 of up to 2000 33 and 38; 256 of up to 1000 67 and 61).
constexpr int kOrdered = 512, kOrderedFrom = 2048;  // requests, tokens
__device__ __forceinline__ int request_of_rank(const int32_t *lens, int N, int max_blocks, int page, int rank)
{
    constexpr int NR = kOrdered / (NW * 32), CL = 128;
    static_assert(CL == NW * 32 && NR * NW <= 32, "a class a thread, four a lane; a count a lane");
    __shared__ __align__(16) int s_count[CL];
    __shared__ int s_here[32], s_request;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len[NR], cl[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const int i = tid + NW * 32 * j;
        len[j] = i < N ? context_len(lens, i, max_blocks, page) : -1;
    }
    s_count[tid] = 0;
    if (tid < 32) s_here[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j) {  // the float's exponent and two bits of its fraction; class 0 are the longest
        cl[j] = len[j] < 0 ? -1 : CL - 1 - (len[j] ? (int)(__float_as_uint((float)len[j]) >> 21) - (127 << 2) : 0);
        if (cl[j] >= 0) atomicAdd(&s_count[cl[j]], 1);
    }
    __syncthreads();
    // every warp: the class of this rank, and the rank within it
    auto scan = [&](int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    const int4 c = reinterpret_cast<const int4 *>(s_count)[lane];
    const int sum = c.x + c.y + c.z + c.w;
    int k = rank - (scan(sum) - sum);  // within the lane's four classes
    const int src = __ffs(__ballot_sync(0xffffffffu, k >= 0 && k < sum)) - 1;
    int want = 4 * lane;
    if (k >= c.x) {
        k -= c.x, ++want;
        if (k >= c.y) {
            k -= c.y, ++want;
            if (k >= c.z) k -= c.z, ++want;
        }
    }
    want = __shfl_sync(0xffffffffu, want, src);
    k = __shfl_sync(0xffffffffu, k, src);
    // the k-th request of the class
    unsigned in[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        in[j] = __ballot_sync(0xffffffffu, cl[j] == want);
        if (lane == 0) s_here[NW * j + warp] = __popc(in[j]);
    }
    __syncthreads();
    const int here = s_here[lane], before = scan(here) - here;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const int at = __shfl_sync(0xffffffffu, before, NW * j + warp) + __popc(in[j] & ((1u << lane) - 1));
        if ((in[j] >> lane & 1) && at == k) s_request = tid + NW * 32 * j;
    }
    __syncthreads();
    return s_request;
}

// Partial results lie in the workspace as [request x query head][split][d + 4]: o, then m and l of the
// frame above (two floats unused).

template <bool F32> __device__ __forceinline__ void store_out(void *out, int64_t at, float4 x)
{
    if (F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = x;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + at) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

template <int D> __host__ __device__ constexpr int stage_bytes() { return 2 * TT * D; }
template <int D> __host__ __device__ constexpr int ring_bytes() { return NW * NSTG * stage_bytes<D>(); }
// What a stage's tile needs besides its bytes, for its tokens 0-15 and 16-31: its pages' key scale, log2 and
// reciprocal of the value scale; one below 0 marks tokens that are left out.
struct alignas(32) TileInfo {
    float ks0, ks1, lg0, lg1, iv0, iv1;
};

// behind the ring: the stages' info, barriers, then the warps' (m, l) for the join
template <int D> __host__ __device__ constexpr int decode_smem()
{
    return 1024 + ring_bytes<D>() + NW * NSTG * ((int)sizeof(TileInfo) + 8) + NW * 16 * 8;
}

// bf16 calls in groups of 8 heads or, with more than 8 on a key head, of 16; fp32 calls in groups of 8, q and the weights
// as sums of two fp16.
enum { kHeads8, kHeads16, kFloat };

// 8 x 8 of 16 bits, transposed: thread (g, c) gives row g, columns 2c and 2c + 1, and gets column g, rows 2c and 2c + 1
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int D, int KIND>
__global__ void __launch_bounds__(NW * 32, OCC)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const AttnDecodeArgs a, int splits, int mtiles, int ordered)
{
    constexpr bool F32 = KIND == kFloat;
    constexpr int NA = KIND == kHeads16 ? 2 : 1;  // groups of 8 heads
    constexpr int NQ = KIND == kHeads8 ? 1 : 2;   // B operands of q: the groups, or q's two parts
    constexpr int MH = 8 * NA;                    // heads of a CTA
    constexpr int KS = D / 16;        // k steps of the score product
    constexpr int ND = D / 16;        // row tiles of the value product
    constexpr int NG = D / 32;        // 4-byte words of a V row per thread
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    unsigned char *ring = sm + warp * NSTG * stage_bytes<D>();
    TileInfo *info = reinterpret_cast<TileInfo *>(sm + ring_bytes<D>()) + warp * NSTG;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + ring_bytes<D>() + NW * NSTG * sizeof(TileInfo)) + warp * NSTG;
    float2 *s_ml = reinterpret_cast<float2 *>(sm + ring_bytes<D>() + NW * NSTG * (sizeof(TileInfo) + 8));

    int idx = blockIdx.x;
    const int split = idx % splits;
    idx /= splits;
    const int mt = idx % mtiles;
    idx /= mtiles;
    const int hk = idx % a.Hk;
    const int n = ordered ? request_of_rank(a.lens, a.N, a.max_blocks, a.page, idx / a.Hk) : idx / a.Hk;
    const int G = a.Hq / a.Hk;
    const int len = context_len(a.lens, n, a.max_blocks, a.page);
    const int per = split_tiles(len, splits);
    const int t0 = (int)min((long long)split * per * TT, (long long)len);
    const int t1 = (int)min(t0 + (long long)per * TT, (long long)len);
    asm volatile("griddepcontrol.launch_dependents;");  // the join waits for this grid's end
    if (t0 >= t1 && split > 0) return;  // split 0 writes the zeros of an empty context

    if (lane == 0) {
        for (int i = 0; i < NSTG; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    __syncwarp();

    const int shift = __ffs(a.page) - 1;
    const int tiles = context_tiles(t1 - t0);           // of this CTA; warp w takes tiles w, w + 4, ...
    const int mine = tiles > warp ? (tiles - warp + NW - 1) / NW : 0;
    const int32_t *table = a.table + (int64_t)n * a.max_blocks;
    const bool small = a.page < TT;

    // Page numbers and scales of 32 own tiles, one tile a lane (two pages where a page has 16
    // tokens), with the next 32 fetched while these are worked on, so that the chain table -> scale
    // is waited for once.
    int pg0, pg1, npg0 = -1, npg1 = -1;
    float nks0 = 0.f, nks1 = 0.f, nvs0 = 0.f, nvs1 = 0.f;
    TileInfo own;
    auto take_scales = [&]() {
        own = TileInfo{nks0, nks1, log2f(nvs0), log2f(nvs1), 1.f / nvs0, 1.f / nvs1};
    };
    auto fetch_pages = [&](int i0, int &p0, int &p1) {
        p0 = p1 = -1;
        if (i0 + lane < mine) {
            const int tok = t0 + (warp + NW * (i0 + lane)) * TT;
            p0 = table[tok >> shift];
            if (small) p1 = tok + 16 < t1 ? table[(tok >> shift) + 1] : -1;
        }
        if (p0 < 0 || p0 >= a.num_pages) p0 = -1;
        if (p1 < 0 || p1 >= a.num_pages) p1 = -1;
        if (!small) p1 = p0;
    };
    auto fetch_scales = [&](int p0, int p1, float &k0, float &k1, float &v0, float &v1) {
        k0 = k1 = v0 = v1 = -1.f;
        if (p0 >= 0) {
            k0 = a.k_scale[(int64_t)p0 * a.Hk + hk];
            v0 = fmaxf(a.v_scale[(int64_t)p0 * a.Hk + hk], 0x1p-60f);
        }
        if (!small) {
            k1 = k0;
            v1 = v0;
        } else if (p1 >= 0) {
            k1 = a.k_scale[(int64_t)p1 * a.Hk + hk];
            v1 = fmaxf(a.v_scale[(int64_t)p1 * a.Hk + hk], 0x1p-60f);
        }
    };
    // Loads of own tile i, in order.  Every tile brings 2 TT D bytes; page 0 stands in for a page
    // out of range, whose tokens are left out.
    auto load = [&](int i) {
        const int at = i & 31;
        if (at == 0 && i > 0) {
            pg0 = npg0, pg1 = npg1;
            take_scales();
        }
        const int p0 = max(__shfl_sync(0xffffffffu, pg0, at), 0), p1 = max(__shfl_sync(0xffffffffu, pg1, at), 0);
        if (lane == 0) {
            unsigned char *st = ring + (i % NSTG) * stage_bytes<D>();
            uint64_t *b = &bar[i % NSTG];
            mbar_arrive_expect_tx(b, stage_bytes<D>());
            const int tok = t0 + (warp + NW * i) * TT;
            const int y = tok & (a.page - 1);
            tma_load_4d(st, &tmK, b, y, hk, p0);
            tma_load_4d(st + TT * D, &tmV, b, y, hk, p0);
            if (small) {
                tma_load_4d(st + 16 * D, &tmK, b, 0, hk, p1);
                tma_load_4d(st + TT * D + 16 * D, &tmV, b, 0, hk, p1);
            }
        }
    };
    // The scales of tile i, behind its loads: they come from memory as its bytes do.
    auto note = [&](int i) {
        const int at = i & 31;
        if (lane == at) info[i % NSTG] = own;
        if (at == 8) fetch_pages(i - 8 + 32, npg0, npg1);
        if (at == 20) fetch_scales(npg0, npg1, nks0, nks1, nvs0, nvs1);
    };
    fetch_pages(0, pg0, pg1);
    int issued = 0;
    for (; issued < NSTG && issued < mine; ++issued) load(issued);
    fetch_scales(pg0, pg1, nks0, nks1, nvs0, nvs1);
    take_scales();
    for (int i = 0; i < issued; ++i) note(i);
    __syncwarp();

    // ---- q as B operands; thread (g, c) holds heads g and g + 8 and, at k step ks, the four d values of its 16-byte
    // chunks of a K row: chunk 2c + i (D = 128) or c (D = 64), word e, ks = 4 i + e ----
    uint32_t qb[NQ][KS][2];
    float unscale[NA][2];  // score = accumulated x unscale x ks, heads 2c and 2c + 1 of a group
    {
        const int h0 = mt * MH + g, h1 = F32 ? h0 : h0 + 8;
        const bool on0 = h0 < G, on1 = KIND == kHeads16 && h1 < G;
        const int64_t r0 = ((int64_t)n * a.Hq + hk * G + h0) * D, r1 = ((int64_t)n * a.Hq + hk * G + h1) * D;
        float x0[KS][4], x1[KS][4];
        float mx0 = 0.f, mx1 = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d0 = 16 * (D == 128 ? 2 * c + (ks >> 2) : c) + 4 * (ks & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) x0[ks][j] = x1[ks][j] = 0.f;
            if (F32) {
                const float *q = static_cast<const float *>(a.q);
                if (on0) {
                    const float4 w = *reinterpret_cast<const float4 *>(q + r0 + d0);
                    x0[ks][0] = w.x, x0[ks][1] = w.y, x0[ks][2] = w.z, x0[ks][3] = w.w;
                }
            } else {
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
                if (on0) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(q + r0 + d0);
                    x0[ks][0] = __uint_as_float(w.x << 16), x0[ks][1] = __uint_as_float(w.x & 0xffff0000u);
                    x0[ks][2] = __uint_as_float(w.y << 16), x0[ks][3] = __uint_as_float(w.y & 0xffff0000u);
                }
                if (on1) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(q + r1 + d0);
                    x1[ks][0] = __uint_as_float(w.x << 16), x1[ks][1] = __uint_as_float(w.x & 0xffff0000u);
                    x1[ks][2] = __uint_as_float(w.y << 16), x1[ks][3] = __uint_as_float(w.y & 0xffff0000u);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mx0 = fmaxf(mx0, fabsf(x0[ks][j]));
                mx1 = fmaxf(mx1, fabsf(x1[ks][j]));
            }
        }
        // a power of two for each head brings its largest |q| into [256, 512): fp16 then holds values down
        // to 2^-22 of it with full precision, whatever the other heads hold
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        auto exponent = [](float mx) {
            return mx > 0.f ? max(-126, min((int)(__float_as_uint(mx) >> 23) - 127 - 8, 126)) : 0;
        };
        auto two_to = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
        const int e0 = exponent(mx0), e1 = exponent(mx1);
        const float down0 = two_to(-e0), down1 = two_to(-e1);
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)  // thread (h, 0) knows head h's
                unscale[i][e] = two_to(__shfl_sync(0xffffffffu, i ? e1 : e0, 4 * (2 * c + e))) * a.scale * kLog2e;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x0[ks][j] *= down0;
                x1[ks][j] *= down1;
            }
            if (F32) {  // the second part: what fp16 rounding left over
#pragma unroll
                for (int j = 0; j < 4; ++j) x1[ks][j] = x0[ks][j] - __half2float(__float2half_rn(x0[ks][j]));
            }
            qb[0][ks][0] = pack_half(x0[ks][0], x0[ks][1]);
            qb[0][ks][1] = pack_half(x0[ks][2], x0[ks][3]);
            if (NQ == 2) {
                qb[NQ - 1][ks][0] = pack_half(x1[ks][0], x1[ks][1]);
                qb[NQ - 1][ks][1] = pack_half(x1[ks][2], x1[ks][3]);
            }
        }
    }

    // o[i][4 rows of V^T, 2 heads]: tile 2x + t, register 2u + e: d = 4 (g + 8 x) + 2 t + u, head 2c + e of group i
    float o[NA][ND][4], m[NA][2], l[NA][2];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int x = 0; x < ND; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][x][j] = 0.f;
    }
    // D = 64: a thread with odd c reads its token pairs in the other order (bank conflicts, below)
    const uint32_t sel_lo = (D == 64 && (c & 1)) ? 0x1504u : 0x5140u, sel_hi = (D == 64 && (c & 1)) ? 0x3726u : 0x7362u;
    const int odd = D == 64 ? (c & 1) : 0;
    bool dead = false;
    int done = 0;

    for (int i = 0; i < mine; ++i, ++done) {
        unsigned char *kt = ring + (i % NSTG) * stage_bytes<D>(), *vt = kt + TT * D;
        if (!mbar_wait_bounded(&bar[i % NSTG], (i / NSTG) & 1, kWaitNs)) {
            if (lane == 0) atomicOr(&g_attn_decode_error, 1);
            dead = true;
            break;
        }
        const int tok = t0 + (warp + NW * i) * TT;
        const int live = min(TT, t1 - tok);
        const TileInfo ti = info[i % NSTG];
        const float iA = ti.iv0, iB = ti.iv1;
        const bool onA = !(iA < 0.f), onB = !(iB < 0.f);
        // V rows that are not part of the context may hold any byte, NaN among them: zero them,
        // since a weight of 0 times NaN is NaN
        const bool partial = live < TT || !onA || !onB;
        if (partial) {
            for (int r = 0; r < TT; ++r)
                if (r >= live || !(r < 16 ? onA : onB))
                    for (int w = lane; w < D / 4; w += 32) reinterpret_cast<uint32_t *>(vt + r * D)[w] = 0u;
            __syncwarp();
        }
        // ---- scores: 2 x 16 tokens x 8 heads: register 2u + e of tile t is token 16 t + 8 u + g, head 2c + e ----
        float s[NA][2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int x = 0; x < NA; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][t][e] = 0.f;
            const int row = 16 * t + g;
#pragma unroll
            for (int i2 = 0; i2 < D / 64; ++i2) {
                // the swizzle XORs the 16-byte chunk with the row (D = 128) or row pair (D = 64):
                // the eight threads of a phase then read eight different chunk columns
                const int ch = D == 128 ? ((2 * c + i2) ^ (row & 7)) : (c ^ ((row >> 1) & 3));
                const uint4 w = *reinterpret_cast<const uint4 *>(kt + row * D + ch * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(kt + (row + 8) * D + ch * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int ks = 4 * i2 + e;
                    const uint32_t a0 = cvt_lo(ww[e]), a1 = cvt_lo(yy[e]), a2 = cvt_hi(ww[e]), a3 = cvt_hi(yy[e]);
#pragma unroll
                    for (int x = 0; x < NQ; ++x) mma_f16(s[x % NA][t], a0, a1, a2, a3, qb[x][ks][0], qb[x][ks][1]);
                }
            }
        }
        // ---- softmax weights ----
        // (the lanes' maxima are joined only where one of them passes the running one)
        float mx[NA][2];
        bool up = false;
#pragma unroll
        for (int x = 0; x < NA; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float fA = unscale[x][e] * ti.ks0, fB = unscale[x][e] * ti.ks1;
                mx[x][e] = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const bool on = (t ? onB : onA) && 16 * t + 8 * u + g < live;
                        float &y = s[x][t][2 * u + e];
                        y = on ? fmaf(y, t ? fB : fA, t ? ti.lg1 : ti.lg0) : -INFINITY;
                        mx[x][e] = fmaxf(mx[x][e], y);
                    }
                up |= mx[x][e] > m[x][e];
            }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int x = 0; x < NA; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int b = 4; b < 32; b <<= 1) mx[x][e] = fmaxf(mx[x][e], __shfl_xor_sync(0xffffffffu, mx[x][e], b));
                    const float to = fmaxf(m[x][e], ceilf(mx[x][e]));
                    const float f = to == -INFINITY ? 1.f : ex2_approx(m[x][e] - to);
                    m[x][e] = to;
                    l[x][e] *= f;
#pragma unroll
                    for (int i3 = 0; i3 < ND; ++i3) {
                        o[x][i3][e] *= f;
                        o[x][i3][2 + e] *= f;
                    }
                }
        }
        uint32_t pb[NQ][2][2];  // weights as B operands of 16 tokens: the groups, or the weights' two parts
#pragma unroll
        for (int x = 0; x < NA; ++x) {
            const float b0 = m[x][0] == -INFINITY ? 0.f : m[x][0] - kFrame, b1 = m[x][1] == -INFINITY ? 0.f : m[x][1] - kFrame;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float y0 = ex2_approx(s[x][t][2 * u] - b0), y1 = ex2_approx(s[x][t][2 * u + 1] - b1);
                    l[x][0] = fmaf(y0, t ? iB : iA, l[x][0]);
                    l[x][1] = fmaf(y1, t ? iB : iA, l[x][1]);
                    const uint32_t w = pack_half(y0, y1);
                    pb[x][t][u] = transposed(w);
                    if (F32) {
                        const __half2 hi = *reinterpret_cast<const __half2 *>(&w);
                        pb[NQ - 1][t][u] = transposed(pack_half(y0 - __low2float(hi), y1 - __high2float(hi)));
                    }
                }
        }
        // ---- o += V^T p: k = 16 tokens a step; thread (g, c) reads words g + 8 x of the rows 2c, 2c + 1,
        // 2c + 8, 2c + 9; bytes 2 t and 2 t + 1 of a word are rows g and g + 8 of tile 2 x + t ----
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                uint32_t w[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // D = 64 packs two rows into 128 bytes; odd c swaps the rows of a pair so that a
                    // phase's rows fall into both halves
                    const int row = 16 * k2 + 2 * c + ((r & 1) ^ odd) + 8 * (r >> 1);
                    const int ch = (g >> 2) + 2 * x;
                    const int pos = D == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
                    w[r] = *reinterpret_cast<const uint32_t *>(vt + row * D + pos * 16 + 4 * (g & 3));
                }
                // bytes of two tokens side by side: (token 2c, token 2c + 1) of each d
                const uint32_t u0 = __byte_perm(w[0], w[1], sel_lo), u1 = __byte_perm(w[0], w[1], sel_hi);
                const uint32_t z0 = __byte_perm(w[2], w[3], sel_lo), z1 = __byte_perm(w[2], w[3], sel_hi);
                const uint32_t a0 = cvt_lo(u0), a1 = cvt_hi(u0), a2 = cvt_lo(z0), a3 = cvt_hi(z0);
                const uint32_t c0 = cvt_lo(u1), c1 = cvt_hi(u1), c2 = cvt_lo(z1), c3 = cvt_hi(z1);
#pragma unroll
                for (int y = 0; y < NQ; ++y) {
                    mma_f16(o[y % NA][2 * x], a0, a1, a2, a3, pb[y][k2][0], pb[y][k2][1]);
                    mma_f16(o[y % NA][2 * x + 1], c0, c1, c2, c3, pb[y][k2][0], pb[y][k2][1]);
                }
            }
        }
        if (partial) fence_proxy_async_smem();  // the zeros, before the stage's next bytes
        __syncwarp();                           // every lane has read the stage
        if (issued < mine) {
            load(issued);
            note(issued++);
        }
        __syncwarp();
    }
    if (dead)  // copies in flight end before the CTA does
        for (int i = done; i < issued; ++i) mbar_wait_bounded(&bar[i % NSTG], (i / NSTG) & 1, kWaitNs);

    // ---- the four warps join through shared memory (their rings are free now) ----
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], x);
    __syncthreads();
    float *so = reinterpret_cast<float *>(sm) + warp * MH * D;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * i + 2 * c + e;
            if (g == 0) s_ml[warp * 16 + r] = make_float2(m[i][e], l[i][e]);
#pragma unroll
            for (int x = 0; x < NG; ++x)
                *reinterpret_cast<float4 *>(so + r * D + 4 * (g + 8 * x)) =
                    make_float4(o[i][2 * x][e], o[i][2 * x][2 + e], o[i][2 * x + 1][e], o[i][2 * x + 1][2 + e]);
        }
    __syncthreads();
    const float *all = reinterpret_cast<const float *>(sm);
    for (int i = tid; i < MH * (D / 4); i += NW * 32) {
        const int r = i / (D / 4), d0 = 4 * (i % (D / 4)), h = mt * MH + r;
        if (h >= G) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w * 16 + r].x);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 ml = s_ml[w * 16 + r];
            const float f = M == -INFINITY ? 1.f : ex2_approx(ml.x - M);
            const float4 y = *reinterpret_cast<const float4 *>(all + (w * MH + r) * D + d0);
            L = fmaf(f, ml.y, L);
            x.x = fmaf(f, y.x, x.x);
            x.y = fmaf(f, y.y, x.y);
            x.z = fmaf(f, y.z, x.z);
            x.w = fmaf(f, y.w, x.w);
        }
        const int64_t row = (int64_t)n * a.Hq + hk * G + h;
        if (splits > 1) {
            float *ws = static_cast<float *>(a.workspace) + (row * splits + split) * (D + 4);
            *reinterpret_cast<float4 *>(ws + d0) = x;
            if (d0 == 0) *reinterpret_cast<float2 *>(ws + D) = make_float2(M, L);
        } else {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            store_out<F32>(a.out, row * D + d0, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        }
    }
}

// Joins the splits of one (request, query head): out = sum_s e_s o_s / sum_s e_s l_s, e_s =
// exp2(m_s - max m).  One CTA a row; warp w takes splits w, w + JW, ...
template <int D, bool F32>
__global__ void __launch_bounds__(JW * 32) attn_decode_join(const AttnDecodeArgs a, int splits)
{
    constexpr int E = D / 32;  // elements of a row per lane
    __shared__ float s_o[JW][D];
    __shared__ float s_l[JW];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int len = context_len(a.lens, (int)(row / a.Hq), a.max_blocks, a.page);
    const int per = split_tiles(len, splits), used = max(1, (context_tiles(len) + per - 1) / per);
    const float *ws = static_cast<const float *>(a.workspace) + row * splits * (D + 4);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float M = -INFINITY;
    for (int s = lane; s < used; s += 32) M = fmaxf(M, ws[(int64_t)s * (D + 4) + D]);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    float o[E], L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int s = warp; s < used; s += JW) {
        const float *w = ws + (int64_t)s * (D + 4);
        const float2 ml = *reinterpret_cast<const float2 *>(w + D);
        const float f = M == -INFINITY ? 1.f : ex2_approx(ml.x - M);
        L = fmaf(f, ml.y, L);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f, w[lane + 32 * e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = o[e];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (threadIdx.x < D / 4) {
        const int d0 = 4 * threadIdx.x, n = min(used, JW);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        L = 0.f;
        for (int w = 0; w < n; ++w) {
            const float4 y = *reinterpret_cast<const float4 *>(&s_o[w][d0]);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            L += s_l[w];
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        store_out<F32>(a.out, row * D + d0, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    }
}

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    return n;
}

int kind_of(int G, int dtype) { return dtype == GDN_DTYPE_F32 ? kFloat : G > 8 ? kHeads16 : kHeads8; }
int head_tiles(int G, int dtype)
{
    const int mh = kind_of(G, dtype) == kHeads16 ? 16 : 8;
    return (G + mh - 1) / mh;
}

// Splits of a context.  A CTA starts with a chain of dependent loads, some 5 us, so splits beyond need cost:
// - few (request, key head) pairs: one CTA for each place on the SMs, down to a tile a warp (one context of
//   65536 tokens, 4 key heads, its cache in L2: 19.3 us in 111 splits, 20.4 in 55, 26 in 27, 25 in 222; now 18.1 in 111,
//   and 22.5 from HBM; of 4096: 7.2 us in 32 splits, 8.2 in 27);
// - more: about 1.5 for each place, down to two tiles a warp (contexts of 128 to 8192 tokens, 8 key heads: 16 of
//   them 34.7 us in 6 splits, 37.9 in 8, 34.8 in 4; 32 of them 56.4 in 3, 59.7 in 4, 57.9 in 2);
// - pairs for all places: two splits only where they leave 16 tiles a warp (64 contexts of 128 to 8192 tokens, 8
//   key heads: 109 us in 2, 103 in 1; of up to 32768: 306 and 357; of up to 2000: 47 and 33).
int split_count(int N, int Hk, int mtiles, int page, int max_blocks)
{
    const long tiles = ((long)max_blocks * page + TT - 1) / TT;
    const long units = (long)N * Hk * mtiles, places = (long)OCC * sm_count();
    const bool few = units * 16 <= places;
    const long s = few ? places / units : (3 * places / 2 + units - 1) / units;
    const long most = few ? tiles / NW : tiles / ((units < places ? 2 : 16) * NW);
    return (int)(s > most ? (most < 1 ? 1 : most) : (s < 1 ? 1 : s));
}

bool cache_map(CUtensorMap *m, const void *base, int num_pages, int Hk, int page, int d)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)Hk, (cuuint64_t)num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)d, (cuuint64_t)d * page, (cuuint64_t)d * page * Hk};
    const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)(page < TT ? page : TT), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND> cudaError_t run_decode(const AttnDecodeArgs &a, cudaStream_t st)
{
    const int mtiles = head_tiles(a.Hq / a.Hk, a.dtype);
    const int splits = split_count(a.N, a.Hk, mtiles, a.page, a.max_blocks);
    constexpr int smem = decode_smem<D>();
    auto kern = attn_decode_kernel<D, KIND>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    CUtensorMap mk, mv;
    if (!cache_map(&mk, a.k_cache, a.num_pages, a.Hk, a.page, D) || !cache_map(&mv, a.v_cache, a.num_pages, a.Hk, a.page, D))
        return cudaErrorInvalidValue;
    const long ctas = (long)a.N * a.Hk * mtiles * splits;
    const int ordered = a.N > 1 && a.N <= kOrdered && (long)a.max_blocks * a.page >= kOrderedFrom && ctas > (long)OCC * sm_count();
    kern<<<(unsigned)ctas, NW * 32, smem, st>>>(mk, mv, a, splits, mtiles, ordered);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    // the join's CTAs may be set up while the last ones above run; they wait for all of them
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * a.Hq));
    cfg.blockDim = dim3(JW * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_decode_join<D, KIND == kFloat>, a, splits);
}

}  // namespace

size_t attn_decode_workspace_bytes(int N, int Hq, int Hk, int d, int page, int max_blocks, int dtype)
{
    const int splits = split_count(N, Hk, head_tiles(Hq / Hk, dtype), page, max_blocks);
    return splits == 1 ? 0 : (size_t)N * Hq * splits * (d + 4) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t st)
{
    switch (kind_of(a.Hq / a.Hk, a.dtype)) {
        case kHeads8: return a.d == 128 ? run_decode<128, kHeads8>(a, st) : run_decode<64, kHeads8>(a, st);
        case kHeads16: return a.d == 128 ? run_decode<128, kHeads16>(a, st) : run_decode<64, kHeads16>(a, st);
        default: return a.d == 128 ? run_decode<128, kFloat>(a, st) : run_decode<64, kFloat>(a, st);
    }
}

int read_and_clear_attn_decode_error()
{
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_decode_error, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_attn_decode_error, &z, sizeof(int));
    return v;
}

}  // namespace gdn
