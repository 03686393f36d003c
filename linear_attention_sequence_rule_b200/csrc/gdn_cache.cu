// gdn_cache.cu -- the paged 8-bit cache of the attention layers: one step's plan (block table,
// slots, positions) from request lengths, and the write of new keys and values.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "gdn_attn.h"
#include "../../include/gdn.h"

namespace gdn {

namespace cg = cooperative_groups;

namespace {

// ---- plan ----------------------------------------------------------------------------------------
//
// Integers only: with held_r = ceil(lens_r / page) and want_r = ceil((lens_r + added_r) / page),
// exclusive prefix sums over the requests give the first row cu_r of each request's new tokens and
// the first entry first_r of the free list it takes; block b >= held_r of request r is
// free_list[head + first_r + b - held_r], and token t of request r has position lens_r + t - cu_r.
//
// The work is a few kilobytes: launch and memory latency bound it.  One cluster of 8 CTAs; every CTA
// forms the prefix sums of all requests in its own shared memory (reading N numbers again from L2
// costs less than a second launch), and after a cluster barrier, behind which no input is read that
// an output may overwrite, the CTAs share the writes.

constexpr int PT = 1024;  // threads per CTA
constexpr int PC = 8;     // CTAs of the cluster

struct Sum2 {
    long long rows, pages;
};

__device__ __forceinline__ Sum2 warp_scan(Sum2 x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x.rows, o), b = __shfl_up_sync(0xffffffffu, x.pages, o);
        if (lane >= o) {
            x.rows += a;
            x.pages += b;
        }
    }
    return x;
}

__global__ void __cluster_dims__(PC, 1, 1) __launch_bounds__(PT) cache_plan_kernel(const CachePlanArgs a)
{
    extern __shared__ int32_t sh[];
    int32_t *s_cu = sh;             // [N + 1]
    int32_t *s_first = sh + a.N + 1;  // [N]
    int32_t *s_lens = s_first + a.N;  // [N]
    __shared__ Sum2 s_warp[PT / 32];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x;
    const int gid = rank * PT + tid;
    if (tid == 0) s_bad = 0x7fffffff;
    __syncthreads();
    const int head = a.free_head[0];
    const long long room = (long long)a.max_blocks * a.page;
    const int shift = __ffs(a.page) - 1;
    Sum2 base = {0, 0};
    for (int r0 = 0; r0 < a.N; r0 += PT) {
        const int r = r0 + tid;
        Sum2 x = {0, 0};
        int len = 0, held = 0;
        if (r < a.N) {
            len = a.lens[r];
            const int add = a.added[r];
            if (len < 0 || add < 0 || (long long)len + add > room) {
                atomicMin(&s_bad, r);
                len = 0;
            } else {
                held = (int)(((long long)len + a.page - 1) >> shift);
                x.rows = add;
                x.pages = (int)(((long long)len + add + a.page - 1) >> shift) - held;
            }
        }
        const Sum2 incl = warp_scan(x, lane);
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const Sum2 w = warp_scan(s_warp[lane], lane);
            s_warp[lane] = w;
        }
        __syncthreads();
        Sum2 ex = {base.rows + incl.rows - x.rows, base.pages + incl.pages - x.pages};
        if (warp > 0) {
            ex.rows += s_warp[warp - 1].rows;
            ex.pages += s_warp[warp - 1].pages;
        }
        if (r < a.N) {  // a plan whose sums pass 32 bits is refused below
            s_cu[r] = (int32_t)ex.rows;
            s_first[r] = (int32_t)ex.pages;
            s_lens[r] = len;
        }
        base.rows += s_warp[PT / 32 - 1].rows;
        base.pages += s_warp[PT / 32 - 1].pages;
        __syncthreads();
    }
    if (tid == 0) s_cu[a.N] = (int32_t)base.rows;
    int code = 0, detail = 0;
    if (head < 0 || head > a.num_free) {
        code = 4;
    } else if (s_bad != 0x7fffffff) {
        code = 2;
        detail = s_bad;
    } else if (base.rows > a.rows) {
        code = 3;
        detail = (int)min(base.rows - a.rows, 0x7fffffffLL);
    } else if (base.pages > a.num_free - head) {
        code = 1;
        detail = (int)min(base.pages - (a.num_free - head), 0x7fffffffLL);
    }
    // lens_out and free_head_out may be lens and free_head: every CTA has read them behind this.
    // lens is read once more below (refused plans) only by the thread that writes lens_out[r].
    cg::this_cluster().sync();
    if (gid == 0) {
        a.free_head_out[0] = code ? head : head + (int)base.pages;
        a.status[0] = code;
        a.status[1] = detail;
    }
    if (code) {
        for (int r = gid; r <= a.N; r += PC * PT) {
            a.cu[r] = 0;
            if (r < a.N) a.lens_out[r] = a.lens[r];
        }
        for (int t = gid; t < a.rows; t += PC * PT) {
            a.slots[t] = -1;
            a.positions[t] = -1;
        }
        return;
    }
    const int total = s_cu[a.N];
    for (int r = gid; r <= a.N; r += PC * PT) {
        a.cu[r] = s_cu[r];
        if (r < a.N) a.lens_out[r] = s_lens[r] + s_cu[r + 1] - s_cu[r];
    }
    // new table entries: a warp per request
    for (int r = rank * (PT / 32) + warp; r < a.N; r += PC * (PT / 32)) {
        const int n = (r + 1 < a.N ? s_first[r + 1] : (int)base.pages) - s_first[r];
        const int held = (int)(((long long)s_lens[r] + a.page - 1) >> shift);
        for (int i = lane; i < n; i += 32)
            a.table[(int64_t)r * a.max_blocks + held + i] = a.free_list[head + s_first[r] + i];
    }
    // slots and positions: four rows a thread, the first row's request by binary search
    for (int t0 = 4 * gid; t0 < a.rows; t0 += 4 * PC * PT) {
        int slot[4], pos[4];
        int lo = 0, hi = a.N;  // s_cu[lo] <= t0 < s_cu[hi] where t0 < total
        if (t0 < total)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t0) lo = mid; else hi = mid;
            }
        int block = -1, page_no = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = t0 + e;
            slot[e] = pos[e] = -1;
            if (t < total) {
                while (t >= s_cu[lo + 1]) {
                    ++lo;
                    block = -1;
                }
                const int p = s_lens[lo] + t - s_cu[lo], b = p >> shift;
                if (b != block) {
                    const int held = (int)(((long long)s_lens[lo] + a.page - 1) >> shift);
                    page_no = b < held ? a.table[(int64_t)lo * a.max_blocks + b]
                                       : a.free_list[head + s_first[lo] + b - held];
                    block = b;
                }
                pos[e] = p;
                // a page number too large for a slot of 32 bits must not come out as another page's
                const int first = (int)((uint32_t)page_no << shift);
                slot[e] = first >> shift == page_no ? first + (p & (a.page - 1)) : -1;
            }
        }
        if (t0 + 3 < a.rows) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int e = 0; t0 + e < a.rows; ++e) {
                a.slots[t0 + e] = slot[e];
                a.positions[t0 + e] = pos[e];
            }
        }
    }
}

// ---- append ---------------------------------------------------------------------------------------
//
// A run is the rows of one page, for one head and for keys or values: the largest magnitude of its rows,
// the page's new scale 2^e, then the quotients.  Dividing by a power of two is exact, so a token that is
// held already changes only where it falls into e4m3's subnormal range, and the plain form's values
// come out bit for bit.
//
// Memory bounds it: 2 or 4 bytes in and 1 out an element.  A CTA takes a block of rows for one head, keys
// or values, and finds the runs that begin there: short ones (a generation step's, of one row) go to
// groups of lanes as wide as a row, side by side; the rows of a long one (a prompt's) are held in registers
// between the maximum and the quotients, so that they are read once, by as many warps as four loads a lane
// take for a page, so that a CTA has several runs of small pages under way.

constexpr int AT = 256;  // threads per CTA

// The least power of two 2^e, e >= -60, with amax <= 448 x 2^e = 1.75 x 2^(e + 8).
__device__ __forceinline__ float scale_of(float amax)
{
    const uint32_t u = __float_as_uint(fminf(amax, 3.402823466e38f));
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -60) + 127) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float4 x)
{
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t w)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 16 bytes of a row: 8 bf16 or 4 fp32
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    // largest magnitude so far, of the even and of the odd elements (their signs mean nothing); a NaN counts for nothing
    typedef uint32_t Max;
    __device__ __forceinline__ void add(Max &m) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(u[i]));
    }
    __device__ __forceinline__ static float value(Max m)
    {
        return fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xffff0000u)));
    }
    __device__ __forceinline__ void store(uint8_t *p, float f) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = to_e4m3x4(make_float4(__uint_as_float(u[2 * i] << 16) * f, __uint_as_float(u[2 * i] & 0xffff0000u) * f,
                                         __uint_as_float(u[2 * i + 1] << 16) * f,
                                         __uint_as_float(u[2 * i + 1] & 0xffff0000u) * f));
        *reinterpret_cast<uint2 *>(p) = make_uint2(r[0], r[1]);
    }
};
template <> struct Vec16<float> {
    static constexpr int N = 4;
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
    typedef float Max;
    __device__ __forceinline__ void add(Max &m) const
    {
        m = fmaxf(fmaxf(m, fmaxf(fabsf(w.x), fabsf(w.y))), fmaxf(fabsf(w.z), fabsf(w.w)));
    }
    __device__ __forceinline__ static float value(Max m) { return m; }
    __device__ __forceinline__ void store(uint8_t *p, float f) const
    {
        *reinterpret_cast<uint32_t *>(p) = to_e4m3x4(make_float4(w.x * f, w.y * f, w.z * f, w.w * f));
    }
};

// Held values of a page after its scale has grown by 1 / f: E bytes from p on in rows r0, r0 + STEP, ...
// below n, eight rows under way at a time.
template <int D, int E, int STEP> __device__ __forceinline__ void shrink_rows(uint8_t *p, int r0, int n, float f)
{
    for (int r = r0; r < n; r += 8 * STEP) {
        uint32_t w[8][E / 4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                if (r + i * STEP < n) w[i][e] = *reinterpret_cast<const uint32_t *>(p + (r + i * STEP) * D + 4 * e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                if (r + i * STEP < n) {
                    const float2 lo = from_e4m3x2(w[i][e]), hi = from_e4m3x2(w[i][e] >> 16);
                    *reinterpret_cast<uint32_t *>(p + (r + i * STEP) * D + 4 * e) =
                        to_e4m3x4(make_float4(lo.x * f, lo.y * f, hi.x * f, hi.y * f));
                }
    }
}

struct Where {
    int shift, nslots;
    __device__ __forceinline__ bool on(int slot) const { return slot >= 0 && slot < nslots; }
    // does a row with slot `b` continue the run of the row before it, with slot `a`?
    __device__ __forceinline__ bool same_page(int a, int b) const { return on(a) && on(b) && (a >> shift) == (b >> shift); }
};

// A run of n rows from x on, by a group of C = D / E lanes (lane c of it, the others in `group`).
template <typename T, int D>
__device__ __forceinline__ void append_run(const T *x, int64_t ld, uint8_t *base, float *scale, int n, int off, int c,
                                           uint32_t group)
{
    constexpr int E = Vec16<T>::N, C = D / E;
    const float was = off ? *scale : 0.f;
    Vec16<T> y;
    typename Vec16<T>::Max top = 0;
    for (int r = n - 1; r >= 0; --r) {
        y.load(x + r * ld);
        y.add(top);
    }
    float mx = Vec16<T>::value(top);
#pragma unroll
    for (int o = C / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(group, mx, o));
    const float to = fmaxf(was, scale_of(mx)), inv = 1.f / to;
    if (off && to != was) shrink_rows<D, E, 1>(base, 0, off, was * inv);
    y.store(base + off * D, inv);  // the run's first row is the last one read
    for (int r = 1; r < n; ++r) {  // the others again, from L2
        y.load(x + r * ld);
        y.store(base + (off + r) * D, inv);
    }
    __syncwarp(group);  // every lane has the old scale
    if (c == 0) *scale = to;
}

// Threads that hold a page's rows of one head, with four loads of 16 bytes each (the whole CTA with up to 16), and
// the loads.  (Prompts of 32768 rows of 4 heads, bf16, d 64, pages of 16: 21 us, and 34 by the CTA with one load a
// thread; now 12.7, since the runs' lengths are found once and not by every thread; all with the rows in L2, from HBM
// now 16.7.)
template <typename T, int D, int PAGE>
constexpr int HOLD = PAGE * (D / Vec16<T>::N) / 4 < AT ? PAGE * (D / Vec16<T>::N) / 4 : AT;
template <typename T, int D, int PAGE> constexpr int NPB = PAGE * (D / Vec16<T>::N) / HOLD<T, D, PAGE>;

// A barrier of the N threads of group `g` of the CTA.
template <int N> __device__ __forceinline__ void group_sync(int g)
{
    if (N == 32) __syncwarp();
    else if (N == AT) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(N) : "memory");
}

template <typename T, int D, int PAGE, int TILE>
__global__ void __launch_bounds__(AT, NPB<T, D, PAGE> <= 4 ? 4 : 3) cache_append_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                          const int32_t *__restrict__ slots, uint8_t *k_cache,
                                                          uint8_t *v_cache, float *k_scale, float *v_scale, int rows,
                                                          int Hk, int num_pages)
{
    constexpr int E = Vec16<T>::N, C = D / E, RP = AT / C;  // threads a row, rows at a time
    constexpr int NP = NPB<T, D, PAGE>;                     // registers: NP x 16 bytes
    constexpr int GT = HOLD<T, D, PAGE>, GW = GT / 32;      // threads and warps that share a long run
    static_assert(GT >= 32 && AT % GT == 0, "whole warps");
    __shared__ float s_max[AT / 32];
    constexpr int kShortRun = 4;                            // up to this length a run goes to a group of lanes
    constexpr int SPAN = (TILE + PAGE + 31) & ~31;          // rows looked at
    static_assert(SPAN <= AT, "one row a thread");
    __shared__ uint32_t s_lead[SPAN / 32], s_cont[SPAN / 32];
    constexpr int TW = (TILE + 31) / 32;
    __shared__ uint32_t s_short[TW], s_long[TW];            // rows that begin a run of up to kShortRun, of more
    __shared__ int s_slot[TILE], s_len[TILE];               // and its length
    const int tid = threadIdx.x, lane = tid & 31, c = tid % C, rr = tid / C;
    const int h = blockIdx.y, tile0 = blockIdx.x * TILE;
    const T *x = (blockIdx.z ? v : k) + (int64_t)h * D + E * c;
    uint8_t *cache = blockIdx.z ? v_cache : k_cache;
    float *scale = blockIdx.z ? v_scale : k_scale;
    const int64_t ld = (int64_t)Hk * D;
    constexpr int shift = PAGE == 16 ? 4 : PAGE == 32 ? 5 : PAGE == 64 ? 6 : 7;
    const Where w{shift, num_pages << shift};
    // rows of this block and a page's worth behind it: which begin a run, which continue the row before them
    if (tid < SPAN) {
        const int t = tile0 + tid;
        const int s = t < rows ? slots[t] : -1, before = t > 0 && t <= rows ? slots[t - 1] : -1;
        const bool paged = w.same_page(before, s);
        const uint32_t lead = __ballot_sync(0xffffffffu, w.on(s) && !paged && tid < TILE);
        const uint32_t cont = __ballot_sync(0xffffffffu, paged && s == before + 1);
        if (lane == 0) {
            s_lead[tid >> 5] = lead;
            s_cont[tid >> 5] = cont;
        }
        if (tid < TILE) s_slot[tid] = s;
    }
    __syncthreads();
    auto leads = [&](int at) { return (s_lead[at >> 5] >> (at & 31)) & 1; };
    auto length = [&](int at) {  // of the run that begins at row `at`: up to the first row that does not continue
        int n = 1;
        for (int i = at + 1; i < SPAN;) {
            const uint32_t gap = ~s_cont[i >> 5] >> (i & 31);
            const int more = gap ? __ffs(gap) - 1 : 32 - (i & 31);
            n += more;
            i += more;
            if (gap) break;
        }
        return min(n, PAGE - (s_slot[at] & (PAGE - 1)));
    };
    if (tid < 32 * TW) {
        const int n = tid < TILE && leads(tid) ? length(tid) : 0;
        if (tid < TILE) s_len[tid] = n;
        const uint32_t few = __ballot_sync(0xffffffffu, n > 0 && n <= kShortRun), many = __ballot_sync(0xffffffffu, n > kShortRun);
        if (lane == 0) {
            s_short[tid >> 5] = few;
            s_long[tid >> 5] = many;
        }
    }
    __syncthreads();
    const uint32_t group = (C == 32 ? 0xffffffffu : (1u << C) - 1) << (lane / C * C);
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < TW; ++q) any |= s_short[q];
    if (any)
        for (int at = rr; at < TILE; at += RP) {
            const int n = s_len[at], slot = s_slot[at];
            if (n == 0 || n > kShortRun) continue;
            const int64_t ph = (int64_t)(slot >> shift) * Hk + h;
            append_run<T, D>(x + (int64_t)(tile0 + at) * ld, ld, cache + (ph << shift) * D + E * c, scale + ph, n,
                             slot & (PAGE - 1), c, group);
        }
    // group `grp` takes every (AT / GT)-th long run; this thread has a part of its rows r0, r0 + RH, ...
    constexpr int RH = GT / C;
    const int grp = tid / GT, r0 = tid % GT / C;
    int turn = 0;
    for (int q = 0; q < TW; ++q)
        for (uint32_t left = s_long[q]; left; left &= left - 1) {
            const int at = 32 * q + __ffs(left) - 1, t = tile0 + at, n = s_len[at];
            if (GT < AT && (turn++ & (AT / GT - 1)) != grp) continue;
            const int slot = s_slot[at], pg = slot >> shift, off = slot & (PAGE - 1);
            const T *xr = x + (int64_t)t * ld;
            Vec16<T> y[NP];
            typename Vec16<T>::Max top = 0;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (r0 + RH * i < n) y[i].load(xr + (int64_t)(r0 + RH * i) * ld);
            const int64_t ph = (int64_t)pg * Hk + h;
            const float was = off ? scale[ph] : 0.f;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (r0 + RH * i < n) y[i].add(top);
            float mx = Vec16<T>::value(top);
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (GW > 1) {
                if (lane == 0) s_max[tid >> 5] = mx;
                group_sync<GT>(grp);
                mx = s_max[grp * GW];
#pragma unroll
                for (int i = 1; i < GW; ++i) mx = fmaxf(mx, s_max[grp * GW + i]);
            }
            const float to = fmaxf(was, scale_of(mx)), inv = 1.f / to;
            uint8_t *base = cache + (ph << shift) * D + E * c;
            if (off && to != was) shrink_rows<D, E, RH>(base, r0, off, was * inv);
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (r0 + RH * i < n) y[i].store(base + (off + r0 + RH * i) * D, inv);
            // s_max is read, and every thread has the old scale
            group_sync<GT>(grp);
            if (tid % GT == 0) scale[ph] = to;
        }
}

template <typename T, int D, int PAGE> cudaError_t run_append(const CacheAppendArgs &a, cudaStream_t st)
{
    // Rows a CTA: few where rows are few, so that a generation step's spread over the SMs (256 rows of 4 heads,
    // d 128, page 64, bf16: 2.3 us with 16, 5.3 with 64), more where they are many (prompts of 32768 rows, d 64:
    // 30 us with 16, 22 with 64, 17 with 128 when that was measured, now 11.2, the rows in L2), but 64 where
    // they all fit the SMs at once (4096 rows, d 64: 4.3 us with 64, 4.7 with 128; d 128: 5.0 and 6.0).  Four CTAs an
    // SM: with five, registers spill (8192 rows of a step, d 128: 13.5 us with four, 17.8 with five).
    const int tile = a.rows <= 2048 ? 16 : (long)a.rows / 64 * a.Hk * 2 <= 4 * 148 ? 64 : 128;
    auto kern = tile == 16 ? cache_append_kernel<T, D, PAGE, 16> : tile == 64 ? cache_append_kernel<T, D, PAGE, 64>
                                                                             : cache_append_kernel<T, D, PAGE, 128>;
    kern<<<dim3((a.rows + tile - 1) / tile, a.Hk, 2), AT, 0, st>>>((const T *)a.k, (const T *)a.v, a.slots, a.k_cache,
                                                                   a.v_cache, a.k_scale, a.v_scale, a.rows, a.Hk,
                                                                   a.num_pages);
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t run_append(const CacheAppendArgs &a, cudaStream_t st)
{
    if (a.page == 16) return run_append<T, D, 16>(a, st);
    if (a.page == 32) return run_append<T, D, 32>(a, st);
    if (a.page == 64) return run_append<T, D, 64>(a, st);
    return run_append<T, D, 128>(a, st);
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanArgs &a, cudaStream_t st)
{
    // Without leave a CTA has 48 KB, the kernel's static arrays (some 500 bytes) among them.  The leave is the kernel's,
    // not the call's: always the largest plan's, so that a call beside this one cannot lower it before the launch.
    auto bytes = [](int n) { return (3 * n + 1) * 4; };
    const int smem = bytes(a.N);
    if (smem > 47 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxPlan));
        if (e != cudaSuccess) return e;
    }
    cache_plan_kernel<<<PC, PT, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t st)
{
    if (a.rows == 0) return cudaSuccess;
    if (a.dtype == GDN_DTYPE_BF16)
        return a.d == 128 ? run_append<__nv_bfloat16, 128>(a, st) : run_append<__nv_bfloat16, 64>(a, st);
    return a.d == 128 ? run_append<float, 128>(a, st) : run_append<float, 64>(a, st);
}

}  // namespace gdn
