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
                slot[e] = page_no * a.page + (p & (a.page - 1));
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
// One CTA takes the runs (rows of one page) that begin in its block of rows, for one head and for
// keys or values: the largest magnitude of the run, the page's new scale 2^e, then the quotients.
// Dividing by a power of two is exact, so a token that is held already changes only where it falls
// into e4m3's subnormal range, and the plain form's values come out bit for bit.

constexpr int AT = 128;  // threads per CTA

__device__ __forceinline__ float4 load_row4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load_row4(const __nv_bfloat16 *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

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

__device__ __forceinline__ float absmax4(float m, float4 x)  // NaN is passed over
{
    return fmaxf(fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
}

template <typename T, int D>
__global__ void __launch_bounds__(AT) cache_append_kernel(const T *__restrict__ k, const T *__restrict__ v,
                                                          const int32_t *__restrict__ slots, uint8_t *k_cache,
                                                          uint8_t *v_cache, float *k_scale, float *v_scale, int rows,
                                                          int Hk, int page, int num_pages, int tile)
{
    constexpr int C = D / 4;            // threads per row, four elements each
    constexpr int RP = AT / C;          // rows at a time
    __shared__ float s_max[AT / 32];
    const int tid = threadIdx.x, c = tid % C, rr = tid / C;
    const int h = blockIdx.y;
    const T *x = blockIdx.z ? v : k;
    uint8_t *cache = blockIdx.z ? v_cache : k_cache;
    float *scale = blockIdx.z ? v_scale : k_scale;
    const int64_t ld = (int64_t)Hk * D;
    const int shift = __ffs(page) - 1;
    const int nslots = num_pages << shift;
    const int t_end = min((int)(blockIdx.x + 1) * tile, rows);
    for (int t = blockIdx.x * tile; t < t_end;) {
        const int slot = slots[t];
        const bool on = slot >= 0 && slot < nslots;
        const int pg = slot >> shift, off = slot & (page - 1);
        if (!on) {
            ++t;
            continue;
        }
        if (t > 0) {  // rows of a run that began before this one
            const int before = slots[t - 1];
            if (before >= 0 && before < nslots && (before >> shift) == pg) {
                ++t;
                continue;
            }
        }
        // the run: at most to the page's end
        int n = 1;
        while (off + n < page && t + n < rows && slots[t + n] == slot + n) ++n;
        const T *xr = x + (int64_t)t * ld + (int64_t)h * D + 4 * c;
        float mx = 0.f;
        for (int r = rr; r < n; r += RP) mx = absmax4(mx, load_row4(xr + (int64_t)r * ld));
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) s_max[tid >> 5] = mx;
        const int64_t ph = (int64_t)pg * Hk + h;
        const float was = off ? scale[ph] : 0.f;
        __syncthreads();
        mx = s_max[0];
#pragma unroll
        for (int w = 1; w < AT / 32; ++w) mx = fmaxf(mx, s_max[w]);
        const float to = fmaxf(was, scale_of(mx)), inv = 1.f / to;
        uint8_t *base = cache + ((ph << shift)) * D + 4 * c;
        if (off && to != was) {
            const float f = was * inv;
            for (int r = rr; r < off; r += RP) {
                uint32_t *w = reinterpret_cast<uint32_t *>(base + r * D);
                const uint32_t old = *w;
                const float2 lo = from_e4m3x2(old), hi = from_e4m3x2(old >> 16);
                *w = to_e4m3x4(make_float4(lo.x * f, lo.y * f, hi.x * f, hi.y * f));
            }
        }
        for (int r = rr; r < n; r += RP) {
            const float4 y = load_row4(xr + (int64_t)r * ld);
            *reinterpret_cast<uint32_t *>(base + (off + r) * D) =
                to_e4m3x4(make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
        __syncthreads();  // s_max is read, and every thread has the old scale
        if (tid == 0) scale[ph] = to;
        t += n;
    }
}

template <typename T, int D> cudaError_t run_append(const CacheAppendArgs &a, cudaStream_t st)
{
    // rows per CTA: one where there are few (a generation step: every row is a run of its own), up
    // to a page where there are many (prompts: one run per page), with about 16 CTAs per SM
    const long want = (long)a.rows * a.Hk * 2 / (148 * 16);
    const int tile = (int)(want < 1 ? 1 : want > a.page ? a.page : want);
    const dim3 grid((a.rows + tile - 1) / tile, a.Hk, 2);
    cache_append_kernel<T, D><<<grid, AT, 0, st>>>((const T *)a.k, (const T *)a.v, a.slots, a.k_cache, a.v_cache,
                                                   a.k_scale, a.v_scale, a.rows, a.Hk, a.page, a.num_pages, tile);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanArgs &a, cudaStream_t st)
{
    const int smem = (3 * a.N + 1) * 4;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
