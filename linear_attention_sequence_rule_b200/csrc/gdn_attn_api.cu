// gdn_attn_api.cu -- the softmax-attention entries of the C-ABI (include/gdn.h): argument checks on the
// host, choice of kernel, launch on the caller's stream.  No call allocates device memory.
#include <math.h>

#include "gdn_attn.h"
#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {

namespace {

template <typename... A> int refuse(int code, const char *fmt, A... args)
{
    set_error(fmt, args...);
    return code;
}

int launched(cudaError_t e, const char *fn)
{
    if (e == cudaSuccess) return GDN_OK;
    return refuse(GDN_ERR_CUDA, "%s: %s (%s)", fn, cudaGetErrorName(e), cudaGetErrorString(e));
}

template <size_t N> int check_pointers(const char *fn, const void *const (&ptrs)[N])
{
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u)
            return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: pointer %p is not 16-byte aligned", fn, p);
    return GDN_OK;
}

int check_types(const char *fn, int d, int dtype)
{
    if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F32) return refuse(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
    if (d != 64 && d != 128) return refuse(GDN_ERR_UNSUPPORTED, "%s: d=%d, supported: 64 or 128", fn, d);
    return GDN_OK;
}

int check_heads(const char *fn, int Hq, int Hk)
{
    if (Hk < 1 || Hq < 1 || Hq % Hk != 0 || Hq > 65535)
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: Hq=%d Hk=%d, need Hk >= 1 and Hq <= 65535 a multiple of Hk", fn, Hq, Hk);
    return GDN_OK;
}

int check_scale(const char *fn, float scale)
{
    if (!(scale > 0.f) || !(scale < INFINITY))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: scale %g, must be finite and > 0", fn, (double)scale);
    return GDN_OK;
}

int check_page(const char *fn, int page)
{
    if (page != 16 && page != 32 && page != 64 && page != 128)
        return refuse(GDN_ERR_UNSUPPORTED, "%s: page=%d, supported: 16, 32, 64 or 128", fn, page);
    return GDN_OK;
}

int check_prompt(const char *fn, int B, int T, int Hq, int Hk, int d, int varlen, int dtype)
{
    int rc = check_types(fn, d, dtype);
    if (rc != GDN_OK || (rc = check_heads(fn, Hq, Hk)) != GDN_OK) return rc;
    if (B < 1 || T < 0 || (!varlen && T < 1))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: B=%d T=%d (B >= 1; dense T >= 1)", fn, B, T);
    const long long tokens = varlen ? (long long)T : (long long)B * T;
    const long long tiles = varlen ? T / 128 + (long long)B : (long long)B * ((T + 127LL) / 128);  // CTAs a head
    if (tokens >= (1LL << 31) || tokens * Hq * d >= (1LL << 40) || B > (1 << 24) || tiles * Hq >= (1LL << 31))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: problem too large", fn);
    return GDN_OK;
}

int check_workspace(const char *fn, const void *workspace, size_t have, size_t need)
{
    if (need == 0) return GDN_OK;
    if (!workspace || have < need)
        return refuse(GDN_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need, workspace ? have : (size_t)0);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: workspace must be 256-byte aligned", fn);
    return GDN_OK;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_attn_fwd(const void *q, const void *k, const void *v, void *out, float *lse, int B, int T, int Hq, int Hk,
                 int d, const int32_t *cu_seqlens, int dtype, float scale, void *stream)
{
    const char *fn = "gdn_attn_fwd";
    set_error("%s", "");
    int rc = check_prompt(fn, B, T, Hq, Hk, d, cu_seqlens != nullptr, dtype);
    if (rc != GDN_OK || (rc = check_scale(fn, scale)) != GDN_OK) return rc;
    if (!q || !k || !v || !out) return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: q, k, v and out are required", fn);
    const void *ptrs[] = {q, k, v, out, lse, cu_seqlens};
    if ((rc = check_pointers(fn, ptrs)) != GDN_OK) return rc;
    if (T == 0) return GDN_OK;  // packed, no token
    AttnArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = out, a.lse = lse;
    a.B = B, a.T = T, a.Hq = Hq, a.Hk = Hk, a.d = d, a.cu = cu_seqlens, a.scale = scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(dtype == GDN_DTYPE_BF16 ? launch_attn_fwd_tc(a, st) : launch_attn_fwd_simt(a, st), fn);
}

size_t gdn_attn_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d, int varlen, int dtype)
{
    if (check_prompt("gdn_attn_bwd", B, T, Hq, Hk, d, varlen, dtype) != GDN_OK) return (size_t)-1;
    // bf16: D and -lse log2 e of every (token, query head)
    const size_t rows = (varlen ? (size_t)T : (size_t)B * T) * Hq;
    const size_t bytes = dtype == GDN_DTYPE_BF16 ? 2 * rows * sizeof(float) : attn_bwd_simt_workspace(B, T, Hq, Hk, d, varlen);
    return (bytes + 255) & ~(size_t)255;
}

int gdn_attn_bwd(const void *q, const void *k, const void *v, const void *out, const float *lse, const void *dout,
                 void *dq, void *dk, void *dv, int B, int T, int Hq, int Hk, int d, const int32_t *cu_seqlens,
                 int dtype, float scale, void *workspace, size_t workspace_bytes, void *stream)
{
    const char *fn = "gdn_attn_bwd";
    set_error("%s", "");
    int rc = check_prompt(fn, B, T, Hq, Hk, d, cu_seqlens != nullptr, dtype);
    if (rc != GDN_OK || (rc = check_scale(fn, scale)) != GDN_OK) return rc;
    if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv)
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: every tensor is required", fn);
    const void *ptrs[] = {q, k, v, out, lse, dout, dq, dk, dv, cu_seqlens};
    if ((rc = check_pointers(fn, ptrs)) != GDN_OK) return rc;
    rc = check_workspace(fn, workspace, workspace_bytes,
                         gdn_attn_bwd_workspace_bytes(B, T, Hq, Hk, d, cu_seqlens != nullptr, dtype));
    if (rc != GDN_OK) return rc;
    if (T == 0) return GDN_OK;
    AttnArgs a{};
    a.q = q, a.k = k, a.v = v, a.out = const_cast<void *>(out), a.lse = const_cast<float *>(lse), a.dout = dout;
    a.dq = dq, a.dk = dk, a.dv = dv, a.workspace = workspace;
    a.B = B, a.T = T, a.Hq = Hq, a.Hk = Hk, a.d = d, a.cu = cu_seqlens, a.scale = scale;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(dtype == GDN_DTYPE_BF16 ? launch_attn_bwd_tc(a, st) : launch_attn_bwd_simt(a, st), fn);
}

int gdn_cache_plan(const int32_t *lens, const int32_t *added, int32_t *block_table, const int32_t *free_list,
                   const int32_t *free_head, int32_t *cu_seqlens, int32_t *slots, int32_t *positions,
                   int32_t *lens_out, int32_t *free_head_out, int32_t *status, int N, int max_blocks, int num_free,
                   int rows, int page, void *stream)
{
    const char *fn = "gdn_cache_plan";
    set_error("%s", "");
    int rc = check_page(fn, page);
    if (rc != GDN_OK) return rc;
    if (N > kMaxPlan) return refuse(GDN_ERR_UNSUPPORTED, "%s: N=%d, supported: up to %d", fn, N, kMaxPlan);
    if (N < 1 || max_blocks < 1 || num_free < 0 || rows < 0 || rows > (1 << 30) || (long long)max_blocks * page >= (1LL << 31))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: N=%d max_blocks=%d num_free=%d rows=%d out of range", fn, N,
                      max_blocks, num_free, rows);
    if (!lens || !added || !block_table || !free_head || !cu_seqlens || !lens_out || !free_head_out || !status ||
        (num_free > 0 && !free_list) || (rows > 0 && (!slots || !positions)))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: every array is required", fn);
    const void *ptrs[] = {lens, added, block_table, free_list, cu_seqlens, slots, positions, lens_out};
    if ((rc = check_pointers(fn, ptrs)) != GDN_OK) return rc;
    for (const void *p : {(const void *)free_head, (const void *)free_head_out, (const void *)status})
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: pointer %p is not 4-byte aligned", fn, p);
    const CachePlanArgs a{lens, added, block_table, free_list, free_head, cu_seqlens, slots, positions, lens_out,
                          free_head_out, status, N, max_blocks, num_free, rows, page};
    return launched(launch_cache_plan(a, static_cast<cudaStream_t>(stream)), fn);
}

int gdn_cache_append(const void *k, const void *v, const int32_t *slots, void *k_cache, void *v_cache, float *k_scale,
                     float *v_scale, int rows, int Hk, int d, int page, int num_pages, int dtype, void *stream)
{
    const char *fn = "gdn_cache_append";
    set_error("%s", "");
    int rc = check_types(fn, d, dtype);
    if (rc != GDN_OK || (rc = check_page(fn, page)) != GDN_OK) return rc;
    if (rows < 0 || rows > (1 << 30) || Hk < 1 || Hk > 65535 || num_pages < 1 || (long long)num_pages * page >= (1LL << 31))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: rows=%d Hk=%d num_pages=%d out of range", fn, rows, Hk, num_pages);
    if (!k_cache || !v_cache || !k_scale || !v_scale || (rows > 0 && (!k || !v || !slots)))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: every array is required", fn);
    const void *ptrs[] = {k, v, slots, k_cache, v_cache, k_scale, v_scale};
    if ((rc = check_pointers(fn, ptrs)) != GDN_OK) return rc;
    const CacheAppendArgs a{k, v, slots, static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale,
                            v_scale, rows, Hk, d, page, num_pages, dtype};
    return launched(launch_cache_append(a, static_cast<cudaStream_t>(stream)), fn);
}

static int check_attn_decode(const char *fn, int N, int Hq, int Hk, int d, int page, int max_blocks, int dtype)
{
    int rc = check_types(fn, d, dtype);
    if (rc != GDN_OK || (rc = check_page(fn, page)) != GDN_OK || (rc = check_heads(fn, Hq, Hk)) != GDN_OK) return rc;
    if (N < 1 || (long long)N * Hq > (1LL << 24) || max_blocks < 1 || (long long)max_blocks * page >= (1LL << 31))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: N=%d max_blocks=%d out of range (N Hq at most 2^24)", fn, N, max_blocks);
    return GDN_OK;
}

size_t gdn_attn_decode_workspace_bytes(int N, int Hq, int Hk, int d, int page, int max_blocks, int dtype)
{
    if (check_attn_decode("gdn_attn_decode", N, Hq, Hk, d, page, max_blocks, dtype) != GDN_OK) return (size_t)-1;
    return attn_decode_workspace_bytes(N, Hq, Hk, d, page, max_blocks, dtype);
}

int gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                    const float *v_scale, const int32_t *block_table, const int32_t *lens, void *out, int N, int Hq,
                    int Hk, int d, int page, int num_pages, int max_blocks, int dtype, float scale, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    const char *fn = "gdn_attn_decode";
    set_error("%s", "");
    int rc = check_attn_decode(fn, N, Hq, Hk, d, page, max_blocks, dtype);
    if (rc != GDN_OK || (rc = check_scale(fn, scale)) != GDN_OK) return rc;
    if (num_pages < 1 || (long long)num_pages * page >= (1LL << 31))
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: num_pages=%d out of range", fn, num_pages);
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !lens || !out)
        return refuse(GDN_ERR_INVALID_ARGUMENT, "%s: every array is required", fn);
    const void *ptrs[] = {q, k_cache, v_cache, k_scale, v_scale, block_table, lens, out};
    if ((rc = check_pointers(fn, ptrs)) != GDN_OK) return rc;
    rc = check_workspace(fn, workspace, workspace_bytes,
                         attn_decode_workspace_bytes(N, Hq, Hk, d, page, max_blocks, dtype));
    if (rc != GDN_OK) return rc;
    const AttnDecodeArgs a{q, static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache), k_scale,
                           v_scale, block_table, lens, out, N, Hq, Hk, d, page, num_pages, max_blocks, dtype, scale,
                           workspace};
    return launched(launch_attn_decode(a, static_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
