// gdn_attn.h -- declarations shared by the softmax-attention entries (gdn_attn_api.cu) and their
// kernels.  Not part of the public C-ABI (include/gdn.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// One prompt-attention call: tensors as gdn_attn_fwd / gdn_attn_bwd take them.
struct AttnArgs {
    const void *q, *k, *v;
    void *out;         // backward: the forward's result
    float *lse;        // forward: may be NULL
    const void *dout;  // backward only, as the rest
    void *dq, *dk, *dv;
    void *workspace;
    int B, T, Hq, Hk, d;
    const int32_t *cu;  // NULL: dense
    float scale;
};

// bf16 on the tcgen05 tensor cores (gdn_attn_tc.cu, gdn_attn_tc_bwd.cu); the device error records of
// their bounded waits, read and cleared.
cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_attn_bwd_tc(const AttnArgs &a, cudaStream_t stream);
int read_and_clear_attn_fwd_error();
int read_and_clear_attn_bwd_error();

// fp32 on CUDA cores (gdn_attn_simt.cu).
cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_attn_bwd_simt(const AttnArgs &a, cudaStream_t stream);
size_t attn_bwd_simt_workspace(int B, int T, int Hq, int Hk, int d, int varlen);

constexpr int kMaxPlan = 16384;  // requests of a plan

struct CachePlanArgs {
    const int32_t *lens, *added;
    int32_t *table;
    const int32_t *free_list, *free_head;
    int32_t *cu, *slots, *positions, *lens_out, *free_head_out, *status;
    int N, max_blocks, num_free, rows, page;
};
cudaError_t launch_cache_plan(const CachePlanArgs &a, cudaStream_t stream);

struct CacheAppendArgs {
    const void *k, *v;
    const int32_t *slots;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int rows, Hk, d, page, num_pages, dtype;
};
cudaError_t launch_cache_append(const CacheAppendArgs &a, cudaStream_t stream);

struct AttnDecodeArgs {
    const void *q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    void *out;
    int N, Hq, Hk, d, page, num_pages, max_blocks, dtype;
    float scale;
    void *workspace;
};
// Scratch of the split over a long context, for the current device.
size_t attn_decode_workspace_bytes(int N, int Hq, int Hk, int d, int page, int max_blocks, int dtype);
cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t stream);
// The decode kernel's device error record (bounded waits that ran out), read and cleared.
int read_and_clear_attn_decode_error();

}  // namespace gdn
