// gdn_attn_tile.cuh -- where a tile of a prompt-attention launch lies.
#pragma once

#include <stdint.h>

namespace gdn {

struct AttnTile {
    int seq;     // -1: this tile does not exist
    int block;   // block of `rows` tokens within the sequence
    int len;     // the sequence's length
    int64_t t0;  // the sequence's first token
};

// Tile `index` of a launch over blocks of `rows` tokens, from last blocks to first ones (under the
// causal mask the last query block has the most work): dense calls (B ceil(T / rows) tiles) block by
// block over all sequences, packed ones (at most T / rows + B tiles; those past the last one are
// empty) sequence by sequence.  Called by whole warps; 32 sequences are looked at at a time.
__device__ __forceinline__ AttnTile attn_tile(const int32_t *__restrict__ cu, int B, int T, int rows, int index)
{
    AttnTile r;
    if (!cu) {
        const int n = (T + rows - 1) / rows;
        r.seq = index % B;
        r.block = n - 1 - index / B;
        r.len = T;
        r.t0 = (int64_t)r.seq * T;
        return r;
    }
    const int lane = threadIdx.x & 31;
    int base = 0;
    r.seq = -1;
    r.block = r.len = 0;
    r.t0 = 0;
    for (int s0 = 0; s0 < B; s0 += 32) {
        const int s = s0 + lane;
        int a = 0, len = 0;
        if (s < B) {
            a = cu[s];
            len = max(0, min(cu[s + 1], T) - a);
            if (a < 0) len = 0;
        }
        const int n = (len + rows - 1) / rows;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const int rel = index - base;
        const unsigned hit = __ballot_sync(0xffffffffu, rel >= incl - n && rel < incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.seq = s0 + src;
            r.block = __shfl_sync(0xffffffffu, incl - 1 - rel, src);
            r.len = __shfl_sync(0xffffffffu, len, src);
            r.t0 = __shfl_sync(0xffffffffu, a, src);
            return r;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

// Tiles of a launch (packed: an upper bound).
inline long attn_tiles(const int32_t *cu, int B, int T, int rows)
{
    return cu ? (long)T / rows + B : (long)B * ((T + rows - 1) / rows);
}

}  // namespace gdn
