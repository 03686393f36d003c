// gdn_attn_tile.cuh -- where a tile of a prompt-attention launch lies.
#pragma once

#include <stdint.h>

namespace gdn {

// Division of n < 2^31 by a number known at launch: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (floor(m n / 2^32) + n) / 2^l (Granlund and Montgomery 1994).  A CTA starts with a handful of divisions by
// heads and sequences, some 100 cycles each in their general form.
struct FastDiv {
    uint32_t d, m, l;
    explicit FastDiv(int by) : d((uint32_t)by), m(0), l(0)
    {
        while ((1ull << l) < d) ++l;
        m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> l); }
};

struct AttnTile {
    int seq;     // -1: this tile does not exist
    int block;   // block of `rows` tokens within the sequence
    int len;     // the sequence's length
    int64_t t0;  // the sequence's first token
};

// Tile `index` of a launch over blocks of `rows` tokens, the tiles with the most work first: block b of
// a sequence attends to b + 1 blocks, so tiles go from the highest block down over all sequences, and the
// launch does not end with a long one alone.  Dense calls have B ceil(T / rows) tiles; a packed launch
// has at most T / rows + B, and the tiles past the last one are empty.  With more than 128 sequences
// (each lane holds four lengths; many sequences of a launch's size are short ones) packed tiles go
// sequence by sequence, each from its last block on: sequence s has the tiles from cu[s] / rows + s on, since
// len / rows rounded up is at most cu[s + 1] / rows - cu[s] / rows + 1.  Called by whole warps.
__device__ __forceinline__ AttnTile attn_tile(const int32_t *__restrict__ cu, const FastDiv &by, int T, int rows, int index)
{
    const int B = (int)by.d;
    AttnTile r;
    if (!cu) {
        const int n = (T + rows - 1) / rows;
        const int turn = by.div(index);
        r.seq = index - turn * B;
        r.block = n - 1 - turn;
        r.len = T;
        r.t0 = (int64_t)r.seq * T;
        return r;
    }
    const int lane = threadIdx.x & 31;
    r.seq = -1;
    r.block = r.len = 0;
    r.t0 = 0;
    if (B <= 128) {
        int n[4], most = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int s = 32 * x + lane;
            n[x] = 0;
            if (s < B) {
                const int a = cu[s], len = min(cu[s + 1], T) - a;
                if (a >= 0 && len > 0) n[x] = (len + rows - 1) / rows;
            }
            most = max(most, n[x]);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        // tiles of block b and above: sum of max(0, n - b); the block sought is the highest with more than `index`
        auto above = [&](int b) {
            int c = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) c += max(0, n[x] - b);
            return __reduce_add_sync(0xffffffffu, c);
        };
        if (index >= above(0)) return r;
        int lo = 0, hi = most;  // above(lo) > index >= above(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (above(mid) > index) lo = mid; else hi = mid;
        }
        int k = index - above(lo + 1);  // among the sequences with a block lo, in their order
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const unsigned has = __ballot_sync(0xffffffffu, n[x] > lo);
            if (r.seq < 0 && k < __popc(has)) r.seq = 32 * x + (int)__fns(has, 0, k + 1);
            k -= __popc(has);
        }
        r.block = lo;
        r.t0 = cu[r.seq];
        r.len = min(cu[r.seq + 1], T) - (int)r.t0;
        return r;
    }
    // largest s with cu[s] / rows + s <= index: 32 of them looked at at once
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int stride = (hi - lo + 31) >> 5, s = lo + lane * stride;
        const unsigned before = __ballot_sync(0xffffffffu, s < hi && max(cu[s], 0) / rows + s <= index);
        const int c = before == 0xffffffffu ? 32 : __ffs(~before) - 1;
        lo += max(0, c - 1) * stride;
        hi = min(hi, lo + stride);
    }
    const int a = cu[lo], len = min(cu[lo + 1], T) - a;
    if (a < 0 || len <= 0) return r;
    const int n = (len + rows - 1) / rows, rel = index - a / rows - lo;
    if (rel < 0 || rel >= n) return r;
    r.seq = lo;
    r.block = n - 1 - rel;
    r.len = len;
    r.t0 = a;
    return r;
}

// Tiles of a launch (packed: an upper bound).
inline long attn_tiles(const int32_t *cu, int B, int T, int rows)
{
    return cu ? (long)T / rows + B : (long)B * ((T + rows - 1) / rows);
}

}  // namespace gdn
