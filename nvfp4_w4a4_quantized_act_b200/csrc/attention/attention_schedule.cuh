// attention_schedule.cuh -- how the attention kernel's CTAs share a batch.
//
// An item is a tile of query rows of one sequence and key head: up to
// 128 / group tokens with all `group` query heads of the key head, so every
// key block loaded serves all of them.  An item costs its keys plus one block
// of 128 (loading the queries, writing the result).  The items of the batch,
// ordered by sequence, key head and row tile, form one line of cost; CTA c of
// n takes the c-th n-th of it, whatever the mix of long and short sequences,
// prompts and single tokens.  A boundary inside an item falls between two of
// its 128-key blocks, and the parts are joined afterwards.  Row tiles of a
// sequence grow by a constant number of keys, so the cost before a row tile
// is an arithmetic series and a CTA finds its start without a table.
#pragma once

#include <cstdint>

#include "paged_batch.cuh"

namespace nvfp4 {
namespace attn {

constexpr int KEY_BLOCK = 128;
constexpr int ROW_TILE = 128;
constexpr int CTAS = 148;   // one per SM; results do not depend on the device's own count

struct SeqItems {
    Seq s;
    int32_t tiles;  // row tiles
    int32_t past;   // len - fresh (may be negative)

    __device__ __forceinline__ void set(const Seq &seq, int tile_tokens)
    {
        s = seq;
        tiles = (seq.fresh + tile_tokens - 1) / tile_tokens;
        past = seq.len - seq.fresh;
    }

    // Cost of row tile m, and of all row tiles before m.
    __device__ __forceinline__ int64_t cost(int m, int tile_tokens) const
    {
        return KEY_BLOCK + max(static_cast<int64_t>(past) + static_cast<int64_t>(tile_tokens) * (m + 1), int64_t(0));
    }
    __device__ __forceinline__ int64_t before(int m, int tile_tokens) const
    {
        // row tiles i with past + tile_tokens * (i + 1) > 0 start at m0
        const int64_t t = tile_tokens;
        const int64_t m0 = past >= 0 ? 0 : static_cast<int64_t>(-past) / tile_tokens;
        int64_t sum = static_cast<int64_t>(KEY_BLOCK) * m;
        if (m > m0) {
            const int64_t n = m - m0;
            sum += n * past + t * (n * m0 + n * (n + 1) / 2);
        }
        return sum;
    }
    __device__ __forceinline__ int64_t total(int tile_tokens) const { return before(tiles, tile_tokens); }

    // Keys that the last row (and the first) of row tile m sees.
    __device__ __forceinline__ int keys(int m, int tile_tokens) const
    {
        return max(past + min(s.fresh, (m + 1) * tile_tokens), 0);
    }
    __device__ __forceinline__ int keys_first(int m, int tile_tokens) const
    {
        return max(past + m * tile_tokens + 1, 0);
    }
};

// A CTA's walk over its part of the line.
struct Walk {
    int b, h, m;
    int64_t x;     // offset in the item
    int64_t left;  // cost left
    SeqItems q;
    // the current item
    int keys, blocks, t0, t1;

    // Moves to the next item with key blocks for this CTA; false at the end.
    // First call: `b, h, m, x, left, q` set by the start.
    __device__ __forceinline__ bool next(const BatchView &v, int kv_heads, int tile_tokens, bool first)
    {
        if (!first)
            step(v, kv_heads, tile_tokens);
        while (left > 0) {
            const int64_t c = q.cost(m, tile_tokens);
            const int64_t x1 = min(c, x + left);
            keys = q.keys(m, tile_tokens);
            blocks = max((keys + KEY_BLOCK - 1) / KEY_BLOCK, 1);
            t0 = static_cast<int>(x * blocks / c);
            t1 = static_cast<int>(x1 * blocks / c);
            left -= x1 - x;
            x = x1;
            if (t1 > t0)
                return true;
            step(v, kv_heads, tile_tokens);
        }
        return false;
    }

private:
    __device__ __forceinline__ void step(const BatchView &v, int kv_heads, int tile_tokens)
    {
        x = 0;
        if (++m < q.tiles)
            return;
        m = 0;
        if (++h < kv_heads)
            return;
        h = 0;
        bool bad = false;
        while (left > 0 && ++b < v.num_seqs) {
            q.set(load_seq(v, b, bad), tile_tokens);
            if (q.tiles > 0)
                return;
        }
        left = 0;
    }
};

struct WalkStart {
    int b, h, m;
    int64_t x, left;
    int64_t total;
};

// Fills `st` (shared memory) with the start of CTA `cta` of CTAS; all THREADS
// threads call it, `scratch`: THREADS / 32 words of shared memory.  Malformed
// offsets or lengths set *bad (this thread's share).
template <int THREADS>
__device__ __forceinline__ void find_start(const BatchView &v, int kv_heads, int tile_tokens, int cta, WalkStart *st,
                                           int64_t *scratch, bool &bad)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (v.num_seqs + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, v.num_seqs), b1 = min(b0 + per, v.num_seqs);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        SeqItems q;
        q.set(load_seq(v, b, bad), tile_tokens);
        mine += q.total(tile_tokens) * kv_heads;
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o)
            scan += up;
    }
    if (lane == 31)
        scratch[warp] = scan;
    __syncthreads();
    int64_t base = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        base += w < warp ? scratch[w] : 0;
        total += scratch[w];
    }
    const int64_t from = total * cta / CTAS, to = total * (cta + 1) / CTAS;
    int64_t at = base + scan - mine;
    if (tid == 0) {
        st->left = to - from;
        st->total = total;
    }
    if (to > from && from >= at && from < at + mine) {
        for (int b = b0; b < b1; ++b) {
            SeqItems q;
            q.set(load_seq(v, b, bad), tile_tokens);
            const int64_t one = q.total(tile_tokens);
            if (from < at + one * kv_heads) {
                int64_t off = from - at;
                st->b = b;
                st->h = static_cast<int>(off / one);
                off -= st->h * one;
                int lo = 0, hi = q.tiles - 1;  // last row tile that starts at or before off
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (q.before(mid, tile_tokens) <= off)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                st->m = lo;
                st->x = off - q.before(lo, tile_tokens);
                break;
            }
            at += one * kv_heads;
        }
    }
    __syncthreads();
}

}  // namespace attn
}  // namespace nvfp4
