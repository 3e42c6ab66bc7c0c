// attention_schedule.cuh -- how the attention kernel's CTAs share a batch.
//
// An item is a tile of query rows of one sequence and key head: up to
// 128 / group tokens with all `group` query heads of the key head, so every
// key block loaded serves all of them.  An item costs its keys plus item_cost
// (loading the queries, filling the pipeline, writing the result).  The items of the batch,
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
    int32_t m0;     // first row tile with keys by the formula of cost()
    int32_t extra;  // cost of an item beside its keys

    __device__ __forceinline__ void set(const Seq &seq, const BatchView &v, int tile_tokens)
    {
        s = seq;
        extra = v.item_cost;
        const bool mine = seq.fresh >= v.fresh_min && seq.fresh <= v.fresh_max;
        tiles = mine ? (seq.fresh + tile_tokens - 1) / tile_tokens : 0;
        past = seq.len - seq.fresh;
        m0 = past >= 0 ? 0 : -past / tile_tokens;
    }

    // Cost of row tile m, and of all row tiles before m.
    __device__ __forceinline__ int64_t cost(int m, int tile_tokens) const
    {
        return extra + max(static_cast<int64_t>(past) + static_cast<int64_t>(tile_tokens) * (m + 1), int64_t(0));
    }
    __device__ __forceinline__ int64_t before(int m, int tile_tokens) const
    {
        int64_t sum = static_cast<int64_t>(extra) * m;
        if (m > m0) {
            const int64_t n = m - m0;
            sum += n * past + tile_tokens * (n * m0 + n * (n + 1) / 2);
        }
        return sum;
    }
    __device__ __forceinline__ int64_t total(int tile_tokens) const { return before(tiles, tile_tokens); }
};

// What the kernel's warps need to know of an item.
struct Item {
    int32_t blocks;      // key blocks of this CTA's part; 0: no more items
    int32_t t0;          // first of them
    int32_t keys;        // keys that the last row sees
    int32_t seen_first;  // and the first row
    int32_t rows;        // rows (tokens x group)
    int32_t past0;       // position of the first token
    int32_t token0;      // first token row
    int32_t head;        // key head
    int32_t seq;
    int32_t part;        // 0: the item is this CTA's alone; 1: begun by an earlier CTA; 2: finished by later ones

    // No work and nothing to address: the end of a CTA's items, and what a warp goes on with when its wait for one
    // ran out.
    __host__ __device__ static Item none()
    {
        Item it;
        it.blocks = it.t0 = it.keys = it.seen_first = it.rows = it.past0 = it.token0 = it.head = it.seq = 0;
        it.part = 1;
        return it;
    }
};

// A CTA's walk over its part of the line.
struct Walk {
    // Key block that a boundary at cost x of an item of cost c falls to.  In
    // fp64 for large items: rounded, but alike for both neighbours of the
    // boundary and never falling as x grows.
    static __device__ __forceinline__ int block_at(int64_t x, int blocks, int64_t c)
    {
        if (c < (1 << 20) && blocks < (1 << 12))
            return static_cast<int>(static_cast<uint32_t>(x) * static_cast<uint32_t>(blocks) / static_cast<uint32_t>(c));
        return static_cast<int>(static_cast<double>(x) * blocks / static_cast<double>(c));
    }

    int b, h, m;
    int64_t x;     // offset in the item
    int64_t left;  // cost left
    SeqItems q;

    // The next item with key blocks for this CTA; Item::none() at the end.  `end_cost`: for part 2, the cost of the
    // item behind this CTA's share.
    __device__ __forceinline__ Item next(const BatchView &v, int kv_heads, int tile_tokens, int group, int64_t &end_cost)
    {
        Item it;
        while (left > 0) {
            if (m >= q.tiles) {
                m = 0;
                x = 0;
                if (++h >= kv_heads) {
                    h = 0;
                    bool ignored = false;
                    do {
                        if (++b >= v.num_seqs) {
                            left = 0;
                            return Item::none();
                        }
                        q.set(load_seq(v, b, ignored), v, tile_tokens);
                    } while (q.tiles == 0);
                }
            }
            const int64_t c = q.cost(m, tile_tokens);
            const int64_t x1 = min(c, x + left);
            const int first = m * tile_tokens;
            const int tokens = min(q.s.fresh - first, tile_tokens);
            it.keys = max(q.past + first + tokens, 0);
            const int blocks = max((it.keys + KEY_BLOCK - 1) / KEY_BLOCK, 1);
            const int t0 = x == 0 ? 0 : block_at(x, blocks, c);
            const int t1 = x1 == c ? blocks : block_at(x1, blocks, c);
            end_cost = c - x1;
            left -= x1 - x;
            it.t0 = t0;
            it.seen_first = max(q.past + first + 1, 0);
            it.rows = tokens * group;
            it.past0 = q.past + first;
            it.token0 = q.s.first + first;
            it.head = h;
            it.seq = b;
            it.part = t0 > 0 ? 1 : t1 < blocks ? 2 : 0;
            x = 0;
            ++m;
            if (t1 > t0) {
                it.blocks = t1 - t0;
                return it;
            }
        }
        return Item::none();
    }
};

struct WalkStart {
    int b, h, m;
    int64_t x, left;
    int64_t total;
    SeqItems q;  // of sequence b
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
    SeqItems q;  // kept where the thread has one sequence alone
    for (int b = b0; b < b1; ++b) {
        q.set(load_seq(v, b, bad), v, tile_tokens);
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
    const int used = min(THREADS / 32, (v.num_seqs + 32 * per - 1) / (32 * per));  // warps with sequences
    for (int w = 0; w < used; ++w) {
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
            if (per > 1)
                q.set(load_seq(v, b, bad), v, tile_tokens);
            const int64_t one = q.total(tile_tokens);
            if (from < at + one * kv_heads) {
                int64_t off = from - at;
                st->b = b;
                st->h = (off | one) >> 32 ? static_cast<int>(off / one)
                                          : static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(one));
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
                st->q = q;
                break;
            }
            at += one * kv_heads;
        }
    }
    __syncthreads();
}

}  // namespace attn
}  // namespace nvfp4
