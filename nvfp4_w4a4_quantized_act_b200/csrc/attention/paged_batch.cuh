// paged_batch.cuh -- the device's view of a step's batch and of the paged
// cache, with every value that comes from device memory checked before it
// becomes an address.
#pragma once

#include <cstdint>

#include "status.cuh"

namespace nvfp4 {
namespace attn {

struct BatchView {
    const int32_t *table;
    const int32_t *cu;
    const int32_t *lens;
    int64_t table_stride;
    int32_t num_seqs;
    int32_t max_pages;
    int32_t page_shift;  // page_size = 1 << page_shift
    int32_t tokens;      // token rows of the call
    int64_t num_pages;
    // how a kernel shares the batch (attention_schedule.cuh): the sequences it takes, by their new tokens, and what
    // an item costs beside its keys
    int32_t fresh_min, fresh_max;
    int32_t item_cost;
};

// One sequence: rows [first, first + fresh) of the call, `len` cached
// positions.  Row j sits at position len - fresh + j.
struct Seq {
    int32_t first, fresh, len;
};

// Sequence b with its offsets (c0, c1) clamped to the call's rows and its
// length n to the table's pages; `bad` is set when a clamp changed something.
__device__ __forceinline__ Seq clamp_seq(const BatchView &v, int b, int32_t c0, int32_t c1, int32_t n, bool &bad)
{
    const int64_t cap = static_cast<int64_t>(v.max_pages) << v.page_shift;
    Seq s;
    s.first = min(max(c0, 0), v.tokens);
    s.fresh = min(max(c1, s.first), v.tokens) - s.first;
    s.len = static_cast<int32_t>(min(static_cast<int64_t>(max(n, 0)), cap));
    bad |= (s.first != c0) | (s.first + s.fresh != c1) | (s.len != n) | (b == 0 && c0 != 0);
    return s;
}

__device__ __forceinline__ Seq load_seq(const BatchView &v, int b, bool &bad)
{
    return clamp_seq(v, b, __ldg(v.cu + b), __ldg(v.cu + b + 1), __ldg(v.lens + b), bad);
}

// Last sequence b with cu[b] <= t (t < cu[num_seqs]), found by the 32 lanes
// of a warp together: each round narrows the range to one of 32 parts, and in
// the last one every lane has what load_seq() reads of its sequence already.
__device__ __forceinline__ Seq warp_find_seq(const BatchView &v, int32_t t, int lane, int &b, bool &bad)
{
    int lo = 0, n = v.num_seqs;  // the answer lies in [lo, lo + n)
    // offsets ascend, so the lanes that hold form a prefix; lane 0 may miss only on malformed offsets
    while (n > 32) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, at < n && __ldg(v.cu + lo + at) <= t);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    int32_t c0 = 0, c1 = 0, len = 0;
    if (lane < n) {
        c0 = __ldg(v.cu + lo + lane);
        c1 = __ldg(v.cu + lo + lane + 1);
        len = __ldg(v.lens + lo + lane);
    }
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, lane < n && c0 <= t);
    const int k = m ? 31 - __clz(m) : 0;
    b = lo + k;
    return clamp_seq(v, b, __shfl_sync(0xFFFFFFFFu, c0, k), __shfl_sync(0xFFFFFFFFu, c1, k), __shfl_sync(0xFFFFFFFFu, len, k), bad);
}

}  // namespace attn
}  // namespace nvfp4
