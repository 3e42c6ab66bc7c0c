// paged_attention_kernel.cuh -- causal attention of new tokens over the paged
// FP8 cache on the tcgen05 tensor cores.
//
//   s_i = c * sum_d q[d] k_code[i][d],  c = softmax_scale * k_scale
//   out = v_scale * sum_i 2^(t_i - r) v_code[i] / sum_i 2^(t_i - r),  t = s log2(e)
//
// Keys and values go from their pages to the tensor cores as they are stored:
// both products run as 8-bit MMAs, K and V tiles unconverted.  The 16-bit
// operand beside them is split into two E4M3 terms, high and low, which
// accumulate into the same fp32 accumulator; two MMAs at the 8-bit rate cost
// what one 16-bit MMA would, without a conversion pass over K and V and with
// half the shared memory for them.
//   Queries: a row is scaled by a power of two to put its largest element in
//   [128, 256); high = E4M3(x), low = E4M3(x - high).  A bf16 value has 8
//   significant bits, two E4M3 values 4 each: exact down to 2^-10 of the row's
//   largest, off by at most 2^-17 of the largest below.
//   Probabilities: 2^(t - r + 8) with r within a few units of the largest t of
//   the block of 128 keys, so the block's largest lies in [2^5, 2^8.75];
//   high keeps 4 significant bits by truncation, low = E4M3(p - high): 8 bits
//   together, as bf16 would keep, and never coarser than 2^-14 of the block's
//   largest.  The reference r follows the block's maximum both ways (not only
//   up, as a running maximum would): after a key far above the rest, a sink,
//   the others keep their precision.  When r moves, the accumulated row is
//   rescaled by the exact difference; r never falls more than 40 below the
//   largest t so far, under which nothing counts in 32 bits anyway.
//
// One CTA per SM; query tile of 128 rows (tokens x query heads of one key
// head) against blocks of 128 keys; work is shared by attention_schedule.cuh.
//   warp 0       loads K and V blocks page by page (4-D TMA, 128-byte
//                swizzle) into a ring of stages
//   warp 1       TMEM; one lane issues the MMAs: scores of block j+1 before
//                the values of block j, so the softmax of one block runs under
//                the MMAs of the next
//   warps 4..11  two threads per row (64 keys each): softmax, probabilities to
//                TMEM over the scores, rescaling, queries to shared memory,
//                results
// TMEM: D columns of output, two buffers of 128 score columns.  P of a block
// replaces its scores: high and low terms, four keys per column.
//
// Keys out of a row's sight must not reach it whatever they hold: scores are
// replaced before the maximum; values meet a zero probability, which only a
// NaN code survives (E4M3 has no infinity), so in blocks that some row does
// not see to the end the softmax threads clear values that no row sees and
// NaN codes in the rest, and remember per dimension the first key with a NaN:
// the rows that see it get their NaN when the result is written.
//
// Every mbarrier wait is bounded in time; when one runs out the kernel
// latches kStatusTimeout and unwinds.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "attention_schedule.cuh"
#include "head_rows_kernels.cuh"
#include "paged_batch.cuh"
#include "ptx_f8.cuh"
#include "status.cuh"

namespace nvfp4 {
namespace attn {

constexpr int ATTN_THREADS = 384;
constexpr int SOFT_WARP0 = 4;
constexpr int SOFT_THREADS = 256;
constexpr uint64_t ATTN_WAIT_NS = 2000000000ull;
constexpr uint32_t TMEM_COLS = 512;
constexpr float P_SHIFT = 8.0f;       // the block's largest probability is near 2^P_SHIFT
constexpr float REF_UP = 0.75f;       // r moves when the block's largest t leaves [r - REF_DOWN, r + REF_UP]
constexpr float REF_DOWN = 3.0f;      // 2^(8 + 0.75) < 448
constexpr float REF_SPAN = 40.0f;

// What a CTA leaves in the workspace: the state of an item it did not do
// alone.  Slot 0: the first item, begun by an earlier CTA; slot 1: the last,
// finished by later ones.
struct PartInfo {
    int32_t continues;  // slot 0 holds a part
    int32_t owns;       // slot 1 holds the first part of an item that ends in CTA `last`
    int32_t last;
    int32_t token0;     // first token row of the item
    int32_t rows;
    int32_t group0;     // first query head
    int32_t past0;      // position of the item's first token
    int32_t pad;
};

struct AttnParams {
    HeadRows q, gate, out;    // gate.data null: no gate
    const float *k_scale, *v_scale;
    int32_t kv_heads, group, tile_tokens;
    float softmax_scale;
    BatchView batch;
    // place of the page's row, head and page coordinate in the tensor maps (1..3)
    int32_t k_row_at, k_head_at, v_row_at, v_head_at;
    PartInfo *parts;          // [CTAS]
    float *part_o;            // [CTAS][2][part_rows][D]
    float *part_ml;           // [CTAS][2][part_rows][2]: r, sum
    int32_t part_rows;
    uint32_t *out_amax;
    uint32_t *status;
};

template <int D>
struct AttnShape {
    static constexpr int SUBS = D / 128;                        // 128-byte wide sub-tiles of a row
    static constexpr uint32_t SUB_BYTES = 128 * 128;
    static constexpr uint32_t Q_BYTES = 2 * SUBS * SUB_BYTES;   // high and low terms
    static constexpr uint32_t STAGE_BYTES = SUBS * SUB_BYTES;   // 128 keys of K or V
    static constexpr int STAGES = D == 256 ? 4 : 8;
    static constexpr uint32_t O_COL = 0;
    static constexpr uint32_t S_COL = 256;
};

template <int D>
struct AttnSmem {
    uint64_t full[AttnShape<D>::STAGES], empty[AttnShape<D>::STAGES];
    uint64_t s_full[2], p_ready[2];
    uint64_t pv_done, q_ready, o_free, drain;
    uint32_t tmem_base;
    volatile int32_t abort_flag;
    WalkStart start;
    int64_t scratch[ATTN_THREADS / 32];
    float red[2][2][ROW_TILE];     // block maximum of each half row, by block parity
    float row_scale[ROW_TILE];     // 1 / (power of two of the query row); NaN: the row is not finite
    float sum[2][ROW_TILE];
    int32_t nan_any[2];            // by item parity
    int32_t nan_key[2][D];         // first key with a NaN value in this dimension
};

template <int D>
constexpr uint32_t attn_smem_bytes()
{
    return AttnShape<D>::Q_BYTES + AttnShape<D>::STAGES * AttnShape<D>::STAGE_BYTES + 1024 + sizeof(AttnSmem<D>);
}

template <int D>
__device__ __forceinline__ void attn_timeout(AttnSmem<D> *sm, uint32_t *status)
{
    sm->abort_flag = 1;
    atomicOr(status, kStatusTimeout);
}

// Order in which K and V blocks of an item of n blocks pass through the ring:
// K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int ring_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int ring_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

__device__ __forceinline__ float block_max64(const uint32_t (&v)[64])
{
    float a = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1])), b = fmaxf(__uint_as_float(v[2]), __uint_as_float(v[3]));
#pragma unroll
    for (int i = 4; i < 64; i += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(v[i])), __uint_as_float(v[i + 1]));
        b = fmaxf(fmaxf(b, __uint_as_float(v[i + 2])), __uint_as_float(v[i + 3]));
    }
    return fmaxf(a, b);
}

// One bf16 query row (8 elements of each lane, D / 8 lanes) as two E4M3 terms.
template <int D>
__device__ __forceinline__ void split_query(const uint4 &v, uint2 &hi, uint2 &lo, float &unscale)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        mag = __vmaxu2(mag, w[i] & 0x7FFF7FFFu);
    mag = max(mag & 0xFFFFu, mag >> 16);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
        mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, o));
    // exponent field e of the largest: scale by 2^(134 - e); at most 2^127
    const int e = static_cast<int>(mag >> 7);
    const int up = min(134 - e, 127);
    const float scale = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    unscale = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
    uint32_t hw[2], lw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = __uint_as_float(w[2 * i] << 16) * scale, b = __uint_as_float(w[2 * i] & 0xFFFF0000u) * scale;
        const float c = __uint_as_float(w[2 * i + 1] << 16) * scale, d = __uint_as_float(w[2 * i + 1] & 0xFFFF0000u) * scale;
        hw[i] = f32_to_e4m3x4(a, b, c, d);
        lw[i] = f32_to_e4m3x4(a - e4m3_to_f32(hw[i]), b - e4m3_to_f32(hw[i] >> 8), c - e4m3_to_f32(hw[i] >> 16),
                              d - e4m3_to_f32(hw[i] >> 24));
    }
    hi = make_uint2(hw[0], hw[1]);
    lo = make_uint2(lw[0], lw[1]);
}

template <int D>
__global__ void __launch_bounds__(ATTN_THREADS, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const AttnParams p)
{
    using A = AttnShape<D>;
    extern __shared__ uint8_t attn_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
    AttnSmem<D> *sm = reinterpret_cast<AttnSmem<D> *>(smem + A::Q_BYTES + A::STAGES * A::STAGE_BYTES);
    const uint32_t q_smem = smem_u32(smem), ring = q_smem + A::Q_BYTES;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < A::STAGES; ++s) {
            mbar_init(smem_u32(&sm->full[s]), 1);
            mbar_init(smem_u32(&sm->empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm->s_full[i]), 1);
            mbar_init(smem_u32(&sm->p_ready[i]), SOFT_THREADS / 32);
            sm->nan_any[i] = 0;
        }
        mbar_init(smem_u32(&sm->pv_done), 1);
        mbar_init(smem_u32(&sm->q_ready), SOFT_THREADS / 32);
        mbar_init(smem_u32(&sm->o_free), SOFT_THREADS / 32);
        mbar_init(smem_u32(&sm->drain), 1);
        sm->abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    for (int i = tid; i < 2 * D; i += ATTN_THREADS)
        sm->nan_key[i / D][i % D] = INT_MAX;
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm->tmem_base), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    grid_dep_wait();
    grid_dep_launch_dependents();

    const float ks = __ldg(p.k_scale), vs = __ldg(p.v_scale);
    const bool scales_ok = valid_scale(ks) && valid_scale(vs);
    bool bad = false;
    find_start<ATTN_THREADS>(p.batch, p.kv_heads, p.tile_tokens, cta, &sm->start, sm->scratch, bad);
    if (cta == 0) {
        if (!scales_ok && tid == 0)
            atomicOr(p.status, kStatusNonFinite);
        if (bad)
            atomicOr(p.status, kStatusBadIndex);
    }
    if (!scales_ok && tid == 0)
        sm->start.left = 0;
    __syncthreads();

    Walk walk;
    walk.b = sm->start.b;
    walk.h = sm->start.h;
    walk.m = sm->start.m;
    walk.x = sm->start.x;
    walk.left = sm->start.left;
    if (walk.left > 0) {
        bool ignored = false;
        walk.q.set(load_seq(p.batch, walk.b, ignored), p.tile_tokens);
    }

    if (warp == 0) {
        // ------------------------------------------------------ loads
        const int shift = p.batch.page_shift, page = 1 << shift;
        const int rows = min(page, KEY_BLOCK);        // rows of a box
        const int boxes = KEY_BLOCK / rows;
        int64_t fills = 0;
        bool ok = true;
        for (bool first = true; ok && walk.next(p.batch, p.kv_heads, p.tile_tokens, first); first = false) {
            const int n = walk.t1 - walk.t0;
            const int32_t *table = p.batch.table + walk.b * p.batch.table_stride;
            // page of this lane's box in block t; -1: nothing to load
            auto page_of = [&](int t) -> int32_t {
                const int key = t * KEY_BLOCK + lane * rows;
                return (t < walk.t1 && lane < boxes && key < walk.keys) ? __ldg(table + (key >> shift)) : -1;
            };
            auto wanted = [&](int t) -> bool {
                return t < walk.t1 && lane < boxes && t * KEY_BLOCK + lane * rows < walk.keys;
            };
            auto load = [&](const CUtensorMap *map, int row_at, int head_at, int t, int32_t id) -> bool {
                const int stage = static_cast<int>(fills % A::STAGES);
                const uint32_t phase = static_cast<uint32_t>(fills / A::STAGES) & 1u;
                const uint32_t bar = smem_u32(&sm->full[stage]);
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, wanted(t)));
                bool good = true;
                if (lane == 0) {
                    good = mbar_wait_bounded(smem_u32(&sm->empty[stage]), phase ^ 1u, ATTN_WAIT_NS);
                    if (good)
                        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(count * rows * D));
                    else
                        attn_timeout(sm, p.status);
                }
                good = __shfl_sync(0xFFFFFFFFu, static_cast<int>(good), 0) != 0 && !sm->abort_flag;
                good = __all_sync(0xFFFFFFFFu, good);
                if (!good)
                    return false;
                if (wanted(t)) {
                    const int row = (t * KEY_BLOCK + lane * rows) & (page - 1);
                    const uint32_t dst = ring + stage * A::STAGE_BYTES + lane * rows * 128;
                    const int32_t c1 = row_at == 1 ? row : head_at == 1 ? walk.h : id;
                    const int32_t c2 = row_at == 2 ? row : head_at == 2 ? walk.h : id;
                    const int32_t c3 = row_at == 3 ? row : head_at == 3 ? walk.h : id;
#pragma unroll
                    for (int s = 0; s < A::SUBS; ++s)
                        tma_load_4d(dst + s * A::SUB_BYTES, map, s * 128, c1, c2, c3, bar);
                }
                ++fills;
                return true;
            };
            int32_t id = page_of(walk.t0), id_next = page_of(walk.t0 + 1);
            bool out_of_pool = false;
            ok = load(&tmK, p.k_row_at, p.k_head_at, walk.t0, id);
            for (int j = 0; ok && j < n; ++j) {
                const int t = walk.t0 + j;
                out_of_pool |= wanted(t) && (id < 0 || id >= p.batch.num_pages);
                const int32_t id_after = page_of(t + 2);
                if (j + 1 < n)
                    ok = load(&tmK, p.k_row_at, p.k_head_at, t + 1, id_next);
                if (ok)
                    ok = load(&tmV, p.v_row_at, p.v_head_at, t, id);
                id = id_next;
                id_next = id_after;
            }
            if (out_of_pool)
                atomicOr(p.status, kStatusBadIndex);
        }
        // when unwinding, copies in flight land before the shared memory goes away
        if (lane == 0 && sm->abort_flag)
            for (int64_t f = max(fills - A::STAGES, int64_t(0)); f < fills; ++f)
                mbar_wait_bounded(smem_u32(&sm->full[f % A::STAGES]), static_cast<uint32_t>(f / A::STAGES) & 1u, ATTN_WAIT_NS);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMAs
        if (lane == 0) {
            // E4M3 x E4M3 -> fp32, M = 128; scores: N = 128 keys, K-major; values: N = D, V's dimensions contiguous
            constexpr uint32_t IDESC_S = (1u << 4) | (uint32_t(KEY_BLOCK >> 3) << 17) | (uint32_t(ROW_TILE >> 4) << 24);
            constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(ROW_TILE >> 4) << 24);
            const uint64_t qdesc = smem_desc(q_smem, 16, 1024, 2);
            const uint64_t kdesc = smem_desc(ring, 16, 1024, 2);
            // V: rows of 128 bytes; 8-key groups 1024 bytes apart, 128-dimension groups a sub-tile apart
            const uint64_t vdesc = smem_desc(ring, A::SUB_BYTES, 1024, 2);
            int64_t fill0 = 0;   // ring position of the item's first block
            int64_t block = 0;   // blocks done
            int item = 0;
            bool ok = true;
            auto wait = [&](uint64_t &bar, uint32_t parity) {
                if (ok && !mbar_wait_bounded(smem_u32(&bar), parity & 1u, ATTN_WAIT_NS)) {
                    attn_timeout(sm, p.status);
                    ok = false;
                }
                ok = ok && !sm->abort_flag;
                return ok;
            };
            auto scores = [&](int j) {
                const int64_t f = fill0 + ring_k(j);
                const int stage = static_cast<int>(f % A::STAGES);
                if (!wait(sm->full[stage], static_cast<uint32_t>(f / A::STAGES)))
                    return;
                tc_fence_after();
                const uint32_t d = tmem + A::S_COL + ((block + j) & 1) * KEY_BLOCK;
                const uint64_t kd = kdesc + ((stage * A::STAGE_BYTES) >> 4);
#pragma unroll
                for (int i = 0; i < 2 * A::SUBS; ++i)  // high terms' sub-tiles, then the low terms'
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f8_ss(d, qdesc + ((i * A::SUB_BYTES) >> 4) + 2 * k,
                                     kd + (((i % A::SUBS) * A::SUB_BYTES) >> 4) + 2 * k, IDESC_S, (i | k) != 0);
                tc_commit(smem_u32(&sm->empty[stage]));
                tc_commit(smem_u32(&sm->s_full[(block + j) & 1]));
            };
            for (bool first = true; ok && walk.next(p.batch, p.kv_heads, p.tile_tokens, first); first = false, ++item) {
                const int n = walk.t1 - walk.t0;
                if (!wait(sm->q_ready, item))
                    break;
                scores(0);
                for (int j = 0; ok && j < n; ++j) {
                    if (j + 1 < n)
                        scores(j + 1);
                    if (j == 0 && item > 0 && !wait(sm->o_free, item - 1))
                        break;
                    const int64_t bl = block + j, f = fill0 + ring_v(j, n);
                    const int stage = static_cast<int>(f % A::STAGES);
                    if (!wait(sm->p_ready[bl & 1], static_cast<uint32_t>(bl >> 1)) ||
                        !wait(sm->full[stage], static_cast<uint32_t>(f / A::STAGES)))
                        break;
                    tc_fence_after();
                    const uint32_t pb = tmem + A::S_COL + (bl & 1) * KEY_BLOCK;
                    const uint64_t vd = vdesc + ((stage * A::STAGE_BYTES) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // 32 keys: 8 columns of high terms, 16 columns on their low terms; each half row has its own 64
                        const uint32_t a = pb + (k >> 1) * 64 + (k & 1) * 8;
                        const uint64_t b = vd + ((k * 4096) >> 4);
                        tc_mma_f8_ts(tmem + A::O_COL, a, b, IDESC_O, (j | k) != 0);
                        tc_mma_f8_ts(tmem + A::O_COL, a + 16, b, IDESC_O, 1);
                    }
                    tc_commit(smem_u32(&sm->empty[stage]));
                    tc_commit(smem_u32(&sm->pv_done));
                }
                block += n;
                fill0 += 2 * n;
            }
            // every tcgen05 operation of this thread ends before TMEM is freed
            tc_commit(smem_u32(&sm->drain));
            if (!mbar_wait_bounded(smem_u32(&sm->drain), 0, ATTN_WAIT_NS))
                attn_timeout(sm, p.status);
        }
    } else if (warp >= SOFT_WARP0) {
        // ------------------------------------------------------ softmax
        const int quarter = warp & 3, half = (warp - SOFT_WARP0) >> 2, sw = warp - SOFT_WARP0;
        const int st = tid - SOFT_WARP0 * 32;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const float c = p.softmax_scale * ks * 1.4426950408889634f;
        PartInfo info;
        info.continues = info.owns = 0;
        info.last = info.token0 = info.rows = info.group0 = info.past0 = info.pad = 0;
        int64_t block = 0, fill0 = 0;
        int item = 0;
        bool fail = false;  // a wait of this thread ran out; the barriers' votes make it everyone's
        uint32_t amax = 0;

        // Queries of row tile (b, h, m) to shared memory, as two E4M3 terms
        auto load_queries = [&](const Walk &w) {
            constexpr int LANES = D / 8, GROUP = 32 / LANES;
            const int col = (lane % LANES) * 8;
            const int rows = min(w.q.s.fresh - w.m * p.tile_tokens, p.tile_tokens) * p.group;
            const int token0 = w.q.s.first + w.m * p.tile_tokens;
#pragma unroll 4
            for (int base = sw * GROUP; base < ROW_TILE; base += 8 * GROUP) {
                if (base >= rows)
                    break;
                const int r = base + lane / LANES;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int t = r / p.group, g = r - t * p.group;
                    v = *reinterpret_cast<const uint4 *>(p.q.data + (token0 + t) * p.q.token_stride +
                                                         (w.h * p.group + g) * p.q.head_stride + col);
                }
                uint2 hi, lo;
                float unscale;
                split_query<D>(v, hi, lo, unscale);
                uint8_t *at = smem + (col >> 7) * A::SUB_BYTES + r * 128 + ((col & 127) ^ ((r & 7) << 4));
                *reinterpret_cast<uint2 *>(at) = hi;
                *reinterpret_cast<uint2 *>(at + A::SUBS * A::SUB_BYTES) = lo;
                if ((lane % LANES) == 0)
                    sm->row_scale[r] = unscale;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm->q_ready));
        };

        bool more = walk.next(p.batch, p.kv_heads, p.tile_tokens, true);
        if (more)
            load_queries(walk);
        while (more) {
            const int n = walk.t1 - walk.t0;
            const int rows = min(walk.q.s.fresh - walk.m * p.tile_tokens, p.tile_tokens) * p.group;
            const int past0 = walk.q.past + walk.m * p.tile_tokens;
            const bool live = row < rows;
            const bool warp_live = quarter * 32 < rows;
            const int seen = live ? max(past0 + row / p.group + 1, 0) : 0;  // keys in this row's sight
            const int seen_first = walk.q.keys_first(walk.m, p.tile_tokens);
            const int np = item & 1;
            float f = 0.0f, ref = 0.0f, top = -INFINITY, sum = 0.0f;
            bool stop = false;
            named_barrier_any(1, SOFT_THREADS, false);  // row_scale of this item is written
            if (live) {
                f = sm->row_scale[row] * c;
                f = f < 1.17549435e-38f ? 1.17549435e-38f : f;  // keeps (-inf) * f; NaN stays
            }
            for (int j = 0; j < n; ++j) {
                const int t = walk.t0 + j;
                const int64_t bl = block + j;
                const int buf = static_cast<int>(bl & 1);
                if (!mbar_wait_bounded(smem_u32(&sm->s_full[buf]), static_cast<uint32_t>(bl >> 1) & 1u, ATTN_WAIT_NS))
                    fail = true;
                __syncwarp();
                tc_fence_after();
                const uint32_t scol = tmem + A::S_COL + buf * KEY_BLOCK + half * 64 + lanes;
                uint32_t v[64];
                float mine = -INFINITY;
                if (warp_live) {
                    tc_ld_32x32b_x64(scol, v);
                    tc_wait_ld();
                    const int vis = seen - t * KEY_BLOCK - half * 64;  // keys of this half row in sight
                    if (__any_sync(0xFFFFFFFFu, vis < 64)) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            v[i] = i < vis ? v[i] : 0xFF800000u;
                    }
                    mine = block_max64(v);
                    sm->red[buf][half][row] = mine;
                }
                stop = named_barrier_any(1, SOFT_THREADS, fail);
                if (stop)
                    break;
                if (warp_live) {
                    const float tm = fmaxf(mine, sm->red[buf][half ^ 1][row]) * f;
                    float turn = 1.0f;
                    if (tm > -INFINITY) {
                        const bool begun = top > -INFINITY;
                        top = fmaxf(top, tm);
                        if (!begun) {
                            ref = tm;
                        } else if (tm > ref + REF_UP || tm < ref - REF_DOWN) {
                            const float to = fmaxf(tm, top - REF_SPAN);
                            turn = exp2_fast(ref - to);
                            sum *= turn;
                            ref = to;
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, turn != 1.0f)) {
                        // the values of the blocks so far are in the accumulator
                        if (!mbar_wait_bounded(smem_u32(&sm->pv_done), static_cast<uint32_t>(bl - 1) & 1u, ATTN_WAIT_NS))
                            fail = true;
                        __syncwarp();
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            uint32_t o[32];
                            const uint32_t oc = tmem + A::O_COL + half * (D / 2) + k * 32 + lanes;
                            tc_ld_32x32b_x32(oc, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * turn);
                            tc_st_32x32b_x32(oc, o);
                        }
                    }
                    const float base = P_SHIFT - ref;
                    float s0 = 0.0f, s1 = 0.0f;
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x[4], y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = exp2_fast(fmaf(__uint_as_float(v[4 * i + e]), f, base));
                            y[e] = __uint_as_float(__float_as_uint(x[e]) & 0xFFF00000u);
                        }
                        s0 += x[0] + x[1];
                        s1 += x[2] + x[3];
                        hi[i] = f32_to_e4m3x4(y[0], y[1], y[2], y[3]);
                        lo[i] = f32_to_e4m3x4(x[0] - y[0], x[1] - y[1], x[2] - y[2], x[3] - y[3]);
                    }
                    sum += s0 + s1;
                    tc_st_32x32b_x16(scol, hi);
                    tc_st_32x32b_x16(scol + 16, lo);
                    tc_wait_st();
                }
                if ((t + 1) * KEY_BLOCK > seen_first) {
                    // some row does not see the block to its end
                    const int64_t fv = fill0 + ring_v(j, n);
                    const int stage = static_cast<int>(fv % A::STAGES);
                    if (!mbar_wait_bounded(smem_u32(&sm->full[stage]), static_cast<uint32_t>(fv / A::STAGES) & 1u, ATTN_WAIT_NS))
                        fail = true;
                    const int none = walk.keys - t * KEY_BLOCK;         // keys from here on: seen by no row
                    const int some = seen_first - t * KEY_BLOCK;        // from here on: not by every row
#pragma unroll 2
                    for (int i = 0; i < A::SUBS * 4; ++i) {
                        const int chunk = st + SOFT_THREADS * i;        // 16 bytes: key row, sub-tile
                        const int key = (chunk >> 3) & 127;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + A::Q_BYTES + stage * A::STAGE_BYTES) + chunk;
                        if (key >= none) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else if (key >= some) {
                            const uint4 x = *at;
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            uint32_t hit = 0;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                hit |= __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            if (hit) {
                                const int dim = (chunk >> 10) * 128 + ((chunk ^ key) & 7) * 16;
                                uint8_t *bytes = reinterpret_cast<uint8_t *>(at);
                                for (int e = 0; e < 16; ++e)
                                    if ((bytes[e] & 0x7F) == 0x7F) {
                                        atomicMin(&sm->nan_key[np][dim + e], t * KEY_BLOCK + key);
                                        bytes[e] = 0;
                                    }
                                sm->nan_any[np] = 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->p_ready[buf]));
            }
            if (!stop) {
                sm->sum[half][row] = sum;
                stop = named_barrier_any(1, SOFT_THREADS, fail);  // sums and NaN marks are written
            }
            if (stop) {
                fail = true;
                break;
            }
            block += n;
            fill0 += 2 * n;
            const Walk done = walk;
            more = walk.next(p.batch, p.kv_heads, p.tile_tokens, false);
            if (more)
                load_queries(walk);  // every score MMA of the item has completed
            if (!mbar_wait_bounded(smem_u32(&sm->pv_done), static_cast<uint32_t>(block - 1) & 1u, ATTN_WAIT_NS))
                fail = true;
            __syncwarp();
            if (named_barrier_any(1, SOFT_THREADS, fail)) {
                fail = true;
                break;
            }
            tc_fence_after();
            // ------------------------------------------------ results
            const float total = sm->sum[0][row] + sm->sum[1][row];
            const bool whole = done.t0 == 0 && done.t1 == done.blocks;
            const int slot = done.t0 == 0 ? 1 : 0;
            const int token0 = done.q.s.first + done.m * p.tile_tokens;
            const bool has_nan = sm->nan_any[np] != 0;
            const int tk = row / p.group, g = row - tk * p.group;
            const float inv = vs / total;
            const int64_t prow = (static_cast<int64_t>(cta) * 2 + slot) * p.part_rows + row;
            if (warp_live) {
#pragma unroll 1
                for (int k = 0; k < D / 64; ++k) {
                    const int col = half * (D / 2) + k * 32;
                    uint32_t o[32];
                    tc_ld_32x32b_x32(tmem + A::O_COL + col + lanes, o);
                    tc_wait_ld();
                    if (has_nan) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (sm->nan_key[np][col + i] < seen)
                                o[i] = 0x7FC00000u;
                    }
                    if (!live) {
                        // a row of the tile that no token fills
                    } else if (whole) {
                        const uint16_t *gp = p.gate.data + (token0 + tk) * p.gate.token_stride +
                                             (done.h * p.group + g) * p.gate.head_stride + col;
                        uint16_t *op = const_cast<uint16_t *>(p.out.data) + (token0 + tk) * p.out.token_stride +
                                       (done.h * p.group + g) * p.out.head_stride + col;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                y[e] = seen > 0 ? __uint_as_float(o[i + e]) * inv : 0.0f;
                            if (p.gate.data != nullptr) {
                                float gx[8];
                                unpack8(*reinterpret_cast<const uint4 *>(gp + i), gx);
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    y[e] = __fdividef(y[e], 1.0f + __expf(-gx[e]));
                            }
                            const uint4 w = pack8(y);
                            *reinterpret_cast<uint4 *>(op + i) = w;
                            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                amax = __vmaxu2(amax, ww[e] & 0x7FFF7FFFu);
                        }
                    } else {
                        float4 *op = reinterpret_cast<float4 *>(p.part_o + prow * D + col);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            op[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                    __syncwarp();
                }
                if (!whole && live && half == 0) {
                    p.part_ml[prow * 2] = top > -INFINITY ? ref : -INFINITY;
                    p.part_ml[prow * 2 + 1] = total;
                }
            }
            if (!whole) {
                if (slot == 0) {
                    info.continues = 1;
                } else {
                    // the item's last CTA: the one that holds the end of its cost
                    const int64_t all = sm->start.total;
                    const int64_t end = all * (cta + 1) / CTAS + done.q.cost(done.m, p.tile_tokens) - done.x;
                    info.owns = 1;
                    info.last = static_cast<int>((end * CTAS - 1) / all);
                    info.token0 = token0;
                    info.rows = rows;
                    info.group0 = done.h * p.group;
                    info.past0 = past0;
                }
            }
            // NaN marks of the next item but one's parity were last read before this item
            for (int i = st; i < D; i += SOFT_THREADS)
                sm->nan_key[np ^ 1][i] = INT_MAX;
            if (st == 0)
                sm->nan_any[np ^ 1] = 0;
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm->o_free));
            ++item;
        }
        if (fail && lane == 0)
            attn_timeout(sm, p.status);
        if (st == 0)
            p.parts[cta] = info;
        if (p.out_amax != nullptr) {
            amax = max(amax & 0xFFFFu, amax >> 16);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            if (lane == 0 && amax != 0)
                atomicMax(p.out_amax, amax);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the parts of the items that several CTAs worked on: CTA c's last
// item, whose later parts are the first items of CTAs c+1 .. last.  One warp
// per row; the parts are added in the order of their keys.
constexpr int JOIN_ROWS = 8;

template <int D>
__global__ void __launch_bounds__(JOIN_ROWS * 32) paged_attention_join_kernel(const AttnParams p)
{
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    const int row = blockIdx.y * JOIN_ROWS + (threadIdx.x >> 5);
    const PartInfo info = p.parts[cta];
    const float ks = __ldg(p.k_scale), vs = __ldg(p.v_scale);
    if (!info.owns || row >= info.rows || !valid_scale(ks) || !valid_scale(vs))
        return;
    auto slot_of = [&](int c) { return (static_cast<int64_t>(c) * 2 + (c == cta ? 1 : 0)) * p.part_rows + row; };
    auto has = [&](int c) { return c == cta || p.parts[c].continues != 0; };
    float top = -INFINITY;
    for (int c = cta; c <= info.last; ++c)
        if (has(c))
            top = fmaxf(top, p.part_ml[slot_of(c) * 2]);
    constexpr int PER = D / 32;
    float o[PER], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        o[i] = 0.0f;
    for (int c = cta; c <= info.last; ++c) {
        if (!has(c))
            continue;
        const int64_t s = slot_of(c);
        // no key in sight in any part: weight 1 keeps the zero or NaN sums
        const float w = top > -INFINITY ? exp2_fast(p.part_ml[s * 2] - top) : 1.0f;
        sum = fmaf(w, p.part_ml[s * 2 + 1], sum);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(p.part_o + s * D + i * 128 + lane * 4);
            o[4 * i] = fmaf(w, x.x, o[4 * i]);
            o[4 * i + 1] = fmaf(w, x.y, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(w, x.z, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(w, x.w, o[4 * i + 3]);
        }
    }
    const int tk = row / p.group, h = info.group0 + row - tk * p.group;
    const bool empty = info.past0 + tk < 0;
    const float inv = vs / sum;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
        const int col = i * 128 + lane * 4;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = empty ? 0.0f : o[4 * i + e] * inv;
        if (p.gate.data != nullptr) {
            const uint2 gw = *reinterpret_cast<const uint2 *>(p.gate.data + (info.token0 + tk) * p.gate.token_stride +
                                                              h * p.gate.head_stride + col);
            const float gx[4] = {__uint_as_float(gw.x << 16), __uint_as_float(gw.x & 0xFFFF0000u),
                                 __uint_as_float(gw.y << 16), __uint_as_float(gw.y & 0xFFFF0000u)};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = __fdividef(y[e], 1.0f + __expf(-gx[e]));
        }
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(y[0], y[1]), b1 = __floats2bfloat162_rn(y[2], y[3]);
        const uint2 w = make_uint2(*reinterpret_cast<const uint32_t *>(&b0), *reinterpret_cast<const uint32_t *>(&b1));
        *reinterpret_cast<uint2 *>(const_cast<uint16_t *>(p.out.data) + (info.token0 + tk) * p.out.token_stride +
                                   h * p.out.head_stride + col) = w;
        amax = __vmaxu2(__vmaxu2(amax, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
    }
    if (p.out_amax != nullptr) {
        amax = max(amax & 0xFFFFu, amax >> 16);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
        if (lane == 0 && amax != 0)
            atomicMax(p.out_amax, amax);
    }
}

}  // namespace attn
}  // namespace nvfp4
