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
//   Probabilities: 2^(t - r + 8), in f16; high keeps 4 significant bits by
//   truncation, low = E4M3(p - high), ties to even: 8 bits together, as bf16
//   would keep, but no finer than 2^-9.  So the reference r has to keep the
//   probabilities up: it follows the blocks of 128 keys both ways, not only up
//   as a running maximum would (after a key far above the rest, a sink, the
//   others would lose their bits).  r moves up when a block's largest t is more than 0.75
//   above it (2^8.75 < 448), and down when it is more than 3 below while the
//   sum so far is under 32 for each block: so the 128 errors of at most 2^-9
//   of a block stay under 2^-7 of its share of the sum, in the worst case of
//   keys that all round the same way.  A new r lies 1.5 above (3 above on the
//   way down) the block's largest, so that the blocks around it fit; the
//   accumulated row is rescaled by the exact difference.  r never falls more
//   than 40 below the largest t so far, under which nothing counts in 32 bits.
//
// One CTA per SM; query tile of 128 rows (tokens x query heads of one key
// head) against blocks of 128 keys; work is shared by attention_schedule.cuh.
//   warps 0, 3   load K blocks and V blocks page by page (4-D TMA, 128-byte
//                swizzle) into a ring of stages
//   warp 1       TMEM; one lane issues the MMAs: scores of block j+1 before
//                the values of block j, so the softmax of one block runs under
//                the MMAs of the next
//   warp 2       walks the CTA's items, four ahead of the others, and brings
//                their queries and gates into L2
//   warps 4..7   one thread per row: rescaling of the accumulated rows, values
//                out of sight, results
//   warps 8..15  two threads per row (64 keys each): softmax, probabilities to
//                TMEM over the scores, queries to shared memory
// The softmax of a block has the time of two products (2 x 1060 cycles at
// D = 256) before the tensor cores would wait for it; everything that is not
// on its path is done by other warps beside it.  An SM's quarter issues such
// code at one instruction in two cycles, so instructions count, not units: a
// block's 2 x 64 scores of a quarter take some 2250 cycles (350 for the
// maximum, 300 for the reference, 2 x 800 for powers and terms), and powers
// moved from the special-function unit to the FMA pipe made it slower.
//
// Measured, the same call again and again (24 query heads on 4 key heads of
// 256): four chunks of 509 tokens over histories to 16384, 354 GFLOP, 314 us,
// 1.13 PFLOP/s; a prompt of 8192, 825 GFLOP, 800 to 850 us, 0.97 to 1.03
// PFLOP/s, where the board's 1.63 for plain 16-bit products is the measure
// (among other calls, with inputs that change, 362 and 858 us).  32 heads on 8
// of 128: a prompt of 4000, 131 GFLOP, 223 us, 0.59 PFLOP/s: the softmax is the
// same for half the products.  At D = 256 a block takes 2300 to 2600 cycles, 2130 of them
// on the tensor cores: the softmax bounds it.  From one item's last block to
// the next one's first go 20 thousand cycles (8 rows of queries a warp split
// into terms, and a row of results a lane, gated): at D = 256 the accumulator
// and two blocks of scores fill TMEM, so nothing of the next item's values can
// begin before.  Eight warps for the results in place of four, with fewer
// registers for the softmax, gained nothing.  With K and V fetched by one warp that
// read the page table block by block, the chunks took 551 thousand cycles a
// CTA, now 454.
// TMEM: D columns of output, two buffers of 128 score columns.  P of a block
// replaces its scores: high and low terms, four keys per column.
//
// Keys out of a row's sight must not reach it whatever they hold: scores are
// replaced before the maximum; values meet a zero probability, which only a
// NaN code survives (E4M3 has no infinity), so in blocks that some row does
// not see to the end warps 4..7 clear values that no row sees and NaN codes in
// the rest, and remember per dimension the first key with a NaN:
// the rows that see it get their NaN when the result is written.
//
// Every mbarrier wait is bounded in time; when one runs out the kernel
// latches kStatusTimeout and unwinds.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_schedule.cuh"
#include "head_rows_kernels.cuh"
#include "paged_batch.cuh"
#include "ptx_f8.cuh"
#include "status.cuh"

namespace nvfp4 {
namespace attn {

constexpr int ATTN_THREADS = 512;
constexpr int ROW_WARP0 = 4;        // warps 4..7: one thread per row
constexpr int SOFT_WARP0 = 8;       // warps 8..15: softmax
constexpr int SOFT_THREADS = 256;
constexpr int STAGE_LD = 36;        // floats of a row of the results' staging: 32 columns, spread over the banks
constexpr uint64_t ATTN_WAIT_NS = 2000000000ull, ATTN_DRAIN_NS = 10000000ull;
constexpr uint32_t TMEM_COLS = 512;
constexpr float P_SHIFT = 8.0f;       // probabilities are 2^(t - r + P_SHIFT)
constexpr float P_UNIT = 256.0f;      // 2^P_SHIFT
constexpr float REF_UP = 0.75f;       // 2^(P_SHIFT + REF_UP) < 448
constexpr float REF_DOWN = 3.0f;
constexpr float BLOCK_SUM = 32.0f;    // 2^(P_SHIFT - REF_DOWN): a block above that edge has it in its largest alone
constexpr float SLACK_UP = 1.5f;      // how far a new r lies above the block's largest t
constexpr float SLACK_DOWN = 3.0f;
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

struct Parts {
    PartInfo *info;  // [CTAS]
    float *o;        // [CTAS][2][rows][D]
    float *ml;       // [CTAS][2][rows][2]: reference, sum
    int32_t rows;
};

struct AttnParams {
    HeadRows q, gate, out;    // gate.data null: no gate
    const float *k_scale, *v_scale;
    int32_t kv_heads, group, tile_tokens;
    float softmax_scale;
    BatchView batch;
    // place of the page's row, head and page coordinate in the tensor maps (1..3)
    int32_t k_row_at, k_head_at, v_row_at, v_head_at;
    Parts parts;
    uint32_t group_inv;       // ceil(2^16 / group): row / group = row * group_inv >> 16 for rows below 128
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

constexpr int ITEMS = 4;  // items known ahead

template <int D>
struct AttnSmem {
    Item items[ITEMS];
    uint64_t item_ready[ITEMS], item_done[ITEMS];
    uint64_t full[AttnShape<D>::STAGES], empty[AttnShape<D>::STAGES];
    uint64_t s_full[2], turn_ready[2], pv_done[2];
    uint64_t p_ready[2], p_rest[2];  // probabilities of the first 32 keys of each half row, of the others
    uint64_t q_ready, o_free, stats_ready, drain;
    uint32_t tmem_base;
    volatile int32_t abort_flag;
    WalkStart start;
    int64_t scratch[ATTN_THREADS / 32];
    float2 red[2][2][ROW_TILE];    // by block parity: each half row's maximum, and its sum so far
    float turn[2][ROW_TILE];       // factor of the accumulated row before this block, by block parity
    // By item parity, 1 / (power of two of the query row); NaN: the row is not finite.  A warp writes rows of every
    // quarter and reads its own after barrier 5; after an item of a block or two it may write the next item's while
    // another quarter has not read this one's, but it cannot pass the next item's barrier 5 before that.
    float row_scale[2][ROW_TILE];
    float sum[2][2][ROW_TILE];     // by item parity: each half row's sum
    float ref[2][ROW_TILE];        // and the row's reference; -inf: no key seen
    int32_t nan_any[2];            // by item parity
    int32_t nan_key[2][D];         // first key with a NaN value in this dimension
    alignas(16) float staging[4][32 * STAGE_LD];
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

// Place of V block j among the K and V blocks of an item of n blocks, which
// pass through the ring as K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int ring_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

__device__ __forceinline__ float block_max64(const uint32_t (&v)[64])
{
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = __uint_as_float(v[k]);
#pragma unroll
        for (int i = k + 4; i + 4 < 64; i += 8)
            m[k] = max3(m[k], __uint_as_float(v[i]), __uint_as_float(v[i + 4]));
        m[k] = fmaxf(m[k], __uint_as_float(v[60 + k]));
    }
    return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

// Scale of a query row whose largest element has the magnitude bits `mag`: the
// power of two that puts it in [128, 256), and its inverse; NaN for a row that
// is not finite.
__device__ __forceinline__ void query_scale(uint32_t mag, float &scale, float &unscale)
{
    const int e = static_cast<int>(mag >> 7);  // exponent field: scale by 2^(134 - e), at most 2^127
    const int up = min(134 - e, 127);
    scale = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    unscale = e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
}

// Eight scaled query elements as two E4M3 terms.  A scaled value is exact in
// f16 (8 bits; below 2^-14 it is far under the low term's step), and so is x -
// high.
__device__ __forceinline__ void split8(const uint4 &v, float scale, uint2 &hi, uint2 &lo)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __floats2half2_rn(__uint_as_float(w[i] << 16) * scale, __uint_as_float(w[i] & 0xFFFF0000u) * scale);
        h[i] = f16x2_to_e4m3x2(x);
        l[i] = f16x2_to_e4m3x2(__hsub2(x, e4m3x2_to_f16x2(h[i])));
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// One bf16 query row (8 elements of each lane, D / 8 lanes) as two E4M3 terms.
template <int D>
__device__ __forceinline__ void split_query(const uint4 &v, uint2 &hi, uint2 &lo, float &unscale)
{
    uint32_t mag = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    mag = max(mag & 0xFFFFu, mag >> 16);
    if (D == 256) {
        mag = __reduce_max_sync(0xFFFFFFFFu, mag);
    } else {
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1)
            mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, o));
    }
    float scale;
    query_scale(mag, scale, unscale);
    split8(v, scale, hi, lo);
}

// Four columns of the gate's row; of no effect without a gate.
__device__ __forceinline__ uint2 load_gate4(const AttnParams &p, int32_t token, int32_t head, int col)
{
    uint2 g = make_uint2(0, 0);
    if (p.gate.data != nullptr)
        g = *reinterpret_cast<const uint2 *>(p.gate.data + token * p.gate.token_stride + head * p.gate.head_stride + col);
    return g;
}

// Four columns of an output row: sums times inv (zeros where the row saw no
// key), the gate, bf16.  Returns the running max|out| (two bf16 magnitudes).
__device__ __forceinline__ uint32_t write_row4(const AttnParams &p, const float (&o)[4], float inv, bool empty, const uint2 &gate,
                                               int32_t token, int32_t head, int col, uint32_t amax)
{
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        y[e] = empty ? 0.0f : o[e] * inv;
    if (p.gate.data != nullptr) {
        const float gx[4] = {__uint_as_float(gate.x << 16), __uint_as_float(gate.x & 0xFFFF0000u),
                             __uint_as_float(gate.y << 16), __uint_as_float(gate.y & 0xFFFF0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = __fdividef(y[e], 1.0f + __expf(-gx[e]));
    }
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(y[0], y[1]), b1 = __floats2bfloat162_rn(y[2], y[3]);
    const uint2 w = make_uint2(*reinterpret_cast<const uint32_t *>(&b0), *reinterpret_cast<const uint32_t *>(&b1));
    *reinterpret_cast<uint2 *>(const_cast<uint16_t *>(p.out.data) + token * p.out.token_stride + head * p.out.head_stride + col) = w;
    return __vmaxu2(__vmaxu2(amax, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
}

// Eight results times sigmoid(gate) = 1 / (1 + 2^(-gate log2 e)).
__device__ __forceinline__ void gate8(float (&y)[8], const uint4 &g)
{
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
    const uint64_t minus_log2e = pack2(-1.4426950408889634f, -1.4426950408889634f), one = pack2(1.0f, 1.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t t = mul2(pack2u(w[k] << 16, w[k] & 0xFFFF0000u), minus_log2e);
        float a, b;
        unpack2(add2(exp2_fast2(t), one), a, b);
        unpack2(mul2(pack2(y[2 * k], y[2 * k + 1]), pack2(rcp_fast(a), rcp_fast(b))), y[2 * k], y[2 * k + 1]);
    }
}

// A warp's max|out| into the caller's word.
__device__ __forceinline__ void store_amax(const AttnParams &p, uint32_t amax, int lane)
{
    if (p.out_amax == nullptr)
        return;
    amax = max(amax & 0xFFFFu, amax >> 16);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (lane == 0 && amax != 0)
        atomicMax(p.out_amax, amax);
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
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // uniform to the compiler too
    const int cta = blockIdx.x;

    // Beside the kernel for single tokens this one may find nothing to do: a look at the offsets alone says so, before
    // anything is set up, and the other kernel reports what is malformed.
    if (p.batch.fresh_min > 1) {
        grid_dep_wait();
        bool some = false;
        for (int b = tid; b < p.batch.num_seqs; b += ATTN_THREADS)
            some |= __ldg(p.batch.cu + b + 1) - __ldg(p.batch.cu + b) >= p.batch.fresh_min;
        if (__syncthreads_or(some) == 0) {
            if (tid == 0) {
                PartInfo none;
                none.continues = none.owns = none.last = none.token0 = none.rows = none.group0 = none.past0 = none.pad = 0;
                p.parts.info[cta] = none;
            }
            return;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < A::STAGES; ++s) {
            mbar_init(smem_u32(&sm->full[s]), 1);
            mbar_init(smem_u32(&sm->empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm->s_full[i]), 1);
            mbar_init(smem_u32(&sm->p_ready[i]), SOFT_THREADS / 32 + 4);
            mbar_init(smem_u32(&sm->p_rest[i]), SOFT_THREADS / 32);
            mbar_init(smem_u32(&sm->turn_ready[i]), 4);
            mbar_init(smem_u32(&sm->pv_done[i]), 1);
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(smem_u32(&sm->item_ready[i]), 1);
            mbar_init(smem_u32(&sm->item_done[i]), 4);
        }
        mbar_init(smem_u32(&sm->q_ready), SOFT_THREADS / 32);
        mbar_init(smem_u32(&sm->o_free), 4);
        mbar_init(smem_u32(&sm->stats_ready), SOFT_THREADS / 32);
        mbar_init(smem_u32(&sm->drain), 1);
        sm->abort_flag = 0;
        sm->nan_any[0] = sm->nan_any[1] = 0;
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

    // The next item, from warp 2; Item::none() at the end and when unwinding.  `fail`: whether a wait of this
    // thread, or with warp_item() of its warp, has run out.
    auto thread_item = [&](int i, bool &fail) -> Item {
        fail = fail || !mbar_wait(smem_u32(&sm->item_ready[i % ITEMS]), (i / ITEMS) & 1, ATTN_WAIT_NS);
        return fail ? Item::none() : sm->items[i % ITEMS];
    };
    auto warp_item = [&](int i, bool &fail) -> Item {
        fail = fail || !mbar_wait(smem_u32(&sm->item_ready[i % ITEMS]), (i / ITEMS) & 1, ATTN_WAIT_NS);
        fail = __any_sync(0xFFFFFFFFu, fail);
        return fail ? Item::none() : sm->items[i % ITEMS];
    };

    uint32_t filled = 0, phases = 0;  // stages that this warp has filled, and the last time's phases
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------ loads
        // Warp 0 fetches the K blocks, warp 3 the V blocks, into the ring in the order K0 K1 V0 K2 V1 .. K(n-1) V(n-2)
        // V(n-1).  A lane holds the page of one box, 32 boxes at a time and the next 32 on their way: read block by
        // block, the page table's latency came between any two fetches.
        const bool is_k = warp == 0;
        const int shift = p.batch.page_shift, page = 1 << shift;
        const int rows = min(page, KEY_BLOCK);        // rows of a box
        const int row_shift = min(shift, 7), boxes_shift = 7 - row_shift, boxes = 1 << boxes_shift;
        const CUtensorMap *map = is_k ? &tmK : &tmV;
        const int row_at = is_k ? p.k_row_at : p.v_row_at, head_at = is_k ? p.k_head_at : p.v_head_at;
        uint32_t base = 0;  // ring stages of the items before
        bool fail = false, out_of_pool = false;
        for (int i = 0;; ++i) {
            const Item it = warp_item(i, fail);
            if (it.blocks == 0)
                break;
            const int32_t *table = p.batch.table + it.seq * p.batch.table_stride;
            const int box0 = it.t0 << boxes_shift, box1 = min((it.t0 + it.blocks) << boxes_shift, (it.keys + rows - 1) >> row_shift);
            auto page_of = [&](int box) { return box < box1 ? __ldg(table + ((box << row_shift) >> shift)) : 0; };
            int32_t ids = page_of(box0 + lane), next = page_of(box0 + 32 + lane);
#pragma unroll 1
            for (int j = 0; j < it.blocks; ++j) {
                const int at = j << boxes_shift;  // first box of the block, from box0
                if (j > 0 && (at & 31) == 0) {
                    ids = next;
                    next = page_of(box0 + at + 32 + lane);
                }
                const int32_t id = __shfl_sync(0xFFFFFFFFu, ids, (at + lane) & 31);
                const int box = box0 + at + lane;
                const bool mine = lane < boxes && box < box1;
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, mine));
                const uint32_t fill = base + (is_k ? max(2 * j - 1, 0) : ring_v(j, it.blocks));
                const uint32_t stage = fill % A::STAGES, phase = (fill / A::STAGES) & 1u;
                const uint32_t bar = smem_u32(&sm->full[stage]);
                if (lane == 0) {
                    if (mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1u, ATTN_WAIT_NS))
                        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(count * rows * D));
                    else
                        fail = true;
                }
                fail = __any_sync(0xFFFFFFFFu, fail || sm->abort_flag);
                if (fail)
                    break;
                if (mine) {
                    const int row = (box << row_shift) & (page - 1);
                    const uint32_t dst = ring + stage * A::STAGE_BYTES + lane * rows * 128;
                    const int32_t c1 = row_at == 1 ? row : head_at == 1 ? it.head : id;
                    const int32_t c2 = row_at == 2 ? row : head_at == 2 ? it.head : id;
                    const int32_t c3 = row_at == 3 ? row : head_at == 3 ? it.head : id;
#pragma unroll
                    for (int s = 0; s < A::SUBS; ++s)
                        tma_load_4d(dst + s * A::SUB_BYTES, map, s * 128, c1, c2, c3, bar);
                    out_of_pool |= id < 0 || id >= p.batch.num_pages;
                }
                filled |= 1u << stage;
                phases = (phases & ~(1u << stage)) | phase << stage;
            }
            base += 2 * it.blocks;
        }
        if (out_of_pool)
            atomicOr(p.status, kStatusBadIndex);
        if (fail && lane == 0)
            attn_timeout(sm, p.status);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMAs
        // One lane, elected: with `lane == 0` in place of the election a prompt of 8192 takes 910 us instead of 800 to
        // 850 and chunks of 509 take 378 instead of 340.
        if (elect_one()) {
            // E4M3 x E4M3 -> fp32, M = 128; scores: N = 128 keys, K-major; values: N = D, V's dimensions contiguous
            constexpr uint32_t IDESC_S = (1u << 4) | (uint32_t(KEY_BLOCK >> 3) << 17) | (uint32_t(ROW_TILE >> 4) << 24);
            constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(ROW_TILE >> 4) << 24);
            const uint64_t qdesc = smem_desc(q_smem, 16, 1024, 2);
            const uint64_t kdesc = smem_desc(ring, 16, 1024, 2);
            // V: rows of 128 bytes; 8-key groups 1024 bytes apart, 128-dimension groups a sub-tile apart
            const uint64_t vdesc = smem_desc(ring, A::SUB_BYTES, 1024, 2);
            uint32_t uses = 0;   // ring stages consumed
            uint32_t block = 0;  // blocks of scores begun
            bool fail = false;
            auto wait = [&](uint64_t &bar, uint32_t phase) {
                fail = fail || !mbar_wait(smem_u32(&bar), phase & 1u, ATTN_WAIT_NS);
            };
            for (int i = 0;; ++i) {
                const Item it = thread_item(i, fail);
                if (it.blocks == 0)
                    break;
                wait(sm->q_ready, i);
                wait(sm->full[uses % A::STAGES], uses / A::STAGES);
                // The tensor pipe queues an MMA or two; a wait costs some 70 cycles even when its phase is over.  So
                // each wait comes ahead of the last MMAs before the ones that need it, not between the products.
#pragma unroll 1
                for (int j = -1; j < it.blocks && !fail; ++j) {
                    const bool more = j + 1 < it.blocks;
                    const uint32_t ks = uses % A::STAGES, sbuf = block & 1u;           // K block j + 1
                    const uint32_t vu = uses + (more ? 1 : 0), vst = vu % A::STAGES;   // V block j
                    const uint32_t bl = block - 1, buf = bl & 1u;                      // scores of block j
                    if (more) {
                        tc_fence_after();
                        const uint32_t d = tmem + A::S_COL + sbuf * KEY_BLOCK;
                        const uint64_t kd = kdesc + ((ks * A::STAGE_BYTES) >> 4);
#pragma unroll
                        for (int m = 0; m < 8 * A::SUBS; ++m) {  // high terms' sub-tiles, then the low terms'
                            const int s = m >> 2, k = m & 3;
                            if (m == 8 * A::SUBS - 3 && j >= 0) {
                                if (j == 0 && i > 0)
                                    wait(sm->o_free, i - 1);
                                wait(sm->full[vst], vu / A::STAGES);
                                wait(sm->p_ready[buf], bl >> 1);
                            }
                            tc_mma_f8_ss(d, qdesc + ((s * A::SUB_BYTES) >> 4) + 2 * k,
                                         kd + (((s % A::SUBS) * A::SUB_BYTES) >> 4) + 2 * k, IDESC_S, m != 0);
                        }
                        tc_commit(smem_u32(&sm->empty[ks]));
                        tc_commit(smem_u32(&sm->s_full[sbuf]));
                        ++uses;
                        ++block;
                    } else {
                        if (j == 0 && i > 0)
                            wait(sm->o_free, i - 1);
                        wait(sm->full[vst], vu / A::STAGES);
                        wait(sm->p_ready[buf], bl >> 1);
                    }
                    if (j >= 0) {
                        tc_fence_after();
                        const uint32_t pb = tmem + A::S_COL + buf * KEY_BLOCK;
                        const uint64_t vd = vdesc + ((vst * A::STAGE_BYTES) >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // 32 keys of a half row: 8 columns of high terms, 16 columns on their low terms; each half
                            // has its own 64 columns.  The first 32 keys of both come first.
                            const uint32_t a = pb + (k & 1) * 64 + (k >> 1) * 8;
                            const uint64_t b = vd + ((((k & 1) * 2 + (k >> 1)) * 4096) >> 4);
                            if (k == 2) {
                                wait(sm->p_rest[buf], bl >> 1);
                                tc_fence_after();
                            }
                            if (k == 3 && j + 2 < it.blocks)
                                wait(sm->full[(uses + 1) % A::STAGES], (uses + 1) / A::STAGES);
                            tc_mma_f8_ts(tmem + A::O_COL, a, b, IDESC_O, (j | k) != 0);
                            tc_mma_f8_ts(tmem + A::O_COL, a + 16, b, IDESC_O, 1);
                        }
                        tc_commit(smem_u32(&sm->empty[vst]));
                        tc_commit(smem_u32(&sm->pv_done[buf]));
                        ++uses;
                    } else if (1 < it.blocks) {
                        wait(sm->full[uses % A::STAGES], uses / A::STAGES);
                    }
                }
                if (fail || sm->abort_flag) {
                    fail = true;
                    break;
                }
            }
            // every tcgen05 operation of this thread ends before TMEM is freed
            tc_commit(smem_u32(&sm->drain));
            if (!mbar_wait(smem_u32(&sm->drain), 0, ATTN_WAIT_NS) || fail)
                attn_timeout(sm, p.status);
        }
    } else if (warp == 2) {
        // ------------------------------------------------- items, prefetches
        Walk walk;
        walk.b = sm->start.b;
        walk.h = sm->start.h;
        walk.m = sm->start.m;
        walk.x = sm->start.x;
        walk.left = sm->start.left;
        walk.q = sm->start.q;
        PartInfo info;
        info.continues = info.owns = 0;
        info.last = info.token0 = info.rows = info.group0 = info.past0 = info.pad = 0;
        bool fail = false;
        for (int i = 0;; ++i) {
            int64_t end_cost = 0;
            const Item it = walk.next(p.batch, p.kv_heads, p.tile_tokens, p.group, end_cost);
            const int slot = i % ITEMS;
            if (i >= ITEMS)
                fail = !mbar_wait(smem_u32(&sm->item_done[slot]), ((i / ITEMS) - 1) & 1, ATTN_WAIT_NS);
            fail = __any_sync(0xFFFFFFFFu, fail || sm->abort_flag);
            if (fail)
                break;
            if (lane == 0) {
                sm->items[slot] = it;
                mbar_arrive(smem_u32(&sm->item_ready[slot]));
            }
            if (it.blocks == 0)
                break;
            if (it.part == 1) {
                info.continues = 1;
            } else if (it.part == 2) {
                // the item's last CTA is the one that holds the end of its cost
                const int64_t all = sm->start.total;
                info.owns = 1;
                info.last = static_cast<int>(((all * (cta + 1) / CTAS + end_cost) * CTAS - 1) / all);
                info.token0 = it.token0;
                info.rows = it.rows;
                info.group0 = it.head * p.group;
                info.past0 = it.past0;
            }
#pragma unroll 1
            for (int which = i > 0 ? 0 : 1; which < 2; ++which) {  // the first item's queries are being read already
                const HeadRows &x = which ? p.gate : p.q;
                if (x.data != nullptr && (which == 0 || it.part == 0))
#pragma unroll 1
                    for (int k = lane; k < it.rows * (D / 64); k += 32) {
                        const uint32_t r = k / (D / 64), tk = r * p.group_inv >> 16, g = r - tk * p.group;
                        const uint16_t *at = x.data + (it.token0 + tk) * x.token_stride +
                                             (it.head * p.group + g) * x.head_stride + (k % (D / 64)) * 64;
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                    }
            }
        }
        if (lane == 0) {
            if (fail)
                attn_timeout(sm, p.status);
            p.parts.info[cta] = info;
        }
    } else if (warp >= ROW_WARP0 && warp < SOFT_WARP0) {
        // ------------------------------------------- rows: rescaling, results
        const int quarter = warp & 3, rt = tid - ROW_WARP0 * 32, row = rt;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        float *stage_rows = sm->staging[quarter];
        uint32_t block = 0, uses = 0;
        bool fail = false;  // a wait of this thread ran out
        uint32_t amax = 0;
        auto wait = [&](uint64_t &bar, uint32_t phase) {
            fail = fail || !mbar_wait(smem_u32(&bar), phase & 1u, ATTN_WAIT_NS);
            __syncwarp();
        };
        // The values of block i are in the accumulator.  A wait by parity tells a phase only from its neighbour, so
        // even and odd blocks have a barrier each: here the scores of block i or i + 1 have been seen, so block
        // i - 2 is done, and block i + 2 waits for these warps.
        auto wait_values = [&](uint32_t i) { wait(sm->pv_done[i & 1], i >> 1); };
        for (int i = 0;; ++i) {
            const Item it = warp_item(i, fail);
            const int ip = i & 1;
            const bool live = row < it.rows;
            // keys in this row's sight
            const int seen = live ? max(it.past0 + static_cast<int>(row * p.group_inv >> 16) + 1, 0) : 0;
#pragma unroll 1
            for (int j = 0; j < it.blocks; ++j, ++block) {
                const int key0 = (it.t0 + j) * KEY_BLOCK;
                const int buf = static_cast<int>(block & 1);
                wait(sm->turn_ready[buf], block >> 1);
                const float turn = live ? sm->turn[buf][row] : 1.0f;
                if (__any_sync(0xFFFFFFFFu, turn != 1.0f)) {
                    wait_values(block - 1);  // not the item's first block
                    tc_fence_after();
                    const uint64_t tt = pack2(turn, turn);
#pragma unroll 1
                    for (int k = 0; k < D; k += 64) {
                        uint32_t o[64];
                        tc_ld_32x32b_x64(tmem + A::O_COL + k + lanes, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            float a, b;
                            unpack2(mul2(pack2u(o[e], o[e + 1]), tt), a, b);
                            o[e] = __float_as_uint(a);
                            o[e + 1] = __float_as_uint(b);
                        }
                        tc_st_32x32b_x64(tmem + A::O_COL + k + lanes, o);
                    }
                    tc_wait_st();
                }
                if (key0 + KEY_BLOCK > it.seen_first) {
                    // some row does not see the block to its end
                    const uint32_t fv = uses + ring_v(j, it.blocks), stage = fv % A::STAGES;
                    wait(sm->full[stage], fv / A::STAGES);
                    const int none = it.keys - key0;         // keys from here on: seen by no row
                    const int some = it.seen_first - key0;   // from here on: not by every row
#pragma unroll 1
                    for (int c = rt; c < A::SUBS * 1024; c += 128) {  // 16 bytes: key row, sub-tile
                        const int key = (c >> 3) & 127;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + A::Q_BYTES + stage * A::STAGE_BYTES) + c;
                        if (key >= none) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else if (key >= some) {
                            const uint4 x = *at;
                            const uint32_t hit = __vcmpeq4(x.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                                                 __vcmpeq4(x.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(x.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            if (hit) {
                                const int dim = (c >> 10) * 128 + ((c ^ key) & 7) * 16;
                                uint8_t *bytes = reinterpret_cast<uint8_t *>(at);
#pragma unroll 1
                                for (int e = 0; e < 16; ++e)
                                    if ((bytes[e] & 0x7F) == 0x7F) {
                                        atomicMin(&sm->nan_key[ip][dim + e], key0 + key);
                                        bytes[e] = 0;
                                    }
                                sm->nan_any[ip] = 1;
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
            uses += 2 * it.blocks;
            // ------------------------------------------------ results
            // 32 columns at a time, a lane 8 columns of every 8th row.  Addresses, and the gate's first columns on their
            // way, while the last values are being added up; then the next columns' while these are worked on.
            const bool whole = it.part == 0, gated = whole && p.gate.data != nullptr;
            const int rows_here = it.rows - quarter * 32, sub = lane >> 2, c8 = (lane & 3) * 8;
            const uint16_t *gate_at[4];
            uint16_t *out_at[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = quarter * 32 + e * 8 + sub, tk = r * p.group_inv >> 16;
                const int32_t t = it.token0 + tk, h = it.head * p.group + (r - tk * p.group);
                gate_at[e] = p.gate.data + t * p.gate.token_stride + h * p.gate.head_stride + c8;
                out_at[e] = const_cast<uint16_t *>(p.out.data) + t * p.out.token_stride + h * p.out.head_stride + c8;
            }
            uint4 gv[4] = {};
            auto load_gate = [&](int col) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (gated && col < D && e * 8 + sub < rows_here)
                        gv[e] = *reinterpret_cast<const uint4 *>(gate_at[e] + col);
            };
            load_gate(0);
            if (it.blocks > 0) {
                wait(sm->stats_ready, i);
                wait_values(block - 1);
            }
            // NaN marks are written.  The vote is taken at the end marker too: a warp whose wait ran out comes here
            // whatever the others were given, and none may leave before it has.
            fail = named_barrier_any(6, 128, fail);
            if (fail || it.blocks == 0)
                break;
            tc_fence_after();
            const float total = sm->sum[ip][0][row] + sm->sum[ip][1][row];
            const bool has_nan = sm->nan_any[ip] != 0;
            const float factor = whole ? vs / total : 1.0f;
            const uint64_t ff = pack2(factor, factor);
            if (rows_here > 0) {
                // The accumulator has a row per lane; memory wants a row's columns together: 32 columns at a time
                // pass through shared memory, and a lane takes 16 bytes of every 8th row (results) or 4th (parts).
                auto stage = [&](int col) {
                    uint32_t o[32];
                    tc_ld_32x32b_x32(tmem + A::O_COL + col + lanes, o);
                    tc_wait_ld();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float4 y;
                        unpack2(mul2(pack2u(o[e], o[e + 1]), ff), y.x, y.y);
                        unpack2(mul2(pack2u(o[e + 2], o[e + 3]), ff), y.z, y.w);
                        *reinterpret_cast<float4 *>(stage_rows + lane * STAGE_LD + e) = y;
                    }
                    if (live && (seen == 0 || has_nan)) {  // no key in sight, or perhaps a NaN
#pragma unroll 1
                        for (int e = 0; e < 32; ++e) {
                            if (whole && seen == 0)
                                stage_rows[lane * STAGE_LD + e] = 0.0f;
                            if (sm->nan_key[ip][col + e] < seen)
                                stage_rows[lane * STAGE_LD + e] = __uint_as_float(0x7FC00000u);
                        }
                    }
                    __syncwarp();
                };
                if (whole) {
#pragma unroll 1
                    for (int col = 0; col < D; col += 32) {
                        stage(col);
                        // all four rows at once: a branch between them would leave their latencies in a row
                        float y[4][8];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int k = 0; k < 8; k += 4)
                                *reinterpret_cast<float4 *>(&y[e][k]) =
                                    *reinterpret_cast<const float4 *>(stage_rows + (e * 8 + sub) * STAGE_LD + c8 + k);
                        if (gated) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                gate8(y[e], gv[e]);
                        }
                        load_gate(col + 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 w = pack8(y[e]);
                            if (e * 8 + sub < rows_here) {
                                *reinterpret_cast<uint4 *>(out_at[e] + col) = w;
                                if (p.out_amax == nullptr)
                                    continue;
                                amax = __vmaxu2(__vmaxu2(amax, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
                                amax = __vmaxu2(__vmaxu2(amax, w.z & 0x7FFF7FFFu), w.w & 0x7FFF7FFFu);
                            }
                        }
                    }
                } else {
                    const int64_t prow0 = (static_cast<int64_t>(cta) * 2 + (it.part == 2 ? 1 : 0)) * p.parts.rows + quarter * 32;
                    float *to = p.parts.o + (prow0 + (lane >> 3)) * D + (lane & 7) * 4;
                    const float *from = stage_rows + (lane >> 3) * STAGE_LD + (lane & 7) * 4;
#pragma unroll 1
                    for (int col = 0; col < D; col += 32) {
                        stage(col);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 a = *reinterpret_cast<const float4 *>(from + e * 4 * STAGE_LD);
                            if (e * 4 + (lane >> 3) < rows_here)
                                *reinterpret_cast<float4 *>(to + e * 4 * D + col) = a;
                        }
                    }
                    if (live) {
                        p.parts.ml[(prow0 + lane) * 2] = sm->ref[ip][row];
                        p.parts.ml[(prow0 + lane) * 2 + 1] = total;
                    }
                }
            }
            tc_fence_before();
            if (has_nan) {  // alike for all 128 threads; the next marks of this parity come behind the next item's barrier
                named_barrier_any(6, 128, false);
#pragma unroll 1
                for (int e = rt; e < D; e += 128)
                    sm->nan_key[ip][e] = INT_MAX;
                if (rt == 0)
                    sm->nan_any[ip] = 0;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm->o_free));
                mbar_arrive(smem_u32(&sm->item_done[i % ITEMS]));
            }
        }
        if (fail && lane == 0)
            attn_timeout(sm, p.status);
        store_amax(p, amax, lane);
    } else if (warp >= SOFT_WARP0) {
        // ------------------------------------------------------ softmax
        const int quarter = warp & 3, half = (warp - SOFT_WARP0) >> 2, sw = warp - SOFT_WARP0;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const float c = p.softmax_scale * ks * 1.4426950408889634f;
        uint32_t block = 0;
        bool fail = false;  // a wait of this thread ran out: no more waits until the item's vote makes it everyone's
        for (int i = 0;; ++i) {
            const Item it = warp_item(i, fail);
            // Queries to shared memory as two E4M3 terms (the score MMAs of the item before have completed): each
            // warp takes every 8th row, or pair of rows, eight rows at a time and the other eight on their way
            if (it.blocks > 0) {
                constexpr int LANES = D / 8, GROUP = 32 / LANES, BATCH = 8 / GROUP;
                const int col = (lane % LANES) * 8;
                const uint16_t *src = p.q.data + it.token0 * p.q.token_stride + it.head * p.group * p.q.head_stride + col;
                auto load = [&](int r0, uint4 (&v)[BATCH]) {
#pragma unroll
                    for (int e = 0; e < BATCH; ++e) {
                        const uint32_t r = r0 + 8 * GROUP * e + lane / LANES, tk = r * p.group_inv >> 16;
                        v[e] = make_uint4(0, 0, 0, 0);
                        if (r < static_cast<uint32_t>(it.rows))
                            v[e] = *reinterpret_cast<const uint4 *>(src + tk * p.q.token_stride + (r - tk * p.group) * p.q.head_stride);
                    }
                };
                uint4 v[BATCH];
                load(sw * GROUP, v);
#pragma unroll 1
                for (int r0 = sw * GROUP; r0 < it.rows; r0 += 8 * GROUP * BATCH) {
                    uint4 next[BATCH];
                    load(r0 + 8 * GROUP * BATCH, next);
#pragma unroll
                    for (int e = 0; e < BATCH; ++e) {
                        const int r = r0 + 8 * GROUP * e + lane / LANES;  // below 128
                        uint2 hi, lo;
                        float unscale;
                        split_query<D>(v[e], hi, lo, unscale);
                        uint8_t *at = smem + (col >> 7) * A::SUB_BYTES + r * 128 + ((col & 127) ^ ((r & 7) << 4));
                        *reinterpret_cast<uint2 *>(at) = hi;
                        *reinterpret_cast<uint2 *>(at + A::SUBS * A::SUB_BYTES) = lo;
                        if ((lane % LANES) == 0)
                            sm->row_scale[i & 1][r] = unscale;
                        v[e] = next[e];
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->q_ready));
            }
            // row_scale of this item is written; a vote at the end marker too, as among the row warps
            fail = named_barrier_any(5, SOFT_THREADS, fail);
            if (fail || it.blocks == 0)
                break;
            const bool live = row < it.rows, warp_live = quarter * 32 < it.rows;
            // keys in sight of this half row, from the current block's first; rows that no token fills need no mask
            int vis = live ? max(it.past0 + static_cast<int>(row * p.group_inv >> 16) + 1, 0) - it.t0 * KEY_BLOCK - half * 64 : INT_MAX;
            float f = 0.0f, ref = -INFINITY, top = -INFINITY;
            if (live) {
                f = sm->row_scale[i & 1][row] * c;
                f = f < 1.17549435e-38f ? 1.17549435e-38f : f;  // keeps (-inf) * f; NaN stays
            }
            const uint64_t ff = pack2(f, f);
            uint64_t sum2 = 0;  // two fp32 sums
            float so_far = 0.0f;
#pragma unroll 1
            for (int j = 0; j < it.blocks; ++j, ++block) {
                const int buf = static_cast<int>(block & 1);
                fail = fail || !mbar_wait(smem_u32(&sm->s_full[buf]), (block >> 1) & 1u, ATTN_WAIT_NS);
                __syncwarp();
                tc_fence_after();
                const uint32_t scol = tmem + A::S_COL + buf * KEY_BLOCK + half * 64 + lanes;
                float mine = -INFINITY, turn = 1.0f;
                if (warp_live) {
                    if (__any_sync(0xFFFFFFFFu, vis < 64)) {  // out of sight: -inf in place of the scores
#pragma unroll 1
                        for (int c32 = 0; c32 < 64; c32 += 32) {
                            uint32_t v[32];
                            tc_ld_32x32b_x32(scol + c32, v);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = c32 + e < vis ? v[e] : 0xFF800000u;
                            tc_st_32x32b_x32(scol + c32, v);
                        }
                        tc_wait_st();
                    }
                    uint32_t v[64];
                    tc_ld_32x32b_x64(scol, v);
                    tc_wait_ld();
                    mine = block_max64(v);
                    sm->red[buf][half][row] = make_float2(mine, so_far);
                }
                vis -= live ? KEY_BLOCK : 0;
                named_barrier_sync(1 + quarter, 64);  // the two warps of these rows
                if (warp_live) {
                    const float2 other = sm->red[buf][half ^ 1][row];
                    const float most = fmaxf(mine, other.x), tm = most * f;
                    // How far the block's largest lies above the reference, rounded as its power's exponent is: from tm,
                    // which is rounded before the difference, scores of millions would pass for smaller ones than they
                    // are, and their power leave E4M3.  ref is -inf until the row has seen a key; one branch for the warp,
                    // few blocks take it.
                    const float above = fmaf(most, f, -ref);
                    const bool up = above > REF_UP;
                    const bool down = above < -REF_DOWN && so_far + other.y < BLOCK_SUM / P_UNIT * static_cast<float>(j) && tm > -INFINITY;
                    top = fmaxf(top, tm);
                    if (__any_sync(0xFFFFFFFFu, up || down)) {
                        if (up || down) {
                            float to = fmaxf(tm + (up ? SLACK_UP : SLACK_DOWN), top - REF_SPAN);
                            if (fmaf(most, f, -to) > REF_UP)  // the steps of fp32 are wider than the slack
                                to = fmaf(fabsf(tm), 0x1p-23f, to);
                            turn = ref > -INFINITY ? exp2_fast(ref - to) : 1.0f;
                            ref = to;
                            sum2 = mul2(sum2, pack2(turn, turn));
                        }
                    }
                }
                if (half == 0) {
                    sm->turn[buf][row] = turn;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&sm->turn_ready[buf]));
                }
                const float minus_ref = ref > -INFINITY ? -ref : 0.0f;
                const uint64_t bb = pack2(minus_ref, minus_ref);
                uint64_t sum_b = 0;
                // A pair of probabilities goes to f16 (11 bits) without its 2^8.  There the byte below the sign holds the
                // E4M3 code of 2^8 times the value cut to 4 bits, subnormal codes too: the high term.  The rest, exact,
                // is converted to the low term, ties to even: it has 7 bits at most, so ties are frequent, and rounded
                // up they made every probability 3.0e-4 too large on average, against a sum that takes them unrounded
                // (that form, a byte shuffle, was 0.7 % faster on chunks of D = 256, 2.3 % at D = 128).
                // Scores are read from TMEM a second time, 32 at a time, instead of being held: the loop's code is
                // half as long, and the warps' loops together have to fit the instruction cache.
#pragma unroll 1
                for (int c32 = 0; c32 < 2; ++c32) {
                    if (warp_live) {
                        uint32_t v[32], hi[8], lo[8];
                        tc_ld_32x32b_x32(scol + c32 * 32, v);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint64_t x[2];
                            uint32_t h[2], l[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                x[e] = exp2_fast2(fma2(pack2u(v[4 * k + 2 * e], v[4 * k + 2 * e + 1]), ff, bb));
                                h[e] = f16x2_of(x[e]);
                                l[e] = e4m3x2_of_rest(sub_f16x2(h[e], h[e] & 0x7F807F80u));
                            }
                            sum2 = add2(sum2, x[0]);
                            sum_b = add2(sum_b, x[1]);
                            hi[k] = __byte_perm(h[0] << 1, h[1] << 1, 0x7531);
                            lo[k] = l[0] | l[1] << 16;
                        }
                        tc_st_32x32b_x8(scol + c32 * 8, hi);
                        tc_st_32x32b_x8(scol + 16 + c32 * 8, lo);
                        tc_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(c32 ? &sm->p_rest[buf] : &sm->p_ready[buf]));
                }
                sum2 = add2(sum2, sum_b);
                float sa, sb;
                unpack2(sum2, sa, sb);
                so_far = sa + sb;
            }
            sm->sum[i & 1][half][row] = so_far * P_UNIT;
            if (half == 0)
                sm->ref[i & 1][row] = top > -INFINITY ? ref : -INFINITY;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sm->stats_ready));
        }
        if (fail && lane == 0)
            attn_timeout(sm, p.status);
    }

    tc_fence_before();
    __syncthreads();
    // When some wait ran out, whosever it was, copies may be in flight that nobody has waited for: they land before
    // the shared memory goes away.
    if ((warp == 0 || warp == 3) && lane == 0 && sm->abort_flag) {
        for (int f = 0; f < A::STAGES; ++f)
            if (filled >> f & 1u)
                mbar_wait(smem_u32(&sm->full[f]), phases >> f & 1u, ATTN_DRAIN_NS);
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the parts of the items that several CTAs worked on: CTA c's last
// item, whose later parts are the first items of CTAs c+1 .. last.  One warp
// per row; the parts are added in the order of their keys.  Where the
// kernel for single tokens ran beside the tile kernel, its parts come first in
// the grid: the tile kernel may have found nothing to do.
//
// The bytes are few (D floats a part and row); what counts is how many loads
// wait for one another and how many rows are in flight.  Once a row's item is
// known, its gate and, where AHEAD CTAs or fewer share it, their sums are asked
// for at once.  After tiles, AHEAD = 4 leaves room for 32 warps on an SM: with
// 107 registers and the loads one after the other the join of 148 x 126 rows
// of 256 took 33 us.  After single tokens alone there are few rows, and an
// item may have many parts: AHEAD = 8.
constexpr int JOIN_ROWS = 8;

template <int D, int AHEAD>
__global__ void __launch_bounds__(JOIN_ROWS * 32, AHEAD > 4 ? 2 : 4) paged_attention_join_kernel(const AttnParams p, const Parts first,
                                                                                                    const int first_blocks)
{
    grid_dep_wait();
    grid_dep_launch_dependents();
    const bool other = static_cast<int>(blockIdx.x) < first_blocks;
    const int block = static_cast<int>(blockIdx.x) - (other ? 0 : first_blocks);
    const Parts parts = other ? first : p.parts;
    const int cta = block % CTAS, lane = threadIdx.x & 31;
    const int row = block / CTAS * JOIN_ROWS + (threadIdx.x >> 5);
    if (row >= parts.rows)
        return;
    auto slot_of = [&](int c) { return (static_cast<int64_t>(c) * 2 + (c == cta ? 1 : 0)) * parts.rows + row; };
    // A lane for every CTA of a span of 32: which hold a part, and their references and sums.  The first span's are
    // asked for together with the row's item, before it is known how far that goes.
    auto state = [&](int c, float2 &ml) {
        ml = make_float2(-INFINITY, 0.0f);
        if (c >= CTAS)
            return false;
        ml = *reinterpret_cast<const float2 *>(parts.ml + slot_of(c) * 2);
        return c == cta || parts.info[c].continues != 0;
    };
    float2 ml;
    bool has = state(cta + lane, ml);
    const PartInfo info = parts.info[cta];
    const float ks = __ldg(p.k_scale), vs = __ldg(p.v_scale);
    // addresses come from the workspace: another call that uses it at the same time must not make them point elsewhere
    const int tk = row / p.group, h = info.group0 + row - tk * p.group;
    const bool outside = (static_cast<uint32_t>(info.last) >= CTAS) | (static_cast<uint32_t>(h) >= static_cast<uint32_t>(p.out.heads)) |
                         (static_cast<uint32_t>(info.token0 + tk) >= static_cast<uint32_t>(p.batch.tokens));
    if ((info.owns == 0) | (row >= info.rows) | outside | !valid_scale(ks) | !valid_scale(vs))
        return;
    has = has && cta + lane <= info.last;
    constexpr int PER = D / 128;
    int pick[AHEAD];  // CTAs whose parts are in x, from the span's first; -1: none
    float4 x[AHEAD][PER];
    auto load = [&](int c0) {
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const float *src = parts.o + slot_of(c0 + max(pick[e], 0)) * D + lane * 4;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (pick[e] >= 0)
                    x[e][i] = *reinterpret_cast<const float4 *>(src + i * 128);
        }
    };
    uint2 gate[PER];
    // Few CTAs: all their sums are read before it is known which of them hold a part
    const bool near = info.last - cta < AHEAD;
    if (near) {
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
            pick[e] = cta + e <= info.last ? e : -1;
        load(cta);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        gate[i] = load_gate4(p, info.token0 + tk, h, i * 128 + lane * 4);
    float top = has ? ml.x : -INFINITY;
    for (int c = cta + 32 + lane; c - lane <= info.last; c += 32) {
        float2 more;
        if (state(c, more) && c <= info.last)
            top = fmaxf(top, more.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    float o[4 * PER], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4 * PER; ++i)
        o[i] = 0.0f;
#pragma unroll 1
    for (int c0 = cta; c0 <= info.last; c0 += 32) {
        if (c0 > cta)
            has = state(c0 + lane, ml) && c0 + lane <= info.last;
        uint32_t todo = __ballot_sync(0xFFFFFFFFu, has);
        const uint32_t there = todo;
        // no key in sight in any part: weight 1 keeps the zero or NaN sums
        const float mine = top > -INFINITY ? exp2_fast(ml.x - top) : 1.0f;
#pragma unroll 1
        while (todo) {
            if (near) {
                todo = 0;
            } else {
#pragma unroll
                for (int e = 0; e < AHEAD; ++e) {
                    pick[e] = todo ? __ffs(todo) - 1 : -1;
                    todo &= todo - 1;
                }
                load(c0);
            }
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                if (pick[e] < 0 || !(there >> pick[e] & 1u))
                    continue;
                const float w = __shfl_sync(0xFFFFFFFFu, mine, pick[e]);
                sum = fmaf(w, __shfl_sync(0xFFFFFFFFu, ml.y, pick[e]), sum);
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    o[4 * i] = fmaf(w, x[e][i].x, o[4 * i]);
                    o[4 * i + 1] = fmaf(w, x[e][i].y, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(w, x[e][i].z, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(w, x[e][i].w, o[4 * i + 3]);
                }
            }
        }
    }
    const float inv = vs / sum;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float y[4] = {o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
        amax = write_row4(p, y, inv, info.past0 + tk < 0, gate[i], info.token0 + tk, h, i * 128 + lane * 4, amax);
    }
    store_amax(p, amax, lane);
}

}  // namespace attn
}  // namespace nvfp4
