// paged_decode_kernel.cuh -- attention of single new tokens over the paged
// FP8 cache.
//
// The formulas, the two-term queries and probabilities and the reference r
// are those of paged_attention_kernel.cuh.  A token's `group` query heads (at
// most 8) read the same keys, so a key block of 64 KB meets 8 rows at most:
// the bytes of the cache bound this kernel, not the products.  A 128-row tile
// on tcgen05 spends some 2100 cycles of tensor time on such a block, close to
// the 2800 that its bytes take, and its pipeline of specialised warps starts
// slowly; here four warps work on their own quarter of every block with
// warp-level MMAs (m16n8k32) and meet once per token.  The MMA's 16 rows hold
// the 8 queries' high terms and their low terms, so the two-term products cost
// nothing extra: the two halves of the accumulator are added at the end.
//
//   warps 0..3   32 keys of every block of 128
//   warp 4       walks the CTA's items (attention_schedule.cuh) and loads their
//                K and V rows (4-D TMA, 128-byte swizzle), each warp's 32 keys
//                into that warp's own ring of stages
//
// Fragments come straight from the stages.  K: the lanes of a key take 16
// bytes each, which are the operands of two MMAs (any order of the dimensions
// serves, the queries take the same).  V: a lane takes 16 dimensions of the 8
// keys whose probabilities it holds; 4x4 byte transposes make the MMA's four
// keys per register.  Column n of a score tile is key n for even n and key
// ((n - 1) ^ 4) + 1 for odd n, which makes both reads free of bank conflicts
// under the swizzle.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "attention_schedule.cuh"
#include "head_rows_kernels.cuh"
#include "paged_attention_kernel.cuh"
#include "paged_batch.cuh"
#include "ptx_f8.cuh"
#include "status.cuh"

namespace nvfp4 {
namespace attn {

constexpr int DECODE_WARPS = 4;
constexpr int DECODE_THREADS = (DECODE_WARPS + 1) * 32;
constexpr int DECODE_ROWS = 8;     // query heads of a key head, at most
constexpr int WARP_KEYS = KEY_BLOCK / DECODE_WARPS;

template <int D>
struct DecodeShape {
    static constexpr uint32_t K_BYTES = WARP_KEYS * D;
    static constexpr uint32_t STAGE_BYTES = 2 * K_BYTES;    // K, then V; each D / 128 sub-tiles of 32 rows x 128 bytes
    static constexpr int STAGES = D == 256 ? 3 : 6;
    static constexpr uint32_t RING_BYTES = STAGES * STAGE_BYTES;
};

template <int D>
struct DecodeSmem {
    float o[DECODE_WARPS][DECODE_ROWS][D];
    float ml[DECODE_WARPS][DECODE_ROWS][2];  // reference (-inf: no key seen), sum
    Item items[ITEMS];
    uint64_t item_ready[ITEMS], item_done[ITEMS];
    uint64_t full[DECODE_WARPS][DecodeShape<D>::STAGES], empty[DECODE_WARPS][DecodeShape<D>::STAGES];
    volatile int32_t abort_flag;
    WalkStart start;
    int64_t scratch[DECODE_THREADS / 32];
};

template <int D>
constexpr uint32_t decode_smem_bytes()
{
    return DECODE_WARPS * DecodeShape<D>::RING_BYTES + 1024 + sizeof(DecodeSmem<D>);
}

// D += A B: 16 x 32 by 32 x 8, E4M3 operands, fp32 accumulator.
__device__ __forceinline__ void mma_16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// Bytes of four words, word i's byte j to word j's byte i.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&t)[4])
{
    const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);
    const uint32_t ab2 = __byte_perm(a, b, 0x7362), cd2 = __byte_perm(c, d, 0x7362);
    t[0] = __byte_perm(ab, cd, 0x5410);
    t[1] = __byte_perm(ab, cd, 0x7632);
    t[2] = __byte_perm(ab2, cd2, 0x5410);
    t[3] = __byte_perm(ab2, cd2, 0x7632);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int D>
__device__ __forceinline__ void decode_timeout(DecodeSmem<D> *sm, uint32_t *status)
{
    sm->abort_flag = 1;
    atomicOr(status, kStatusTimeout);
}

template <int D>
__global__ void __launch_bounds__(DECODE_THREADS, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p)
{
    using A = DecodeShape<D>;
    constexpr int SUBS = D / 128;
    extern __shared__ uint8_t attn_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
    DecodeSmem<D> *sm = reinterpret_cast<DecodeSmem<D> *>(smem + DECODE_WARPS * A::RING_BYTES);
    const uint32_t ring0 = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int cta = blockIdx.x;

    if (tid == 0) {
        for (int w = 0; w < DECODE_WARPS; ++w)
            for (int s = 0; s < A::STAGES; ++s) {
                mbar_init(smem_u32(&sm->full[w][s]), 1);
                mbar_init(smem_u32(&sm->empty[w][s]), 1);
            }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(smem_u32(&sm->item_ready[i]), 1);
            mbar_init(smem_u32(&sm->item_done[i]), DECODE_WARPS);
        }
        sm->abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch_dependents();

    const float ks = __ldg(p.k_scale), vs = __ldg(p.v_scale);
    const bool scales_ok = valid_scale(ks) && valid_scale(vs);
    bool bad = false;
    find_start<DECODE_THREADS>(p.batch, p.kv_heads, p.tile_tokens, cta, &sm->start, sm->scratch, bad);
    if (cta == 0) {
        if (!scales_ok && tid == 0)
            atomicOr(p.status, kStatusNonFinite);
        if (bad)
            atomicOr(p.status, kStatusBadIndex);
    }

    if (warp == DECODE_WARPS) {
        // ------------------------------------------------ items, loads
        Walk walk;
        walk.b = sm->start.b;
        walk.h = sm->start.h;
        walk.m = sm->start.m;
        walk.x = sm->start.x;
        walk.left = scales_ok ? sm->start.left : 0;
        if (walk.left > 0) {
            bool ignored = false;
            walk.q.set(load_seq(p.batch, walk.b, ignored), p.batch, p.tile_tokens);
        }
        PartInfo info;
        info.continues = info.owns = 0;
        info.last = info.token0 = info.rows = info.group0 = info.past0 = info.pad = 0;
        const int shift = p.batch.page_shift, page = 1 << shift;
        const int rows = min(page, WARP_KEYS);        // rows of a box
        const int boxes = KEY_BLOCK / rows, per_warp = WARP_KEYS / rows;
        const int to = lane / per_warp;               // warp that this lane's box is for
        const bool leader = lane < boxes && lane % per_warp == 0;
        uint32_t fills = 0;
        bool fail = false, out_of_pool = false;
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
            const int32_t *table = p.batch.table + it.seq * p.batch.table_stride;
            const int t1 = it.t0 + it.blocks;
            auto wanted = [&](int t) { return t < t1 && lane < boxes && t * KEY_BLOCK + lane * rows < it.keys; };
            auto page_of = [&](int t) { return wanted(t) ? __ldg(table + ((t * KEY_BLOCK + lane * rows) >> shift)) : 0; };
            int32_t id = page_of(it.t0);
#pragma unroll 1
            for (int t = it.t0; t < t1; ++t, ++fills) {
                const int32_t id_next = page_of(t + 1);
                const uint32_t stage = fills % A::STAGES, phase = (fills / A::STAGES) & 1u;
                const bool mine = wanted(t);
                const uint32_t any = __ballot_sync(0xFFFFFFFFu, mine);
                if (leader) {
                    const int count = __popc(any >> lane & ((per_warp < 32 ? 1u << per_warp : 0u) - 1u));
                    if (mbar_wait(smem_u32(&sm->empty[to][stage]), phase ^ 1u, ATTN_WAIT_NS))
                        mbar_arrive_expect_tx(smem_u32(&sm->full[to][stage]), static_cast<uint32_t>(count * rows * D * 2));
                    else
                        fail = true;
                }
                fail = __any_sync(0xFFFFFFFFu, fail || sm->abort_flag);
                if (fail)
                    break;
                if (mine) {
                    const int row = (t * KEY_BLOCK + lane * rows) & (page - 1);
                    const uint32_t dst = ring0 + to * A::RING_BYTES + stage * A::STAGE_BYTES + (lane % per_warp) * rows * 128;
                    const uint32_t bar = smem_u32(&sm->full[to][stage]);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const CUtensorMap *map = kv ? &tmV : &tmK;
                        const int row_at = kv ? p.v_row_at : p.k_row_at, head_at = kv ? p.v_head_at : p.k_head_at;
                        const int32_t c1 = row_at == 1 ? row : head_at == 1 ? it.head : id;
                        const int32_t c2 = row_at == 2 ? row : head_at == 2 ? it.head : id;
                        const int32_t c3 = row_at == 3 ? row : head_at == 3 ? it.head : id;
#pragma unroll
                        for (int s = 0; s < SUBS; ++s)
                            tma_load_4d(dst + kv * A::K_BYTES + s * (WARP_KEYS * 128), map, s * 128, c1, c2, c3, bar);
                    }
                    out_of_pool |= id < 0 || id >= p.batch.num_pages;
                }
                id = id_next;
            }
            if (fail)
                break;
        }
        if (out_of_pool)
            atomicOr(p.status, kStatusBadIndex);
        if (fail && lane == 0)
            decode_timeout(sm, p.status);
        if (fail && leader)  // copies in flight land before the shared memory goes away
            for (uint32_t f = fills > A::STAGES ? fills - A::STAGES : 0; f < fills; ++f)
                mbar_wait(smem_u32(&sm->full[to][f % A::STAGES]), (f / A::STAGES) & 1u, ATTN_WAIT_NS);
        if (lane == 0)
            p.parts.info[cta] = info;
    } else {
        // ------------------------------------------------ products, softmax
        const int g = lane >> 2, q = lane & 3;
        // key rows of this lane: of the score tiles' operands, and of the 8 probabilities that it holds (4 tiles x 2)
        const int krow = (g & 1) ? ((g - 1) ^ 4) + 1 : g;
        const int prow[2] = {2 * q, ((2 * q) ^ 4) + 1};
        const float c = p.softmax_scale * ks * 1.4426950408889634f;
        const uint32_t ring = ring0 + warp * A::RING_BYTES;
        uint32_t uses = 0, amax = 0;
        bool fail = false;
        for (int i = 0;; ++i) {
            Item it;
            it.blocks = 0;
            if (mbar_wait(smem_u32(&sm->item_ready[i % ITEMS]), (i / ITEMS) & 1, ATTN_WAIT_NS))
                it = sm->items[i % ITEMS];
            else
                fail = true;
            fail = __any_sync(0xFFFFFFFFu, fail);
            if (!fail && it.blocks == 0)
                break;
            // Queries: row g, 16 dimensions at 64 s + 16 q for every s, as the MMAs' A operands
            uint32_t qa[D / 32][4];
            float f = 0.0f;
            if (!fail) {
                uint4 v[D / 32];
#pragma unroll
                for (int s = 0; s < D / 32; ++s)
                    v[s] = make_uint4(0, 0, 0, 0);
                if (g < it.rows) {
                    const uint16_t *src = p.q.data + it.token0 * p.q.token_stride +
                                          static_cast<int64_t>(it.head * p.group + g) * p.q.head_stride + 16 * q;
#pragma unroll
                    for (int s = 0; s < D / 32; ++s)
                        v[s] = *reinterpret_cast<const uint4 *>(src + 64 * (s >> 1) + 8 * (s & 1));
                }
                uint32_t mag = 0;
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    mag = __vmaxu2(__vmaxu2(mag, v[s].x & 0x7FFF7FFFu), v[s].y & 0x7FFF7FFFu);
                    mag = __vmaxu2(__vmaxu2(mag, v[s].z & 0x7FFF7FFFu), v[s].w & 0x7FFF7FFFu);
                }
                mag = max(mag & 0xFFFFu, mag >> 16);
                mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
                mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
                float scale, unscale;
                query_scale(mag, scale, unscale);
                f = unscale * c;
                f = f < 1.17549435e-38f ? 1.17549435e-38f : f;  // keeps (-inf) * f; NaN stays
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    uint2 hi, lo;
                    split8(v[s], scale, hi, lo);
                    qa[s][0] = hi.x, qa[s][1] = lo.x, qa[s][2] = hi.y, qa[s][3] = lo.y;
                }
            }
            float o[D / 8][4];
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
            float ref = 0.0f, top = -INFINITY, sum = 0.0f;
#pragma unroll 1
            for (int j = 0; j < it.blocks; ++j, ++uses) {
                const uint32_t stage = uses % A::STAGES;
                fail = fail || !mbar_wait(smem_u32(&sm->full[warp][stage]), (uses / A::STAGES) & 1u, ATTN_WAIT_NS);
                __syncwarp();
                const int key0 = (it.t0 + j) * KEY_BLOCK + warp * WARP_KEYS;
                const int left = it.keys - key0;  // keys of this warp's share
                const uint32_t kb = ring + stage * A::STAGE_BYTES, vb = kb + A::K_BYTES;
                if (left > 0) {
                    float acc[4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
#pragma unroll
                    for (int s = 0; s < D / 64; ++s)
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const uint4 k = lds128(kb + (s >> 1) * (WARP_KEYS * 128) + (n * 8 + krow) * 128 +
                                                   ((((s & 1) * 4 + q) ^ krow) << 4));
                            mma_16832(acc[n], qa[2 * s], k.x, k.y);
                            mma_16832(acc[n], qa[2 * s + 1], k.z, k.w);
                        }
                    float x[4][2], mx = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[n][e] = n * 8 + prow[e] < left ? acc[n][e] + acc[n][e + 2] : -INFINITY;
                            mx = fmaxf(mx, x[n][e]);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                    float all = sum + __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                    all += __shfl_xor_sync(0xFFFFFFFFu, all, 2);
                    const float tm = mx * f;
                    float turn = 1.0f;
                    if (tm > -INFINITY) {
                        const bool begun = top > -INFINITY;
                        top = fmaxf(top, tm);
                        if (!begun) {
                            ref = tm + SLACK_UP;
                        } else {
                            // a warp's share of a block is a quarter, and so is its share of the bound on the sum
                            const bool up = tm > ref + REF_UP;
                            if (up || (tm < ref - REF_DOWN && all < BLOCK_SUM * 0.25f * static_cast<float>(j))) {
                                const float next = fmaxf(tm + (up ? SLACK_UP : SLACK_DOWN), top - REF_SPAN);
                                turn = exp2_fast(ref - next);
                                sum *= turn;
                                ref = next;
                            }
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, turn != 1.0f)) {
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][0] *= turn, o[n][1] *= turn, o[n][2] *= turn, o[n][3] *= turn;
                        }
                    }
                    const float base = P_SHIFT - ref;
                    float hi[4][2], lo[4][2];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float w = exp2_fast(fmaf(x[n][e], f, base));
                            sum += w;
                            hi[n][e] = __uint_as_float(__float_as_uint(w) & 0xFFF00000u);
                            lo[n][e] = w - hi[n][e];
                        }
                    uint32_t pa[4];
                    pa[0] = f32_to_e4m3x4(hi[0][0], hi[0][1], hi[1][0], hi[1][1]);
                    pa[1] = f32_to_e4m3x4(lo[0][0], lo[0][1], lo[1][0], lo[1][1]);
                    pa[2] = f32_to_e4m3x4(hi[2][0], hi[2][1], hi[3][0], hi[3][1]);
                    pa[3] = f32_to_e4m3x4(lo[2][0], lo[2][1], lo[3][0], lo[3][1]);
#pragma unroll
                    for (int s = 0; s < SUBS; ++s) {
                        uint4 w[4][2];
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                w[n][e] = lds128(vb + s * (WARP_KEYS * 128) + (n * 8 + prow[e]) * 128 + ((g ^ prow[e]) << 4));
                        if (left < WARP_KEYS) {  // what lies behind the keys may be anything, a NaN included
#pragma unroll
                            for (int n = 0; n < 4; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (n * 8 + prow[e] >= left)
                                        w[n][e] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t b0[4], b1[4];
                            transpose4(word(w[0][0], k), word(w[0][1], k), word(w[1][0], k), word(w[1][1], k), b0);
                            transpose4(word(w[2][0], k), word(w[2][1], k), word(w[3][0], k), word(w[3][1], k), b1);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mma_16832(o[s * 16 + k * 4 + e], pa, b0[e], b1[e]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->empty[warp][stage]));
            }
            // ------------------------------------------------ results: the four warps' sums meet
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            // column n = 2 q + e of tile (s, k): dimension 128 s + 16 n + k; neighbouring k lie together
#pragma unroll
            for (int s = 0; s < SUBS; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        float4 y;
                        y.x = o[s * 16 + k][e] + o[s * 16 + k][e + 2];
                        y.y = o[s * 16 + k + 1][e] + o[s * 16 + k + 1][e + 2];
                        y.z = o[s * 16 + k + 2][e] + o[s * 16 + k + 2][e + 2];
                        y.w = o[s * 16 + k + 3][e] + o[s * 16 + k + 3][e + 2];
                        *reinterpret_cast<float4 *>(&sm->o[warp][g][128 * s + 16 * (2 * q + e) + k]) = y;
                    }
            if (q == 0) {
                sm->ml[warp][g][0] = top > -INFINITY ? ref : -INFINITY;
                sm->ml[warp][g][1] = sum;
            }
            fail = named_barrier_any(1, DECODE_WARPS * 32, fail);
            if (fail)
                break;
            const bool whole = it.part == 0;
            const int64_t prow0 = (static_cast<int64_t>(cta) * 2 + (it.part == 2 ? 1 : 0)) * p.parts.rows;
#pragma unroll 1
            for (int k = tid; k < it.rows * (D / 4); k += DECODE_WARPS * 32) {
                const int r = k / (D / 4), col = (k % (D / 4)) * 4;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < DECODE_WARPS; ++w)
                    m = fmaxf(m, sm->ml[w][r][0]);
                float total = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < DECODE_WARPS; ++w) {
                    // no key in sight of any warp: weight 1 keeps the zero or NaN sums
                    const float a = m > -INFINITY ? exp2_fast(sm->ml[w][r][0] - m) : 1.0f;
                    const float4 x = *reinterpret_cast<const float4 *>(&sm->o[w][r][col]);
                    total = fmaf(a, sm->ml[w][r][1], total);
                    y[0] = fmaf(a, x.x, y[0]);
                    y[1] = fmaf(a, x.y, y[1]);
                    y[2] = fmaf(a, x.z, y[2]);
                    y[3] = fmaf(a, x.w, y[3]);
                }
                if (whole) {
                    amax = write_row4(p, y, vs / total, it.past0 < 0, it.token0, it.head * p.group + r, col, amax);
                } else {
                    *reinterpret_cast<float4 *>(p.parts.o + (prow0 + r) * D + col) = make_float4(y[0], y[1], y[2], y[3]);
                    if (col == 0) {
                        p.parts.ml[(prow0 + r) * 2] = m;
                        p.parts.ml[(prow0 + r) * 2 + 1] = total;
                    }
                }
            }
            __syncwarp();
            named_barrier_sync(1, DECODE_WARPS * 32);  // the sums are read before the next item's come
            if (lane == 0)
                mbar_arrive(smem_u32(&sm->item_done[i % ITEMS]));
        }
        if (fail && lane == 0)
            decode_timeout(sm, p.status);
        store_amax(p, amax, lane);
    }
    __syncthreads();
}

}  // namespace attn
}  // namespace nvfp4
