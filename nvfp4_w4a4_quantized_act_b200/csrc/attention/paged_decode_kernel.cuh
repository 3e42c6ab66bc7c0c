// paged_decode_kernel.cuh -- attention of single new tokens over the paged
// FP8 cache.
//
//   s_i = c * sum_d q[d] k_code[i][d],  c = softmax_scale * k_scale
//   out = v_scale * sum_i 2^(t_i - r) v_code[i] / sum_i 2^(t_i - r),  t = s log2(e)
//
// A token's `group` query heads (at most 8) read the same keys, so a key block
// of 64 KB meets 8 rows at most: the bytes of the cache bound this kernel, not
// the products.  A 128-row tile on tcgen05 spends some 2100 cycles of tensor
// time on such a block, close to the 2800 that its bytes take, and its
// pipeline of specialised warps starts slowly; here the warps work on their
// own part of every block with warp-level MMAs (m16n8k16) and meet once per
// token.  Keys are the MMA's 16 rows and queries its 8 columns, so nothing is
// padded; the value product is taken the same way round.  There is no 8-bit
// warp-level MMA on this part (one is emulated by conversions), so codes are
// converted to f16, which is exact; scaled queries are exact in f16 too, and
// probabilities keep 11 bits over 2^-14 .. 2^15 (a reference r that moves only
// when a block's largest is 2^7 above it; a sink 2^22 above the rest still
// leaves those their bits).
//
//   warps 0..7   16 keys of every block of 128
//   warp 8       walks the CTA's items (attention_schedule.cuh) and loads K and
//                V blocks page by page (4-D TMA, 128-byte swizzle) into a ring
//   warps 9..11  add the warps' sums of an item and write its result, while
//                warps 0..7 are at the next item
//
// Fragments come straight from the stages.  K: a lane takes 16 bytes of a key
// at a time, the operands of four MMAs (any order of the dimensions serves, the
// queries take the same).  V: a lane takes 16 dimensions of the four keys whose
// probabilities it holds after the 8 x 8 transposes that turn the score tile
// into the product's operand; a byte shuffle puts two keys of a dimension side
// by side.  MMA row n stands for key n for even n and key ((n - 1) ^ 4) + 1 for
// odd n, which makes both reads free of bank conflicts under the swizzle.
//
// Measured (24 query heads on 4 key heads of 256, parts joined): 64 sequences
// of up to 8192 keys, 527 MB, 99 us, 5.3 TB/s; 2 of 131072, 537 MB, 96 us, 5.6
// TB/s (a copy on this board runs at 6.45).  A CTA's start (offsets, page table,
// first keys: three loads that wait for one another), the join and the launches
// take some 13 us of each; one sequence of 777 keys takes 11 us for them alone,
// 13.5 with an idle tile kernel beside it.
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

constexpr int DECODE_WARPS = 8;
constexpr int WRITE_WARPS = 3;
constexpr int DECODE_THREADS = (DECODE_WARPS + 1 + WRITE_WARPS) * 32;
constexpr int DECODE_ROWS = 8;     // query heads of a key head, at most
constexpr int WARP_KEYS = KEY_BLOCK / DECODE_WARPS;
constexpr int KEY_PARTS = DECODE_WARPS / 2;   // sums of two warps that meet in shared memory
constexpr float P_ROOM = 7.0f;                // 2^(P_SHIFT + P_ROOM) < 65504

template <int D>
struct DecodeShape {
    static constexpr int SUBS = D / 128;                    // 128-byte wide sub-tiles of a row
    static constexpr uint32_t SUB_BYTES = KEY_BLOCK * 128;
    static constexpr uint32_t K_BYTES = SUBS * SUB_BYTES;
    static constexpr uint32_t STAGE_BYTES = 2 * K_BYTES;    // 128 keys of K, then of V
    static constexpr int STAGES = D == 256 ? 3 : 6;
    static constexpr int TILES = D / 16;                    // of 16 value dimensions
};

template <int D>
struct DecodeSmem {
    float o[KEY_PARTS][DECODE_ROWS][D];
    float2 ml[KEY_PARTS][DECODE_ROWS];  // reference (-inf: no key seen), sum
    Item items[ITEMS];
    uint64_t item_ready[ITEMS], item_done[ITEMS];
    uint64_t full[DecodeShape<D>::STAGES], empty[DecodeShape<D>::STAGES];
    uint64_t pair_ready[KEY_PARTS], o_ready, o_free;
    volatile int32_t abort_flag;
    WalkStart start;
    int64_t scratch[DECODE_THREADS / 32];
};

template <int D>
constexpr uint32_t decode_smem_bytes()
{
    return DecodeShape<D>::STAGES * DecodeShape<D>::STAGE_BYTES + 1024 + sizeof(DecodeSmem<D>);
}

// D += A B: 16 x 16 by 16 x 8, f16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values (a lane holds two of a row).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// f16 values of the lower and of the upper two E4M3 codes of a word.
__device__ __forceinline__ void unpack_e4m3x4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

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
    extern __shared__ uint8_t attn_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(attn_smem_raw) + 1023) & ~uintptr_t(1023));
    DecodeSmem<D> *sm = reinterpret_cast<DecodeSmem<D> *>(smem + A::STAGES * A::STAGE_BYTES);
    const uint32_t ring = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int cta = blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < A::STAGES; ++s) {
            mbar_init(smem_u32(&sm->full[s]), 1);
            mbar_init(smem_u32(&sm->empty[s]), DECODE_WARPS);
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(smem_u32(&sm->item_ready[i]), 1);
            mbar_init(smem_u32(&sm->item_done[i]), WRITE_WARPS);
        }
        for (int i = 0; i < KEY_PARTS; ++i)
            mbar_init(smem_u32(&sm->pair_ready[i]), 1);
        mbar_init(smem_u32(&sm->o_ready), KEY_PARTS);
        mbar_init(smem_u32(&sm->o_free), WRITE_WARPS);
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

    uint32_t fills = 0;  // of the loading warp: stages filled so far
    if (warp == DECODE_WARPS) {
        // ------------------------------------------------ items, loads
        Walk walk;
        walk.b = sm->start.b;
        walk.h = sm->start.h;
        walk.m = sm->start.m;
        walk.x = sm->start.x;
        walk.left = scales_ok ? sm->start.left : 0;
        walk.q = sm->start.q;
        PartInfo info;
        info.continues = info.owns = 0;
        info.last = info.token0 = info.rows = info.group0 = info.past0 = info.pad = 0;
        const int shift = p.batch.page_shift, page = 1 << shift;
        const int rows = min(page, KEY_BLOCK);        // rows of a box
        const int boxes = KEY_BLOCK / rows;
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
            if (lane < it.rows * (D / 64)) {  // the rows that the other warps will read
                const int64_t h = it.head * p.group + lane / (D / 64);
                const int col = (lane % (D / 64)) * 64;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q.data + it.token0 * p.q.token_stride + h * p.q.head_stride + col));
                if (p.gate.data != nullptr)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.gate.data + it.token0 * p.gate.token_stride +
                                                                 h * p.gate.head_stride + col));
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
                const uint32_t bar = smem_u32(&sm->full[stage]);
                const bool mine = wanted(t);
                const int count = __popc(__ballot_sync(0xFFFFFFFFu, mine));
                if (lane == 0) {
                    if (mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1u, ATTN_WAIT_NS))
                        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(count * rows * D * 2));
                    else
                        fail = true;
                }
                fail = __any_sync(0xFFFFFFFFu, fail || sm->abort_flag);
                if (fail)
                    break;
                if (mine) {
                    const int row = (t * KEY_BLOCK + lane * rows) & (page - 1);
                    const uint32_t dst = ring + stage * A::STAGE_BYTES + lane * rows * 128;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const CUtensorMap *map = kv ? &tmV : &tmK;
                        const int row_at = kv ? p.v_row_at : p.k_row_at, head_at = kv ? p.v_head_at : p.k_head_at;
                        const int32_t c1 = row_at == 1 ? row : head_at == 1 ? it.head : id;
                        const int32_t c2 = row_at == 2 ? row : head_at == 2 ? it.head : id;
                        const int32_t c3 = row_at == 3 ? row : head_at == 3 ? it.head : id;
#pragma unroll
                        for (int s = 0; s < A::SUBS; ++s)
                            tma_load_4d(dst + kv * A::K_BYTES + s * A::SUB_BYTES, map, s * 128, c1, c2, c3, bar);
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
        if (lane == 0)
            p.parts.info[cta] = info;
    } else if (warp < DECODE_WARPS) {
        // ------------------------------------------------ products, softmax
        const int g = lane >> 2, q = lane & 3;
        auto key_of = [](int n) { return (n & 1) ? ((n - 1) ^ 4) + 1 : n; };
        const int krow = key_of(g), vrow0 = key_of(2 * q), vrow1 = key_of(2 * q + 1);
        const float c = p.softmax_scale * ks * 1.4426950408889634f;
        const uint8_t *my_k = smem + warp * WARP_KEYS * 128;
        uint32_t uses = 0;
        bool fail = false;
        for (int i = 0;; ++i) {
            Item it;
            it.blocks = 0;
            if (mbar_wait(smem_u32(&sm->item_ready[i % ITEMS]), (i / ITEMS) & 1, ATTN_WAIT_NS))
                it = sm->items[i % ITEMS];
            else
                fail = true;
            fail = __any_sync(0xFFFFFFFFu, fail);
            if (fail || it.blocks == 0)
                break;
            // Queries as the MMAs' B operands: column g, 16 dimensions at 64 s + 16 q for every s
            uint32_t qb[D / 2 / 4];
            float f[2];
            {
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
                const float fg = unscale * c;
                // of the two queries whose scores this lane holds; the bound keeps (-inf) * f, a NaN stays
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = __shfl_sync(0xFFFFFFFFu, fg, (2 * q + e) * 4);
                    f[e] = f[e] < 1.17549435e-38f ? 1.17549435e-38f : f[e];
                }
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2 x = __floats2half2_rn(__uint_as_float(w[k] << 16) * scale,
                                                            __uint_as_float(w[k] & 0xFFFF0000u) * scale);
                        qb[s * 4 + k] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                }
            }
            float o[A::TILES][4];
#pragma unroll
            for (int n = 0; n < A::TILES; ++n)
                o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
            float ref[2] = {0.0f, 0.0f}, sum[2] = {0.0f, 0.0f};
            bool begun[2] = {false, false};
#pragma unroll 1
            for (int j = 0; j < it.blocks; ++j, ++uses) {
                const uint32_t stage = uses % A::STAGES;
                fail = fail || !mbar_wait(smem_u32(&sm->full[stage]), (uses / A::STAGES) & 1u, ATTN_WAIT_NS);
                __syncwarp();
                const int left = it.keys - (it.t0 + j) * KEY_BLOCK - warp * WARP_KEYS;  // keys of this warp's share
                const uint8_t *kb = my_k + stage * A::STAGE_BYTES, *vb = kb + A::K_BYTES;
                if (left > 0) {
                    float acc[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.0f;
#pragma unroll
                    for (int s = 0; s < D / 64; ++s) {
                        const uint8_t *at = kb + (s >> 1) * A::SUB_BYTES + krow * 128 + ((((s & 1) * 4 + q) ^ krow) << 4);
                        const uint4 x = *reinterpret_cast<const uint4 *>(at), y = *reinterpret_cast<const uint4 *>(at + 8 * 128);
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t a0, a1, a2, a3;
                            unpack_e4m3x4(xw[k], a0, a2);
                            unpack_e4m3x4(yw[k], a1, a3);
                            mma_16816(acc[k & 1], a0, a1, a2, a3, qb[s * 8 + 2 * k], qb[s * 8 + 2 * k + 1]);
                        }
                    }
                    // scores of keys krow and krow + 8 (h), queries 2 q and 2 q + 1 (e)
                    float x[2][2], mx[2];
                    const bool in[2] = {krow < left, krow + 8 < left};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            x[h][e] = in[h] ? acc[0][2 * h + e] + acc[1][2 * h + e] : -INFINITY;
                        mx[e] = fmaxf(x[0][e], x[1][e]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], off));
                    }
                    float turn[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // the difference is rounded as the powers' exponents are (paged_attention_kernel.cuh)
                        const float tm = mx[e] * f[e];
                        const bool move = tm > -INFINITY && (!begun[e] || fmaf(mx[e], f[e], -ref[e]) > P_ROOM);
                        turn[e] = move && begun[e] ? exp2_fast(ref[e] - tm) : 1.0f;
                        ref[e] = move ? tm : ref[e];
                        begun[e] = begun[e] || move;
                        sum[e] *= turn[e];
                    }
                    if (__any_sync(0xFFFFFFFFu, turn[0] != 1.0f || turn[1] != 1.0f)) {
#pragma unroll
                        for (int n = 0; n < A::TILES; ++n) {
                            o[n][0] *= turn[0], o[n][1] *= turn[1], o[n][2] *= turn[0], o[n][3] *= turn[1];
                        }
                    }
                    uint32_t pb[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float u = exp2_fast(fmaf(x[h][0], f[0], P_SHIFT - ref[0]));
                        const float w = exp2_fast(fmaf(x[h][1], f[1], P_SHIFT - ref[1]));
                        sum[0] += u;
                        sum[1] += w;
                        const __half2 uw = __floats2half2_rn(u, w);
                        pb[h] = transpose8x8(*reinterpret_cast<const uint32_t *>(&uw));
                    }
#pragma unroll
                    for (int s = 0; s < A::SUBS; ++s) {
                        // 16 dimensions of the keys of rows 2 q, 2 q + 1, 2 q + 8, 2 q + 9
                        uint32_t w[4][4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = (k & 1) ? vrow1 : vrow0, row = r + (k >> 1) * 8;
                            const uint4 v = *reinterpret_cast<const uint4 *>(vb + s * A::SUB_BYTES + row * 128 + ((g ^ r) << 4));
                            w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
                        }
                        if (left < WARP_KEYS) {  // what lies behind the keys may be anything, a NaN included
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (((k & 1) ? vrow1 : vrow0) + (k >> 1) * 8 >= left)
                                    w[k][0] = w[k][1] = w[k][2] = w[k][3] = 0;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t a[4][2];  // dimension, pair of keys
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                unpack_e4m3x4(__byte_perm(w[2 * h][k], w[2 * h + 1][k], 0x5140), a[0][h], a[1][h]);
                                unpack_e4m3x4(__byte_perm(w[2 * h][k], w[2 * h + 1][k], 0x7362), a[2][h], a[3][h]);
                            }
                            // MMA rows g and g + 8: dimensions 16 g + 4 k + 2 m and the next
                            mma_16816(o[s * 8 + 2 * k], a[0][0], a[1][0], a[0][1], a[1][1], pb[0], pb[1]);
                            mma_16816(o[s * 8 + 2 * k + 1], a[2][0], a[3][0], a[2][1], a[3][1], pb[0], pb[1]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->empty[stage]));
            }
            // ------------------------------------------------ results: the warps' sums meet, first in pairs
            float2 ml[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], off);
                ml[e] = make_float2(begun[e] ? ref[e] : -INFINITY, sum[e]);
            }
            const int part = warp % KEY_PARTS;
            float4 *frag = reinterpret_cast<float4 *>(&sm->o[part][0][0]);  // [tile][lane]
            if (i > 0)  // the item before has been written
                fail = fail || !mbar_wait(smem_u32(&sm->o_free), (i - 1) & 1, ATTN_WAIT_NS);
            if (warp >= KEY_PARTS) {
#pragma unroll
                for (int n = 0; n < A::TILES; ++n)
                    frag[n * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
                if (g == 0) {
                    sm->ml[part][2 * q] = ml[0];
                    sm->ml[part][2 * q + 1] = ml[1];
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->pair_ready[part]));
            } else {
                fail = fail || !mbar_wait(smem_u32(&sm->pair_ready[part]), i & 1, ATTN_WAIT_NS);
            }
            fail = __any_sync(0xFFFFFFFFu, fail);
            if (fail)
                break;
            if (warp < KEY_PARTS) {
                float a[2], b[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 other = sm->ml[part][2 * q + e];
                    const float m = fmaxf(ml[e].x, other.x);
                    // no key in sight of either: weight 1 keeps the zero or NaN sums
                    a[e] = m > -INFINITY ? exp2_fast(ml[e].x - m) : 1.0f;
                    b[e] = m > -INFINITY ? exp2_fast(other.x - m) : 1.0f;
                    ml[e] = make_float2(m, ml[e].y * a[e] + other.y * b[e]);
                }
#pragma unroll
                for (int n = 0; n < A::TILES; ++n) {
                    const float4 y = frag[n * 32 + lane];
                    o[n][0] = o[n][0] * a[0] + y.x * b[0];
                    o[n][1] = o[n][1] * a[1] + y.y * b[1];
                    o[n][2] = o[n][2] * a[0] + y.z * b[0];
                    o[n][3] = o[n][3] * a[1] + y.w * b[1];
                }
                __syncwarp();
                // tile 8 s + m: dimensions 128 s + 16 g + 2 m and the next, of two queries
#pragma unroll
                for (int n = 0; n < A::TILES; ++n) {
                    const int dim = (n >> 3) * 128 + 16 * g + 2 * (n & 7);
                    *reinterpret_cast<float2 *>(&sm->o[part][2 * q][dim]) = make_float2(o[n][0], o[n][2]);
                    *reinterpret_cast<float2 *>(&sm->o[part][2 * q + 1][dim]) = make_float2(o[n][1], o[n][3]);
                }
                if (g == 0) {
                    sm->ml[part][2 * q] = ml[0];
                    sm->ml[part][2 * q + 1] = ml[1];
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&sm->o_ready));
            }
        }
        if (fail && lane == 0)
            decode_timeout(sm, p.status);
    } else {
        // ------------------------------------------------ results
        uint32_t amax = 0;
        bool fail = false;
        for (int i = 0;; ++i) {
            Item it;
            it.blocks = 0;
            if (mbar_wait(smem_u32(&sm->item_ready[i % ITEMS]), (i / ITEMS) & 1, ATTN_WAIT_NS))
                it = sm->items[i % ITEMS];
            else
                fail = true;
            fail = __any_sync(0xFFFFFFFFu, fail);
            if (fail || it.blocks == 0)
                break;
            fail = __any_sync(0xFFFFFFFFu, !mbar_wait(smem_u32(&sm->o_ready), i & 1, ATTN_WAIT_NS));
            if (fail)
                break;
            const bool whole = it.part == 0;
            const int64_t prow0 = (static_cast<int64_t>(cta) * 2 + (it.part == 2 ? 1 : 0)) * p.parts.rows;
#pragma unroll 1
            for (int k = tid - (DECODE_WARPS + 1) * 32; k < it.rows * (D / 4); k += WRITE_WARPS * 32) {
                const int r = k / (D / 4), col = (k % (D / 4)) * 4;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < KEY_PARTS; ++w)
                    m = fmaxf(m, sm->ml[w][r].x);
                float total = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < KEY_PARTS; ++w) {
                    // no key in sight of any warp: weight 1 keeps the zero or NaN sums
                    const float a = m > -INFINITY ? exp2_fast(sm->ml[w][r].x - m) : 1.0f;
                    const float4 x = *reinterpret_cast<const float4 *>(&sm->o[w][r][col]);
                    total = fmaf(a, sm->ml[w][r].y, total);
                    y[0] = fmaf(a, x.x, y[0]);
                    y[1] = fmaf(a, x.y, y[1]);
                    y[2] = fmaf(a, x.z, y[2]);
                    y[3] = fmaf(a, x.w, y[3]);
                }
                if (whole) {
                    const int32_t h = it.head * p.group + r;
                    amax = write_row4(p, y, vs / total, it.past0 < 0, load_gate4(p, it.token0, h, col), it.token0, h, col, amax);
                } else {
                    *reinterpret_cast<float4 *>(p.parts.o + (prow0 + r) * D + col) = make_float4(y[0], y[1], y[2], y[3]);
                    if (col == 0) {
                        p.parts.ml[(prow0 + r) * 2] = m;
                        p.parts.ml[(prow0 + r) * 2 + 1] = total;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm->o_free));
                mbar_arrive(smem_u32(&sm->item_done[i % ITEMS]));
            }
        }
        if (fail && lane == 0)
            decode_timeout(sm, p.status);
        store_amax(p, amax, lane);
    }
    __syncthreads();
    // when some wait ran out: copies in flight land before the shared memory goes away
    if (warp == DECODE_WARPS && lane == 0 && sm->abort_flag) {
        for (uint32_t f = fills > A::STAGES ? fills - A::STAGES : 0; f < fills; ++f)
            mbar_wait(smem_u32(&sm->full[f % A::STAGES]), (f / A::STAGES) & 1u, ATTN_DRAIN_NS);
    }
}

}  // namespace attn
}  // namespace nvfp4
