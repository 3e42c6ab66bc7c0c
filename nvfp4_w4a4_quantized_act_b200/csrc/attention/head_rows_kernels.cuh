// head_rows_kernels.cuh -- the per-head row operators of an attention layer:
// RMS norm with the position rotation (queries and keys), and the append of
// keys and values to the paged FP8 cache with both applied on the way.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (w, or 1 + w; absent: y = x)
//   (y[i], y[i+R/2]) turned by position * inv_freq[i],  i < R/2
//   out = bf16_RNE(y)   or   code = E4M3_RNE_satfinite(fl32(y / scale))
//
// Both are bound by memory: a row is read once and written once.  A warp takes
// one token and a few of its heads, and needs no other warp; all its rows are
// asked for at once, into shared memory: held in registers, one row ahead, too
// little was in flight (8192 tokens x 28 heads of 256: 54 us, now 45, 5.3 TB/s
// of 6.45; append of 8192 tokens x 4 heads: 16.4, now 15.1, 3.3 TB/s, where
// the IEEE division and the conversions of 8 elements a lane count too).  A
// row of 256 (128) elements is held by 32 (16) lanes, 8 elements each.  The
// lanes of the rotated part hold 4 elements of the first half and their 4
// partners of the second, so a pair turns inside a lane; the others hold 8
// neighbours.  The angle is the expensive part (an fp64 product
// and reduction, a sine and cosine) and the same for every head: the warp
// computes its token's angles once, a lane each, while the rows are on their
// way.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "fp_div.cuh"
#include "paged_batch.cuh"
#include "ptx_sm100.cuh"

namespace nvfp4 {
namespace attn {

constexpr int ROW_WARPS = 4;        // warps of a block
constexpr int MAX_HALF = 128;       // rotated pairs of a head (head_dim <= 256)
constexpr int UNIT_BYTES = 4096;    // of the rows that a warp takes at most

// cos and sin of pos * f.  The product of a 31-bit position and a 24-bit
// frequency is held in fp64, multiplied by 1 / 2 pi (in two parts) and reduced
// to less than half a turn by exact steps; fp32 keeps the rest to 2^-25.
__device__ __forceinline__ float2 rotation(int32_t pos, float f)
{
    const double a = static_cast<double>(pos) * static_cast<double>(f);
    const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;  // hi + lo = 1 / 2 pi
    const double turns = rint(a * hi);
    const float t = static_cast<float>(fma(a, lo, fma(a, hi, -turns)));
    float2 cs;
    sincospif(2.0f * t, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a lane's 8 elements of a row lie: 4 at `a` and 4 at `b`; rotated: b is
// a's partner.
struct LaneMap {
    int a, b;
    bool turned;

    __device__ __forceinline__ LaneMap(int lane_of_row, int half)
    {
        turned = lane_of_row < (half >> 2);
        a = lane_of_row * (turned ? 4 : 8);
        b = turned ? half + a : a + 4;
    }
};

__device__ __forceinline__ uint4 load_row(const uint16_t *row, const LaneMap &m)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(row + m.a), v = *reinterpret_cast<const uint2 *>(row + m.b);
    return make_uint4(u.x, u.y, v.x, v.y);
}

// 16 bytes to shared memory, asynchronously, and the wait for all of them.
__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// The token's rotations to shared memory (one warp's share), then the lane's 4.
__device__ __forceinline__ void load_rotations(float2 *cs, int32_t pos, const float *inv_freq, int half, const LaneMap &m,
                                               int lane, float (&c)[4], float (&s)[4])
{
    for (int i = lane; i < half; i += 32)
        cs[i] = rotation(pos, __ldg(inv_freq + i));
    __syncwarp();
    if (m.turned) {
        const float4 u = *reinterpret_cast<const float4 *>(cs + m.a), v = *reinterpret_cast<const float4 *>(cs + m.a + 2);
        c[0] = u.x, s[0] = u.y, c[1] = u.z, s[1] = u.w, c[2] = v.x, s[2] = v.y, c[3] = v.z, s[3] = v.w;
    }
}

// Norm and rotation of one row spread over D / 8 lanes, in place.  All 32
// lanes call it (with D = 128 for two rows).
template <int D>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool norm, const float (&w)[8], float eps, bool turned,
                                            const float (&c)[4], const float (&s)[4])
{
    if (norm) {
        float ss = 0.0f, st = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ss = fmaf(x[i], x[i], ss);
            st = fmaf(x[i + 4], x[i + 4], st);
        }
        ss += st;
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = x[i] * r * w[i];
    }
    if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[i], b = x[i + 4];
            x[i] = fmaf(a, c[i], -(b * s[i]));
            x[i + 4] = fmaf(b, c[i], a * s[i]);
        }
    }
}

__device__ __forceinline__ void load_weights(const uint16_t *w, const LaneMap &m, float one, float (&out)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[i] = 1.0f;
    if (w != nullptr) {
        unpack8(load_row(w, m), out);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            out[i] += one;
    }
}

struct HeadRows {
    const uint16_t *data;
    int64_t token_stride, head_stride;
    int32_t heads;
};

struct NormRopeParams {
    HeadRows in[2], out[2];   // queries, keys (heads = 0: absent)
    const uint16_t *weight[2];
    const int32_t *positions;
    const float *inv_freq;
    int32_t half;             // rotary_dim / 2
    float eps;
    float one;                // 1 with NVFP4_NORM_PLUS_ONE, else 0
    int32_t tokens;
    int32_t unit_heads;       // heads of a warp
    int32_t units[2];         // warps of a token: for its queries, for its keys
};

template <int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) qk_norm_rope_kernel(const NormRopeParams p)
{
    constexpr int LANES = D / 8;               // lanes of a row
    constexpr int GROUP = 32 / LANES;          // rows of a warp at a time
    __shared__ alignas(16) float2 cs[ROW_WARPS][MAX_HALF];
    __shared__ alignas(16) uint16_t in_rows[ROW_WARPS][UNIT_BYTES / 2];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = p.units[0] + p.units[1];
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * ROW_WARPS + warp;
    const int t = static_cast<int>(unit / per);
    if (t >= p.tokens)
        return;
    int u = static_cast<int>(unit - static_cast<int64_t>(t) * per);
    const int which = u >= p.units[0];
    u -= which ? p.units[0] : 0;
    const HeadRows in = p.in[which], out = p.out[which];
    const int h1 = min((u + 1) * p.unit_heads, in.heads);
    const LaneMap m(lane % LANES, p.half);
    const uint16_t *src = in.data + t * in.token_stride;
    uint16_t *dst = const_cast<uint16_t *>(out.data) + t * out.token_stride;
    int h = u * p.unit_heads + lane / LANES;
    const int lane8 = lane % LANES * 8;
    uint16_t *row = in_rows[warp] + lane / LANES * D;
    for (int i = 0; h + i < h1; i += GROUP)
        copy16(row + i * D + lane8, src + (h + i) * in.head_stride + lane8);
    float w[8], c[4], s[4];
    load_weights(p.weight[which], m, p.one, w);
    if (p.half > 0)
        load_rotations(cs[warp], __ldg(p.positions + t), p.inv_freq, p.half, m, lane, c, s);
    copies_done();
    for (int i = u * p.unit_heads; i < h1; i += GROUP, h += GROUP, row += GROUP * D) {  // alike for all lanes
        float x[8];
        unpack8(load_row(row, m), x);
        norm_rotate<D>(x, p.weight[which] != nullptr, w, p.eps, m.turned, c, s);
        if (h < h1) {
            const uint4 y = pack8(x);
            *reinterpret_cast<uint2 *>(dst + h * out.head_stride + m.a) = make_uint2(y.x, y.y);
            *reinterpret_cast<uint2 *>(dst + h * out.head_stride + m.b) = make_uint2(y.z, y.w);
        }
    }
}

struct AppendParams {
    HeadRows in[2];           // keys, values
    uint8_t *pages[2];
    const float *scale[2];
    int64_t page_stride[2], token_stride[2], head_stride[2];
    const uint16_t *weight;   // of the keys
    const int32_t *positions; // null: cache positions
    const float *inv_freq;
    int32_t half;
    float eps;
    float one;
    int32_t unit_heads, units;
    BatchView batch;
    uint32_t *status;
};

// Four E4M3 codes (round to nearest even, saturating at +-448), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ bool valid_scale(float s) { return s > 0.0f && s <= 3.40282347e38f; }

// Codes of 8 elements divided by s (inv = RN(1 / s)), the IEEE quotients.
__device__ __forceinline__ uint2 codes8(float (&x)[8], float s, float inv)
{
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        big = fmaxf(big, fabsf(x[i]));
    if (div_shared_ok(s, big)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = div_shared(x[i], s, inv);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __fdiv_rn(x[i], s);
    }
    return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) kv_append_kernel(const AppendParams p)
{
    constexpr int LANES = D / 8;
    constexpr int GROUP = 32 / LANES;
    __shared__ alignas(16) float2 cs[ROW_WARPS][MAX_HALF];
    __shared__ alignas(16) uint16_t in_rows[ROW_WARPS][UNIT_BYTES / 2];  // keys, and values in the other half
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float s0 = __ldg(p.scale[0]), s1 = __ldg(p.scale[1]);
    if (!valid_scale(s0) || !valid_scale(s1)) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(p.status, kStatusNonFinite);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * ROW_WARPS + warp;
    const int t = static_cast<int>(unit / p.units);
    if (t >= p.batch.tokens)
        return;
    const int u = static_cast<int>(unit - static_cast<int64_t>(t) * p.units);
    const int h1 = min((u + 1) * p.unit_heads, p.in[0].heads);
    const LaneMap m(lane % LANES, p.half);
    const uint16_t *k_src = p.in[0].data + t * p.in[0].token_stride, *v_src = p.in[1].data + t * p.in[1].token_stride;
    int h = u * p.unit_heads + lane / LANES;
    // the rows are on their way while the token's place is looked up
    const int lane8 = lane % LANES * 8;
    uint16_t *k_row = in_rows[warp] + lane / LANES * D, *v_row = k_row + UNIT_BYTES / 4;
    for (int i = 0; h + i < h1; i += GROUP) {
        copy16(k_row + i * D + lane8, k_src + (h + i) * p.in[0].head_stride + lane8);
        copy16(v_row + i * D + lane8, v_src + (h + i) * p.in[1].head_stride + lane8);
    }
    int b;
    bool bad = false;
    const Seq seq = warp_find_seq(p.batch, t, lane, b, bad);
    const int j = t - seq.first, pos = seq.len - seq.fresh + j;
    int64_t id = -1;
    if (j >= 0 && j < seq.fresh && pos >= 0) {
        id = __ldg(p.batch.table + b * p.batch.table_stride + (pos >> p.batch.page_shift));
        if (id < 0 || id >= p.batch.num_pages) {
            bad = true;
            id = -1;
        }
    }
    if (bad && lane == 0)
        atomicOr(p.status, kStatusBadIndex);
    copies_done();
    if (id < 0)
        return;  // the token belongs to no sequence, or has no place in the cache
    const int64_t row = pos & ((1 << p.batch.page_shift) - 1);
    uint8_t *k_dst = p.pages[0] + id * p.page_stride[0] + row * p.token_stride[0];
    uint8_t *v_dst = p.pages[1] + id * p.page_stride[1] + row * p.token_stride[1];
    float w[8], c[4], s[4];
    load_weights(p.weight, m, p.one, w);
    if (p.half > 0)
        load_rotations(cs[warp], p.positions != nullptr ? __ldg(p.positions + t) : pos, p.inv_freq, p.half, m, lane, c, s);
    const float r0 = __frcp_rn(s0), r1 = __frcp_rn(s1);
    for (int i = u * p.unit_heads; i < h1; i += GROUP, h += GROUP, k_row += GROUP * D, v_row += GROUP * D) {  // alike for all lanes
        float x[8], y[8];
        unpack8(load_row(k_row, m), x);
        unpack8(*reinterpret_cast<const uint4 *>(v_row + lane8), y);
        norm_rotate<D>(x, p.weight != nullptr, w, p.eps, m.turned, c, s);
        const uint2 kc = codes8(x, s0, r0), vc = codes8(y, s1, r1);
        if (h < h1) {
            *reinterpret_cast<uint32_t *>(k_dst + h * p.head_stride[0] + m.a) = kc.x;
            *reinterpret_cast<uint32_t *>(k_dst + h * p.head_stride[0] + m.b) = kc.y;
            *reinterpret_cast<uint2 *>(v_dst + h * p.head_stride[1] + lane8) = vc;
        }
    }
}

}  // namespace attn
}  // namespace nvfp4
