// head_rows_kernels.cuh -- the per-head row operators of an attention layer:
// RMS norm with the position rotation (queries and keys), and the append of
// keys and values to the paged FP8 cache with both applied on the way.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (w, or 1 + w; absent: y = x)
//   (y[i], y[i+R/2]) turned by position * inv_freq[i],  i < R/2
//   out = bf16_RNE(y)   or   code = E4M3_RNE_satfinite(fl32(y / scale))
//
// Both are bound by memory: a row is read once and written once, held in
// registers in between.  A row of 128 (256) elements is taken by 16 (32)
// lanes, 8 elements = one 16-byte load each, so a warp's load covers 512
// contiguous bytes; the mean is a 4- (5-) step shuffle, and since R/2 is a
// multiple of 8 an element's partner sits at the same place of another lane.
// The angle is the expensive part -- an fp64 product and reduction and a
// sincosf -- and the same for every head, so a block computes the angles of
// its tokens once, one thread each, into shared memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "fp_div.cuh"
#include "paged_batch.cuh"
#include "ptx_sm100.cuh"

namespace nvfp4 {
namespace attn {

constexpr int ROW_THREADS = 256;
constexpr int MAX_HALF = 128;       // rotated pairs of a head (head_dim <= 256)
constexpr int BLOCK_TOKENS = 4;     // tokens of a block for large batches

// cos and sin of pos * f.  fp64 holds the product of a 31-bit position and a
// 24-bit frequency to 2^-53 of its value; after whole turns are taken off the
// remainder is below pi and fp32 keeps it to 2^-25 of pi.
__device__ __forceinline__ float2 rotation(int32_t pos, float f)
{
    const double a = static_cast<double>(pos) * static_cast<double>(f);
    const double turns = rint(a * 0.15915494309189533577);
    const float r = static_cast<float>(fma(turns, -2.4492935982947064e-16, fma(turns, -6.283185307179586232, a)));
    float2 cs;
    sincosf(r, &cs.y, &cs.x);
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

// Norm and rotation of one row spread over D / 8 lanes, in place.  `w`: the
// lane's 8 norm weights; cs: the token's rotations; col: the lane's first
// element.  All 32 lanes call it.
template <int D>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool norm, const float (&w)[8], float eps, const float2 *cs,
                                            int half, int col, int lane)
{
    if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = D / 16; o > 0; o >>= 1)
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = x[i] * r * w[i];
    }
    if (half > 0) {
        const bool low = col < half, turned = col < 2 * half;
        const int src = turned ? (low ? lane + (half >> 3) : lane - (half >> 3)) : lane;
        const float2 *my = cs + (turned ? (low ? col : col - half) : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl_sync(0xFFFFFFFFu, x[i], src);
            if (turned) {
                const float2 c = my[i];
                x[i] = low ? fmaf(x[i], c.x, -(other * c.y)) : fmaf(x[i], c.x, other * c.y);
            }
        }
    }
}

__device__ __forceinline__ void load_weights(const uint16_t *w, int col, float one, float (&out)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[i] = 1.0f;
    if (w != nullptr) {
        float x[8];
        unpack8(__ldg(reinterpret_cast<const uint4 *>(w + col)), x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            out[i] = x[i] + one;
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
    int32_t block_tokens;
};

template <int D>
__global__ void __launch_bounds__(ROW_THREADS) qk_norm_rope_kernel(const NormRopeParams p)
{
    constexpr int LANES = D / 8;               // lanes of a row
    constexpr int GROUP = 32 / LANES;          // rows of a warp at a time
    constexpr int STEP = ROW_THREADS / LANES;  // rows of the block at a time
    __shared__ float2 cs[BLOCK_TOKENS * MAX_HALF];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int col = (lane % LANES) * 8;
    const int heads = p.in[0].heads + p.in[1].heads;
    const int t0 = blockIdx.x * p.block_tokens;
    const int nt = min(p.block_tokens, p.tokens - t0);
    for (int i = threadIdx.x; i < nt * p.half; i += ROW_THREADS) {
        const int t = i / p.half;
        cs[t * MAX_HALF + (i - t * p.half)] = rotation(__ldg(p.positions + t0 + t), __ldg(p.inv_freq + (i - t * p.half)));
    }
    float w[2][8];
    load_weights(p.weight[0], col, p.one, w[0]);
    load_weights(p.weight[1], col, p.one, w[1]);
    __syncthreads();
    const int rows = nt * heads;
    for (int base = (threadIdx.x >> 5) * GROUP; base < rows; base += STEP) {
        const int row = base + lane / LANES;
        const bool live = row < rows;
        const int t = live ? row / heads : 0;
        int h = live ? row - t * heads : 0;
        const int which = h >= p.in[0].heads;
        h -= which ? p.in[0].heads : 0;
        float x[8];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live)
            v = *reinterpret_cast<const uint4 *>(p.in[which].data + (t0 + t) * p.in[which].token_stride +
                                                  h * p.in[which].head_stride + col);
        unpack8(v, x);
        float wr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            wr[i] = which ? w[1][i] : w[0][i];
        norm_rotate<D>(x, p.weight[which] != nullptr, wr, p.eps, cs + t * MAX_HALF, p.half, col, lane);
        if (live)
            *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(p.out[which].data) + (t0 + t) * p.out[which].token_stride +
                                       h * p.out[which].head_stride + col) = pack8(x);
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
    int32_t block_tokens;
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

template <int D>
__global__ void __launch_bounds__(ROW_THREADS) kv_append_kernel(const AppendParams p)
{
    constexpr int LANES = D / 8;
    constexpr int GROUP = 32 / LANES;
    constexpr int STEP = ROW_THREADS / LANES;
    __shared__ float2 cs[BLOCK_TOKENS * MAX_HALF];
    __shared__ int64_t slot[BLOCK_TOKENS];  // page << 32 | row in the page; -1: the token is not cached
    __shared__ int32_t turn[BLOCK_TOKENS];  // position of the rotation
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (lane % LANES) * 8;
    const float s0 = __ldg(p.scale[0]), s1 = __ldg(p.scale[1]);
    if (!valid_scale(s0) || !valid_scale(s1)) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            atomicOr(p.status, kStatusNonFinite);
        return;
    }
    const int t0 = blockIdx.x * p.block_tokens;
    const int nt = min(p.block_tokens, p.batch.tokens - t0);
    if (warp < nt) {  // one warp finds one token's place
        const int t = t0 + warp;
        const int b = warp_find_seq(p.batch, t, lane);
        if (lane == 0) {
            bool bad = false;
            const Seq s = load_seq(p.batch, b, bad);
            const int j = t - s.first;
            const int pos = s.len - s.fresh + j;
            int64_t at = -1;
            if (j >= 0 && j < s.fresh && pos >= 0) {
                const int32_t id = __ldg(p.batch.table + b * p.batch.table_stride + (pos >> p.batch.page_shift));
                if (id >= 0 && id < p.batch.num_pages)
                    at = (static_cast<int64_t>(id) << 32) | (pos & ((1 << p.batch.page_shift) - 1));
                else
                    bad = true;
            }
            slot[warp] = at;
            turn[warp] = p.positions != nullptr ? __ldg(p.positions + t) : max(pos, 0);
            if (bad)
                atomicOr(p.status, kStatusBadIndex);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * p.half; i += ROW_THREADS) {
        const int t = i / p.half;
        cs[t * MAX_HALF + (i - t * p.half)] = rotation(turn[t], __ldg(p.inv_freq + (i - t * p.half)));
    }
    float w[8];
    load_weights(p.weight, col, p.one, w);
    __syncthreads();
    const int heads = p.in[0].heads;
    const int rows = nt * heads * 2;
    for (int base = warp * GROUP; base < rows; base += STEP) {
        const int row = base + lane / LANES;
        const bool live = row < rows;
        const int t = live ? row / (2 * heads) : 0;
        int h = live ? row - t * 2 * heads : 0;
        const int which = h >= heads;
        h -= which ? heads : 0;
        const int64_t at = slot[t];
        float x[8];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && at >= 0)
            v = __ldg(reinterpret_cast<const uint4 *>(p.in[which].data + (t0 + t) * p.in[which].token_stride +
                                                      h * p.in[which].head_stride + col));
        unpack8(v, x);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = x[i];
        norm_rotate<D>(y, p.weight != nullptr, w, p.eps, cs + t * MAX_HALF, p.half, col, lane);
        const float s = which ? s1 : s0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = __fdiv_rn(which ? x[i] : y[i], s);
        if (live && at >= 0)
            *reinterpret_cast<uint2 *>(p.pages[which] + (at >> 32) * p.page_stride[which] +
                                       (at & 0xFFFFFFFF) * p.token_stride[which] + h * p.head_stride[which] + col) =
                make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
    }
}

}  // namespace attn
}  // namespace nvfp4
