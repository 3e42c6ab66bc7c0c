// paged_attention_simple.cuh -- causal attention of new tokens over the paged
// FP8 cache, one block per token and query head.
//
//   s_i = c * sum_d q[d] k_code[i][d],  c = softmax_scale * k_scale
//   out = v_scale * sum_i e^(s_i - m) v_code[i] / sum_i e^(s_i - m)
//
// Keys are taken 128 at a time: one thread per key for the scores, one thread
// per D / 128 output dimensions for the sums, with the running maximum m and
// sum of the softmax carried over the blocks of keys in fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "head_rows_kernels.cuh"
#include "paged_batch.cuh"
#include "ptx_sm100.cuh"

namespace nvfp4 {
namespace attn {

struct AttnParams {
    HeadRows q, gate, out;    // gate.data null: no gate
    const uint8_t *k_pages, *v_pages;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    const float *k_scale, *v_scale;
    int32_t kv_heads, group;
    float softmax_scale;
    BatchView batch;
    uint32_t *out_amax;
    uint32_t *status;
};

template <int D>
__global__ void __launch_bounds__(128) paged_attention_simple_kernel(const AttnParams p)
{
    constexpr int DIMS = D / 128;
    __shared__ float qs[D];
    __shared__ float ps[128];
    __shared__ int64_t vrow[128];
    __shared__ float red[4];
    __shared__ int32_t found[3];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = blockIdx.x, h = blockIdx.y, hk = h / p.group;
    const float ks = __ldg(p.k_scale), vs = __ldg(p.v_scale);
    if (!valid_scale(ks) || !valid_scale(vs)) {
        if (t == 0 && h == 0 && tid == 0)
            atomicOr(p.status, kStatusNonFinite);
        return;
    }
    if (warp == 0) {
        const int b = warp_find_seq(p.batch, t, lane);
        if (lane == 0) {
            bool bad = false;
            const Seq s = load_seq(p.batch, b, bad);
            const int j = t - s.first;
            found[0] = (j >= 0 && j < s.fresh) ? 1 : 0;
            found[1] = max(s.len - s.fresh + j + 1, 0);  // keys in sight
            found[2] = b;
            if (bad)
                atomicOr(p.status, kStatusBadIndex);
        }
    }
    for (int i = tid; i < D; i += 128)
        qs[i] = __uint_as_float(static_cast<uint32_t>(p.q.data[t * p.q.token_stride + h * p.q.head_stride + i]) << 16);
    __syncthreads();
    if (!found[0])
        return;
    const int n = found[1];
    const int32_t *table = p.batch.table + found[2] * p.batch.table_stride;
    const float c = p.softmax_scale * ks;
    float m = -INFINITY, l = 0.0f, o[DIMS];
    for (int i = 0; i < DIMS; ++i)
        o[i] = 0.0f;
    for (int k0 = 0; k0 < n; k0 += 128) {
        const int key = k0 + tid;
        float s = -INFINITY;
        if (key < n) {
            int64_t id = __ldg(table + (key >> p.batch.page_shift));
            if (id < 0 || id >= p.batch.num_pages) {
                atomicOr(p.status, kStatusBadIndex);
                id = 0;
            }
            const int64_t r = key & ((1 << p.batch.page_shift) - 1);
            const uint8_t *kr = p.k_pages + id * p.k_page_stride + r * p.k_token_stride + hk * p.k_head_stride;
            vrow[tid] = id * p.v_page_stride + r * p.v_token_stride + hk * p.v_head_stride;
            s = 0.0f;
            for (int d = 0; d < D; d += 16) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(kr + d));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                for (int e = 0; e < 16; ++e)
                    s = fmaf(qs[d + e], e4m3_to_f32(w[e >> 2] >> (8 * (e & 3))), s);
            }
            s *= c;
        }
        float mx = s;
        for (int off = 16; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        if (lane == 0)
            red[warp] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float m2 = fmaxf(m, mx), w = expf(m - m2);
        m = m2;
        ps[tid] = key < n ? expf(s - m) : 0.0f;
        __syncthreads();
        l *= w;
        for (int i = 0; i < DIMS; ++i)
            o[i] *= w;
        const int cnt = min(128, n - k0);
        for (int k = 0; k < cnt; ++k) {
            l += ps[k];
            for (int i = 0; i < DIMS; ++i)
                o[i] = fmaf(ps[k], e4m3_to_f32(__ldg(p.v_pages + vrow[k] + tid + 128 * i)), o[i]);
        }
        __syncthreads();
    }
    uint32_t mag = 0;
    for (int i = 0; i < DIMS; ++i) {
        const int d = tid + 128 * i;
        float y = n > 0 ? o[i] / l * vs : 0.0f;
        if (p.gate.data != nullptr) {
            const float g =
                __uint_as_float(static_cast<uint32_t>(p.gate.data[t * p.gate.token_stride + h * p.gate.head_stride + d]) << 16);
            y = y / (1.0f + expf(-g));
        }
        const unsigned short b = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        const_cast<uint16_t *>(p.out.data)[t * p.out.token_stride + h * p.out.head_stride + d] = b;
        mag = max(mag, static_cast<uint32_t>(b & 0x7FFFu));
    }
    if (p.out_amax != nullptr) {
        for (int off = 16; off > 0; off >>= 1)
            mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, off));
        if (lane == 0)
            atomicMax(p.out_amax, mag);
    }
}

}  // namespace attn
}  // namespace nvfp4
