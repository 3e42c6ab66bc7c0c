// attention_api.cu -- the attention layer's entry points of the C ABI: head
// norms and rotation, the paged FP8 cache's append, attention over it.
// Argument checks and launches; declared and documented in include/nvfp4.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include <cuda.h>
#include <cuda_runtime.h>

#include "nvfp4.h"
#include "head_rows_kernels.cuh"
#include "host.h"
#include "paged_attention_kernel.cuh"
#include "paged_batch.cuh"
#include "paged_decode_kernel.cuh"

namespace {

using nvfp4::host::launch;
namespace attn = nvfp4::attn;

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Status of a call whose last launch this was, which is counted if it took place.
int launched()
{
    if (nvfp4::host::launch_failed())
        return NVFP4_ERR_CUDA;
    nvfp4::host::count_launch();
    return NVFP4_OK;
}

int check_head_dim(int64_t d) { return (d == 128 || d == 256) ? NVFP4_OK : NVFP4_ERR_UNSUPPORTED_SHAPE; }

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxHeads = 1024;

int check_heads(const nvfp4_heads *x, int64_t tokens)
{
    if (x == nullptr || x->heads < 1 || (tokens > 0 && x->data == nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (x->heads > kMaxHeads)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(x->data, 16) || x->token_stride % 8 != 0 || x->head_stride % 8 != 0)
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

// Bytes [lo, hi) that head rows span, gaps between them included.
struct Span {
    __int128 lo, hi;
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

Span span_of(const void *p, __int128 bytes)
{
    const __int128 lo = static_cast<__int128>(reinterpret_cast<uintptr_t>(p));
    return {lo, lo + bytes};
}

Span span_of(const nvfp4_heads &x, int64_t tokens, int64_t head_dim)
{
    Span s = span_of(x.data, 2 * head_dim);
    for (const __int128 reach : {static_cast<__int128>(tokens - 1) * x.token_stride, static_cast<__int128>(x.heads - 1) * x.head_stride})
        (reach < 0 ? s.lo : s.hi) += 2 * reach;
    return s;
}

bool same_rows(const nvfp4_heads &a, const nvfp4_heads &b, int64_t tokens)
{
    return a.data == b.data && a.heads == b.heads && (tokens == 1 || a.token_stride == b.token_stride) &&
           (a.heads == 1 || a.head_stride == b.head_stride);
}

// Whether some row of `a` and some row of `b` share an element.  Views of one
// projection's output have one token stride: there the answer is exact.  With
// two token strides, spans that meet count as an overlap.
bool rows_meet(const nvfp4_heads &a, const nvfp4_heads &b, int64_t tokens, int64_t head_dim)
{
    const Span sa = span_of(a, tokens, head_dim), sb = span_of(b, tokens, head_dim);
    if (!sa.meets(sb))
        return false;
    if (tokens > 1 && a.token_stride != b.token_stride)
        return true;
    constexpr int64_t kFar = int64_t(1) << 50;  // beyond any memory, and the sums below stay in 64 bits
    if (sa.hi - sa.lo > kFar || sb.hi - sb.lo > kFar)
        return true;
    const int64_t step = tokens > 1 ? std::abs(a.token_stride) : 0;
    const int64_t apart = (static_cast<const char *>(b.data) - static_cast<const char *>(a.data)) / 2;
    const int64_t ha = a.heads > 1 ? a.head_stride : 0, hb = b.heads > 1 ? b.head_stride : 0;
    // rows of one token next to those of the other within a token's stride: columns of one projection's output
    const int64_t wide_a = (a.heads - 1) * ha + head_dim, wide_b = (b.heads - 1) * hb + head_dim;
    if (step > 0 && ha >= 0 && hb >= 0) {
        const int64_t at = ((apart % step) + step) % step;
        if (wide_a <= at && at + wide_b <= step)
            return false;
    }
    // a row of b that lies `d` elements behind one of a, at the same token or at tokens - 1 others at most
    auto near = [&](int64_t d) {
        if (step == 0)
            return std::abs(d) < head_dim;
        const int64_t n = std::min<int64_t>(std::abs(d) / step, tokens - 1), rest = std::abs(d) - n * step;
        return rest < head_dim || (n + 1 < tokens && step - rest < head_dim);
    };
    if (ha == hb) {  // only the difference of two heads counts
        for (int64_t h = 1 - a.heads; h < b.heads; ++h)
            if (near(apart + h * ha))
                return true;
        return false;
    }
    for (int64_t i = 0; i < a.heads; ++i)
        for (int64_t k = 0; k < b.heads; ++k)
            if (near(apart + k * hb - i * ha))
                return true;
    return false;
}

int check_tokens(int64_t tokens)
{
    if (tokens < 0)
        return NVFP4_ERR_INVALID_ARG;
    return tokens <= kMaxTokens ? NVFP4_OK : NVFP4_ERR_UNSUPPORTED_SHAPE;
}

// `weight`: the norm weight that this call reads.
int check_norm_rope(const nvfp4_norm_rope *n, int64_t head_dim)
{
    if (n == nullptr || (n->flags & ~NVFP4_NORM_PLUS_ONE) != 0 || n->rotary_dim < 0 || !(n->eps >= 0.0f) ||
        !std::isfinite(n->eps) || (n->rotary_dim > 0 && n->inv_freq == nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (n->rotary_dim % 16 != 0 || n->rotary_dim > head_dim)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(n->q_weight, 16) || !aligned(n->k_weight, 16) || !aligned(n->inv_freq, 4))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

// Strides of a tensor map in the order of their size, each a multiple of the
// one before it, as the map's definition asks.
bool strides_nest(int64_t a, int64_t b, int64_t c)
{
    int64_t s[3] = {a, b, c};
    std::sort(s, s + 3);
    return s[0] > 0 && s[1] % s[0] == 0 && s[2] % s[1] == 0;
}

int check_pages(const nvfp4_kv_pages *c)
{
    if (c == nullptr || c->k_pages == nullptr || c->v_pages == nullptr || c->k_scale == nullptr ||
        c->v_scale == nullptr || c->num_pages < 1 || c->kv_heads < 1)
        return NVFP4_ERR_INVALID_ARG;
    int rc = check_head_dim(c->head_dim);
    if (rc != NVFP4_OK)
        return rc;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0 ||
        c->kv_heads > kMaxHeads || c->num_pages >= (int64_t(1) << 31))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    const int64_t strides[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                                c->v_page_stride, c->v_token_stride, c->v_head_stride};
    for (int64_t s : strides) {
        if (s < c->head_dim)
            return NVFP4_ERR_INVALID_ARG;
        if (s % 16 != 0)
            return NVFP4_ERR_MISALIGNED;
        if (s >= (int64_t(1) << 40))
            return NVFP4_ERR_UNSUPPORTED_SHAPE;
    }
    if (!strides_nest(c->k_page_stride, c->k_token_stride, c->k_head_stride) ||
        !strides_nest(c->v_page_stride, c->v_token_stride, c->v_head_stride) || !aligned(c->k_pages, 16) ||
        !aligned(c->v_pages, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

int check_batch(const nvfp4_kv_batch *b, int32_t page_size)
{
    if (b == nullptr || b->num_seqs < 0 || b->max_pages < 0)
        return NVFP4_ERR_INVALID_ARG;
    if (b->num_seqs > 0 && (b->cu_tokens == nullptr || b->seq_lens == nullptr ||
                            (b->max_pages > 0 && b->page_table == nullptr) || b->table_stride < b->max_pages))
        return NVFP4_ERR_INVALID_ARG;
    // positions are 32-bit, and so are they rounded up to the end of a key block and the block behind it
    if (b->num_seqs > (1 << 20) || int64_t(b->max_pages) * page_size > (int64_t(1) << 31) - 2 * attn::KEY_BLOCK)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(b->cu_tokens, 4) || !aligned(b->seq_lens, 4) || !aligned(b->page_table, 4))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

attn::HeadRows rows_of(const nvfp4_heads *x)
{
    attn::HeadRows r;
    r.data = x == nullptr ? nullptr : static_cast<const uint16_t *>(x->data);
    r.token_stride = x == nullptr ? 0 : x->token_stride;
    r.head_stride = x == nullptr ? 0 : x->head_stride;
    r.heads = x == nullptr ? 0 : static_cast<int32_t>(x->heads);
    return r;
}

int32_t log2_of(int32_t v)
{
    int32_t s = 0;
    while ((1 << s) < v)
        ++s;
    return s;
}

attn::BatchView batch_view(const nvfp4_kv_batch *b, const nvfp4_kv_pages *c, int64_t tokens)
{
    attn::BatchView v;
    v.table = b->page_table;
    v.cu = b->cu_tokens;
    v.lens = b->seq_lens;
    v.table_stride = b->table_stride;
    v.num_seqs = b->num_seqs;
    v.max_pages = b->max_pages;
    v.page_shift = log2_of(c->page_size);
    v.tokens = static_cast<int32_t>(tokens);
    v.num_pages = c->num_pages;
    v.fresh_min = 1;
    v.fresh_max = INT32_MAX;
    v.item_cost = 0;
    return v;
}

// The pages of K or V as a 4-D byte tensor, dimensions in the order of their
// strides behind the contiguous head_dim; row_at and head_at say where the
// page's rows and the heads ended up.  A box is one page's rows (128 at most)
// by 128 bytes of one head.
int make_page_map(const nvfp4::host::Device &d, CUtensorMap *map, const void *base, const nvfp4_kv_pages *c,
                  int64_t page_stride, int64_t row_stride, int64_t head_stride, int32_t *row_at, int32_t *head_at)
{
    struct Dim {
        int64_t stride, size;
        int which;  // 0 row, 1 head, 2 page
    } dims[3] = {{row_stride, c->page_size, 0}, {head_stride, c->kv_heads, 1}, {page_stride, c->num_pages, 2}};
    std::sort(dims, dims + 3, [](const Dim &a, const Dim &b) {
        return a.stride != b.stride ? a.stride < b.stride : a.which < b.which;
    });
    cuuint64_t size[4] = {static_cast<cuuint64_t>(c->head_dim), 0, 0, 0};
    cuuint64_t stride[3];
    cuuint32_t box[4] = {128, 1, 1, 1}, unit[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        size[i + 1] = static_cast<cuuint64_t>(dims[i].size);
        stride[i] = static_cast<cuuint64_t>(dims[i].stride);
        if (dims[i].which == 0) {
            box[i + 1] = static_cast<cuuint32_t>(std::min(c->page_size, attn::KEY_BLOCK));
            *row_at = i + 1;
        } else if (dims[i].which == 1) {
            *head_at = i + 1;
        }
    }
    const CUresult r = d.encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), size, stride, box,
                                      unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? NVFP4_OK : NVFP4_ERR_CUDA;
}

// Shared memory beyond the default, once per device.
int allow_smem(int device)
{
    static std::atomic<bool> done[64];
    if (device < 0 || device >= 64)
        return NVFP4_ERR_CUDA;
    if (done[device].load(std::memory_order_acquire))
        return NVFP4_OK;
    if (cudaFuncSetAttribute(attn::paged_attention_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::attn_smem_bytes<128>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::paged_attention_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::attn_smem_bytes<256>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::paged_decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::decode_smem_bytes<128>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::paged_decode_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::decode_smem_bytes<256>()) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    done[device].store(true, std::memory_order_release);
    return NVFP4_OK;
}

// Workspace: two sets of parts (the tile kernel's, the single-token kernel's).
// A set: a PartInfo per CTA, then the two parts of each CTA: per row its
// reference and sum, then its sums of values.
constexpr int64_t kPartsBytes = (attn::CTAS * sizeof(attn::PartInfo) + 255) / 256 * 256;

int64_t part_rows(int64_t tokens, int64_t group) { return std::min<int64_t>(attn::ROW_TILE / group, tokens) * group; }

int64_t part_ml_bytes(int64_t rows) { return (attn::CTAS * 2 * rows * 8 + 255) / 256 * 256; }

int64_t parts_bytes(int64_t rows, int64_t head_dim)
{
    return kPartsBytes + part_ml_bytes(rows) + attn::CTAS * 2 * rows * head_dim * 4;
}

attn::Parts parts_at(uint8_t *base, int64_t rows)
{
    attn::Parts p;
    p.info = reinterpret_cast<attn::PartInfo *>(base);
    p.ml = reinterpret_cast<float *>(base + kPartsBytes);
    p.o = reinterpret_cast<float *>(base + kPartsBytes + part_ml_bytes(rows));
    p.rows = static_cast<int32_t>(rows);
    return p;
}

// Where a batch may hold both kinds of sequences, the single tokens get their
// own kernel beside the tile kernel from this many single items on (sequences
// x key heads).  Measured (us, both kernels against the tile kernel alone):
// 64 x 4 heads of 256, 8192 keys, a chunk of 512: 201 against 203; 16 x 4, 4000
// keys, a chunk of 1000: 144 against 121; 200 x 4, 2000 keys, 512: 138 against
// 189; 8 heads of 128, 4000 keys, a chunk of 500: 32 x 8: 104 against 107; 48 x
// 8: 120 against 131; 128 x 8: 192 against 235.
constexpr int32_t kMixedItems = 370;
// Rows beyond the sequences up to which a batch counts as padded single
// tokens.  For padded single tokens alone (us, both kernels against the tile
// kernel alone): 64 x 8192 keys of 4 heads of 256: 98 against 123; 64 x 500: 25
// against 44; 1 x 777: 13.4 against 16.3; 256 x 1000 keys of 8 heads of 128: 85
// against 184.
constexpr int32_t kPadRows = 8;
// What an item costs beside its keys, in keys: the time from one item's last
// block to the next one's first.  Tile kernel, D = 256: 20 thousand cycles (a
// block of 128 keys: 2300 to 2600); a prompt of 8192 takes 1010 us at 512, 917
// at 768, 800 to 850 at 1152.  D = 128 (32 heads on 8), at 256, 384, 512, 768
// and 1024: a prompt of 4000 takes 271, 244, 223, 219 and 226 us, four chunks of
// 509 with up to 16384 keys 329, 320, 312, 304 and 307, 1000 tokens beside 23
// single ones 145, 137, 136, 137 and 139.  Single tokens, D = 256: 64 x 8192
// takes 105 us at 32, 102 at 128, 99 at 320; D = 128: 256 x 1000 takes 101 at
// 32, 85 at 128, 92 at 320.
constexpr int32_t kTileItemCost256 = 1152, kTileItemCost128 = 512, kDecodeItemCost256 = 320, kDecodeItemCost128 = 128;

// Heads that one warp of the row kernels takes, sharing the token's angles:
// one while the rows do not fill the GPU, then as many as leave 16 warps an
// SM, up to `most`.  Measured (us): 16 tokens x 28 heads 2.6 with one, 4.2
// with 8; 1337 tokens 7.2 with 3, 5.2 with 8; 8192 tokens 62 with 2, 49 with
// 4, 45 with 8.
int unit_heads(int64_t rows, int64_t heads, int sm_count, int64_t most)
{
    return static_cast<int>(std::max<int64_t>(1, std::min({most, heads, rows / (int64_t(sm_count) * 16)})));
}

int64_t row_blocks(int64_t units) { return cdiv(units, attn::ROW_WARPS); }

}  // namespace

extern "C" int nvfp4_qk_norm_rope(const nvfp4_heads *q, const nvfp4_heads *k, const nvfp4_heads *q_out,
                                  const nvfp4_heads *k_out, int64_t tokens, int64_t head_dim, const int32_t *positions,
                                  const nvfp4_norm_rope *norm_rope, void *stream)
{
    int rc = check_tokens(tokens);
    if (rc == NVFP4_OK)
        rc = check_head_dim(head_dim);
    if (rc == NVFP4_OK)
        rc = check_norm_rope(norm_rope, head_dim);
    if (rc == NVFP4_OK)
        rc = check_heads(q, tokens);
    if (rc == NVFP4_OK)
        rc = check_heads(q_out, tokens);
    if (rc != NVFP4_OK)
        return rc;
    if (q_out->heads != q->heads || (k == nullptr) != (k_out == nullptr) ||
        (k != nullptr && k->heads != k_out->heads) ||
        (tokens > 0 && norm_rope->rotary_dim > 0 && positions == nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (k != nullptr) {
        rc = check_heads(k, tokens);
        if (rc == NVFP4_OK)
            rc = check_heads(k_out, tokens);
        if (rc != NVFP4_OK)
            return rc;
    }
    if (!aligned(positions, 4))
        return NVFP4_ERR_MISALIGNED;
    if (tokens == 0)
        return NVFP4_OK;
    // warps read rows while others write theirs; a row that is its own output is read before it is written
    if ((!same_rows(*q, *q_out, tokens) && rows_meet(*q, *q_out, tokens, head_dim)) ||
        (k != nullptr && ((!same_rows(*k, *k_out, tokens) && rows_meet(*k, *k_out, tokens, head_dim)) ||
                          rows_meet(*q_out, *k_out, tokens, head_dim) || rows_meet(*q, *k_out, tokens, head_dim) ||
                          rows_meet(*k, *q_out, tokens, head_dim))))
        return NVFP4_ERR_INVALID_ARG;
    nvfp4::host::Device d;
    rc = nvfp4::host::device(&d);
    if (rc != NVFP4_OK)
        return rc;
    attn::NormRopeParams p;
    p.in[0] = rows_of(q);
    p.in[1] = rows_of(k);
    p.out[0] = rows_of(q_out);
    p.out[1] = rows_of(k_out);
    p.weight[0] = static_cast<const uint16_t *>(norm_rope->q_weight);
    p.weight[1] = static_cast<const uint16_t *>(norm_rope->k_weight);
    p.positions = positions;
    p.inv_freq = norm_rope->inv_freq;
    p.half = norm_rope->rotary_dim / 2;
    p.eps = norm_rope->eps;
    p.one = (norm_rope->flags & NVFP4_NORM_PLUS_ONE) ? 1.0f : 0.0f;
    p.tokens = static_cast<int32_t>(tokens);
    const int64_t rows = tokens * (p.in[0].heads + p.in[1].heads) * head_dim / 256;
    p.unit_heads = unit_heads(rows, std::max(p.in[0].heads, p.in[1].heads), d.sm_count, 8) * static_cast<int>(256 / head_dim);
    p.units[0] = static_cast<int32_t>(cdiv(p.in[0].heads, p.unit_heads));
    p.units[1] = static_cast<int32_t>(cdiv(p.in[1].heads, p.unit_heads));
    const dim3 grid(static_cast<unsigned>(row_blocks(tokens * (p.units[0] + p.units[1]))));
    launch(head_dim == 256 ? attn::qk_norm_rope_kernel<256> : attn::qk_norm_rope_kernel<128>, grid,
           dim3(attn::ROW_WARPS * 32), 0, static_cast<cudaStream_t>(stream), p);
    return launched();
}

extern "C" int nvfp4_fp8_kv_append(const nvfp4_heads *k, const nvfp4_heads *v, int64_t tokens,
                                   const nvfp4_kv_pages *cache, const nvfp4_kv_batch *batch, const int32_t *positions,
                                   const nvfp4_norm_rope *norm_rope, void *stream)
{
    int rc = check_tokens(tokens);
    if (rc == NVFP4_OK)
        rc = check_pages(cache);
    if (rc == NVFP4_OK)
        rc = check_batch(batch, cache->page_size);
    if (rc == NVFP4_OK)
        rc = check_norm_rope(norm_rope, cache->head_dim);
    if (rc == NVFP4_OK)
        rc = check_heads(k, tokens);
    if (rc == NVFP4_OK)
        rc = check_heads(v, tokens);
    if (rc != NVFP4_OK)
        return rc;
    if (k->heads != cache->kv_heads || v->heads != cache->kv_heads)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned(positions, 4))
        return NVFP4_ERR_MISALIGNED;
    if (tokens == 0 || batch->num_seqs == 0)
        return NVFP4_OK;
    nvfp4::host::Device d;
    rc = nvfp4::host::device(&d);
    if (rc != NVFP4_OK)
        return rc;
    attn::AppendParams p;
    p.in[0] = rows_of(k);
    p.in[1] = rows_of(v);
    p.pages[0] = static_cast<uint8_t *>(cache->k_pages);
    p.pages[1] = static_cast<uint8_t *>(cache->v_pages);
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.page_stride[0] = cache->k_page_stride;
    p.page_stride[1] = cache->v_page_stride;
    p.token_stride[0] = cache->k_token_stride;
    p.token_stride[1] = cache->v_token_stride;
    p.head_stride[0] = cache->k_head_stride;
    p.head_stride[1] = cache->v_head_stride;
    p.weight = static_cast<const uint16_t *>(norm_rope->k_weight);
    p.positions = positions;
    p.inv_freq = norm_rope->inv_freq;
    p.half = norm_rope->rotary_dim / 2;
    p.eps = norm_rope->eps;
    p.one = (norm_rope->flags & NVFP4_NORM_PLUS_ONE) ? 1.0f : 0.0f;
    p.batch = batch_view(batch, cache, tokens);
    p.status = d.status;
    const int64_t rows = tokens * cache->kv_heads * 2 * cache->head_dim / 256;
    p.unit_heads = unit_heads(rows, cache->kv_heads, d.sm_count, 4) * (256 / cache->head_dim);
    p.units = static_cast<int32_t>(cdiv(cache->kv_heads, p.unit_heads));
    const dim3 grid(static_cast<unsigned>(row_blocks(tokens * p.units)));
    launch(cache->head_dim == 256 ? attn::kv_append_kernel<256> : attn::kv_append_kernel<128>, grid,
           dim3(attn::ROW_WARPS * 32), 0, static_cast<cudaStream_t>(stream), p);
    return launched();
}

extern "C" size_t nvfp4_fp8_kv_attention_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads,
                                                         int64_t head_dim)
{
    if (check_tokens(tokens) != NVFP4_OK || check_head_dim(head_dim) != NVFP4_OK || q_heads < 1 || kv_heads < 1 ||
        q_heads > kMaxHeads || q_heads % kv_heads != 0 || q_heads / kv_heads > 128)
        return 0;
    const int64_t group = q_heads / kv_heads;
    return static_cast<size_t>(parts_bytes(part_rows(tokens, group), head_dim) +
                               (group <= attn::DECODE_ROWS ? parts_bytes(group, head_dim) : 0));
}

extern "C" int nvfp4_fp8_kv_attention(const nvfp4_heads *q, const nvfp4_heads *gate, const nvfp4_heads *out,
                                      int64_t tokens, const nvfp4_kv_pages *cache, const nvfp4_kv_batch *batch,
                                      const nvfp4_attention_opts *opts, uint32_t *out_amax, void *ws, size_t ws_bytes,
                                      void *stream)
{
    int rc = check_tokens(tokens);
    if (rc == NVFP4_OK)
        rc = check_pages(cache);
    if (rc == NVFP4_OK)
        rc = check_batch(batch, cache->page_size);
    if (rc == NVFP4_OK)
        rc = check_heads(q, tokens);
    if (rc == NVFP4_OK)
        rc = check_heads(out, tokens);
    if (rc == NVFP4_OK && gate != nullptr)
        rc = check_heads(gate, tokens);
    if (rc != NVFP4_OK)
        return rc;
    if (opts == nullptr || (opts->flags & ~NVFP4_SINGLE_TOKENS) != 0 || !(opts->softmax_scale > 0.0f) || !std::isfinite(opts->softmax_scale) ||
        out->heads != q->heads || (gate != nullptr && gate->heads != q->heads))
        return NVFP4_ERR_INVALID_ARG;
    if (q->heads % cache->kv_heads != 0 || q->heads / cache->kv_heads > 128)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    // The line of cost, times the number of CTAs, stays in 64 bits whatever the offsets and lengths hold: an item for
    // every sequence, row and key head, each with the longest length.
    const double line = double(batch->num_seqs) * double(tokens) * cache->kv_heads *
                        (double(batch->max_pages) * cache->page_size + attn::ROW_TILE + kTileItemCost256);
    if (line * attn::CTAS > 9e18)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(out_amax, 4) || !aligned(ws, 16))
        return NVFP4_ERR_MISALIGNED;
    if (ws == nullptr ||
        ws_bytes < nvfp4_fp8_kv_attention_workspace_bytes(tokens, q->heads, cache->kv_heads, cache->head_dim))
        return NVFP4_ERR_WORKSPACE;
    const int64_t dim = cache->head_dim;
    const Span scratch = span_of(ws, nvfp4_fp8_kv_attention_workspace_bytes(tokens, q->heads, cache->kv_heads, dim));
    if (out_amax != nullptr && scratch.meets(span_of(out_amax, 4)))
        return NVFP4_ERR_INVALID_ARG;
    // CTAs read an item's queries and gates while others write their results
    if (tokens > 0 && (rows_meet(*q, *out, tokens, dim) || (gate != nullptr && rows_meet(*gate, *out, tokens, dim)) ||
                       scratch.meets(span_of(*out, tokens, dim)) || scratch.meets(span_of(*q, tokens, dim)) ||
                       (gate != nullptr && scratch.meets(span_of(*gate, tokens, dim)))))
        return NVFP4_ERR_INVALID_ARG;
    nvfp4::host::Device d;
    rc = nvfp4::host::device(&d);
    if (rc != NVFP4_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (out_amax != nullptr) {
        rc = nvfp4::host::clear_words(out_amax, 1, s);
        if (rc != NVFP4_OK)
            return rc;
    }
    if (tokens == 0 || batch->num_seqs == 0)
        return NVFP4_OK;
    // Sequences with one new token go to the kernel for single tokens where the
    // heads that share a key fit its rows.  The lengths are on the device, so
    // the sizes have to say which kernels may find work.  One row alone is a
    // single token.  As many rows as sequences, fewer or a few more may be
    // single tokens, padded or not, or a chunk among sequences that stand
    // still, and many sequences hold both kinds: both kernels.  Else the tile
    // kernel takes everything.  Where the caller expects single tokens, their
    // kernel takes everything: it is right for more tokens too, but reads their
    // keys again for each.  Measured (us, both kernels against that one alone):
    // 2 x 777 keys of 4 heads of 256: 13.4 against 11.5; 64 x 500: 24.4 against
    // 21.1; 64 x 8192: 117.8 against 113.3; a chunk of 64 tokens at 8192 beside
    // 63 sequences that stand still: 44.8 against 138.8.
    const int64_t group = q->heads / cache->kv_heads;
    const bool expected = (opts->flags & NVFP4_SINGLE_TOKENS) != 0;
    const bool single = group <= attn::DECODE_ROWS &&
                        (expected || int64_t(batch->num_seqs) * cache->kv_heads >= kMixedItems || tokens <= int64_t(batch->num_seqs) + kPadRows);
    const bool tiled = !single || (tokens > 1 && !expected);
    attn::AttnParams p;
    p.q = rows_of(q);
    p.gate = rows_of(gate);
    p.out = rows_of(out);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.kv_heads = cache->kv_heads;
    p.group = static_cast<int32_t>(group);
    p.group_inv = static_cast<uint32_t>((65536 + group - 1) / group);
    p.softmax_scale = opts->softmax_scale;
    p.batch = batch_view(batch, cache, tokens);
    p.out_amax = out_amax;
    p.status = d.status;
    uint8_t *base = static_cast<uint8_t *>(ws);
    const attn::Parts parts[2] = {
        parts_at(base, part_rows(tokens, group)),
        parts_at(base + parts_bytes(part_rows(tokens, group), cache->head_dim), group)};
    if (allow_smem(d.index) != NVFP4_OK)
        return NVFP4_ERR_CUDA;
    CUtensorMap tm_k, tm_v;
    if (make_page_map(d, &tm_k, cache->k_pages, cache, cache->k_page_stride, cache->k_token_stride, cache->k_head_stride,
                      &p.k_row_at, &p.k_head_at) != NVFP4_OK ||
        make_page_map(d, &tm_v, cache->v_pages, cache, cache->v_page_stride, cache->v_token_stride, cache->v_head_stride,
                      &p.v_row_at, &p.v_head_at) != NVFP4_OK)
        return NVFP4_ERR_CUDA;
    int sets = 0;
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? tiled : single))
            continue;
        p.parts = parts[k];
        p.tile_tokens = k == 0 ? attn::ROW_TILE / p.group : 1;
        p.batch.fresh_min = k == 0 && single ? 2 : 1;
        p.batch.fresh_max = k == 0 || !tiled ? INT32_MAX : 1;
        p.batch.item_cost = cache->head_dim == 256 ? (k ? kDecodeItemCost256 : kTileItemCost256) : (k ? kDecodeItemCost128 : kTileItemCost128);
        if (k == 0)
            launch(cache->head_dim == 256 ? attn::paged_attention_kernel<256> : attn::paged_attention_kernel<128>,
                   dim3(attn::CTAS), dim3(attn::ATTN_THREADS),
                   cache->head_dim == 256 ? attn::attn_smem_bytes<256>() : attn::attn_smem_bytes<128>(), s, tm_k, tm_v, p);
        else
            launch(cache->head_dim == 256 ? attn::paged_decode_kernel<256> : attn::paged_decode_kernel<128>,
                   dim3(attn::CTAS), dim3(attn::DECODE_THREADS),
                   cache->head_dim == 256 ? attn::decode_smem_bytes<256>() : attn::decode_smem_bytes<128>(), s, tm_k, tm_v, p);
        // The join takes addresses from what these kernels leave in the workspace: refused, they leave anything.
        if (nvfp4::host::launch_failed())
            return NVFP4_ERR_CUDA;
        nvfp4::host::count_launch();
        ++sets;
    }
    p.parts = parts[tiled ? 0 : 1];
    const int first_blocks = sets == 2 ? static_cast<int>(attn::CTAS * cdiv(parts[1].rows, attn::JOIN_ROWS)) : 0;
    const dim3 join_grid(static_cast<unsigned>(first_blocks + attn::CTAS * cdiv(p.parts.rows, attn::JOIN_ROWS)));
    const bool wide = cache->head_dim == 256;
    launch(tiled ? (wide ? attn::paged_attention_join_kernel<256, 4> : attn::paged_attention_join_kernel<128, 4>)
                 : (wide ? attn::paged_attention_join_kernel<256, 8> : attn::paged_attention_join_kernel<128, 8>),
           join_grid, dim3(attn::JOIN_ROWS * 32), 0, s, p, parts[1], first_blocks);
    return launched();
}
