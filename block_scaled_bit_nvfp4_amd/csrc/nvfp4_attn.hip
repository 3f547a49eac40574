// nvfp4_attn.hip -- nvfp4_kv_attention: argument checks, the launch's shape, and
// the choice of kernel.
#include <limits.h>

#include <algorithm>

#include "nvfp4_attn.h"

namespace nvfp4 {

// Sequences of at most so many rows (new tokens x group) go to the narrow kernel.
constexpr int kNarrowMost = 64;
constexpr int kCus = 256;

// Which kernels a call needs and how each cuts its work.
struct AttnPlan {
    AttnSplit split[2];
    int narrow_rows;
    bool narrow, wide;
    int splits() const { return std::max(split[0].splits, split[1].splits); }
};

// Splits of `keys` keys, a multiple of 128, over a context; its start is rounded
// down to a multiple of 64.
static AttnSplit cut_keys(int tile_rows, int64_t context, int64_t keys) {
    keys = ceil_div(std::max<int64_t>(keys, 128), 128) * 128;
    int64_t splits = ceil_div(context + 63, keys);
    if (splits > kMaxSplits) {
        keys = ceil_div(ceil_div(context + 63, kMaxSplits), 128) * 128;
        splits = ceil_div(context + 63, keys);
    }
    return AttnSplit{tile_rows, int(keys), int(splits)};
}

static AttnPlan attn_plan(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads) {
    const int group = q_heads / c->heads;
    const int64_t most = int64_t(std::max(b->max_new, 1)) * group;
    const int64_t context = std::max(b->max_context, 1);
    AttnPlan p;
    p.wide = most > kNarrowMost;
    p.narrow = !p.wide || b->tokens < int64_t(b->seqs) * b->max_new;     // all the same length otherwise
    p.narrow_rows = !p.wide ? INT_MAX : p.narrow ? kNarrowMost : -1;
    p.split[0] = p.split[1] = AttnSplit{kNarrowRows, 128, 1};
    if (p.narrow) {
        constexpr int64_t kTarget = 768, kLeast = 256;
        const int64_t tiles = tile_items(p.wide ? 0 : b->tokens, group, b->seqs, kNarrowRows) * c->heads;
        p.split[0] = cut_keys(kNarrowRows, context, std::max(ceil_div(context, ceil_div(kTarget, tiles)), kLeast));
    }
    if (p.wide) {
        // the number of splits that takes the fewest key tiles in all, a CU
        // taking one workgroup at a time, a split costing about 256 keys more
        const int rows = wide_rows(c->head_dim);
        const int64_t tiles = (ceil_div(b->tokens * group, rows) + (p.narrow ? 0 : b->seqs - 1)) * c->heads;
        int64_t best = 0, keys = context;
        for (int n = 1; n <= 16; ++n) {
            const int64_t each = ceil_div(context, n);
            if (n > 1 && each < 256) break;
            const int64_t cost = ceil_div(tiles * n, kCus) * (each + 256);
            if (n == 1 || cost < best) {
                best = cost;
                keys = each;
            }
        }
        p.split[1] = cut_keys(rows, context, keys + 63);
    }
    return p;
}

static int attn_check(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads, KvView &v) {
    if (int st = kv_check(c, b, v)) return st;
    if (q_heads < 1 || q_heads % c->heads != 0) return NVFP4_ESHAPE;
    if (b->tokens > (int64_t(1) << 30) / q_heads) return NVFP4_ESHAPE;
    return NVFP4_OK;
}

static size_t attn_bytes(const AttnPlan &p, int64_t tokens, int q_heads, int dim) {
    return p.splits() <= 1 ? 0 : size_t(p.splits()) * size_t(tokens) * q_heads * (dim + 4) * sizeof(float);
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API size_t nvfp4_kv_attention_workspace_bytes(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch,
                                                    int q_heads) {
    KvView v;
    if (attn_check(cache, batch, q_heads, v) != NVFP4_OK) return 0;
    return attn_bytes(attn_plan(cache, batch, q_heads), batch->tokens, q_heads, cache->head_dim);
}

NVFP4_API int nvfp4_kv_attention(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, const uint16_t *q,
                                 int64_t q_stride, int q_heads, float scale, int window, const uint64_t *tree,
                                 uint16_t *out, int64_t out_stride, float *lse, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    AttnArgs a;
    if (int st = attn_check(cache, batch, q_heads, a.kv)) return st;
    if (!q || !out || !tscale_ok(scale) || window < 0) return NVFP4_EINVAL;
    if (tree && (window > 0 || batch->max_new > 64)) return NVFP4_EINVAL;
    const int64_t wide = int64_t(q_heads) * cache->head_dim;
    if (q_stride < wide || out_stride < wide || q_stride > (int64_t(1) << 40) || out_stride > (int64_t(1) << 40))
        return NVFP4_ESHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8 || (lse && !aligned(lse, 4)) ||
        (tree && !aligned(tree, 8)))
        return NVFP4_EALIGN;
    if (batch->tokens == 0) return NVFP4_OK;
    const AttnPlan plan = attn_plan(cache, batch, q_heads);
    const size_t need = attn_bytes(plan, batch->tokens, q_heads, cache->head_dim);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return NVFP4_EWORKSPACE;
        if (!aligned(workspace, 16)) return NVFP4_EALIGN;
    }
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.tree = reinterpret_cast<const unsigned long long *>(tree);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.q_heads = q_heads;
    a.group = q_heads / cache->heads;
    a.window = window;
    a.scale_log2 = scale * kLog2e;
    a.split[0] = plan.split[0];
    a.split[1] = plan.split[1];
    a.narrow_rows = plan.narrow_rows;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + size_t(plan.splits()) * batch->tokens * wide;
    const int dim = cache->head_dim;
    if (plan.narrow)
        if (int st = launch_attn_narrow(a, dim, cache->k_format, cache->v_format, stream)) return st;
    if (plan.wide)
        if (int st = launch_attn_wide(a, dim, cache->k_format, cache->v_format, stream)) return st;
    return plan.splits() > 1 ? launch_attn_join(a, dim, stream) : NVFP4_OK;
}
