// nvfp4_attn.hip -- nvfp4_kv_attention: argument checks, the launch's shape, and
// the choice of kernel.
#include "nvfp4_attn.h"

namespace nvfp4 {

// How the keys are split: as many splits as bring the launch to about kTarget
// workgroups, none shorter than kLeast keys.
struct AttnPlan {
    int split_keys, splits;
};
static AttnPlan attn_plan(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads) {
    constexpr int64_t kTarget = 1024, kLeast = 256;
    const int group = q_heads / c->heads;
    const int64_t tiles = (tile_items<16>(b->tokens, group, 0) + b->seqs) * c->heads;
    const int64_t context = b->max_context < 1 ? 1 : b->max_context;
    int64_t splits = ceil_div(kTarget, tiles);
    int64_t keys = ceil_div(ceil_div(context, splits), 128) * 128;
    if (keys < kLeast) keys = kLeast;
    // the range's start is rounded down to a multiple of 64
    splits = ceil_div(context + 63, keys);
    if (splits > kMaxSplits) {
        splits = kMaxSplits;
        keys = ceil_div(ceil_div(context + 63, splits), 128) * 128;
    }
    return AttnPlan{int(keys), int(splits)};
}

static int attn_check(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads, KvView &v) {
    if (int st = kv_check(c, b, v)) return st;
    if (q_heads < 1 || q_heads % c->heads != 0) return NVFP4_ESHAPE;
    if (b->tokens > (int64_t(1) << 30) / q_heads) return NVFP4_ESHAPE;
    return NVFP4_OK;
}

static size_t attn_bytes(const AttnPlan &p, int64_t tokens, int q_heads, int dim) {
    return p.splits <= 1 ? 0 : size_t(p.splits) * size_t(tokens) * q_heads * (dim + 4) * sizeof(float);
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
    a.split_keys = plan.split_keys;
    a.splits = plan.splits;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + size_t(plan.splits) * batch->tokens * wide;
    if (int st = launch_attn_narrow(a, cache->head_dim, cache->k_format, cache->v_format, stream)) return st;
    if (plan.splits > 1) return launch_attn_join(a, cache->head_dim, 16, stream);
    return NVFP4_OK;
}
