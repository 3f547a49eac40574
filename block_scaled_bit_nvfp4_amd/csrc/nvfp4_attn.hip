// nvfp4_attn.hip -- nvfp4_kv_attention: argument checks, the launch's shape, and
// the choice of kernel.
#include <limits.h>

#include <algorithm>

#include "nvfp4_attn.h"

namespace nvfp4 {

// Sequences of at most so many rows (new tokens x group) go to the narrow kernel,
// whatever the others need.
constexpr int kNarrowMost = 64;
constexpr int kCus = 256;

// Which kernels a call needs and how each cuts its work.
struct AttnPlan {
    AttnCut cut[2];
    int64_t tiles[2];      // tile indexes; 0: the kernel is not needed
    int64_t part_rows;     // of the workspace; 0: no tile is split
    bool many;             // how the splits are joined
    int narrow_rows;
};

// Splits of about `keys` keys of tiles that span `span` (the range's start is rounded
// down to a multiple of 64 where a window moves it).
static void cut_keys(AttnCut &c, int64_t span, int64_t keys, bool window, int most_splits) {
    if (window) span += 63;
    keys = ceil_div(std::max(keys, ceil_div(span, most_splits)), 128) * 128;
    c.keys = int(keys);
    c.splits = int(ceil_div(span, keys));
}

// us that the parts of n splits take on their way out and back (at 4 TB/s), and
// the join's launch.
static double parts_us(const nvfp4_kv_batch *b, int q_heads, int dim, int64_t n) {
    return n == 1 ? 0 : 4 + double(b->tokens) * q_heads * dim * 4 * 2 * n / 4e6;
}

// The narrow kernel's cut for `tiles` tile indexes; returns the us that it should take.
static double cut_narrow(AttnCut &c, const nvfp4_kv_batch *b, int q_heads, int heads, int dim, int64_t tiles, int64_t keys,
                         bool window, int most_splits) {
    // Workgroups to aim at: two for each CU where one sequence is split (more
    // cost the join more than they gain: 131008 keys 51 us, with twice as many 56),
    // up to twelve where several sequences of unknown lengths balance each
    // other (64 ragged sequences: 85.5 us at six for each CU, 84.3 at twelve).
    const int64_t items = tiles * heads, target = 2 * kCus * std::min(b->seqs, 6);
    // No split of fewer keys than a workgroup's start and the join are worth, which
    // grows with the items that fill the card by themselves (one sequence of 1037
    // keys: 9.6 us in splits of 128, 10.3 of 256, 11.9 whole; 900 keys: 8 sequences 12.0
    // in splits of 512, 12.6 of 256; 64 sequences 33.5 of 256, 26.8 whole; past 4096
    // keys splits of 128 would be too many: 8001 keys 13.6, of 256 11.8); up to 512
    // keys (8.4 us whole, 9.4 split) nothing is split.
    int64_t least = items >= 256 ? 1024 : items >= 64 ? 512 : keys <= 4096 ? 128 : 256;
    if (keys <= 512) least = std::max(least, keys + 63);
    cut_keys(c, keys, std::max(ceil_div(keys, ceil_div(target, items)), least), window, most_splits);
    // Launch 6 us; then whichever is longer: all SIMDs' tiles of 16 rows and 32 keys
    // with the workgroups' starts, or one workgroup's walk (measured at 64, 128, 256).
    const double per_tile = 0.15 + 0.0035 * dim, per_step = 0.6 + 0.005 * dim;
    const int64_t groups = items * c.splits, at_once = kCus * (dim == 256 ? 2 : dim == 128 ? 3 : 4);
    const double all = 4.0 * double(groups) / double(at_once) + per_tile * double(items) * double(keys) / 32 / (4 * kCus);
    const double one = 4 + per_step * double(std::min<int64_t>(c.keys, keys)) / 128;
    return 6 + std::max(all, one) + parts_us(b, q_heads, dim, c.splits);
}

// The wide kernel's cut, the same way: the number of splits that should take the
// least time, a CU taking one workgroup at a time.
static double cut_wide(AttnCut &c, const nvfp4_kv_batch *b, int q_heads, int dim, int64_t tiles, int64_t keys, bool window,
                       int most_splits) {
    const double per_tile = dim == 64 ? 2.5 : dim == 128 ? 1.75 : 1.25;       // us of 8192 / dim keys
    double best = 0;
    int64_t each = keys;
    for (int n = 1; n <= kMaxSplits / 2; n += std::max(1, n / 4)) {
        const int64_t of = ceil_div(ceil_div(keys, n), 128) * 128;
        if (n > 1 && of < 32768 / dim) break;
        const double cost = double(ceil_div(tiles * n, kCus)) * (double(of) * dim / 8192 * per_tile + 5) + parts_us(b, q_heads, dim, n);
        if (n == 1 || cost < best) {
            best = cost;
            each = of;
        }
    }
    cut_keys(c, keys, each, window, most_splits);
    return 5 + best;
}

static AttnPlan attn_plan(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads, int window, int64_t most_parts) {
    const int group = q_heads / c->heads, dim = c->head_dim;
    // A caller asks for the workspace without saying the window: with one, no more
    // splits, and no more parts, than without.
    int most_splits[2] = {kMaxSplits, kMaxSplits};
    if (window > 0) {
        const AttnPlan without = attn_plan(c, b, q_heads, 0, INT_MAX);
        for (int cls = 0; cls < 2; ++cls)
            if (without.tiles[cls] > 0) most_splits[cls] = without.cut[cls].splits;
        most_parts = without.part_rows;
    }
    const int64_t most = int64_t(std::max(b->max_new, 1)) * group;
    AttnPlan p = {};
    // a tile sees its window and its own tokens; a bound past every position would
    // pass 32 bits once rounded to whole splits
    const auto span = [&](int rows) {
        const int64_t context = std::min(std::max(b->max_context, 1), kKvMaxPositions);
        return window > 0 ? std::min<int64_t>(context, int64_t(window) + rows / group + 1) : context;
    };
    const bool even = b->tokens == int64_t(b->seqs) * b->max_new;         // all of the same length
    p.cut[0] = AttnCut{kNarrowRows, 128, 1, 0, 0};
    p.cut[1] = AttnCut{wide_rows(dim), 128, 1, 0, 0};
    // All by the narrow kernel, or the long sequences by the wide one.
    const int64_t all_narrow = b->tokens * group / kNarrowRows + b->seqs;
    const double narrow_us = cut_narrow(p.cut[0], b, q_heads, c->heads, dim, all_narrow, span(kNarrowRows), window > 0, most_splits[0]);
    bool wide = most > kNarrowMost;
    if (wide) {
        // tiles of the sequences, each with a last one that is half full on average
        const int rows = p.cut[1].rows;
        const int64_t tiles = c->heads * (even ? b->seqs * ceil_div(most, rows) : ceil_div(b->tokens * group, rows) + b->seqs / 2);
        wide = cut_wide(p.cut[1], b, q_heads, dim, tiles, span(rows), window > 0, most_splits[1]) < narrow_us;
    }
    p.narrow_rows = !wide ? INT_MAX : even ? -1 : kNarrowMost;
    if (!wide) {
        p.tiles[0] = all_narrow;
        p.cut[1].splits = 1;
    } else {
        p.tiles[1] = b->tokens * group / p.cut[1].rows + b->seqs;
        p.cut[0].splits = 1;
        if (!even) {
            p.cut[0].tiles_per_seq = kNarrowMost / kNarrowRows;
            p.tiles[0] = int64_t(b->seqs) * p.cut[0].tiles_per_seq;
            cut_narrow(p.cut[0], b, q_heads, c->heads, dim, p.tiles[0], span(kNarrowRows), window > 0, most_splits[0]);
        }
    }
    int64_t rows = 0;
    for (int cls = 0; cls < 2; ++cls) {
        AttnCut &k = p.cut[cls];
        k.first_row = int(rows);
        if (p.tiles[cls] == 0 || k.splits == 1) continue;
        const int64_t more = p.tiles[cls] * c->heads * k.splits * k.rows;
        if (rows + more > most_parts) {        // part rows are 32-bit: whole tiles then
            k.splits = 1;
            continue;
        }
        rows += more;
    }
    p.part_rows = rows;
    // a workgroup for a row from seven splits on (12 splits: 10.3 us, a thread for four
    // elements 12.7; 5 splits: the same); among many rows few are in many splits
    p.many = !wide && p.cut[0].splits > 6;
    return p;
}

// Bytes of the workspace: the rows' facts, and the parts.
static size_t info_bytes(const nvfp4_kv_batch *b, int q_heads) {
    return size_t(b->tokens) * q_heads * sizeof(RowInfo);
}
static size_t plan_bytes(const AttnPlan &p, const nvfp4_kv_batch *b, int q_heads, int dim) {
    return p.part_rows == 0 ? 0 : info_bytes(b, q_heads) + size_t(p.part_rows) * (dim + 4) * sizeof(float);
}

static int attn_check(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, int q_heads, KvView &v) {
    if (int st = kv_check(c, b, v)) return st;
    if (q_heads < 1 || q_heads % c->heads != 0) return NVFP4_ESHAPE;
    if (b->tokens > (int64_t(1) << 30) / q_heads) return NVFP4_ESHAPE;
    return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API size_t nvfp4_kv_attention_workspace_bytes(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch,
                                                    int q_heads) {
    KvView v;
    if (attn_check(cache, batch, q_heads, v) != NVFP4_OK) return 0;
    return plan_bytes(attn_plan(cache, batch, q_heads, 0, INT_MAX), batch, q_heads, cache->head_dim);
}

NVFP4_API int nvfp4_kv_attention(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, const uint16_t *q,
                                 int64_t q_stride, int q_heads, float scale, int window, const uint64_t *tree,
                                 uint16_t *out, int64_t out_stride, float *lse, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    AttnArgs a;
    if (int st = attn_check(cache, batch, q_heads, a.kv)) return st;
    if ((batch->tokens > 0 && (!q || !out)) || !tscale_ok(scale) || window < 0) return NVFP4_EINVAL;
    if (tree && (window > 0 || batch->max_new > 64)) return NVFP4_EINVAL;
    const int64_t wide = int64_t(q_heads) * cache->head_dim;
    if (q_stride < wide || out_stride < wide || q_stride > (int64_t(1) << 40) || out_stride > (int64_t(1) << 40))
        return NVFP4_ESHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8 || (lse && !aligned(lse, 4)) ||
        (tree && !aligned(tree, 8)))
        return NVFP4_EALIGN;
    if (batch->tokens == 0) return NVFP4_OK;
    const AttnPlan plan = attn_plan(cache, batch, q_heads, window, INT_MAX);
    const size_t need = plan_bytes(plan, batch, q_heads, cache->head_dim);
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
    a.narrow_rows = plan.narrow_rows;
    a.reused = batch->max_new > kNarrowRows / a.group;
    a.cut[0] = plan.cut[0];
    a.cut[1] = plan.cut[1];
    const int dim = cache->head_dim;
    const bool cut = plan.part_rows > 0;
    a.part_rows = int(plan.part_rows);
    a.info = cut ? static_cast<RowInfo *>(workspace) : nullptr;
    a.part_o = cut ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + info_bytes(batch, q_heads)) : nullptr;
    a.part_ml = cut ? a.part_o + size_t(plan.part_rows) * dim : nullptr;
    if (plan.tiles[0] > 0)
        if (int st = launch_attn_narrow(a, plan.tiles[0], dim, cache->k_format, cache->v_format, stream)) return st;
    if (plan.tiles[1] > 0)
        if (int st = launch_attn_wide(a, plan.tiles[1], dim, cache->k_format, cache->v_format, stream)) return st;
    return cut ? launch_attn_join(a, plan.many, dim, stream) : NVFP4_OK;
}
