"""The attention's plan, which is host code: compiled by itself, with stand-ins for the
launches, and asked over small and extreme batches for what the kernels rely on."""
import itertools
import os
import subprocess

import pytest

from block_scaled_bit_nvfp4_amd import build as B

# Reads "dim heads group tokens seqs table_width max_new max_context window" lines; answers
# with the status, the workspace, and for each kernel tiles, rows, keys, splits and first
# part row, then the part rows.
MAIN = r"""
#include "nvfp4_attn.hip"
#include <stdio.h>
namespace nvfp4 {
int kv_check(const nvfp4_kv_cache *, const nvfp4_kv_batch *, KvView &) { return NVFP4_OK; }
int wide_rows(int dim) { return dim == 256 ? 128 : 256; }
int launch_attn_narrow(const AttnArgs &, int64_t, int, int, int, hipStream_t) { return NVFP4_OK; }
int launch_attn_wide(const AttnArgs &, int64_t, int, int, int, hipStream_t) { return NVFP4_OK; }
int launch_attn_join(const AttnArgs &, bool, int, hipStream_t) { return NVFP4_OK; }
}
int main() {
    long dim, heads, group, tokens, seqs, width, max_new, context, window;
    while (scanf("%ld %ld %ld %ld %ld %ld %ld %ld %ld", &dim, &heads, &group, &tokens, &seqs, &width, &max_new, &context,
                 &window) == 9) {
        nvfp4_kv_cache c = {};
        c.pages = 1 << 20; c.page_tokens = 64; c.heads = int(heads); c.head_dim = int(dim);
        nvfp4_kv_batch b = {};
        b.tokens = tokens; b.seqs = int(seqs); b.table_width = int(width);
        b.max_new = int(max_new); b.max_context = int(context);
        const int q = int(heads * group);
        const AttnPlan p = attn_plan(&c, &b, q, int(window), INT_MAX);
        printf("%zu %zu", plan_bytes(p, &b, q, int(dim)), nvfp4_kv_attention_workspace_bytes(&c, &b, q));
        for (int k = 0; k < 2; ++k)
            printf(" %ld %d %d %d %d", long(p.tiles[k]), p.cut[k].rows, p.cut[k].keys, p.cut[k].splits, p.cut[k].first_row);
        printf(" %ld\n", long(p.part_rows));
    }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.hip").write_text(MAIN)
    flags = [f for f in B.CFLAGS if f.startswith(("-std", "-I", "-Wno"))]
    subprocess.run([B.HIPCC, "--offload-arch=" + B.ARCH, "--offload-host-only", "-O1", "-w", *flags, str(at / "plan.hip"),
                    "-o", str(at / "plan")], check=True, capture_output=True, text=True)

    def ask(cases):
        lines = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([str(at / "plan")], input=lines, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return ask


BOUNDS = [0, 1, 127, 5000, 131072, 1 << 30, (1 << 31) - 1]


def test_a_plan_is_one_that_the_kernels_can_follow(plans):
    """Splits of whole 128 keys, no more of them than the join takes, parts in 32 bits that
    do not overlap, and a workspace that one asked for without a window covers."""
    cases = [(dim, heads, group, tokens, seqs, 1 << 14, new, context, window)
             for dim, (heads, group), (tokens, seqs, new), context, window in itertools.product(
                 (64, 128, 256), ((1, 1), (8, 5), (1, 128), (64, 1)),
                 ((1, 1, 1), (8, 1, 8), (512, 1, 512), (2048, 1, 2048), (64, 64, 1), (3000, 4096, 1), (1500, 7, 301),
                  (1 << 16, 1 << 16, 1), (1 << 20, 3, (1 << 31) - 1), (5, 1, 0), (1 << 16, 600, 1 << 14)),
                 BOUNDS, (0, 1, 1024, (1 << 31) - 1))]
    answers = plans(cases)
    assert len(answers) == len(cases)
    for case, (need, without, *rest) in zip(cases, answers):
        dim, heads, group, tokens, _, _, _, context, window = case
        cuts, part_rows = [rest[:5], rest[5:10]], rest[10]
        end = 0
        for tiles, rows, keys, splits, first in cuts:
            if tiles == 0:
                continue
            assert keys > 0 and keys % 128 == 0 and 1 <= splits <= 256, (case, rest)
            span = min(max(context, 1), 1 << 30, window + rows // group + 1 if window else 1 << 30)
            assert keys * splits >= span or splits == 1, (case, rest)
            if splits > 1:
                assert first == end, (case, rest)
                end += tiles * heads * splits * rows
        assert end == part_rows < 1 << 31, (case, rest)
        assert need <= without, (case, rest)


def test_bounds_past_every_position_plan_as_the_last_position(plans):
    """No table names more than 2^30 positions."""
    shapes = [(128, 8, 5, 1, 1), (64, 8, 1, 4096, 4096), (256, 1, 16, 2000, 1), (128, 8, 4, 1500, 7)]
    last, past = (plans([(*s[:4], s[4], 1 << 14, s[3] // s[4], bound, 0) for s in shapes])
                  for bound in (1 << 30, (1 << 31) - 1))
    assert last == past
