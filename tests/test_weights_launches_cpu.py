"""How many kernels argus_attn_weights launches (test_launches_cpu.py has the stand-ins for the runtime's launch calls)."""

from test_launches_cpu import run_with_fakes

LAUNCHES = r"""
/* per line: sequences, query tokens, the pool's codec */
static const int cases[][3] = {CASES};
int main(void) {
  for (unsigned i = 0; i < sizeof cases / sizeof cases[0]; ++i) {
    argus_pool pool = {cases[i][2], 0, (void*)64, (void*)64, 400};
    argus_extend_args a;
    memset(&a, 0, sizeof a);
    a.g = (argus_geom){8, 2, 128, 16};
    a.batch = cases[i][0]; a.total_q = cases[i][1]; a.q_dtype = ARGUS_BF16; a.causal = 1;
    a.q = (void*)64; a.q_start = (void*)64; a.pools = &pool; a.n_pools = 1; a.max_pages = 100;
    a.page_codec = (void*)64; a.block_table = (void*)64; a.seq_lens = (void*)64; a.lse2_out = (void*)(2 << 20);
    a.softmax_scale = 0.5f;
    launches = 0;
    const int st = argus_attn_weights(&a, (void*)(16 << 20), 1600, 1.f, 0);
    printf("%d %d\n", st, launches);
  }
  (void)extend; (void)rope; (void)compact;
  return 0;
}
"""

BF16, FP8, INT8, INT4 = 1, 2, 3, 4


def test_one_sequence_may_have_all_the_rows(tmp_path):
    """Fewer tokens than sequences says nothing about how many one sequence has: with more than 16 rows per KV head in
    the call (4 heads each), or 8 over group codes, one may have them all, and a kernel of their own takes the sequences
    of so many.  As many tokens as sequences is a decode step."""
    want = [((64, 32, FP8), 2), ((64, 32, BF16), 2), ((64, 63, INT8), 2), ((64, 65, FP8), 2), ((64, 5, FP8), 2), ((64, 4, FP8), 1), ((64, 0, FP8), 1),
            ((64, 64, FP8), 1), ((1, 1, FP8), 1), ((1, 32, BF16), 2), ((64, 32, INT4), 2), ((64, 2, INT4), 1), ((64, 64, INT4), 1), ((1, 32, INT4), 1)]
    rows = ", ".join("{%d, %d, %d}" % c for c, _ in want)
    assert run_with_fakes(LAUNCHES.replace("CASES", rows), tmp_path) == [(0, n) for _, n in want]
