"""What the cache operators launch: a C program links the library, stands in for the runtime's launch calls, and lets
chosen ones fail.  Nothing reaches a GPU; no pointer is followed."""

import os
import shutil
import subprocess

import pytest

import mixed_precision_paged_argus_gb300.argus as argus

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKES = r"""
#include <stdio.h>
#include <string.h>
#include "argus.h"
/* the runtime's calls that the library makes on its way to a launch; launches are numbered from 0 */
static int fail_at = -1, launches = 0, last = 0;
static int launch(void) {
  if (launches++ != fail_at) return 0;
  return last = 701;                       /* too many resources requested: the kernel does not run */
}
int __cudaGetKernel(void** k, const void* f) { *k = (void*)f; return 0; }
int __cudaLaunchKernel(void* k, ...) { (void)k; return launch(); }
int cudaLaunchKernelExC(const void* c, const void* f, void** a) { (void)c; (void)f; (void)a; return launch(); }
int cudaLaunchCooperativeKernel(const void* f, ...) { (void)f; return launch(); }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
const char* cudaGetErrorString(int e) { (void)e; return "refused"; }
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int a, int d) { (void)a; (void)d; *v = 152; return 0; }
int cudaFuncSetAttribute(const void* f, int a, int v) { (void)f; (void)a; (void)v; return 0; }
int cudaGetDriverEntryPointByVersion(const char* s, void** f, unsigned v, unsigned long long g, int* q) {
  (void)s; (void)v; (void)g; *f = 0; if (q) *q = 1; return 1;
}
static int extend(void) {
  argus_pool pool = {ARGUS_FP8_E4M3, 0, (void*)64, (void*)64, 400};
  argus_extend_args a;
  memset(&a, 0, sizeof a);
  a.g = (argus_geom){8, 2, 128, 16};
  a.batch = 2; a.total_q = 5; a.q_dtype = ARGUS_BF16; a.causal = 1;
  a.q = (void*)64; a.q_start = (void*)64; a.pools = &pool; a.n_pools = 1; a.max_pages = 100;
  a.page_codec = (void*)64; a.block_table = (void*)64; a.seq_lens = (void*)64; a.out = (void*)(1 << 20);
  a.softmax_scale = 0.5f;
  return argus_paged_extend_attn(&a, (void*)64, (size_t)1 << 40, 0);
}
static argus_rope_args rope_args(void) {
  static argus_pool pool = {ARGUS_FP16, 0, (void*)64, 0, 400};
  argus_rope_args a;
  memset(&a, 0, sizeof a);
  a.g = (argus_geom){8, 2, 128, 16};
  a.batch = 2; a.total_q = 5; a.dtype = ARGUS_FP16; a.rot_dim = 64; a.n_axes = 1;
  a.q = (void*)(1 << 16); a.k = (void*)(2 << 16); a.v = (void*)(3 << 16); a.q_out = (void*)(4 << 16);
  a.positions = (void*)64; a.inv_freq = (void*)64; a.q_start = (void*)64; a.seq_lens = (void*)64; a.pool = &pool;
  a.page_codec = (void*)64; a.block_table = (void*)64; a.max_pages = 4;
  return a;
}
static int rope(void) {
  const argus_rope_args a = rope_args();
  return argus_rope_append(&a, 0);
}
static int compact(void) {
  argus_pool pool = {ARGUS_FP16, 0, (void*)64, 0, 40};
  argus_geom g = {2, 2, 64, 16};
  return argus_compact_pages(&g, 3, &pool, (void*)64, (void*)(1 << 12), (void*)64, (void*)64, (void*)64, (void*)(2 << 12), 4,
                             (void*)(3 << 12), (void*)(4 << 12), (size_t)1 << 40, 0, 0);
}
"""

REFUSED = r"""
int main(void) {
  int (*calls[])(void) = {extend, rope, compact};
  for (int c = 0; c < 3; ++c)
    for (int at = -1; at < 2; ++at) {
      fail_at = at; launches = 0; last = 0;
      const int st = calls[c]();
      /* the call's status, its launches, and whether an error is left for the next call to trip over */
      printf("%d %d %d\n", st, launches, last != 0);
    }
  return 0;
}
"""


def run_with_fakes(main, tmp_path):
    """The numbers that the program prints, line by line."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    from mixed_precision_paged_argus_gb300 import build
    lib = build.build()
    assert os.path.samefile(lib, argus.lib_path())
    src, exe = tmp_path / "launches.c", tmp_path / "launches"
    src.write_text(FAKES + main)
    subprocess.run([cc, "-std=c11", "-rdynamic", "-I", os.path.join(ROOT, "include"), str(src), lib, "-o", str(exe),
                    "-Wl,-rpath," + os.path.dirname(lib), "-Wl,--allow-shlib-undefined"], check=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "lib64")
    env = dict(os.environ, LD_LIBRARY_PATH=cuda + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, env=env).stdout.split("\n")
    return [tuple(int(x) for x in line.split()) for line in out if line]


def test_a_refused_launch_ends_the_call_and_leaves_no_error(tmp_path):
    """The join of ragged attention reads what its first kernel describes: without that kernel it must not be launched."""
    got = run_with_fakes(REFUSED, tmp_path)
    ok, failed = 0, 4
    extend = [(ok, 2, 0), (failed, 1, 0), (failed, 2, 0)]      # none, the first kernel, the join refused
    single = [(ok, 1, 0), (failed, 1, 0), (ok, 1, 0)]
    assert got == extend + single + single


ROPE_PLACES = r"""
/* address and token stride, in elements of two bytes, of q, k, v and q_out; tokens */
static const long long cases[][9] = {CASES};
int main(void) {
  for (unsigned i = 0; i < sizeof cases / sizeof cases[0]; ++i) {
    const long long* c = cases[i];
    argus_rope_args a = rope_args();
    a.q = (void*)(2 * c[0]); a.k = (void*)(2 * c[2]); a.v = (void*)(2 * c[4]); a.q_out = (void*)(2 * c[6]);
    a.q_stride = c[1]; a.k_stride = c[3]; a.v_stride = c[5]; a.q_out_stride = c[7]; a.total_q = (int)c[8];
    launches = 0;
    const int st = argus_rope_append(&a, 0);
    printf("%d %d\n", st, launches);
  }
  return 0;
}
"""


def test_rotated_queries_do_not_overlap_what_is_read(tmp_path):
    """q_out is q itself or meets none of the tokens of q, k and v, whose bytes are marked one by one here."""
    import numpy as np
    rng = np.random.default_rng(1)
    q_len, kv_len, base = 8 * 128, 2 * 128, 1 << 15
    cases = [  # a fused projection's rows: in place, beside, over k, over v's last elements
        (base, 1536, base + 1024, 1536, base + 1280, 1536, base, 1536, 5),
        (base, 2560, base + 1024, 2560, base + 1280, 2560, base + 1536, 2560, 5),
        (base, 2560, base + 1024, 2560, base + 1280, 2560, base + 1528, 2560, 5),
        (base, 2560, base + 1024, 2560, base + 1280, 2560, base + 1024, 2560, 5),
        (base, 2560, base + 1024, 2560, base + 1280, 2560, base + 1536 - 3 * 2560, 2560, 5),
        (base, 2560, base + 1024, 2560, base + 1280, 2560, base + 1528 - 4 * 2560, 2560, 5),
        (base, 0, 3 * base, 0, 4 * base, 0, base + 5 * 1024, 0, 5), (base, 0, 3 * base, 0, 4 * base, 0, base + 5 * 1024 - 8, 0, 5),
        # another stride: between q's tokens, and not
        (base, 4096, 3 * base, 0, 4 * base, 0, base + 1024, 8192, 5), (base, 4096, 3 * base, 0, 4 * base, 0, base + 1024, 2048, 5),
        (base, 4096, 3 * base, 0, 4 * base, 0, base + 1024, 1024, 3), (base, 4096, 3 * base, 0, 4 * base, 0, base + 1024, 1024, 4),
        # far larger strides than anything there
        (base, 1 << 40, 3 * base, 0, 4 * base, 0, base, 1 << 41, 5), (base, 1 << 40, 3 * base, 0, 4 * base, 0, base + 1024, 1 << 41, 5)]
    for _ in range(400):
        where = lambda: int(base + 8 * rng.integers(0, 1 << 10))  # noqa: E731
        strides = [int(8 * rng.integers(n // 8, 3 * n // 8 + 2)) for n in (q_len, kv_len, kv_len, q_len)]
        if rng.random() < 0.6:                          # one buffer's rows
            strides = [int(8 * rng.integers(q_len // 8, 512))] * 4
        at = [where() for _ in range(4)]
        if rng.random() < 0.2:
            at[3], strides[3] = at[0], strides[0]
        cases.append((at[0], strides[0], at[1], strides[1], at[2], strides[2], at[3], strides[3], int(rng.integers(1, 7))))

    def meets(c):
        def mark(at, stride, n):
            return {at + t * (stride or n) + 8 * e for t in range(c[8]) for e in range(n // 8)}
        out = mark(c[6], c[7], q_len)
        same = c[0] == c[6] and (c[1] or q_len) == (c[7] or q_len)
        return bool(out & mark(c[2], c[3], kv_len) or out & mark(c[4], c[5], kv_len) or (not same and out & mark(c[0], c[1], q_len)))

    rows = ", ".join("{%s}" % ", ".join("%dLL" % x for x in c) for c in cases)
    got = run_with_fakes(ROPE_PLACES.replace("CASES", rows), tmp_path)
    want = [(1, 0) if meets(c) else (0, 1) for c in cases]
    assert 100 < sum(w[0] for w in want) < 380
    assert [c for c, g, w in zip(cases, got, want) if g != w] == []


EMPTY_TABLES = r"""
int main(void) {
  argus_rope_args a = rope_args();
  a.page_codec = 0; a.block_table = 0;
  printf("%d\n", argus_rope_append(&a, 0));
  a.max_pages = 0;
  printf("%d\n", argus_rope_append(&a, 0));
  return 0;
}
"""


def test_a_table_without_pages_needs_no_memory(tmp_path):
    """An empty table has no address: its tokens have no place, which *status counts, and q_out is written all the same."""
    assert run_with_fakes(EMPTY_TABLES, tmp_path) == [(1,), (0,)]


TABLES = r"""
/* addresses of fork: parents, n_new, counts in / out of two pools, codecs, table, lengths in and out, workspace */
static const long long cases[][14] = {CASES};
int main(void) {
  for (unsigned i = 0; i < sizeof cases / sizeof cases[0]; ++i) {
    void* c[14];
    for (int k = 0; k < 14; ++k) c[k] = (void*)cases[i][k];
    argus_geom g = {2, 2, 64, 16};
    argus_pool pools[2] = {{ARGUS_FP16, 0, (void*)64, 0, 40}, {ARGUS_INT8, 0, (void*)64, (void*)64, 50}};
    const int32_t* in[2] = {c[2], c[3]};
    int32_t* out[2] = {c[4], c[5]};
    launches = 0;
    int st = argus_fork_pages(&g, 6, c[0], c[1], ARGUS_FP16, pools, 2, in, out, c[6], c[7], c[8], c[9], c[10], c[11], 4, c[12], 4096, 0, 0);
    printf("%d %d ", st, launches);
    /* compaction of the first pool: counts, codecs, table, lengths, the new table, n_live at parents, workspace */
    launches = 0;
    st = argus_compact_pages(&g, 6, &pools[0], c[2], c[4], c[6], c[7], c[8], c[10], 4, c[0], c[12], 4096, 0, 0);
    printf("%d %d\n", st, launches);
  }
  return 0;
}
"""


def test_new_tables_do_not_overlap_the_old(tmp_path):
    """Six rows of four pages, pools of 40 and 50 slots: every pair of arrays, apart, touching and overlapping."""
    names = ["parents", "n_new", "in0", "in1", "out0", "out1", "codec", "table", "lens", "codec_out", "table_out", "lens_out", "ws"]
    size = dict(zip(names, [24, 24, 160, 200, 160, 200, 24, 96, 24, 24, 96, 24, 4096]))
    base = {n: (1 << 20) + (i << 14) for i, n in enumerate(names)}
    cases, want = [], []

    def add(place):
        def bad(out, ins, sizes):
            spans = {n: (place[n], place[n] + sizes[n]) for n in out + ins if place[n]}
            return any(spans[a][0] < spans[b][1] and spans[b][0] < spans[a][1] for a in out if a in spans for b in spans if b != a)
        cases.append([place[n] for n in names] + [0])
        f = bad(["out0", "out1", "codec_out", "table_out", "lens_out", "ws"], ["parents", "n_new", "in0", "in1", "codec", "table", "lens"],
                dict(size, ws=FORK_WS))
        c = bad(["out0", "table_out", "parents", "ws"], ["in0", "codec", "table", "lens"], dict(size, ws=COMPACT_WS, parents=4))
        want.append(((1, 0) if f else (0, 1)) + ((1, 0) if c else (0, 1)))

    # the workspaces' sizes, as the library states them
    sizes = run_with_fakes(r"""
int main(void) {
  argus_pool pools[2] = {{ARGUS_FP16, 0, (void*)64, 0, 40}, {ARGUS_INT8, 0, (void*)64, (void*)64, 50}};
  size_t a, b;
  argus_fork_workspace_bytes(6, pools, 2, &a);
  argus_compact_workspace_bytes(&pools[0], &b);
  printf("%zu %zu\n", a, b);
  return 0;
}
""", tmp_path)
    FORK_WS, COMPACT_WS = sizes[0]
    add(base)
    add(dict(base, n_new=0))
    for a in names:
        for b in names:
            if a != b and not (a == "parents" and b == "ws"):
                for shift in (0, 4 * (size[b] // 4) - 4, size[b], -4, -size[a]):
                    if a != "ws" or shift % 16 == 0:
                        add(dict(base, **{a: base[b] + shift}))
    rows = ", ".join("{%s}" % ", ".join("%dLL" % x for x in c) for c in cases)
    got = run_with_fakes(TABLES.replace("CASES", rows), tmp_path)
    assert [(c, g, w) for c, g, w in zip(cases, got, want) if g != w] == []
    assert sum(w[0] for w in want) > 100 and sum(w[0] == 0 for w in want) > 100


NOTHING = r"""
int main(void) {
  argus_geom g = {2, 2, 64, 16};
  argus_pool pools[2] = {{ARGUS_FP16, 0, (void*)64, 0, 40}, {ARGUS_INT8, 0, (void*)64, (void*)64, 0}};
  /* the empty pool's counts lie at an address inside the other's, and those of compaction inside the table */
  const int32_t* in[2] = {(void*)(1 << 12), (void*)((1 << 12) + 8)};
  int32_t* out[2] = {(void*)(2 << 12), (void*)((2 << 12) + 8)};
  printf("%d\n", argus_fork_pages(&g, 6, (void*)(3 << 12), 0, ARGUS_FP16, pools, 2, in, out, (void*)(4 << 12), (void*)(5 << 12), (void*)(6 << 12),
                                  (void*)(7 << 12), (void*)(8 << 12), (void*)(9 << 12), 4, (void*)(10 << 12), 4096, 0, 0));
  printf("%d\n", argus_compact_pages(&g, 6, &pools[1], (void*)((5 << 12) + 8), (void*)((5 << 12) + 8), (void*)(4 << 12), (void*)(5 << 12),
                                     (void*)(6 << 12), (void*)(8 << 12), 4, (void*)(3 << 12), (void*)(10 << 12), 4096, 0, 0));
  return 0;
}
"""


def test_arrays_without_elements_overlap_nothing(tmp_path):
    assert run_with_fakes(NOTHING, tmp_path) == [(0,), (0,)]


STALE = r"""
int main(void) {
  int (*calls[])(void) = {extend, rope, compact};
  for (int c = 0; c < 3; ++c) {
    last = 701;                              /* somebody else's launch failed before this call */
    printf("%d\n", calls[c]());
  }
  return 0;
}
"""


def test_an_error_from_before_is_not_the_calls(tmp_path):
    assert run_with_fakes(STALE, tmp_path) == [(0,), (0,), (0,)]
