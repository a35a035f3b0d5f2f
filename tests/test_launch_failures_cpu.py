"""What the cache operators do when the CUDA runtime refuses a launch: a C program links the library, stands in for
the runtime's launch calls, and lets chosen ones fail.  Nothing reaches a GPU; no pointer is followed."""

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
static int rope(void) {
  argus_pool pool = {ARGUS_FP16, 0, (void*)64, 0, 400};
  argus_rope_args a;
  memset(&a, 0, sizeof a);
  a.g = (argus_geom){8, 2, 128, 16};
  a.batch = 2; a.total_q = 5; a.dtype = ARGUS_FP16; a.rot_dim = 64; a.n_axes = 1;
  a.q = (void*)(1 << 16); a.k = (void*)(2 << 16); a.v = (void*)(3 << 16); a.q_out = (void*)(4 << 16);
  a.positions = (void*)64; a.inv_freq = (void*)64; a.q_start = (void*)64; a.seq_lens = (void*)64; a.pool = &pool;
  a.page_codec = (void*)64; a.block_table = (void*)64; a.max_pages = 4;
  return argus_rope_append(&a, 0);
}
static int compact(void) {
  argus_pool pool = {ARGUS_FP16, 0, (void*)64, 0, 40};
  argus_geom g = {2, 2, 64, 16};
  return argus_compact_pages(&g, 3, &pool, (void*)64, (void*)(1 << 12), (void*)64, (void*)64, (void*)64, (void*)(1 << 13), 4, (void*)64,
                             (void*)64, (size_t)1 << 40, 0, 0);
}
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


def test_a_refused_launch_ends_the_call_and_leaves_no_error(tmp_path):
    """The join of ragged attention reads what its first kernel describes: without that kernel it must not be launched."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    from mixed_precision_paged_argus_gb300 import build
    lib = build.build()
    assert os.path.samefile(lib, argus.lib_path())
    src, exe = tmp_path / "launches.c", tmp_path / "launches"
    src.write_text(FAKES)
    subprocess.run([cc, "-std=c11", "-rdynamic", "-I", os.path.join(ROOT, "include"), str(src), lib, "-o", str(exe),
                    "-Wl,-rpath," + os.path.dirname(lib), "-Wl,--allow-shlib-undefined"], check=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "lib64")
    env = dict(os.environ, LD_LIBRARY_PATH=cuda + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, env=env).stdout.split("\n")
    got = [tuple(int(x) for x in line.split()) for line in out if line]
    ok, failed = 0, 4
    extend = [(ok, 2, 0), (failed, 1, 0), (failed, 2, 0)]      # none, the first kernel, the join refused
    single = [(ok, 1, 0), (failed, 1, 0), (ok, 1, 0)]
    assert got == extend + single + single
