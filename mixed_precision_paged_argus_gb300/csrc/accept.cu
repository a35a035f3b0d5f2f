// argus_accept_tokens: the K and V rows of a drafted tree's accepted path moved to where the
// sequence goes on.
//
// Mathematics: path token k of a sequence, the drafted token x_k (x_0 < x_1 < ...), goes from
// cached position base + x_k to base + k.  x_k >= k, and a later token's source lies
// behind every earlier destination (x_{k+1} > x_k >= k): a thread that moves the same bytes of
// all rows in order of k, some at a time, reads nothing that it wrote.  So the move is done
// in place without a buffer or a barrier between reads and writes.
//
// What bounds it: latency.  A sequence moves a few rows (some KB); a block has one, every
// 16 bytes of its 2 Hkv rows a thread, and what is left are dependent reads: lengths, path,
// table, rows.  The path and the table are looked up by a warp for 32 tokens at once.
//
// Measured (GB300, replayed from a graph, L2 flushed): one tree's path of 6 tokens, 2 KV heads of 64: 6 us, launch
// included; 256 paths of up to 10 tokens, 8 KV heads of 128: 8.6 us (10 MB).  Called from Python the
// host's 16 us are what counts.
#include "common.cuh"

namespace argus {
namespace accept {

constexpr int kThreads = 256;
constexpr int kAhead = 8;              // rows on their way at once

struct AParams {
  int Hkv, P, B, max_pages, codec, width;
  uint4* codes;
  long long n_slots;
  const uint8_t* page_codec;
  const int32_t *block_table, *q_start, *seq_lens, *path, *n_path;
  int32_t* seq_lens_out;
  uint32_t* status;
};

// A cached position's place, in rows of the pool's first KV head; -1 if it has none.
__device__ __forceinline__ long long place(const AParams& p, int b, long long pos) {
  if (pos >= (long long)p.max_pages * p.P) return -1;
  const int page = (int)((unsigned long long)pos / (unsigned)p.P);
  const size_t e = (size_t)b * p.max_pages + page;
  const long long slot = p.block_table[e];
  if (p.page_codec[e] != p.codec || slot < 0 || slot >= p.n_slots) return -1;
  return slot * 2 * p.Hkv * p.P + (pos - (long long)page * p.P);
}

template <int V>                       // 16-byte vectors of a row
__global__ void __launch_bounds__(kThreads) accept_kernel(const AParams p) {
  __shared__ long long s_from[32], s_to[32];
  __shared__ int s_count;              // of the 32 tokens: those before the path ends
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.seq_lens[b], n = max(p.q_start[b + 1] - p.q_start[b], 0), want = p.n_path[b];
  const int m = len < n ? 0 : min(max(want, 0), p.width);
  const long long base = (long long)len - n;
  int taken = 0, bad = (len < n) + (want != min(max(want, 0), p.width));
  for (int k0 = 0; k0 < m; k0 += 32) {
    if (warp == 0) {
      const int k = k0 + lane;
      const bool in = k < m;
      const int32_t* path = p.path + (size_t)b * p.width;
      const int x = in ? path[k] : 0, before = in && k > 0 ? path[k - 1] : -1;
      const unsigned wrong = __ballot_sync(0xffffffffu, in && (x <= before || x >= n));
      const int cnt = wrong ? __ffs(wrong) - 1 : min(32, m - k0);
      long long from = -1, to = -1;
      bool lost = false;
      if (lane < cnt && x != k) {
        from = place(p, b, base + x);
        to = place(p, b, base + k);
        lost = from < 0 || to < 0;
      }
      s_from[lane] = lost ? -1 : from;
      s_to[lane] = to;
      bad += __popc(__ballot_sync(0xffffffffu, lost)) + (wrong != 0);
      if (lane == 0) s_count = cnt;
    }
    __syncthreads();
    const int cnt = s_count;
    for (int u = threadIdx.x / V; u < 2 * p.Hkv; u += kThreads / V) {
      const long long off = (long long)u * p.P;
      for (int i0 = 0; i0 < cnt; i0 += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i0 + i < cnt && s_from[i0 + i] >= 0) v[i] = p.codes[(s_from[i0 + i] + off) * V + threadIdx.x % V];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i0 + i < cnt && s_from[i0 + i] >= 0) p.codes[(s_to[i0 + i] + off) * V + threadIdx.x % V] = v[i];
      }
    }
    taken += cnt;
    if (cnt < min(32, m - k0)) break;
    __syncthreads();                   // the places have been read
  }
  if (threadIdx.x == 0) {
    p.seq_lens_out[b] = len < n ? len : (int)base + taken;
    if (bad && p.status) atomicAdd(p.status, (uint32_t)bad);
  }
}

static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && a && b && x < y + nb && y < x + na;
}

}  // namespace accept
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_accept_tokens(const argus_geom* g, int32_t batch, const argus_pool* pool, const uint8_t* page_codec,
                                            const int32_t* block_table, int32_t max_pages, const int32_t* q_start,
                                            const int32_t* seq_lens, const int32_t* path, int32_t path_width, const int32_t* n_path,
                                            int32_t* seq_lens_out, uint32_t* status, void* stream) {
  if (!g || !pool) return fail(ARGUS_E_INVALID, "accept: geometry or pool is NULL");
  if (g->n_kv_heads <= 0 || g->page_tokens <= 0) return fail(ARGUS_E_INVALID, "accept: bad head counts or page_tokens");
  if (g->head_dim != 64 && g->head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "accept: head_dim %d (supported: 64, 128)", g->head_dim);
  if (g->page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "accept: page_tokens %d not a multiple of 16", g->page_tokens);
  if (batch < 0 || max_pages < 0 || path_width < 0) return fail(ARGUS_E_INVALID, "accept: negative size");
  if (pool->codec != ARGUS_FP16 && pool->codec != ARGUS_BF16)
    return fail(ARGUS_E_UNSUPPORTED, "accept: pages of codec %d (supported: 16-bit)", pool->codec);
  if (pool->placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "accept: the pool must lie in device memory");
  if (pool->n_slots < 0 || (pool->n_slots > 0 && !pool->codes)) return fail(ARGUS_E_INVALID, "accept: bad pool");
  if (reinterpret_cast<uintptr_t>(pool->codes) & 15) return fail(ARGUS_E_INVALID, "accept: codes must be 16-byte aligned");
  if (batch == 0) return ARGUS_OK;
  if (!q_start || !seq_lens || !n_path || !seq_lens_out || (path_width > 0 && !path)) return fail(ARGUS_E_INVALID, "accept: NULL pointer");
  if (max_pages > 0 && (!page_codec || !block_table)) return fail(ARGUS_E_INVALID, "accept: NULL page_codec or block_table");
  // a block writes its length while others still read theirs
  const size_t n = (size_t)batch * 4, entries = (size_t)batch * max_pages;
  if (accept::overlap(seq_lens_out, n, seq_lens, n) || accept::overlap(seq_lens_out, n, q_start, n + 4) ||
      accept::overlap(seq_lens_out, n, n_path, n) || accept::overlap(seq_lens_out, n, path, n * path_width) ||
      accept::overlap(seq_lens_out, n, block_table, 4 * entries) || accept::overlap(seq_lens_out, n, page_codec, entries))
    return fail(ARGUS_E_INVALID, "accept: seq_lens_out overlaps an input");
  accept::AParams p{};
  p.Hkv = g->n_kv_heads;
  p.P = g->page_tokens;
  p.B = batch;
  p.max_pages = max_pages;
  p.codec = pool->codec;
  p.width = path_width;
  p.codes = static_cast<uint4*>(pool->codes);
  p.n_slots = pool->n_slots;
  p.page_codec = page_codec;
  p.block_table = block_table;
  p.q_start = q_start;
  p.seq_lens = seq_lens;
  p.path = path;
  p.n_path = n_path;
  p.seq_lens_out = seq_lens_out;
  p.status = status;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch);
  cfg.blockDim = dim3(accept::kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = g->head_dim == 64 ? cudaLaunchKernelEx(&cfg, accept::accept_kernel<8>, p) : cudaLaunchKernelEx(&cfg, accept::accept_kernel<16>, p);
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_accept_tokens: launch failed: %s", cudaGetErrorString(e));
}
