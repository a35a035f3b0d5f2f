// argus_paged_extend_attn: several query tokens per sequence attend to the
// paged cache, read in place.  One warp per (query token, query head): an online
// softmax over the keys, D / 32 dims per lane, everything in fp32.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace argus {
namespace extend {

struct PoolRef {
  const uint8_t* codes;
  const float* meta;
  long long n_slots;
};

struct EParams {
  int Hq, Hkv, G, P, B, total_q, causal, max_pages, q_codec;
  const uint16_t* q;
  long long qs;
  const int32_t *q_start, *seq_lens;
  PoolRef pool[4];                   // by codec: FP16, BF16, FP8, INT8
  const uint8_t* page_codec;
  const int32_t* block_table;
  uint16_t* out;
  float* lse2;
  uint32_t* status;
  float scale_log2;
};

__device__ __forceinline__ float value16(uint16_t x, bool bf) {
  return bf ? __uint_as_float((uint32_t)x << 16) : __half2float(*reinterpret_cast<__half*>(&x));
}

template <int D>
__global__ void __launch_bounds__(256) simple_kernel(const EParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (long long)p.total_q * p.Hq) return;
  const int t = (int)(w / p.Hq), hq = (int)(w % p.Hq), h = hq / p.G;
  int b = -1;
  for (int i = 0; i < p.B; ++i)
    if (p.q_start[i] <= t && t < p.q_start[i + 1]) b = i;
  if (b < 0) return;
  const long long cap = (long long)p.max_pages * p.P;
  const int len = (int)min(max((long long)p.seq_lens[b], 0ll), cap);
  const int n = p.q_start[b + 1] - p.q_start[b], i = t - p.q_start[b];
  const int keys = p.causal ? max(0, len - n + i + 1) : len;
  const bool bf = p.q_codec == ARGUS_BF16;
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = value16(p.q[t * p.qs + hq * D + lane * E + e], bf);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < keys; ++j) {
    const size_t entry = (size_t)b * p.max_pages + j / p.P;
    const int codec = p.page_codec[entry];
    const int slot = p.block_table[entry];
    if (codec > 3 || slot < 0 || slot >= p.pool[codec].n_slots) continue;
    const PoolRef& r = p.pool[codec];
    const size_t unit = ((size_t)slot * 2) * p.Hkv + h;
    float k[E], v[E];
    for (int kv = 0; kv < 2; ++kv) {
      const size_t u = unit + (size_t)kv * p.Hkv;
      const size_t at = (u * p.P + j % p.P) * D + lane * E;
      float* x = kv ? v : k;
      for (int e = 0; e < E; ++e) {
        if (codec <= ARGUS_BF16) x[e] = value16(reinterpret_cast<const uint16_t*>(r.codes)[at + e], codec == ARGUS_BF16);
        else if (codec == ARGUS_INT8) x[e] = (float)(int8_t)r.codes[at + e] * r.meta[u];
        else {
          const uint32_t two = e4m3x2_to_f16x2(r.codes[at + e]);
          x[e] = __low2float(*reinterpret_cast<const __half2*>(&two)) * r.meta[u];
        }
      }
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), pr = exp2f(s - mn);
    l = l * a + pr;
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + pr * v[e];
    m = mn;
  }
  // the row that sees every page counts the ones it cannot read
  if (hq == 0 && i == n - 1 && p.status) {
    int bad = 0;
    for (int pg = lane; pg < (len + p.P - 1) / p.P; pg += 32) {
      const size_t entry = (size_t)b * p.max_pages + pg;
      const int codec = p.page_codec[entry], slot = p.block_table[entry];
      bad += codec > 3 || slot < 0 || slot >= p.pool[codec].n_slots;
    }
    for (int x = 16; x > 0; x >>= 1) bad += __shfl_xor_sync(0xffffffffu, bad, x);
    if (lane == 0 && bad) atomicAdd(p.status, bad);
  }
  const size_t row = (size_t)t * p.Hq + hq;
  for (int e = 0; e < E; ++e) {
    const float x = l > 0.f ? o[e] / l : 0.f;
    const uint32_t y = bf ? pack_bf16x2(x, 0.f) : pack_f16x2(x, 0.f);
    p.out[row * D + lane * E + e] = (uint16_t)y;
  }
  if (lane == 0 && p.lse2) p.lse2[row] = l > 0.f ? m + log2f(l) : -INFINITY;
}

static argus_status check(const argus_extend_args* a) {
  if (!a) return fail(ARGUS_E_INVALID, "extend: args is NULL");
  const argus_geom& g = a->g;
  if (g.n_q_heads <= 0 || g.n_kv_heads <= 0 || g.n_q_heads % g.n_kv_heads || g.page_tokens <= 0)
    return fail(ARGUS_E_INVALID, "extend: bad head counts or page_tokens");
  if (g.head_dim != 64 && g.head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "extend: head_dim %d (supported: 64, 128)", g.head_dim);
  if (g.n_q_heads / g.n_kv_heads > 8)
    return fail(ARGUS_E_UNSUPPORTED, "extend: %d query heads per KV head (supported: 1..8)", g.n_q_heads / g.n_kv_heads);
  if (g.page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "extend: page_tokens %d not a multiple of 16", g.page_tokens);
  if (a->q_dtype != ARGUS_FP16 && a->q_dtype != ARGUS_BF16) return fail(ARGUS_E_INVALID, "extend: q_dtype must be FP16 or BF16");
  if (a->causal != 0 && a->causal != 1) return fail(ARGUS_E_INVALID, "extend: causal must be 0 or 1");
  if (a->batch < 0 || a->total_q < 0 || a->max_pages < 0 || a->n_pools < 0) return fail(ARGUS_E_INVALID, "extend: negative size");
  if (a->batch > 65535) return fail(ARGUS_E_UNSUPPORTED, "extend: batch %d above 65535", a->batch);
  if ((long long)a->total_q * g.n_q_heads > 0x7fffffffll - 128) return fail(ARGUS_E_UNSUPPORTED, "extend: 2^31 query rows or more");
  if ((long long)a->max_pages * g.page_tokens > 0x7fffffffll - 256)
    return fail(ARGUS_E_UNSUPPORTED, "extend: 2^31 cached tokens per sequence or more");
  if (!(a->softmax_scale >= 0.f) || !std::isfinite(a->softmax_scale))
    return fail(ARGUS_E_INVALID, "extend: softmax_scale must be finite and >= 0");
  if (a->n_pools > 0 && !a->pools) return fail(ARGUS_E_INVALID, "extend: pools is NULL");
  uint32_t seen = 0;
  for (int i = 0; i < a->n_pools; ++i) {
    const argus_pool& pl = a->pools[i];
    if (pl.codec < 0 || pl.codec > ARGUS_INT1_G32) return fail(ARGUS_E_INVALID, "extend: bad codec %d", pl.codec);
    if (seen >> pl.codec & 1) return fail(ARGUS_E_INVALID, "extend: more than one pool of codec %d", pl.codec);
    seen |= 1u << pl.codec;
    if (pl.codec > ARGUS_INT8) return fail(ARGUS_E_UNSUPPORTED, "extend: pages of codec %d (supported: 16-bit, FP8, INT8)", pl.codec);
    if (pl.codec <= ARGUS_BF16 && pl.codec != a->q_dtype)
      return fail(ARGUS_E_UNSUPPORTED, "extend: 16-bit pages must be of the query's type");
    if (pl.placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "extend: pools must lie in device memory");
    if (pl.n_slots < 0) return fail(ARGUS_E_INVALID, "extend: negative n_slots");
    if (pl.n_slots > 0 && (!pl.codes || (pl.codec >= ARGUS_FP8_E4M3 && !pl.meta)))
      return fail(ARGUS_E_INVALID, "extend: NULL codes or meta (codec %d)", pl.codec);
    if (reinterpret_cast<uintptr_t>(pl.codes) & 15) return fail(ARGUS_E_INVALID, "extend: codes must be 16-byte aligned");
    if (pl.codec >= ARGUS_FP8_E4M3 && (reinterpret_cast<uintptr_t>(pl.meta) & 3))
      return fail(ARGUS_E_INVALID, "extend: meta must be 4-byte aligned");
  }
  return ARGUS_OK;
}

static size_t workspace(const argus_extend_args*) { return 16; }

}  // namespace extend
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_extend_workspace_bytes(const argus_extend_args* a, size_t* bytes) {
  if (!bytes) return fail(ARGUS_E_INVALID, "extend: bytes is NULL");
  argus_status st = extend::check(a);
  if (st != ARGUS_OK) return st;
  *bytes = extend::workspace(a);
  return ARGUS_OK;
}

extern "C" argus_status argus_paged_extend_attn(const argus_extend_args* a, void* ws, size_t ws_bytes, void* stream) {
  argus_status st = extend::check(a);
  if (st != ARGUS_OK) return st;
  if (a->batch == 0 || a->total_q == 0) return ARGUS_OK;
  const argus_geom& g = a->g;
  const int D = g.head_dim;
  if (!a->q || !a->q_start || !a->seq_lens || !a->out) return fail(ARGUS_E_INVALID, "extend: NULL pointer");
  if (a->max_pages > 0 && (!a->page_codec || !a->block_table)) return fail(ARGUS_E_INVALID, "extend: NULL page_codec or block_table");
  const long long qs = a->q_stride ? a->q_stride : (long long)g.n_q_heads * D;
  if (qs < (long long)g.n_q_heads * D) return fail(ARGUS_E_INVALID, "extend: q_stride is smaller than a token");
  if (qs & 7) return fail(ARGUS_E_INVALID, "extend: q_stride must be a multiple of 8 elements");
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) & 15)
    return fail(ARGUS_E_INVALID, "extend: q and out must be 16-byte aligned");
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15)) return fail(ARGUS_E_INVALID, "extend: ws must be a 16-byte aligned device pointer");
  if (ws_bytes < extend::workspace(a))
    return fail(ARGUS_E_WORKSPACE, "extend: workspace of %zu bytes, %zu needed", ws_bytes, extend::workspace(a));
  extend::EParams p{};
  p.Hq = g.n_q_heads;
  p.Hkv = g.n_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.P = g.page_tokens;
  p.B = a->batch;
  p.total_q = a->total_q;
  p.causal = a->causal;
  p.max_pages = a->max_pages;
  p.q_codec = a->q_dtype;
  p.q = static_cast<const uint16_t*>(a->q);
  p.qs = qs;
  p.q_start = a->q_start;
  p.seq_lens = a->seq_lens;
  for (int i = 0; i < a->n_pools; ++i)
    p.pool[a->pools[i].codec] = {static_cast<const uint8_t*>(a->pools[i].codes), static_cast<const float*>(a->pools[i].meta), a->pools[i].n_slots};
  p.page_codec = a->page_codec;
  p.block_table = a->block_table;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse2 = a->lse2_out;
  p.status = a->status;
  p.scale_log2 = (float)((double)a->softmax_scale * 1.4426950408889634);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long warps = (long long)p.total_q * p.Hq;
  const unsigned blocks = (unsigned)((warps + 7) / 8);
  if (D == 64) extend::simple_kernel<64><<<blocks, 256, 0, s>>>(p);
  else extend::simple_kernel<128><<<blocks, 256, 0, s>>>(p);
  return launch_status("argus_paged_extend_attn");
}
