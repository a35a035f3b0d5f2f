// argus_paged_extend_attn, argus_paged_window_extend_attn and argus_paged_tree_attn: the host's
// side.  The kernels and what they measured stand in extend.cuh.
#include <algorithm>
#include <cmath>
#include <numeric>

#include "extend.cuh"

namespace argus {
namespace extend {

ARGUS_EXTEND_FORM(kPlain)
template <>
argus_status launch_mask<kWindow>(int D, bool bf, bool w16, const EParams& p, cudaStream_t s);
template <>
argus_status launch_mask<kTree>(int D, bool bf, bool w16, const EParams& p, cudaStream_t s);

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

// Upper bound of the key blocks of a call: every query tile has at most all of
// its sequence's (fewer than 2^31 rows and 2^31 tokens: the product is below 2^63).
static long long max_blocks(const argus_extend_args* a) {
  const long long G = a->g.n_q_heads / a->g.n_kv_heads;
  const long long tiles = ((long long)a->total_q * G + kBM - 1) / kBM + a->batch;
  return tiles * a->g.n_kv_heads * std::max(1ll, ((long long)a->max_pages * a->g.page_tokens + kBN - 1) / kBN);
}

// One CTA per SM, and no more than there can be blocks.
static int grid_size(const argus_extend_args* a) { return (int)std::min<long long>(device_sm_count(), std::max(1ll, max_blocks(a))); }

static size_t workspace(const argus_extend_args* a) {
  const size_t n = (size_t)grid_size(a);
  return 2 * n * kBM * (a->g.head_dim + 1) * sizeof(float) + n * sizeof(Cut);
}

// The arguments that all forms share, checked and brought into the kernels' form (p.n_ctas
// stays 0 where there is nothing to do).
static argus_status params(const argus_extend_args* a, void* ws, size_t ws_bytes, EParams& p) {
  argus_status st = check(a);
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
  if (ws_bytes < workspace(a))
    return fail(ARGUS_E_WORKSPACE, "extend: workspace of %zu bytes, %zu needed", ws_bytes, workspace(a));
  // an item that two CTAs share has its queries read while rows of others are written
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(a->q), o0 = reinterpret_cast<uintptr_t>(a->out);
  const uintptr_t token = (uintptr_t)g.n_q_heads * D * 2, q_bytes = (uintptr_t)(a->total_q - 1) * qs * 2 + token;
  if (q0 < o0 + a->total_q * token && o0 < q0 + q_bytes) return fail(ARGUS_E_INVALID, "extend: out overlaps q");
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
  p.n_ctas = grid_size(a);
  int bits = 0;
  while ((1 << bits) < p.G) ++bits;
  if (bits) {
    p.g_mul = (uint32_t)(((1ull << (31 + bits)) + p.G - 1) / p.G);
    p.g_shift = bits - 1;
  }
  if (max_blocks(a) / p.n_ctas >= 0x7fffffffll) return fail(ARGUS_E_UNSUPPORTED, "extend: too many key blocks");
  p.ws = static_cast<float*>(ws);
  return ARGUS_OK;
}

template <int MASK>
static argus_status run(const argus_extend_args* a, const EParams& p, void* stream) {
  if (p.n_ctas == 0) return ARGUS_OK;
  return launch_mask<MASK>(a->g.head_dim, a->q_dtype == ARGUS_BF16, p.pool[a->q_dtype].n_slots > 0, p, static_cast<cudaStream_t>(stream));
}

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
  extend::EParams p{};
  const argus_status st = extend::params(a, ws, ws_bytes, p);
  return st != ARGUS_OK ? st : extend::run<extend::kPlain>(a, p, stream);
}

extern "C" argus_status argus_paged_window_extend_attn(const argus_extend_args* a, int32_t window_tokens, int32_t sink_tokens, void* ws,
                                                       size_t ws_bytes, void* stream) {
  extend::EParams p{};
  const argus_status st = extend::params(a, ws, ws_bytes, p);
  if (st != ARGUS_OK) return st;
  if (window_tokens < 1 || sink_tokens < 0) return fail(ARGUS_E_INVALID, "extend: window_tokens must be >= 1 and sink_tokens >= 0");
  if (!a->causal) return fail(ARGUS_E_INVALID, "extend: a window needs causal = 1");
  if (p.n_ctas == 0) return ARGUS_OK;  // nothing to do: p holds no sizes
  p.window = window_tokens;
  p.sinks = sink_tokens;
  // A tile's rows belong to at most `tokens` tokens: its first row is a multiple of gcd(128, G) into a token.
  // The positions that they see behind the first ones, one less than the window and a position per token, touch
  // at most `chunks` chunks of 16.  (2^24 blocks hold every sequence.)
  const long long first = ((long long)p.G - std::gcd(extend::kBM, p.G) + extend::kBM - 1) / p.G, tokens = first + 1;
  const long long chunks = (window_tokens - 1 + tokens + 14) / 16 + 1, sunk = ((long long)sink_tokens + 15) / 16;
  p.sink_chunks = (int)std::min(sunk, (1ll << 27) - 1);
  p.window_blocks = (int)std::min((sunk + chunks + 7) / 8, 1ll << 24);
  return extend::run<extend::kWindow>(a, p, stream);
}

extern "C" argus_status argus_paged_tree_attn(const argus_extend_args* a, const uint32_t* tree_mask, int32_t mask_words, void* ws,
                                              size_t ws_bytes, void* stream) {
  extend::EParams p{};
  const argus_status st = extend::params(a, ws, ws_bytes, p);
  if (st != ARGUS_OK) return st;
  if (mask_words < 1) return fail(ARGUS_E_INVALID, "extend: mask_words must be >= 1");
  if (!a->causal) return fail(ARGUS_E_INVALID, "extend: a tree's mask needs causal = 1");
  if (p.n_ctas > 0 && !tree_mask) return fail(ARGUS_E_INVALID, "extend: tree_mask is NULL");
  if (reinterpret_cast<uintptr_t>(tree_mask) & 3) return fail(ARGUS_E_INVALID, "extend: tree_mask must be 4-byte aligned");
  p.tree = tree_mask;
  p.tree_words = mask_words;
  p.causal = 0;                        // every tile reads the whole cache; the mask says what its rows see
  return extend::run<extend::kTree>(a, p, stream);
}
