// argus_rope_append: rotary positions (one or several axes) on the new tokens'
// queries and keys, and the append of keys and values to the paged cache.
//
// Mathematics: pair i of a token turns by a = pos[axis(i)] * inv_freq[i].  Only
// a mod 2 pi matters, and at a far position the product has no fraction left in
// fp32 (position 10^6 times 1 rad is known to 0.06 rad).  So the frequency is
// taken in turns, as a 64-bit fixed-point fraction F = frac(inv_freq / 2 pi) 2^64,
// and pos * F in wrapping 64-bit integers IS the angle modulo one turn, exactly
// up to F's own rounding.  sincospif of twice the signed fraction follows.
//
// What bounds it: bytes (q, k, v read, q', k', v written once).  One CTA takes
// one token: its sines and cosines (rot_dim / 2 of them) are computed once in
// shared memory and used by all Hq + Hkv heads; every thread moves two 16-byte
// vectors per step, the two that hold a pair's halves.
#include <algorithm>

#include "common.cuh"

namespace argus {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;

struct RParams {
  int Hq, Hkv, P, B, total, rot, adjacent, n_axes, max_pages, codec;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  long long qs, ks, vs, qos;
  const int32_t* pos;
  const double* inv_freq;
  const uint8_t* pair_axis;
  const int32_t *q_start, *seq_lens;
  uint16_t* codes;
  long long n_slots;
  const uint8_t* page_codec;
  const int32_t* block_table;
  uint32_t* status;
};

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return BF ? pack_bf16x2(a, b) : pack_f16x2(a, b);
}

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RParams p) {
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  __shared__ int s_seq, s_bad;
  const int t = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) { s_seq = -1; s_bad = 0; }
  __syncthreads();
  // the sequence b with q_start[b] <= t < q_start[b + 1]: blocks of `step`
  // sequences first, then one block
  const int step = (p.B + kThreads - 1) / kThreads;
  {
    const int b = tid * step;
    if (b < p.B && p.q_start[b] <= t && t < p.q_start[min(b + step, p.B)]) s_seq = b;
  }
  if (tid < p.rot / 2) {
    const int ax = p.pair_axis ? p.pair_axis[tid] : 0;
    float c = 1.f, s = 0.f;
    if (ax < p.n_axes) {
      const double turns = p.inv_freq[tid] * 0.15915494309189535;   // 1 / (2 pi)
      const unsigned long long f = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
      const unsigned long long u = (unsigned long long)(long long)p.pos[(size_t)ax * p.total + t] * f;
      sincospif((float)(long long)u * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
    } else {
      s_bad = 1;
    }
    s_cos[tid] = c;
    s_sin[tid] = s;
  }
  __syncthreads();
  int b = s_seq;
  if (b < 0) return;                 // a row of no sequence
  if (step > 1) {
    const int b0 = b, b1 = min(b + step, p.B);
    __syncthreads();
    for (int i = b0 + tid; i < b1; i += kThreads)
      if (p.q_start[i] <= t && t < p.q_start[i + 1]) s_seq = i;
    __syncthreads();
    b = s_seq;
  }
  const int start = p.q_start[b], n = p.q_start[b + 1] - start;
  const long long c = (long long)p.seq_lens[b] - n + (t - start);
  long long slot = -1;
  int row = 0;
  if (c >= 0 && c < (long long)p.max_pages * p.P) {
    const int page = (int)(c / p.P);
    row = (int)(c - (long long)page * p.P);
    const size_t e = (size_t)b * p.max_pages + page;
    if (p.page_codec[e] == p.codec) slot = p.block_table[e];
    if (slot >= p.n_slots) slot = -1;
  }
  if (tid == 0 && p.status && (slot < 0 || s_bad)) atomicAdd(p.status, (slot < 0) + (s_bad != 0));

  constexpr int U = D / 16;          // units of 16 elements (two vectors) per head
  const int n_items = (p.Hq + 2 * p.Hkv) * U;
  const int ru = p.rot / 16;
  for (int it = tid; it < n_items; it += kThreads) {
    const int head = it / U, u = it % U;
    const bool turn = u < ru && head < p.Hq + p.Hkv;
    const int e0 = (turn && !p.adjacent) ? 8 * u : 16 * u;
    const int e1 = (turn && !p.adjacent) ? p.rot / 2 + 8 * u : 16 * u + 8;
    const uint16_t* src;
    uint16_t* dst = nullptr;
    if (head < p.Hq) {
      src = p.q + t * p.qs + head * D;
      dst = p.q_out + t * p.qos + head * D;
    } else {
      const bool is_v = head >= p.Hq + p.Hkv;
      const int h = head - p.Hq - (is_v ? p.Hkv : 0);
      src = is_v ? p.v + t * p.vs + h * D : p.k + t * p.ks + h * D;
      if (slot >= 0) dst = p.codes + (((size_t)slot * 2 + is_v) * p.Hkv + h) * ((size_t)p.P * D) + (size_t)row * D;
    }
    if (!dst) continue;
    uint4 a4 = *reinterpret_cast<const uint4*>(src + e0), b4 = *reinterpret_cast<const uint4*>(src + e1);
    if (turn) {
      uint32_t* a = reinterpret_cast<uint32_t*>(&a4);
      uint32_t* bb = reinterpret_cast<uint32_t*>(&b4);
      if (p.adjacent) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<BF>(a[j]), y = unpack2<BF>(bb[j]);
          const float c0 = s_cos[8 * u + j], s0 = s_sin[8 * u + j];
          const float c1 = s_cos[8 * u + 4 + j], s1 = s_sin[8 * u + 4 + j];
          a[j] = pack2<BF>(x.x * c0 - x.y * s0, x.y * c0 + x.x * s0);
          bb[j] = pack2<BF>(y.x * c1 - y.y * s1, y.y * c1 + y.x * s1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack2<BF>(a[j]), y = unpack2<BF>(bb[j]);
          const float c0 = s_cos[8 * u + 2 * j], s0 = s_sin[8 * u + 2 * j];
          const float c1 = s_cos[8 * u + 2 * j + 1], s1 = s_sin[8 * u + 2 * j + 1];
          a[j] = pack2<BF>(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
          bb[j] = pack2<BF>(y.x * c0 + x.x * s0, y.y * c1 + x.y * s1);
        }
      }
    }
    *reinterpret_cast<uint4*>(dst + e0) = a4;
    *reinterpret_cast<uint4*>(dst + e1) = b4;
  }
}

}  // namespace rope
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_rope_append(const argus_rope_args* a, void* stream) {
  if (!a) return fail(ARGUS_E_INVALID, "rope: args is NULL");
  const argus_geom& g = a->g;
  if (g.n_q_heads <= 0 || g.n_kv_heads <= 0 || g.n_q_heads % g.n_kv_heads || g.page_tokens <= 0)
    return fail(ARGUS_E_INVALID, "rope: bad head counts or page_tokens");
  if (g.head_dim != 64 && g.head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "rope: head_dim %d (supported: 64, 128)", g.head_dim);
  if (g.page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "rope: page_tokens %d not a multiple of 16", g.page_tokens);
  if (a->dtype != ARGUS_FP16 && a->dtype != ARGUS_BF16) return fail(ARGUS_E_INVALID, "rope: dtype must be FP16 or BF16");
  if (a->batch < 0 || a->total_q < 0 || a->max_pages < 0) return fail(ARGUS_E_INVALID, "rope: negative size");
  if (a->n_axes < 1 || a->n_axes > rope::kMaxAxes) return fail(ARGUS_E_INVALID, "rope: n_axes %d not in 1..4", a->n_axes);
  if (a->adjacent != 0 && a->adjacent != 1) return fail(ARGUS_E_INVALID, "rope: adjacent must be 0 or 1");
  if (a->rot_dim <= 0 || a->rot_dim > g.head_dim) return fail(ARGUS_E_INVALID, "rope: rot_dim %d not in 1..head_dim", a->rot_dim);
  if (a->rot_dim % 16) return fail(ARGUS_E_UNSUPPORTED, "rope: rot_dim %d not a multiple of 16", a->rot_dim);
  if (a->batch == 0 || a->total_q == 0) return ARGUS_OK;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->positions || !a->inv_freq || !a->q_start || !a->seq_lens || !a->pool ||
      !a->page_codec || !a->block_table)
    return fail(ARGUS_E_INVALID, "rope: NULL pointer");
  if (a->pool->codec != a->dtype) return fail(ARGUS_E_UNSUPPORTED, "rope: the pool's codec %d is not the tokens' type", a->pool->codec);
  if (a->pool->placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "rope: the pool must lie in device memory");
  if (a->pool->n_slots < 0 || (a->pool->n_slots > 0 && !a->pool->codes)) return fail(ARGUS_E_INVALID, "rope: bad pool");
  rope::RParams p{};
  p.Hq = g.n_q_heads;
  p.Hkv = g.n_kv_heads;
  p.P = g.page_tokens;
  const int D = g.head_dim;
  p.qs = a->q_stride ? a->q_stride : (long long)p.Hq * D;
  p.ks = a->k_stride ? a->k_stride : (long long)p.Hkv * D;
  p.vs = a->v_stride ? a->v_stride : (long long)p.Hkv * D;
  p.qos = a->q_out_stride ? a->q_out_stride : (long long)p.Hq * D;
  if (p.qs < (long long)p.Hq * D || p.qos < (long long)p.Hq * D || p.ks < (long long)p.Hkv * D || p.vs < (long long)p.Hkv * D)
    return fail(ARGUS_E_INVALID, "rope: a token stride is smaller than the token");
  if ((p.qs | p.ks | p.vs | p.qos) & 7) return fail(ARGUS_E_INVALID, "rope: token strides must be multiples of 8 elements");
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->k) | reinterpret_cast<uintptr_t>(a->v) |
       reinterpret_cast<uintptr_t>(a->q_out) | reinterpret_cast<uintptr_t>(a->pool->codes)) & 15)
    return fail(ARGUS_E_INVALID, "rope: q, k, v, q_out and the pool must be 16-byte aligned");
  if (a->q_out == a->q && p.qs != p.qos) return fail(ARGUS_E_INVALID, "rope: q_out in place needs q's stride");
  p.B = a->batch;
  p.total = a->total_q;
  p.rot = a->rot_dim;
  p.adjacent = a->adjacent;
  p.n_axes = a->n_axes;
  p.max_pages = a->max_pages;
  p.codec = a->dtype;
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.pos = a->positions;
  p.inv_freq = a->inv_freq;
  p.pair_axis = a->pair_axis;
  p.q_start = a->q_start;
  p.seq_lens = a->seq_lens;
  p.codes = static_cast<uint16_t*>(a->pool->codes);
  p.n_slots = a->pool->n_slots;
  p.page_codec = a->page_codec;
  p.block_table = a->block_table;
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = a->dtype == ARGUS_BF16;
  if (D == 64) {
    if (bf) rope::rope_kernel<64, true><<<p.total, rope::kThreads, 0, s>>>(p);
    else rope::rope_kernel<64, false><<<p.total, rope::kThreads, 0, s>>>(p);
  } else {
    if (bf) rope::rope_kernel<128, true><<<p.total, rope::kThreads, 0, s>>>(p);
    else rope::rope_kernel<128, false><<<p.total, rope::kThreads, 0, s>>>(p);
  }
  return launch_status("argus_rope_append");
}
