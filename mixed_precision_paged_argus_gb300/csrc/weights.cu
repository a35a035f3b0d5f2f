// argus_attn_weights: the attention weights of a batch's query tokens, summed per cached
// position and KV head.
//
// Mathematics: after the attention, its row's log-sum L (log2) makes every weight of the row
// a function of one score: p = 2^(s - L).  So the sum over the rows that share a KV head,
//   w_j <- decay w_j + sum_rows 2^(scale log2e q.k_j - L_row),
// needs K once and nothing of V, and no position depends on another.
//
// What bounds it: with few rows the bytes of K; with many the products and exponentials.
//  * All 16-token chunks of all (sequence, KV head) are dealt to the warps in equal
//    contiguous ranges, found on the device.  A warp looks up to 32 chunks up at once,
//    a lane each.
//  * Scores by mma m16n8k16, 16 keys by 8 query rows.  A dot product does not mind
//    the order of its dims: each lane loads 16-byte vectors of its two key rows, and the
//    query's fragments are loaded in the order that makes these the operand.  8-bit codes become 16
//    bits in registers, exactly; of INT4, INT2 and INT1 the codes are multiplied, and a
//    token's scale and zero are applied per group of 32 dims.
//  * The weights of a batch of chunks are summed in shared memory and added to the old ones
//    in whole lines.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace argus {
namespace weights {

struct PoolRef {
  const uint8_t* codes;
  const uint8_t* meta;
  long long n_slots;
};

struct WParams {
  int Hq, Hkv, G, P, B, total_q, causal, max_pages;
  const uint16_t* q;
  long long qs;
  const int32_t *q_start, *seq_lens;
  PoolRef pool[7];
  const uint8_t* page_codec;
  const int32_t* block_table;
  const float* lse2;
  float* weights;
  long long row_len;
  float decay, scale_log2;
  uint32_t* status;
};

constexpr int kWarps = 8;
constexpr int kBatch = 32;             // chunks looked up at once

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ long long warp_scan(long long x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ int length(const WParams& p, int b) {
  return (int)min((long long)max(p.seq_lens[b], 0), (long long)p.max_pages * p.P);
}
__device__ __forceinline__ long long chunks_of(const WParams& p, int b) { return (long long)p.Hkv * ((length(p, b) + 15) / 16); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// How a page's operands are formed: 16-bit as they are, 8-bit codes as fp16, group codes as fp16.
enum Form { kNone = -1, k16 = 0, k8 = 1, kGroup = 2 };
__device__ __forceinline__ int form_of(int codec) { return codec <= ARGUS_BF16 ? k16 : codec <= ARGUS_INT8 ? k8 : kGroup; }

// Eight query rows as the MMA's B operand, in the dims' order of a form.
template <int D>
struct Query {
  uint32_t f[D / 16][2];
  float fac[2];                        // of columns 2c, 2c + 1: undoes the fp16 query's power of two
  float sum[D / 32][2];                // kGroup: sums of a group's elements
};

template <int D, bool BF>
__device__ __forceinline__ void load_query(const uint16_t* row, bool real, int form, int lane, Query<D>& out) {
  const int c = lane & 3;
  uint4 v[D / 32];                     // 8 elements each
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    // k8: two vectors next to each other, 16 codes; else every fourth
    const int at = form == k8 ? (i / 2) * 64 + c * 16 + (i & 1) * 8 : i * 32 + c * 8;
    v[i] = real ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0, 0, 0, 0);
  }
  float fac = 1.f;
  if (BF && form != k16) {
    // the row's largest magnitude comes to [2^14, 2^15): its 8 bits fit fp16
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t a = max_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), b = max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu);
      mx = max_u16x2(mx, max_u16x2(a, b));
    }
    mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const uint32_t ex = max(max(mx >> 16, mx & 0xFFFFu) >> 7, 15u);
    const float up = __uint_as_float((268 - ex) << 23);
    fac = __uint_as_float((ex - 14) << 23);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
    }
  }
  if (form == kGroup) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
        s += y.x + y.y;
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      out.sum[i][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      out.sum[i][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
      // codes come out of their word in pairs (j, j + 4)
      v[i] = make_uint4(prmt(w[0], w[2], 0x5410), prmt(w[0], w[2], 0x7632), prmt(w[1], w[3], 0x5410), prmt(w[1], w[3], 0x7632));
    }
  }
  out.fac[0] = __shfl_sync(0xffffffffu, fac, 8 * c);
  out.fac[1] = __shfl_sync(0xffffffffu, fac, 8 * c + 4);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    out.f[2 * i][0] = v[i].x;
    out.f[2 * i][1] = v[i].y;
    out.f[2 * i + 1][0] = v[i].z;
    out.f[2 * i + 1][1] = v[i].w;
  }
}

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void int8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;  // 1024 + (code + 128), minus 1152
  lo = hsub2_u32(prmt(u, 0x64646464u, 0x4140), 0x64806480u);
  hi = hsub2_u32(prmt(u, 0x64646464u, 0x4342), 0x64806480u);
}

// Scores of 16 keys by 8 rows: d[0], d[1] key lane / 4, columns 2c and 2c + 1; d[2], d[3] eight keys
// further down.
template <int D, bool BF>
__device__ __forceinline__ void scores(const uint8_t* src, const uint8_t* meta, int codec, int lane, const Query<D>& q, float (&d)[4]) {
  const int r = lane >> 2, c = lane & 3;
  d[0] = d[1] = d[2] = d[3] = 0.f;
  if (codec <= ARGUS_BF16) {
    uint4 a[D / 32], b[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      a[i] = ldg16(src + r * 2 * D + i * 64 + c * 16);
      b[i] = ldg16(src + (r + 8) * 2 * D + i * 64 + c * 16);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if (BF) {
        mma_bf16(d, a[i].x, b[i].x, a[i].y, b[i].y, q.f[2 * i][0], q.f[2 * i][1]);
        mma_bf16(d, a[i].z, b[i].z, a[i].w, b[i].w, q.f[2 * i + 1][0], q.f[2 * i + 1][1]);
      } else {
        mma_f16(d, a[i].x, b[i].x, a[i].y, b[i].y, q.f[2 * i][0], q.f[2 * i][1]);
        mma_f16(d, a[i].z, b[i].z, a[i].w, b[i].w, q.f[2 * i + 1][0], q.f[2 * i + 1][1]);
      }
    }
  } else if (codec <= ARGUS_INT8) {
    uint4 a[D / 64], b[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      a[i] = ldg16(src + r * D + i * 64 + c * 16);
      b[i] = ldg16(src + (r + 8) * D + i * 64 + c * 16);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t a0, a1, b0, b1;
        if (codec == ARGUS_FP8_E4M3) {
          a0 = e4m3x2_to_f16x2(wa[e]);
          a1 = e4m3x2_to_f16x2(wa[e] >> 16);
          b0 = e4m3x2_to_f16x2(wb[e]);
          b1 = e4m3x2_to_f16x2(wb[e] >> 16);
        } else {
          int8_to_f16(wa[e], a0, a1);
          int8_to_f16(wb[e], b0, b1);
        }
        mma_f16(d, a0, b0, a1, b1, q.f[4 * i + e][0], q.f[4 * i + e][1]);
      }
    }
  } else {
    const int bits = codec == ARGUS_INT4_G32 ? 4 : codec == ARGUS_INT2_G32 ? 2 : 1, row = D * bits / 8;
    const uint32_t mask = ((1u << bits) - 1) * 0x10001u;
    uint32_t w[2][D / 32];
    uint32_t sz[2][D / 32];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* at = src + (r + 8 * x) * row;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // eight codes of group i: elements j and j + 4 in the two halves, j codes up
        if (codec == ARGUS_INT4_G32) {
          w[x][i] = __ldg(reinterpret_cast<const uint32_t*>(at + i * 16 + c * 4));
        } else if (codec == ARGUS_INT2_G32) {
          const uint32_t y = __ldg(reinterpret_cast<const uint16_t*>(at + i * 8 + c * 2));
          w[x][i] = (y & 0xFF) | (y >> 8) << 16;
        } else {
          const uint32_t y = __ldg(at + i * 4 + c);
          w[x][i] = (y & 0xF) | (y >> 4) << 16;
        }
        sz[x][i] = __ldg(reinterpret_cast<const uint32_t*>(meta) + (r + 8 * x) * (D / 32) + i);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t o[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j)                      // 1024 + code, minus 1024
          o[x][j] = hsub2_u32(((w[x][i] >> (bits * j)) & mask) | 0x64006400u, 0x64006400u);
      }
      float g[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(g, o[0][0], o[1][0], o[0][1], o[1][1], q.f[2 * i][0], q.f[2 * i][1]);
      mma_f16(g, o[0][2], o[1][2], o[0][3], o[1][3], q.f[2 * i + 1][0], q.f[2 * i + 1][1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&sz[x][i]));
#pragma unroll
        for (int k = 0; k < 2; ++k) d[2 * x + k] = fmaf(y.x, g[2 * x + k], fmaf(y.y, q.sum[i][k], d[2 * x + k]));
      }
    }
  }
}

// BF: the queries' (and 16-bit pages') type.
template <int D, bool BF>
__global__ void __launch_bounds__(32 * kWarps) weights_kernel(const WParams p) {
  __shared__ __align__(16) float s_sum[kWarps][kBatch * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
  float* sums = s_sum[warp];
  // this warp's range of chunks
  const int nw = gridDim.x * kWarps, w = blockIdx.x * kWarps + warp;
  const long long first = lane < p.B ? chunks_of(p, lane) : 0;
  long long total = first;
  for (int x = lane + 32; x < p.B; x += 32) total += chunks_of(p, x);
  total = warp_sum(total);
  const long long u0 = total / nw * w + total % nw * w / nw, u1 = total / nw * (w + 1) + total % nw * (w + 1) / nw;
  long long left = u1 - u0;
  if (left <= 0) return;
  int b = 0;
  long long at = 0;                                      // the chunk of sequence b, its KV heads one after the other
  {
    long long before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const long long mine = b0 == 0 ? first : b0 + lane < p.B ? chunks_of(p, b0 + lane) : 0, incl = warp_scan(mine);
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > u0);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        at = u0 - before - __shfl_sync(0xffffffffu, incl - mine, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  Query<D> q;
  int have_b = -1, have_h = -1, have_t = -1, have_form = kNone;   // what q holds
  float lse[2] = {0.f, 0.f};
  int see[2] = {0, 0};                                   // the columns' last visible key
  while (left > 0) {
    const int len = length(p, b), per = (len + 15) / 16;
    if (at >= (long long)per * p.Hkv) {                  // the next sequence that has any
      at = 0;
      ++b;
      continue;
    }
    const int h = (int)(at / per), c0 = (int)(at - (long long)h * per);
    const int n = (int)min(left, (long long)min(kBatch, per - c0));
    left -= n;
    at += n;
    // a chunk per lane
    const uint8_t *src = nullptr, *meta = nullptr;
    int codec = -1;
    float ks = 1.f;
    if (lane < n) {
      const int key = (c0 + lane) * 16, page = (int)((uint32_t)key / (uint32_t)p.P), row = key - page * p.P;
      const size_t e = (size_t)b * p.max_pages + page;
      const int k = p.page_codec[e];
      const long long slot = p.block_table[e];
      const PoolRef r = p.pool[k <= ARGUS_INT1_G32 ? k : 0];
      if (k > ARGUS_INT1_G32 || slot < 0 || slot >= r.n_slots) {
        if (h == 0 && row == 0 && p.status) atomicAdd(p.status, 1u);
      } else {
        codec = k;
        const long long unit = slot * 2 * p.Hkv + h, token = unit * p.P + row;
        const int bytes = k <= ARGUS_BF16 ? 2 * D : k <= ARGUS_INT8 ? D : D >> (k - ARGUS_INT8);
        src = r.codes + token * bytes;
        if (k >= ARGUS_INT4_G32) meta = r.meta + token * (D / 32) * 4;
        else if (k >= ARGUS_FP8_E4M3) ks = __ldg(reinterpret_cast<const float*>(r.meta) + unit);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kBatch * 16 / 128; ++i) reinterpret_cast<float4*>(sums)[i * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
    const int t0 = min(max(p.q_start[b], 0), p.total_q), t1 = min(max(p.q_start[b + 1], 0), p.total_q), nq = max(t1 - t0, 0);
    const long long rows = (long long)nq * p.G;
    for (int t = 0; (long long)t * 8 < rows; ++t) {
      for (int i = 0; i < n; ++i) {
        const int k = __shfl_sync(0xffffffffu, codec, i);
        if (k < 0) continue;
        const int form = form_of(k);
        if (have_form != form || have_t != t || have_h != h || have_b != b) {
          have_form = form;
          have_t = t;
          have_h = h;
          have_b = b;
          const long long mine = (long long)t * 8 + (lane >> 2);
          const bool real = mine < rows;
          const int tok = real ? (int)(mine / p.G) : 0, g = real ? (int)(mine - (long long)tok * p.G) : 0;
          load_query<D, BF>(p.q + (t0 + tok) * p.qs + (long long)(h * p.G + g) * D, real, form, lane, q);
          float L = INFINITY;                            // a row that sees nothing gives nothing
          if (real) {
            L = p.lse2[(size_t)(t0 + tok) * p.Hq + h * p.G + g];
            if (L == -INFINITY) L = INFINITY;
          }
          const int last = !real ? -1 : p.causal ? min(len - nq + tok, len - 1) : len - 1;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            lse[x] = __shfl_sync(0xffffffffu, L, 8 * c + 4 * x);
            see[x] = __shfl_sync(0xffffffffu, last, 8 * c + 4 * x);
          }
        }
        const unsigned long long a = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), i);
        const unsigned long long m = form == kGroup ? __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(meta), i) : 0ull;
        const float f = __shfl_sync(0xffffffffu, ks, i) * p.scale_log2;
        float d[4];
        scores<D, BF>(reinterpret_cast<const uint8_t*>(a), reinterpret_cast<const uint8_t*>(m), k, lane, q, d);
        const int key = (c0 + i) * 16 + (lane >> 2);
        float s[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {                    // selected, not multiplied: rows behind the end may hold anything
          const float p0 = key + 8 * x <= see[0] ? fast_exp2(fmaf(d[2 * x], f * q.fac[0], -lse[0])) : 0.f;
          const float p1 = key + 8 * x <= see[1] ? fast_exp2(fmaf(d[2 * x + 1], f * q.fac[1], -lse[1])) : 0.f;
          s[x] = p0 + p1;
          s[x] += __shfl_xor_sync(0xffffffffu, s[x], 1);
          s[x] += __shfl_xor_sync(0xffffffffu, s[x], 2);
        }
        if (c < 2) sums[i * 16 + (lane >> 2) + 8 * c] += c ? s[1] : s[0];
      }
    }
    __syncwarp();
    float* out = p.weights + ((size_t)b * p.Hkv + h) * p.row_len + (size_t)c0 * 16;
    const int keys = min(len - c0 * 16, n * 16);
    for (int i = lane; i < keys; i += 32) {
      float x = sums[i];
      if (p.decay != 0.f) x = fmaf(p.decay, out[i], x);
      out[i] = x;
    }
  }
}

template <int D, bool BF>
static argus_status launch(const WParams& p, cudaStream_t s) {
  const long long chunks = (long long)p.B * p.Hkv * (((long long)p.max_pages * p.P + 15) / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(1ll, std::min(chunks, device_sm_count() * 3ll)));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weights_kernel<D, BF>, p);
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_attn_weights: launch failed: %s", cudaGetErrorString(e));
}

}  // namespace weights
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_attn_weights(const argus_extend_args* a, float* weights, int64_t row_len, float decay, void* stream) {
  if (!a) return fail(ARGUS_E_INVALID, "weights: args is NULL");
  const argus_geom& g = a->g;
  if (g.n_q_heads <= 0 || g.n_kv_heads <= 0 || g.n_q_heads % g.n_kv_heads || g.page_tokens <= 0)
    return fail(ARGUS_E_INVALID, "weights: bad head counts or page_tokens");
  const int D = g.head_dim;
  if (D != 64 && D != 128) return fail(ARGUS_E_UNSUPPORTED, "weights: head_dim %d (supported: 64, 128)", D);
  if (g.n_q_heads / g.n_kv_heads > 8)
    return fail(ARGUS_E_UNSUPPORTED, "weights: %d query heads per KV head (supported: 1..8)", g.n_q_heads / g.n_kv_heads);
  if (g.page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "weights: page_tokens %d not a multiple of 16", g.page_tokens);
  if (a->q_dtype != ARGUS_FP16 && a->q_dtype != ARGUS_BF16) return fail(ARGUS_E_INVALID, "weights: q_dtype must be FP16 or BF16");
  if (a->causal != 0 && a->causal != 1) return fail(ARGUS_E_INVALID, "weights: causal must be 0 or 1");
  if (a->batch < 0 || a->total_q < 0 || a->max_pages < 0 || a->n_pools < 0) return fail(ARGUS_E_INVALID, "weights: negative size");
  if (a->batch > 65535) return fail(ARGUS_E_UNSUPPORTED, "weights: batch %d above 65535", a->batch);
  if ((long long)a->total_q * g.n_q_heads > 0x7fffffffll - 128) return fail(ARGUS_E_UNSUPPORTED, "weights: 2^31 query rows or more");
  const long long positions = (long long)a->max_pages * g.page_tokens;
  if (positions > 0x7fffffffll - 256) return fail(ARGUS_E_UNSUPPORTED, "weights: 2^31 cached tokens per sequence or more");
  if (!(a->softmax_scale >= 0.f) || !std::isfinite(a->softmax_scale))
    return fail(ARGUS_E_INVALID, "weights: softmax_scale must be finite and >= 0");
  if (!std::isfinite(decay)) return fail(ARGUS_E_INVALID, "weights: decay must be finite");
  if (row_len < positions) return fail(ARGUS_E_INVALID, "weights: rows shorter than the cache");
  if (a->n_pools > 0 && !a->pools) return fail(ARGUS_E_INVALID, "weights: pools is NULL");
  weights::WParams p{};
  uint32_t seen = 0;
  for (int i = 0; i < a->n_pools; ++i) {
    const argus_pool& pl = a->pools[i];
    if (pl.codec < 0 || pl.codec > ARGUS_INT1_G32) return fail(ARGUS_E_INVALID, "weights: bad codec %d", pl.codec);
    if (seen >> pl.codec & 1) return fail(ARGUS_E_INVALID, "weights: more than one pool of codec %d", pl.codec);
    seen |= 1u << pl.codec;
    if (pl.codec <= ARGUS_BF16 && pl.codec != a->q_dtype)
      return fail(ARGUS_E_UNSUPPORTED, "weights: 16-bit pages must be of the query's type");
    if (pl.placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "weights: pools must lie in device memory");
    if (pl.n_slots < 0) return fail(ARGUS_E_INVALID, "weights: negative n_slots");
    if (pl.n_slots > 0 && (!pl.codes || (pl.codec >= ARGUS_FP8_E4M3 && !pl.meta)))
      return fail(ARGUS_E_INVALID, "weights: NULL codes or meta (codec %d)", pl.codec);
    if (reinterpret_cast<uintptr_t>(pl.codes) & 15) return fail(ARGUS_E_INVALID, "weights: codes must be 16-byte aligned");
    if (pl.codec >= ARGUS_FP8_E4M3 && (reinterpret_cast<uintptr_t>(pl.meta) & 3))
      return fail(ARGUS_E_INVALID, "weights: meta must be 4-byte aligned");
    p.pool[pl.codec] = {static_cast<const uint8_t*>(pl.codes), static_cast<const uint8_t*>(pl.meta), pl.n_slots};
  }
  if (a->batch == 0 || positions == 0) return ARGUS_OK;
  if (!a->q_start || !a->seq_lens || !weights || !a->page_codec || !a->block_table || (a->total_q > 0 && (!a->q || !a->lse2_out)))
    return fail(ARGUS_E_INVALID, "weights: NULL pointer");
  const long long qs = a->q_stride ? a->q_stride : (long long)g.n_q_heads * D;
  if (qs < (long long)g.n_q_heads * D) return fail(ARGUS_E_INVALID, "weights: q_stride is smaller than a token");
  if (qs & 7) return fail(ARGUS_E_INVALID, "weights: q_stride must be a multiple of 8 elements");
  if (reinterpret_cast<uintptr_t>(a->q) & 15) return fail(ARGUS_E_INVALID, "weights: q must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(a->lse2_out)) & 3)
    return fail(ARGUS_E_INVALID, "weights: weights and lse2 must be 4-byte aligned");
  // positions are written while others' queries and sums are read
  const uintptr_t w0 = reinterpret_cast<uintptr_t>(weights), w1 = w0 + (uintptr_t)a->batch * g.n_kv_heads * row_len * 4;
  const auto over = [&](const void* x, unsigned long long bytes) {
    const uintptr_t y = reinterpret_cast<uintptr_t>(x);
    return y && bytes && w0 < y + bytes && y < w1;
  };
  const unsigned long long tokens = a->total_q, entries = (unsigned long long)a->batch * a->max_pages;
  if (over(a->q, tokens ? 2 * ((tokens - 1) * qs + (long long)g.n_q_heads * D) : 0) || over(a->lse2_out, 4 * tokens * g.n_q_heads) ||
      over(a->q_start, 4ull * a->batch + 4) || over(a->seq_lens, 4ull * a->batch) || over(a->page_codec, entries) || over(a->block_table, 4 * entries))
    return fail(ARGUS_E_INVALID, "weights: weights overlaps an input");
  p.Hq = g.n_q_heads;
  p.Hkv = g.n_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.P = g.page_tokens;
  p.B = a->batch;
  p.total_q = a->total_q;
  p.causal = a->causal;
  p.max_pages = a->max_pages;
  p.q = static_cast<const uint16_t*>(a->q);
  p.qs = qs;
  p.q_start = a->q_start;
  p.seq_lens = a->seq_lens;
  p.page_codec = a->page_codec;
  p.block_table = a->block_table;
  p.lse2 = a->lse2_out;
  p.weights = weights;
  p.row_len = row_len;
  p.decay = decay;
  p.scale_log2 = (float)((double)a->softmax_scale * 1.4426950408889634);
  p.status = a->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = a->q_dtype == ARGUS_BF16;
  if (D == 64) return bf ? weights::launch<64, true>(p, s) : weights::launch<64, false>(p, s);
  return bf ? weights::launch<128, true>(p, s) : weights::launch<128, false>(p, s);
}
