// argus_rope_append: rotary positions (one or several axes) on the new tokens'
// queries and keys, and the append of keys and values to the paged cache; and
// argus_norm_rope_append, which norms the queries and keys of each head first.
//
// Mathematics: pair i of a token turns by a = pos[axis(i)] * inv_freq[i].  Only
// a mod 2 pi matters, and at a far position the product has no fraction left in
// fp32 (position 10^6 times 1 rad is known to 0.06 rad).  So the frequency is
// taken in turns, as a 64-bit fixed-point fraction F = frac(inv_freq / 2 pi) 2^64
// (off by at most 1 for frequencies below 2^40), and pos * F in wrapping 64-bit integers
// IS the angle modulo one turn: off by at most 2^-33 of a turn at position 2^31.
// sincospif of twice the signed fraction follows.
//
// What bounds it: bytes (q, k, v read, q', k', v written once).  A token is
// taken by a group of W warps (W = 1 when there are many tokens, up to 8 when there
// are few), which loop over tokens.  Each block turns the frequencies into fixed
// point once; a warp computes a token's sines and cosines into
// shared memory of its own (no block barrier), and uses them for all Hq + Hkv heads; a lane moves
// two 16-byte vectors per item, the two that hold a pair's halves, four items in flight.
//
// Measured (GB300, CUDA events, buffers rotated past the L2): two video prompts of 52,768
// tokens together, 14/2 heads of 64, three axes: 54 us, 4.5 TB/s (66% of a plain copy);
// five prompts of 777 to 2,048 tokens, 32/8 heads of 128: 35 us, 5.1 TB/s (75%); a
// decode step of 32 rows: 4.4 us in a graph (7.9 with the L2 flushed, with norms 8.6), its launch and two dependent reads.  Warps on
// runs of neighbouring tokens (sequence and page looked up once) were no faster, nor
// sines and cosines kept in registers: 36 and 52 us at best, with more registers.
//
// The norm, y = x w / sqrt(mean x^2 + eps) over a head's D elements, is one more
// value per head: an item's sum of squares goes around the D / 16 neighbouring lanes that
// hold the head, in fp32, between the loads and the rotation; nothing is read twice and
// nothing rounded in between.  Six prompts of 777 to 2,500 tokens, 32/4 heads of 128: 46 us, 4.4 TB/s (65% of
// a copy): latency, with half of the issue slots used and a third of the warps there; with four items in flight, as
// without norms, two blocks fit an SM: 69 us.
#include <algorithm>
#include <cmath>

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
  const float *q_weight, *k_weight;  // [D] or NULL (ones)
  float eps_4;                       // a quarter of eps: its sum with a quarter of the mean stays in fp32's range
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

// The last sequence that starts at or before token t, by a whole warp: 32
// candidates per step.
__device__ __forceinline__ int seq_of(const RParams& p, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.B;               // it is one of lo .. lo + n - 1, if any is
  while (n > 1) {
    const int step = (n + 31) / 32, b = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && p.q_start[b] <= t);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// frac(f / 2 pi) 2^64.  The product with 1 / (2 pi) has 106 bits, in two doubles: the
// fraction of one double would be off by 2^-54 of the product itself, and a
// position multiplies that.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / (2 pi), its first 53 bits and the next 53
  const double hi = f * kHi, lo = fma(f, kHi, -hi) + f * kLo;
  return __double2ull_rn((hi - floor(hi)) * 0x1p64) + (unsigned long long)__double2ll_rn((lo - rint(lo)) * 0x1p64);
}

template <bool BF>
__device__ __forceinline__ void turn_pair(uint4& a4, uint4& b4, const float* cs, const float* sn, int u, bool adjacent) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&a4);
  uint32_t* b = reinterpret_cast<uint32_t*>(&b4);
  const float4 c0 = *reinterpret_cast<const float4*>(cs + 8 * u), c1 = *reinterpret_cast<const float4*>(cs + 8 * u + 4);
  const float4 s0 = *reinterpret_cast<const float4*>(sn + 8 * u), s1 = *reinterpret_cast<const float4*>(sn + 8 * u + 4);
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = unpack2<BF>(a[j]), y = unpack2<BF>(b[j]);
    if (adjacent) {
      a[j] = pack2<BF>(x.x * c[j] - x.y * s[j], x.y * c[j] + x.x * s[j]);
      b[j] = pack2<BF>(y.x * c[4 + j] - y.y * s[4 + j], y.y * c[4 + j] + y.x * s[4 + j]);
    } else {
      a[j] = pack2<BF>(x.x * c[2 * j] - y.x * s[2 * j], x.y * c[2 * j + 1] - y.y * s[2 * j + 1]);
      b[j] = pack2<BF>(y.x * c[2 * j] + x.x * s[2 * j], y.y * c[2 * j + 1] + x.y * s[2 * j + 1]);
    }
  }
}

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight eight(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The same two vectors by their norm: r = 1 / sqrt(mean + eps) of the head (its values times `pre`, if `far`), wa and wb
// the weights of their elements; turned by the pairs of item u unless u < 0.
template <bool BF>
__device__ __forceinline__ void norm_pair(uint4& a4, uint4& b4, bool far, float pre, float r, const float* wa, const float* wb, const float* cs,
                                          const float* sn, int u, bool adjacent) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&a4);
  uint32_t* b = reinterpret_cast<uint32_t*>(&b4);
  float x[8], y[8];
  const Eight v = eight(wa), w = eight(wb);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = unpack2<BF>(a[j]), q = unpack2<BF>(b[j]);
    x[2 * j] = p.x;
    x[2 * j + 1] = p.y;
    y[2 * j] = q.x;
    y[2 * j + 1] = q.y;
  }
  if (BF && far) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] *= pre;
      y[j] *= pre;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {                       // r first: it brings the values to a few units
    f2_mul(x[j], x[j + 1], x[j], x[j + 1], r, r);
    f2_mul(y[j], y[j + 1], y[j], y[j + 1], r, r);
    f2_mul(x[j], x[j + 1], x[j], x[j + 1], v.v[j], v.v[j + 1]);
    f2_mul(y[j], y[j + 1], y[j], y[j + 1], w.v[j], w.v[j + 1]);
  }
  if (u >= 0) {
    const Eight c = eight(cs + 8 * u), s = eight(sn + 8 * u);
    if (adjacent) {                                      // pairs of neighbours, four in each vector
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = x[2 * j], q = y[2 * j];
        x[2 * j] = p * c.v[j] - x[2 * j + 1] * s.v[j];
        x[2 * j + 1] = x[2 * j + 1] * c.v[j] + p * s.v[j];
        y[2 * j] = q * c.v[4 + j] - y[2 * j + 1] * s.v[4 + j];
        y[2 * j + 1] = y[2 * j + 1] * c.v[4 + j] + q * s.v[4 + j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float t[2], z[2];
        f2_mul(t[0], t[1], y[j], y[j + 1], s.v[j], s.v[j + 1]);
        f2_mul(z[0], z[1], x[j], x[j + 1], s.v[j], s.v[j + 1]);
        f2_mul(x[j], x[j + 1], x[j], x[j + 1], c.v[j], c.v[j + 1]);
        f2_sub(x[j], x[j + 1], x[j], x[j + 1], t[0], t[1]);
        f2_fma(y[j], y[j + 1], y[j], y[j + 1], c.v[j], c.v[j + 1], z[0], z[1]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = pack2<BF>(x[2 * j], x[2 * j + 1]);
    b[j] = pack2<BF>(y[2 * j], y[2 * j + 1]);
  }
}

template <bool BF>
__device__ __forceinline__ float squares(const uint4& a4, bool far, float pre) {
  const uint32_t* a = reinterpret_cast<const uint32_t*>(&a4);
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 x = unpack2<BF>(a[j]);
    if (far) x = make_float2(x.x * pre, x.y * pre);
    f2_fma(s0, s1, x.x, x.y, x.x, x.y, s0, s1);
  }
  return s0 + s1;
}

template <int D, bool BF, bool NORM>
__device__ __forceinline__ void rope_tokens(const RParams& p, int W) {
  __shared__ __align__(16) float s_cs[kThreads / 32][2][D / 2];
  __shared__ unsigned long long s_freq[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* cs = s_cs[warp][0];
  float* sn = s_cs[warp][1];
  const int gw = blockIdx.x * (kThreads / 32) + warp, part = gw % W, groups = gridDim.x * (kThreads / 32) / W;
  // this lane's frequencies, pairs lane and lane + 32, as fractions of a turn: found
  // once per block, as double precision runs at a few results per cycle and SM (in
  // every warp it took 2 us)
  __shared__ __align__(16) float s_weight[NORM ? 2 : 1][NORM ? D : 4];
  if (NORM && threadIdx.x < 2 * D) {
    const float* w = threadIdx.x < D ? p.q_weight : p.k_weight;
    s_weight[threadIdx.x / D][threadIdx.x % D] = w ? w[threadIdx.x % D] : 1.f;
  }
  if (threadIdx.x < p.rot / 2) s_freq[threadIdx.x] = turn_fraction(p.inv_freq[threadIdx.x]);
  __syncthreads();
  constexpr int N = D / 64;
  unsigned long long freq[N];
  int axis[N];
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const int i = lane + 32 * x;
    freq[x] = 0;
    axis[x] = 0;
    if (i < p.rot / 2) {
      freq[x] = s_freq[i];
      if (p.pair_axis) axis[x] = p.pair_axis[i];
    }
  }
  bool bad_axis = false;
#pragma unroll
  for (int x = 0; x < N; ++x) bad_axis |= axis[x] >= p.n_axes;
  bad_axis = __any_sync(0xffffffffu, bad_axis);
  constexpr int U = D / 16;          // items of 16 elements (two vectors) per head
  const int n_items = (p.Hq + 2 * p.Hkv) * U, ru = p.rot / 16;

  for (int t = gw / W; t < p.total; t += groups) {
    int pos[N];
#pragma unroll
    for (int x = 0; x < N; ++x) pos[x] = axis[x] < p.n_axes ? p.pos[(size_t)axis[x] * p.total + t] : 0;
    const int b = seq_of(p, t), start = max(p.q_start[b], 0), end = min(p.q_start[b + 1], p.total);   // 0 <= t < total between
    if (t < start || t >= end) continue;                 // a row of no sequence
    const long long c = (long long)p.seq_lens[b] - (end - start) + (t - start);
    long long slot = -1;
    int row = 0;
    if (c >= 0 && c < (long long)p.max_pages * p.P) {
      const int page = (int)((unsigned long long)c / (unsigned)p.P);
      row = (int)(c - (long long)page * p.P);
      const size_t e = (size_t)b * p.max_pages + page;
      if (p.page_codec[e] == p.codec) slot = p.block_table[e];
      if (slot >= p.n_slots) slot = -1;
    }
    if (part == 0 && lane == 0 && p.status && (slot < 0 || bad_axis)) atomicAdd(p.status, (slot < 0) + bad_axis);
    __syncwarp();                                        // the token before has been read
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int i = lane + 32 * x;
      if (i < p.rot / 2) {
        const unsigned long long turn = (unsigned long long)(long long)pos[x] * freq[x];
        float s, co;
        sincospif((float)(long long)turn * 1.0842021724855044e-19f, &s, &co);   // 2^-63: half turns
        cs[i] = co;
        sn[i] = s;
      }
    }
    __syncwarp();
    uint16_t* page = p.codes + (size_t)(slot < 0 ? 0 : slot) * 2 * p.Hkv * p.P * D + (size_t)row * D;
    constexpr int M = NORM ? 2 : 4;                      // items in flight: what three blocks per SM have registers for
    for (int it0 = part * 32 + lane; it0 - (NORM ? lane : 0) < n_items; it0 += 32 * W * M) {   // NORM: by whole warps
      uint4 a[M], bb[M];
      uint16_t* dst[M];
      int un[M];                                         // >= 0: turned, with these pairs
      int hw[M];                                         // NORM: 0 a query's head, 1 a key's, else V's
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int it = it0 + m * 32 * W;
        dst[m] = nullptr;
        if (NORM) {
          hw[m] = 2;
          a[m] = bb[m] = make_uint4(0, 0, 0, 0);
        }
        if (it >= n_items) continue;
        const int head = it / U, u = it % U;
        const bool turned = u < ru && head < p.Hq + p.Hkv, halves = turned && !p.adjacent;
        un[m] = turned ? u : -1;
        if (NORM) hw[m] = head < p.Hq ? 0 : head < p.Hq + p.Hkv ? 1 : 2;
        const int e0 = halves ? 8 * u : 16 * u, e1 = halves ? p.rot / 2 + 8 * u : 16 * u + 8;
        const uint16_t* src;
        if (head < p.Hq) {
          src = p.q + t * p.qs + head * D;
          dst[m] = p.q_out + t * p.qos + head * D + e0;
        } else {
          const bool is_v = head >= p.Hq + p.Hkv;
          const int h = head - p.Hq - (is_v ? p.Hkv : 0);
          src = is_v ? p.v + t * p.vs + h * D : p.k + t * p.ks + h * D;
          if (slot >= 0) dst[m] = page + (size_t)(head - p.Hq) * p.P * D + e0;   // K heads, then V heads
        }
        a[m] = *reinterpret_cast<const uint4*>(src + e0);
        bb[m] = *reinterpret_cast<const uint4*>(src + e1);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float pre = 1.f, ss = squares<BF>(a[m], false, 1.f) + squares<BF>(bb[m], false, 1.f);
#pragma unroll
          for (int o = 1; o < U; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const bool far = BF && __any_sync(0xffffffffu, ss > 3e38f);   // squares beyond fp32's range (bf16 reaches as far as fp32)
          if (far) {
            float less = squares<BF>(a[m], true, 0x1p-70f) + squares<BF>(bb[m], true, 0x1p-70f);
#pragma unroll
            for (int o = 1; o < U; o *= 2) less += __shfl_xor_sync(0xffffffffu, less, o);
            if (ss > 3e38f) {
              ss = less;
              pre = 0x1p-70f;
            }
          }
          if (hw[m] < 2) {
            const int u = (it0 + m * 32 * W) % U;
            const bool halves = un[m] >= 0 && !p.adjacent;
            const float* w = s_weight[hw[m]];
            norm_pair<BF>(a[m], bb[m], far, pre, 0.5f * rsqrtf(ss * (0.25f / D) + (pre == 1.f ? p.eps_4 : p.eps_4 * 0x1p-140f)), w + (halves ? 8 : 16) * u,
                          w + (halves ? p.rot / 2 + 8 * u : 16 * u + 8), cs, sn, un[m], p.adjacent);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (!dst[m]) continue;
        if (!NORM && un[m] >= 0) turn_pair<BF>(a[m], bb[m], cs, sn, un[m], p.adjacent);
        *reinterpret_cast<uint4*>(dst[m]) = a[m];
        *reinterpret_cast<uint4*>(dst[m] + ((un[m] >= 0 && !p.adjacent) ? p.rot / 2 : 8)) = bb[m];
      }
    }
  }
}

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RParams p, int W) { rope_tokens<D, BF, false>(p, W); }
template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const RParams p, int W) { rope_tokens<D, BF, true>(p, W); }

template <int D, bool BF, bool NORM>
static argus_status launch(const RParams& p, cudaStream_t s) {
  constexpr int kWarps = kThreads / 32;
  const long long sms = device_sm_count();
  // warps per token: enough of them for every SM to hold some, no more than have an item each
  const int items = (p.Hq + 2 * p.Hkv) * (D / 16);
  int W = 1;
  while (W < kWarps && (long long)p.total * W < sms * 16 && 32 * W < items) W *= 2;
  const long long blocks = ((long long)p.total * W + kWarps - 1) / kWarps;
  // three blocks are resident per SM at this register count
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((int)std::min(blocks, sms * 3));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, NORM ? norm_rope_kernel<D, BF> : rope_kernel<D, BF>, p, W);
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_%srope_append: launch failed: %s", NORM ? "norm_" : "", cudaGetErrorString(e));
}

// Whether two tensors of n tokens share memory: tokens of la and lb bytes, sa >= la and
// sb >= lb bytes apart, from a and from b on.
static bool tokens_meet(uintptr_t a, long long la, long long sa, uintptr_t b, long long lb, long long sb, long long n) {
  typedef __int128 wide;
  const wide d = (wide)b - (wide)a;                    // token i of one meets token j of the other: -lb < d + j sb - i sa < la
  if (d >= (n - 1) * (wide)sa + la || -d >= (n - 1) * (wide)sb + lb) return false;
  if (sa == sb) {                                      // (slices of one buffer's rows): for some k = i - j, d - la < k s < d + lb
    const wide low = d - la;
    wide k = (low >= 0 ? low / sa : -((-low + sa - 1) / sa)) + 1;
    if (k < 1 - n) k = 1 - n;
    return k <= n - 1 && k * sa < d + lb;
  }
  for (long long i = 0, j = 0; i < n && j < n;) {      // the one that ends first meets none behind the other's
    const wide gap = d + j * (wide)sb - i * (wide)sa;
    if (gap >= la) ++i;
    else if (gap <= -lb) ++j;
    else return true;
  }
  return false;
}

// The arguments that both forms share, checked and brought into the kernel's form; p.total stays 0
// where there is nothing to do.
static argus_status params(const argus_rope_args* a, RParams& p) {
  if (!a) return fail(ARGUS_E_INVALID, "rope: args is NULL");
  const argus_geom& g = a->g;
  if (g.n_q_heads <= 0 || g.n_kv_heads <= 0 || g.n_q_heads % g.n_kv_heads || g.page_tokens <= 0)
    return fail(ARGUS_E_INVALID, "rope: bad head counts or page_tokens");
  if (g.head_dim != 64 && g.head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "rope: head_dim %d (supported: 64, 128)", g.head_dim);
  if (g.page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "rope: page_tokens %d not a multiple of 16", g.page_tokens);
  if (a->dtype != ARGUS_FP16 && a->dtype != ARGUS_BF16) return fail(ARGUS_E_INVALID, "rope: dtype must be FP16 or BF16");
  if (a->batch < 0 || a->total_q < 0 || a->max_pages < 0) return fail(ARGUS_E_INVALID, "rope: negative size");
  if (a->n_axes < 1 || a->n_axes > kMaxAxes) return fail(ARGUS_E_INVALID, "rope: n_axes %d not in 1..4", a->n_axes);
  if (a->adjacent != 0 && a->adjacent != 1) return fail(ARGUS_E_INVALID, "rope: adjacent must be 0 or 1");
  if (a->rot_dim <= 0 || a->rot_dim > g.head_dim) return fail(ARGUS_E_INVALID, "rope: rot_dim %d not in 1..head_dim", a->rot_dim);
  if (a->rot_dim % 16) return fail(ARGUS_E_UNSUPPORTED, "rope: rot_dim %d not a multiple of 16", a->rot_dim);
  if (a->batch == 0 || a->total_q == 0) return ARGUS_OK;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->positions || !a->inv_freq || !a->q_start || !a->seq_lens || !a->pool)
    return fail(ARGUS_E_INVALID, "rope: NULL pointer");
  if (a->max_pages > 0 && (!a->page_codec || !a->block_table)) return fail(ARGUS_E_INVALID, "rope: NULL page_codec or block_table");
  if (a->pool->codec != a->dtype) return fail(ARGUS_E_UNSUPPORTED, "rope: the pool's codec %d is not the tokens' type", a->pool->codec);
  if (a->pool->placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "rope: the pool must lie in device memory");
  if (a->pool->n_slots < 0 || (a->pool->n_slots > 0 && !a->pool->codes)) return fail(ARGUS_E_INVALID, "rope: bad pool");
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
  // a token is turned while others are still read
  const auto over = [&](const void* x, int heads, long long stride) {
    return tokens_meet(reinterpret_cast<uintptr_t>(a->q_out), 2ll * p.Hq * D, 2 * p.qos, reinterpret_cast<uintptr_t>(x), 2ll * heads * D,
                             2 * stride, a->total_q);
  };
  if ((a->q_out != a->q && over(a->q, p.Hq, p.qs)) || over(a->k, p.Hkv, p.ks) || over(a->v, p.Hkv, p.vs))
    return fail(ARGUS_E_INVALID, "rope: q_out overlaps the tokens of q, k or v");
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
  return ARGUS_OK;
}

template <bool NORM>
static argus_status run(const argus_rope_args* a, const RParams& p, void* stream) {
  if (p.total == 0) return ARGUS_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = a->dtype == ARGUS_BF16;
  if (a->g.head_dim == 64) return bf ? launch<64, true, NORM>(p, s) : launch<64, false, NORM>(p, s);
  return bf ? launch<128, true, NORM>(p, s) : launch<128, false, NORM>(p, s);
}

}  // namespace rope
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_rope_append(const argus_rope_args* a, void* stream) {
  rope::RParams p{};
  const argus_status st = rope::params(a, p);
  return st != ARGUS_OK ? st : rope::run<false>(a, p, stream);
}

extern "C" argus_status argus_norm_rope_append(const argus_rope_args* a, const float* q_weight, const float* k_weight, float eps, void* stream) {
  rope::RParams p{};
  const argus_status st = rope::params(a, p);
  if (st != ARGUS_OK) return st;
  // below 2^-100 squares that fp32 cannot hold would count beside it
  if (!(eps >= 0x1p-100f) || !std::isfinite(eps)) return fail(ARGUS_E_INVALID, "rope: eps must be finite and at least 2^-100");
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 3)
    return fail(ARGUS_E_INVALID, "rope: the norms' weights must be 4-byte aligned");
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps_4 = 0.25f * eps;
  return rope::run<true>(a, p, stream);
}
