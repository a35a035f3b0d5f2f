// argus_evict_tokens: the cached positions of least accumulated attention weight dropped, the
// rest gathered into new pages.
//
// Mathematics: of a sequence of L positions and one KV head, the first S and the last R stay, and
// of those between the k = budget - S - R of largest weight, ties to the lower position.
// Floats are mapped to integers of the same order (NaN below all, -0 = +0); the k-th largest
// key T is found bit by bit, two at a time: with c_d keys at or above each of the three next
// digits, the largest d with c_d >= k is T's.  Where a count is k exactly, the search ends.
// Positions above T stay, and of those at T the first k - #(above T).
//
// Selection: a thread block (or a cluster of them for long rows) per sequence and KV head holds
// the keys in registers, read once; a round is three compares a key, a reduction within
// the warps and one over them.  A warp's positions are neighbours, so the ranks that put the kept
// ones in order are ballots and one scan over the warps.
//
// Gathering: a warp takes 16 rows of a new page and KV head, looks their places up at once
// and has K's (then V's) 16-byte vectors on their way together.  8-bit pages have one scale
// per page, KV head and K | V: a team of warps shares the page's largest magnitude.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace argus {
namespace evict {

namespace cg = cooperative_groups;

struct PoolRef {
  const uint8_t* codes;
  const uint8_t* meta;
  long long n_slots;
};

struct VParams {
  int Hkv, P, B, max_pages, budget, sinks, recent, dst_codec, dst_pages;
  PoolRef pool[7];
  const uint8_t* page_codec;
  const int32_t *block_table, *seq_lens;
  const float* weights;
  long long row_len, row_len_out;
  uint8_t* dst_codes;
  float* dst_meta;
  long long dst_slots;
  const int32_t* dst_table;
  int32_t* seq_lens_out;
  int32_t* kept;
  float* weights_out;
  uint32_t* status;
};

__device__ __forceinline__ int length(const VParams& p, int b) {
  return (int)min((long long)max(p.seq_lens[b], 0), (long long)p.max_pages * p.P);
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kRegKeys = 32;           // keys per thread that stay in registers, at most
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t order(float w) {
  const uint32_t u = __float_as_uint(w);
  if (w != w) return 0u;
  if (w == 0.f) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct Counts {
  uint32_t a, b, c;
};
__device__ __forceinline__ Counts warp_sum(Counts x) {
  x.a = __reduce_add_sync(0xffffffffu, x.a);
  x.b = __reduce_add_sync(0xffffffffu, x.b);
  x.c = __reduce_add_sync(0xffffffffu, x.c);
  return x;
}

// KEYS: a thread's keys, which stay in registers; 0: they are read again in every round.
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const VParams p) {
  __shared__ Counts s_warp[2][kSelWarps];
  __shared__ Counts s_block[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x;          // the cluster spans the grid's first dimension
  const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)b * p.Hkv + h;
  const float* w = p.weights + row * p.row_len;
  int32_t* kept = p.kept + row * p.budget;
  const int len = length(p, b), m = min(len, p.budget);
  if (threadIdx.x == 0 && rank == 0 && h == 0) p.seq_lens_out[b] = m;
  // behind the kept positions
  const int tid = rank * kSelThreads + threadIdx.x, all = C * kSelThreads;
  for (int i = m + tid; i < p.budget; i += all) kept[i] = -1;
  float* w_out = p.weights_out + row * p.row_len_out;
  for (long long i = m + tid; i < p.row_len_out; i += all) w_out[i] = 0.f;
  if (len <= p.budget) {                               // the same in the whole cluster
    for (int i = tid; i < m; i += all) kept[i] = i;
    return;
  }
  const int lo = p.sinks, hi = len - p.recent, k = p.budget - p.sinks - p.recent;   // candidates lo .. hi-1: more than k
  // this warp's positions: steps of 32 neighbours
  const long long all_steps = (long long)C * kSelThreads;
  const int steps = KEYS > 0 ? KEYS : (int)((len + all_steps - 1) / all_steps);
  const long long start = ((long long)rank * kSelWarps + warp) * steps * 32 + lane;
  auto load = [&](int i) -> float {                    // NaN (below all) for what is not a candidate
    const long long pos = start + i * 32ll;
    return pos >= lo && pos < hi ? __ldg(w + pos) : __uint_as_float(0x7FC00000u);
  };
  uint32_t key[KEYS > 0 ? KEYS : 1];
  if constexpr (KEYS > 0) {
    float x[KEYS];                                     // all on their way at once
#pragma unroll
    for (int i = 0; i < KEYS; ++i) x[i] = load(i);
#pragma unroll
    for (int i = 0; i < KEYS; ++i) key[i] = order(x[i]);
  }
  auto each = [&](auto f) {
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) f(i, key[i]);
    } else {
      for (int i = 0; i < steps; ++i) f(i, order(load(i)));
    }
  };
  int turn = 0;
  // sums over the cluster; with `before`, those over the warps in front of this one too
  auto total = [&](Counts x, Counts* before) {
    const int t = turn;
    turn ^= 1;                                         // the other buffer may still be read
    if (lane == 0) s_warp[t][warp] = x;
    __syncthreads();
    Counts y = s_warp[t][lane];
    Counts in = {0, 0, 0};
    if (before) {
      in = {lane < warp ? y.a : 0, lane < warp ? y.b : 0, lane < warp ? y.c : 0};
      in = warp_sum(in);
    }
    y = warp_sum(y);
    if (C > 1) {
      if (threadIdx.x == 0) s_block[t] = y;
      cluster.sync();
      Counts z = {0, 0, 0};
      if (lane < C) z = *cluster.map_shared_rank(&s_block[t], lane);
      if (before) {
        const bool f = lane < rank;
        const Counts g = warp_sum({f ? z.a : 0, f ? z.b : 0, f ? z.c : 0});
        in = {in.a + g.a, in.b + g.b, in.c + g.c};
      }
      y = warp_sum(z);
    }
    if (before) *before = in;
    return y;
  };
  uint32_t T = 0xFFFFFFFFu, ties = 0;                  // keys above T stay, and the first `ties` at T
  if (k > 0) {
    uint32_t prefix = 0, upper = 0;                    // keys at or above the prefix's successor
    bool exact = false;
    for (int s = 30; s >= 0; s -= 2) {
      const uint32_t t1 = prefix | (1u << s), t2 = prefix | (2u << s), t3 = prefix | (3u << s);
      Counts c = {0, 0, 0};
      each([&](int, uint32_t x) {
        c.a += x >= t1;
        c.b += x >= t2;
        c.c += x >= t3;
      });
      c = total(warp_sum(c), nullptr);
      uint32_t at;                                     // keys at or above the new prefix
      if (c.c >= (uint32_t)k) { prefix = t3; at = c.c; }
      else if (c.b >= (uint32_t)k) { prefix = t2; upper = c.c; at = c.b; }
      else if (c.a >= (uint32_t)k) { prefix = t1; upper = c.b; at = c.a; }
      else { upper = c.a; at = 0; }                    // the count at the old prefix: not k, or the search had ended
      if (at == (uint32_t)k) { exact = true; break; }
    }
    T = prefix;
    ties = exact ? 0xFFFFFFFFu : (uint32_t)k - upper;
  }
  auto stays = [&](int i, uint32_t x, bool& tie) {
    const long long pos = start + i * 32ll;
    const bool mid = pos >= lo && pos < hi;
    tie = mid && x == T && ties > 0;
    return (pos < lo || (pos >= hi && pos < len)) || (mid && x > T);
  };
  Counts mine = {0, 0, 0};
  each([&](int i, uint32_t x) {
    bool tie;
    const bool stay = stays(i, x, tie);
    mine.a += __popc(__ballot_sync(0xffffffffu, stay));
    mine.b += __popc(__ballot_sync(0xffffffffu, tie));
  });
  Counts before;
  total(mine, &before);
  uint32_t at = before.a + min(before.b, ties), tied = before.b;
  const uint32_t lt = (1u << lane) - 1;
  each([&](int i, uint32_t x) {
    bool tie;
    const bool stay = stays(i, x, tie);
    const uint32_t eq = __ballot_sync(0xffffffffu, tie);
    const bool keep = stay || (tie && tied + __popc(eq & lt) < ties);
    const uint32_t mask = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      kept[at + __popc(mask & lt)] = (int32_t)(start + i * 32ll);
    }
    at += __popc(mask);
    tied += __popc(eq);
  });
  if (C > 1) cluster.sync();                           // the others may still read this block's sums
}

// ---------------------------------------------------------------- gathering
constexpr int kWarps = 8;

// 16 values of a row, as they lie in the page; in a 16-bit page 32 bytes, else 16 at most and
// the scale (and zero).
template <bool WIDE>
struct Raw {
  uint4 a;
  uint4 b;
};
template <>
struct Raw<false> {
  uint4 a;
  uint32_t s;
};

template <bool BF>
__device__ __forceinline__ float2 two(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// Where a kept row lies: its unit (slot, K | V, KV head), the row in it, its codec (-1: nowhere).
struct Place {
  long long unit;
  int row, codec;
};

template <int D, bool WIDE>
__device__ __forceinline__ Raw<WIDE> fetch(const VParams& p, const Place& s, int kv, int v) {
  Raw<WIDE> r = {};
  uint32_t scale = 0;
  if (s.codec < 0) return r;
  const long long at = ((s.unit + (kv ? p.Hkv : 0)) * p.P + s.row) * D + 16 * v;   // in values
  const uint8_t* c = p.pool[s.codec].codes;
  if constexpr (WIDE) {
    if (s.codec <= ARGUS_BF16) {
      r.a = __ldg(reinterpret_cast<const uint4*>(c + 2 * at));
      r.b = __ldg(reinterpret_cast<const uint4*>(c + 2 * at) + 1);
      return r;
    }
  }
  if (s.codec <= ARGUS_INT8) {
    r.a = __ldg(reinterpret_cast<const uint4*>(c + at));
    scale = __ldg(reinterpret_cast<const uint32_t*>(p.pool[s.codec].meta) + s.unit + (kv ? p.Hkv : 0));
  } else {
    if (s.codec == ARGUS_INT4_G32) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(c + at / 2));
      r.a.x = x.x;
      r.a.y = x.y;
    } else if (s.codec == ARGUS_INT2_G32) {
      r.a.x = __ldg(reinterpret_cast<const uint32_t*>(c + at / 4));
    } else {
      r.a.x = __ldg(reinterpret_cast<const uint16_t*>(c + at / 8));
    }
    scale = __ldg(reinterpret_cast<const uint32_t*>(p.pool[s.codec].meta) + at / 32);   // scale, zero
  }
  if constexpr (WIDE) r.b.x = scale;
  else r.s = scale;
  return r;
}

template <bool WIDE>
__device__ __forceinline__ void values(const Raw<WIDE>& r, int codec, float (&x)[16]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  uint32_t scale;
  if constexpr (WIDE) {
    scale = r.b.x;
    if (codec == ARGUS_FP16 || codec == ARGUS_BF16) {
      const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 y = codec == ARGUS_BF16 ? two<true>(u[i]) : two<false>(u[i]);
        x[2 * i] = y.x;
        x[2 * i + 1] = y.y;
      }
      return;
    }
  } else {
    scale = r.s;
  }
  if (codec == ARGUS_FP8_E4M3) {
    const float s = __uint_as_float(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = two<false>(e4m3x2_to_f16x2(w[i / 2] >> (16 * (i & 1))));
      f2_mul(x[2 * i], x[2 * i + 1], y.x, y.y, s, s);
    }
  } else if (codec == ARGUS_INT8) {
    const float s = __uint_as_float(scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = (float)(int8_t)(w[i / 4] >> (8 * (i & 3))) * s;
  } else if (codec > 0) {
    const float2 sz = two<false>(scale);
    const int bits = codec == ARGUS_INT4_G32 ? 4 : codec == ARGUS_INT2_G32 ? 2 : 1;
    const unsigned long long q = (unsigned long long)w[1] << 32 | w[0];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf((float)((uint32_t)(q >> (bits * i)) & ((1u << bits) - 1)), sz.x, sz.y);   // the product is exact
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
}

// The largest magnitude of 16 values.  Of an e4m3 row it is the largest code's: a product with
// the same scale keeps the order.
template <bool WIDE>
__device__ __forceinline__ float largest(const Raw<WIDE>& r, int codec) {
  float top = 0.f;
  if (codec == ARGUS_FP8_E4M3) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    __half2 m = __float2half2_rn(0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t y = e4m3x2_to_f16x2(w[i / 2] >> (16 * (i & 1)));
      m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&y)));
    }
    uint32_t scale;
    if constexpr (WIDE) scale = r.b.x;
    else scale = r.s;
    top = fabsf(fmaxf(__low2float(m), __high2float(m)) * __uint_as_float(scale));
  } else {
    float x[16];
    values(r, codec, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
  }
  return top;
}

// Four codes of y = RN(x / scale).  x times the reciprocal is off by at most 3 2^-24 of y, so
// y lies between x rcp (1 - 2^-21) and x rcp (1 + 2^-21); both codes are formed, and as
// encoding keeps the order, y's is theirs where they agree.
template <int DST>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (DST == ARGUS_FP8_E4M3) return f32x2_to_e4m3x2(a, b) | f32x2_to_e4m3x2(c, d) << 16;
  const float x[4] = {a, b, c, d};
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) o |= ((uint32_t)(int)fminf(fmaxf(rintf(x[j]), -127.f), 127.f) & 0xFFu) << (8 * j);
  return o;
}
template <int DST>
__device__ __forceinline__ uint4 encode(const float (&x)[16], float scale) {
  uint32_t o[4] = {0, 0, 0, 0};
  if (scale > 0.f) {
    const float rcp = 1.f / scale, lo = rcp * (1.f - 0x1p-21f), hi = rcp * (1.f + 0x1p-21f);
    bool same = scale >= 0x1p-120f && scale <= 0x1p120f;   // outside the reciprocal could lose bits
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a[4], b[4];
      f2_mul(a[0], a[1], x[4 * e], x[4 * e + 1], lo, lo);
      f2_mul(a[2], a[3], x[4 * e + 2], x[4 * e + 3], lo, lo);
      f2_mul(b[0], b[1], x[4 * e], x[4 * e + 1], hi, hi);
      f2_mul(b[2], b[3], x[4 * e + 2], x[4 * e + 3], hi, hi);
      o[e] = encode4<DST>(a[0], a[1], a[2], a[3]);
      same &= o[e] == encode4<DST>(b[0], b[1], b[2], b[3]);
    }
    if (!same) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = encode4<DST>(x[4 * e] / scale, x[4 * e + 1] / scale, x[4 * e + 2] / scale, x[4 * e + 3] / scale);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows row0 .. row0 + 15 of KV head h of sequence b's new cache, by a warp: the places, a row per lane
// (lanes 16 to 31 hold those of 0 to 15).  `first`: their weights are copied, and rows
// without a place counted.
__device__ __forceinline__ Place find(const VParams& p, int b, int h, int row0, int m, int lane, bool first) {
  Place s = {0, 0, -1};
  const int r = row0 + (lane & 15);
  const long long unit = (long long)b * p.Hkv + h;
  bool lost = false;
  if (r < m) {
    const int pos = p.kept[unit * p.budget + r];
    const int page = (int)((unsigned)pos / (unsigned)p.P);
    const size_t e = (size_t)b * p.max_pages + page;
    const int codec = p.page_codec[e];
    const long long slot = p.block_table[e];
    lost = codec > ARGUS_INT1_G32 || slot < 0 || slot >= p.pool[codec > ARGUS_INT1_G32 ? 0 : codec].n_slots;
    if (!lost) s = {slot * 2 * p.Hkv + h, pos - page * p.P, codec};
    if (first && lane < 16) p.weights_out[unit * p.row_len_out + r] = __ldg(p.weights + unit * p.row_len + pos);
  }
  if (first) {
    const unsigned x = __ballot_sync(0xffffffffu, lost && lane < 16);
    if (x && lane == 0 && p.status) atomicAdd(p.status, __popc(x));
  }
  return s;
}

// DST: the new pages' codec; WIDE: there are 16-bit pages among the old.  T warps share a page (1
// where rows need no scale): teams of 1, 2, 4 or 8, so that a page of up to 128 tokens
// has a warp per 16 rows and is read once.
template <int D, int DST, bool WIDE>
__global__ void __launch_bounds__(32 * kWarps) gather_kernel(const VParams p, int T, int units) {
  constexpr bool kScaled = DST == ARGUS_FP8_E4M3 || DST == ARGUS_INT8;
  constexpr int V = D / 16, RS = 32 / V, STEPS = 16 / RS;   // lanes per row, rows per step
  __shared__ float s_max[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / T, tw = warp % T;
  const int unit = blockIdx.x * (kWarps / T) + team;        // KV heads fastest, then pages (or 16-row groups), then sequences
  if (unit >= units) return;                                // whole teams
  const int h = unit % p.Hkv, rows = kScaled ? p.P : 16, groups = (p.budget + p.P - 1) / p.P * (p.P / rows);
  const int g = unit / p.Hkv % groups, b = unit / p.Hkv / groups;
  const int m = min(length(p, b), p.budget), row0 = g * rows;
  const int page = row0 / p.P, in_page = row0 - page * p.P;
  if (row0 - in_page >= m) return;                          // a page that holds something is written whole
  const long long slot = p.dst_table[(size_t)b * p.dst_pages + page];
  const int subs = rows / 16;
  const bool once = subs <= T;                              // every warp has one group of 16 rows at most
  const int v = lane % V;
  Place s = {0, 0, -1};
  auto place_of = [&](int step) {
    const int r = step * RS + lane / V;
    Place y;
    y.unit = __shfl_sync(0xffffffffu, s.unit, r);
    y.row = __shfl_sync(0xffffffffu, s.row, r);
    y.codec = __shfl_sync(0xffffffffu, s.codec, r);
    return y;
  };
  for (int sub = tw; sub < subs; sub += T) s = find(p, b, h, row0 + 16 * sub, m, lane, true);
  if (slot < 0 || slot >= p.dst_slots) {                    // the whole team
    if (p.status && h == 0 && in_page == 0 && tw == 0 && lane == 0) atomicAdd(p.status, 1u);
    return;
  }
  Raw<WIDE> raw[2][STEPS];                                  // K and V on their way together where they are narrow
  auto read = [&](int kv) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) raw[WIDE ? 0 : kv][i] = fetch<D, WIDE>(p, place_of(i), kv, v);
  };
  auto write = [&](int sub, int kv, float scale) {
    const long long at = (((slot * 2 + kv) * p.Hkv + h) * p.P + in_page + 16 * sub) * D + 16 * v;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = i * RS + lane / V, codec = __shfl_sync(0xffffffffu, s.codec, r);
      const long long to = at + (long long)r * D;
      const Raw<WIDE>& y = raw[WIDE ? 0 : kv][i];
      if constexpr (!kScaled) {
        uint4* d = reinterpret_cast<uint4*>(p.dst_codes + 2 * to);
        if constexpr (WIDE) {
          if (codec == DST) {                               // as it is
            d[0] = y.a;
            d[1] = y.b;
            continue;
          }
        }
        float x[16];
        uint32_t o[8];
        values(y, codec, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = DST == ARGUS_BF16 ? pack_bf16x2(x[2 * e], x[2 * e + 1]) : pack_f16x2(x[2 * e], x[2 * e + 1]);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        float x[16];
        values(y, codec, x);
        *reinterpret_cast<uint4*>(p.dst_codes + to) = encode<DST>(x, scale);
      }
    }
  };
  if constexpr (!kScaled) {
    if (!WIDE) {
      read(0);
      read(1);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (WIDE) read(kv);
      write(0, kv, 0.f);
    }
  } else {
    if (!WIDE && once && tw < subs) {
      read(0);
      read(1);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float top = 0.f;
      for (int sub = tw; sub < subs; sub += T) {
        if (!once) s = find(p, b, h, row0 + 16 * sub, m, lane, false);
        if (WIDE || !once) read(kv);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) top = fmaxf(top, largest(raw[WIDE ? 0 : kv][i], __shfl_sync(0xffffffffu, s.codec, i * RS + lane / V)));
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));   // bits of magnitudes order like them
      if (T > 1) {
        if (lane == 0) s_max[kv][warp] = top;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * T) : "memory");
        for (int i = 0; i < T; ++i) top = fmaxf(top, s_max[kv][team * T + i]);
      }
      const float scale = top / (DST == ARGUS_FP8_E4M3 ? 448.f : 127.f);
      if (tw == 0 && lane == 0) p.dst_meta[(slot * 2 + kv) * p.Hkv + h] = scale;
      for (int sub = tw; sub < subs; sub += T) {
        if (!once) {
          s = find(p, b, h, row0 + 16 * sub, m, lane, false);
          read(kv);
        }
        write(sub, kv, scale);
      }
    }
  }
}

template <int D>
static cudaError_t launch_gather(const VParams& p, cudaStream_t s) {
  const bool scaled = p.dst_codec >= ARGUS_FP8_E4M3;
  const int rows = scaled ? p.P : 16;
  int T = 1;
  while (scaled && T < kWarps && 16 * T < p.P) T *= 2;
  const long long units = (long long)p.B * p.Hkv * ((p.budget + p.P - 1) / p.P) * (p.P / rows), per = kWarps / T;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + per - 1) / per));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  const bool wide = p.pool[ARGUS_FP16].n_slots > 0 || p.pool[ARGUS_BF16].n_slots > 0;
  const auto go = [&](auto dst) {
    constexpr int DST = decltype(dst)::value;
    return wide ? cudaLaunchKernelEx(&cfg, gather_kernel<D, DST, true>, p, T, (int)units) : cudaLaunchKernelEx(&cfg, gather_kernel<D, DST, false>, p, T, (int)units);
  };
  switch (p.dst_codec) {
    case ARGUS_FP16: return go(std::integral_constant<int, ARGUS_FP16>{});
    case ARGUS_BF16: return go(std::integral_constant<int, ARGUS_BF16>{});
    case ARGUS_FP8_E4M3: return go(std::integral_constant<int, ARGUS_FP8_E4M3>{});
    default: return go(std::integral_constant<int, ARGUS_INT8>{});
  }
}

static argus_status status_of(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_evict_tokens: launch of the %s failed: %s", what, cudaGetErrorString(e));
}

static argus_status launch(const VParams& p, int D, cudaStream_t s) {
  // blocks per row: one holds 32,768 keys; more than 8 times that are read again in every round
  const long long keys = (long long)kSelThreads * kRegKeys, longest = (long long)p.max_pages * p.P;
  int C = 1;
  while (C < kMaxCluster && C * keys < longest) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, p.Hkv, p.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const auto go = [&](auto n) { return cudaLaunchKernelEx(&cfg, select_kernel<decltype(n)::value>, p); };
  const long long per = (longest + C * kSelThreads - 1) / (C * kSelThreads);
  const argus_status st = status_of(per <= 4 ? go(std::integral_constant<int, 4>{}) : per <= 8 ? go(std::integral_constant<int, 8>{})
                                    : per <= 16 ? go(std::integral_constant<int, 16>{}) : per <= 32 ? go(std::integral_constant<int, 32>{})
                                                : go(std::integral_constant<int, 0>{}), "selection");
  // without the selection the gathering would follow whatever `kept` holds
  if (st != ARGUS_OK || p.budget == 0) return st;
  return status_of(D == 64 ? launch_gather<64>(p, s) : launch_gather<128>(p, s), "gathering");
}

struct Span {
  const void* at;
  unsigned long long bytes;
};
static bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace evict
}  // namespace argus

using namespace argus;

extern "C" argus_status argus_evict_tokens(const argus_geom* g, int32_t batch, const argus_pool* pools, int32_t n_pools, const uint8_t* page_codec,
                                           const int32_t* block_table, const int32_t* seq_lens, int32_t max_pages, const float* weights,
                                           int64_t row_len, int32_t budget, int32_t sink_tokens, int32_t recent_tokens, const argus_pool* dst,
                                           const int32_t* dst_table, int32_t dst_pages, int32_t* seq_lens_out, int32_t* kept,
                                           float* weights_out, int64_t row_len_out, uint32_t* status, void* stream) {
  if (!g || !dst) return fail(ARGUS_E_INVALID, "evict: geometry or dst is NULL");
  if (g->n_kv_heads <= 0 || g->page_tokens <= 0) return fail(ARGUS_E_INVALID, "evict: bad head counts or page_tokens");
  if (g->head_dim != 64 && g->head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "evict: head_dim %d (supported: 64, 128)", g->head_dim);
  if (g->page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "evict: page_tokens %d not a multiple of 16", g->page_tokens);
  if (batch < 0 || max_pages < 0 || n_pools < 0 || dst_pages < 0) return fail(ARGUS_E_INVALID, "evict: negative size");
  if (batch > 65535 || g->n_kv_heads > 65535) return fail(ARGUS_E_UNSUPPORTED, "evict: batch or n_kv_heads above 65535");
  const long long positions = (long long)max_pages * g->page_tokens;
  if (positions > 0x7fffffffll - 65536) return fail(ARGUS_E_UNSUPPORTED, "evict: 2^31 cached tokens per sequence or more");
  if (budget < 0 || sink_tokens < 0 || recent_tokens < 0 || (long long)sink_tokens + recent_tokens > budget)
    return fail(ARGUS_E_INVALID, "evict: budget must hold sink_tokens and recent_tokens (all >= 0)");
  if ((long long)dst_pages * g->page_tokens < budget) return fail(ARGUS_E_INVALID, "evict: dst_pages do not hold the budget");
  if (row_len < positions || row_len_out < budget) return fail(ARGUS_E_INVALID, "evict: rows of weights shorter than the cache, or weights_out than the budget");
  if ((long long)batch * g->n_kv_heads > 0x7fffffffll / std::max(1ll, ((long long)budget + g->page_tokens - 1) / g->page_tokens * (g->page_tokens / 16))) return fail(ARGUS_E_UNSUPPORTED, "evict: 2^31 groups of 16 rows or more");
  if (n_pools > 0 && !pools) return fail(ARGUS_E_INVALID, "evict: pools is NULL");
  if (dst->codec < 0 || dst->codec > ARGUS_INT1_G32) return fail(ARGUS_E_INVALID, "evict: bad codec %d", dst->codec);
  if (dst->codec > ARGUS_INT8) return fail(ARGUS_E_UNSUPPORTED, "evict: new pages of codec %d (supported: 16-bit, FP8, INT8)", dst->codec);
  evict::VParams p{};
  uint32_t seen = 0;
  for (int i = 0; i <= n_pools; ++i) {
    const argus_pool& pl = i < n_pools ? pools[i] : *dst;
    if (pl.codec < 0 || pl.codec > ARGUS_INT1_G32) return fail(ARGUS_E_INVALID, "evict: bad codec %d", pl.codec);
    if (pl.placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "evict: pools must lie in device memory");
    if (pl.n_slots < 0) return fail(ARGUS_E_INVALID, "evict: negative n_slots");
    if (pl.n_slots > 0 && (!pl.codes || (pl.codec >= ARGUS_FP8_E4M3 && !pl.meta)))
      return fail(ARGUS_E_INVALID, "evict: NULL codes or meta (codec %d)", pl.codec);
    if (reinterpret_cast<uintptr_t>(pl.codes) & 15) return fail(ARGUS_E_INVALID, "evict: codes must be 16-byte aligned");
    if (pl.codec >= ARGUS_FP8_E4M3 && (reinterpret_cast<uintptr_t>(pl.meta) & 3)) return fail(ARGUS_E_INVALID, "evict: meta must be 4-byte aligned");
    if (i == n_pools) break;
    if (seen >> pl.codec & 1) return fail(ARGUS_E_INVALID, "evict: more than one pool of codec %d", pl.codec);
    seen |= 1u << pl.codec;
    if (pl.codec <= ARGUS_BF16 && dst->codec <= ARGUS_BF16 && pl.codec != dst->codec)
      return fail(ARGUS_E_UNSUPPORTED, "evict: 16-bit pages must be of the new pages' type");
    p.pool[pl.codec] = {static_cast<const uint8_t*>(pl.codes), static_cast<const uint8_t*>(pl.meta), pl.n_slots};
  }
  if (batch == 0) return ARGUS_OK;
  if (!seq_lens || !seq_lens_out) return fail(ARGUS_E_INVALID, "evict: NULL pointer");
  if ((positions > 0 && (!weights || !page_codec || !block_table)) || (budget > 0 && (!kept || !dst_table)) || (row_len_out > 0 && !weights_out))
    return fail(ARGUS_E_INVALID, "evict: NULL pointer");
  // what is written lies apart from what is read, and from each other
  const unsigned long long rows = (unsigned long long)batch * g->n_kv_heads, entries = (unsigned long long)batch * max_pages;
  const evict::Span out[3] = {{seq_lens_out, 4ull * batch}, {kept, 4ull * rows * budget}, {weights_out, 4ull * rows * row_len_out}};
  const evict::Span in[5] = {{seq_lens, 4ull * batch}, {weights, 4ull * rows * row_len}, {page_codec, entries}, {block_table, 4 * entries},
                             {dst_table, 4ull * batch * dst_pages}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (evict::meet(out[i], in[j])) return fail(ARGUS_E_INVALID, "evict: seq_lens_out, kept or weights_out overlaps an input");
    for (int j = 0; j < i; ++j)
      if (evict::meet(out[i], out[j])) return fail(ARGUS_E_INVALID, "evict: seq_lens_out, kept and weights_out overlap");
  }
  p.Hkv = g->n_kv_heads;
  p.P = g->page_tokens;
  p.B = batch;
  p.max_pages = max_pages;
  p.budget = budget;
  p.sinks = sink_tokens;
  p.recent = recent_tokens;
  p.dst_codec = dst->codec;
  p.dst_pages = dst_pages;
  p.page_codec = page_codec;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.row_len = row_len;
  p.row_len_out = row_len_out;
  p.dst_codes = static_cast<uint8_t*>(dst->codes);
  p.dst_meta = static_cast<float*>(dst->meta);
  p.dst_slots = dst->n_slots;
  p.dst_table = dst_table;
  p.seq_lens_out = seq_lens_out;
  p.kept = kept;
  p.weights_out = weights_out;
  p.status = status;
  return evict::launch(p, g->head_dim, static_cast<cudaStream_t>(stream));
}
