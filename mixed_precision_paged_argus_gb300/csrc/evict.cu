// argus_evict_tokens: the cached positions of least accumulated attention weight dropped, the
// rest gathered into new pages.
//
// Mathematics: of a sequence of L positions and one KV head, the first S and the last R stay, and
// of those between the k = budget - S - R of largest weight, ties to the lower position.
// Floats are mapped to integers of the same order (NaN below all, -0 = +0); the k-th largest
// key T is found bit by bit, two at a time: with c_d keys at or above each of the three next
// digits, the largest d with c_d >= k is T's.  Where a count is k exactly, the search ends; where few
// keys share T's bits so far, the rest of it looks at these alone.
// Positions above T stay, and of those at T the first k - #(above T).
//
// Selection: a thread block (or a cluster of them for long rows) per sequence and KV head holds
// the keys in registers, read once; a round is three compares a key, a reduction within
// the warps and one over them.  The first seven rounds count on the keys' first 15 bits, two in a register;
// once 4,096 keys share T's bits they go to a list of four a lane, and once 128 do one warp goes on alone.
// A warp's positions are neighbours, so the ranks that put the kept
// ones in order are ballots and one scan over the warps.
//
// Gathering: a warp takes 16 rows of a new page and KV head, looks their places up at once
// and has K's (then V's) 16-byte vectors on their way together.  8-bit pages have one scale
// per page, KV head and K | V: a team of warps shares the page's largest magnitude.
//
// Measured (GB300, L2 flushed).  16 sequences of 8,192 to 32,768 FP8 tokens to 4,096, 8 KV heads of 128: 89 us.
// Selection 21 us (128 rows, one block each): a round over 32 keys a thread takes 1.2 us (1.9 on whole keys), one over the
// list 0.5 and by one warp 0.25; reading, and the latency of the first loads, 5.  (Before: 71 us with keys loaded one
// by one and all rounds on all keys; 30 with whole keys, one atomic a warp and key for the list, and the zeros behind the kept
// weights stored four bytes at a time in front of the loads.  Counting the list's digits by atomics in shared
// memory, eight bits at once: 26.)  Gathering 67 us for 268 MB, 4.0 TB/s (60% of a copy): converting, and
// dependent reads that four blocks per SM hide in part, at the price of spills (64 registers a thread; 100 to 330 bytes
// read back) (three blocks with the pairs kept in registers instead of the
// codes 76 us, five 71; two blocks with V fetched behind K 122 us in all; blocks of four warps 120; V's rows fetched
// to the L2 beside K's, or the kernel launched early: no faster).  Divisions as the compiler makes them cost 24 us more, two
// encodings from both sides of the quotient with a division where they differ 22: rows of the page's largest
// scale often hit ties.  One sequence of 16,384 fp16 tokens to 2,048, 2 KV heads of 64: 19 us, the rounds' barriers
// (by a cluster of eight blocks 37 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "codes.cuh"
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
  uint32_t p_mul, p_shift;             // division by P (page_of)
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

// x / P for 0 <= x < 2^31.  With s = ceil(log2 P) and mul = ceil(2^(31 + s) / P), x mul is above
// x 2^(31 + s) / P by less than 2^(31 + s) / P: the quotient's whole part is the same.
__device__ __forceinline__ int page_of(const VParams& p, int x) { return (int)(__umulhi((uint32_t)x, p.p_mul) >> p.p_shift); }

__device__ __forceinline__ int length(const VParams& p, int b) {
  return (int)min((long long)max(p.seq_lens[b], 0), (long long)p.max_pages * p.P);
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kRegKeys = 32;           // keys per thread that stay in registers, at most
constexpr int kMaxCluster = 8;
constexpr int kList = 4 * kSelThreads; // keys that share T's first bits, from which on the others are left alone

// Keys of the weights' order: NaN 1, -inf 0x7FFFFF, zeros 0x80000000, inf 0xFF800000.  A position that
// stays in any case has the key kAlways, one that is not there 0.
constexpr uint32_t kAlways = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);         // -0 becomes 0
  return w != w ? 1u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

struct Counts {
  uint32_t a, b, c;
};
// SMALL: the sums are below 2^16, and two go as one.
template <bool SMALL>
__device__ __forceinline__ Counts warp_sum(Counts x) {
  if (SMALL) {
    const uint32_t ab = __reduce_add_sync(0xffffffffu, x.a | x.b << 16);
    x.a = ab & 0xFFFFu;
    x.b = ab >> 16;
  } else {
    x.a = __reduce_add_sync(0xffffffffu, x.a);
    x.b = __reduce_add_sync(0xffffffffu, x.b);
  }
  x.c = __reduce_add_sync(0xffffffffu, x.c);
  return x;
}

// KEYS: a thread's keys, which stay in registers; 0: they are read again in every round.
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const VParams p) {
  constexpr bool kSmall = KEYS > 0;                    // a block's counts are at most 32,768
  __shared__ Counts s_warp[2][kSelWarps];
  __shared__ Counts s_block[2];
  __shared__ uint32_t s_list[kList], s_listed, s_close, s_few[2][kSelWarps], s_found[3];
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = gridDim.x, rank = blockIdx.x;          // the cluster spans the grid's first dimension
  const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)b * p.Hkv + h;
  const float* w = p.weights + row * p.row_len;
  int32_t* kept = p.kept + row * p.budget;
  const int len = length(p, b), m = min(len, p.budget);
  if (threadIdx.x == 0 && rank == 0 && h == 0) p.seq_lens_out[b] = m;
  const int tid = rank * kSelThreads + threadIdx.x, all = C * kSelThreads;
  // behind the kept positions
  auto clear = [&]() {
    for (int i = m + tid; i < p.budget; i += all) kept[i] = -1;
    // the weights 16 bytes at a time: up to the first whole vector, the vectors, the rest
    float* w_out = p.weights_out + row * p.row_len_out;
    const uintptr_t end = reinterpret_cast<uintptr_t>(w_out + p.row_len_out), from = reinterpret_cast<uintptr_t>(w_out + m);
    const uintptr_t first = min(end, (from + 15) & ~(uintptr_t)15), last = max(first, end & ~(uintptr_t)15);
    uint4* to = reinterpret_cast<uint4*>(first) + tid;
    const uint4* stop = reinterpret_cast<const uint4*>(last);
    for (; to < stop; to += all) *to = make_uint4(0, 0, 0, 0);
    if (tid < 4 && from + 4 * tid < first) reinterpret_cast<float*>(from)[tid] = 0.f;
    if (tid < 4 && last + 4 * tid < end) reinterpret_cast<float*>(last)[tid] = 0.f;
  };
  if (p.budget == 0 || len <= p.budget) {              // the same in the whole cluster
    for (int i = tid; i < m; i += all) kept[i] = i;
    clear();
    return;
  }
  const int lo = p.sinks, hi = len - p.recent, k = p.budget;   // what lies outside lo .. hi-1 is among the k, and less than len are
  // this warp's positions: steps of 32 neighbours (all within 8,192 of the row's end)
  const int steps = KEYS > 0 ? KEYS : (int)(((long long)len + C * kSelThreads - 1) / (C * kSelThreads));
  const int start = (rank * kSelWarps + warp) * steps * 32 + lane;
  auto load = [&](int i) -> float {
    const int pos = start + i * 32;
    return pos >= lo && pos < hi ? __ldg(w + pos) : 0.f;
  };
  auto key_of = [&](int i, float x) {
    const int pos = start + i * 32;
    return pos >= lo && pos < hi ? order(x) : pos < len ? kAlways : 0u;
  };
  uint32_t key[KEYS > 0 ? KEYS : 1];
  // the first 15 bits of two keys each: the early rounds take less than half of the instructions on these
  [[maybe_unused]] uint32_t high[KEYS > 0 ? KEYS / 2 : 1];
  if constexpr (KEYS > 0) {
    float x[KEYS];                                     // all on their way at once
    const bool inner = start - lane >= lo && start - lane + KEYS * 32 <= hi;   // the whole warp's
    if (inner) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) x[i] = __ldg(w + start + i * 32);
    } else {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) x[i] = load(i);
    }
    clear();
    if (inner) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) key[i] = order(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) key[i] = key_of(i, x[i]);
    }
#pragma unroll
    for (int i = 0; i < KEYS / 2; ++i) high[i] = prmt(key[2 * i], key[2 * i + 1], 0x7632) >> 1 & 0x7FFF7FFFu;
  } else {
    clear();
  }
  auto each = [&](auto f) {
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) f(i, key[i]);
    } else {
      for (int i = 0; i < steps; ++i) f(i, key_of(i, load(i)));
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
      in = warp_sum<kSmall>(in);
    }
    y = warp_sum<kSmall>(y);
    if (C > 1) {
      if (threadIdx.x == 0) s_block[t] = y;
      cluster.sync();
      Counts z = {0, 0, 0};
      if (lane < C) z = *cluster.map_shared_rank(&s_block[t], lane);
      if (before) {
        const bool f = lane < rank;
        const Counts g = warp_sum<false>({f ? z.a : 0, f ? z.b : 0, f ? z.c : 0});
        in = {in.a + g.a, in.b + g.b, in.c + g.c};
      }
      y = warp_sum<false>(z);
    }
    if (before) *before = in;
    return y;
  };
  uint32_t T = 0, ties = 0;                            // keys above T stay, and the first `ties` at T
  {
    uint32_t prefix = 0, upper = 0, at = 0xFFFFFFFFu;  // T's bits so far; keys at or above the prefix's successor, and the prefix
    int s = 32;                                        // bits still open
    // two more bits from the counts of keys at or above the three next prefixes; true: the search is over
    auto narrow = [&](Counts c) {
      const bool a = c.a >= (uint32_t)k, b = c.b >= (uint32_t)k, d = c.c >= (uint32_t)k;
      prefix |= ((uint32_t)a + b + d) << s;
      upper = d ? upper : b ? c.c : a ? c.b : c.a;
      at = d ? c.c : b ? c.b : a ? c.a : at;
      return at == (uint32_t)k;
    };
    auto count = [&](Counts& c, uint32_t x) {
      c.a += x >= (prefix | 1u << s);
      c.b += x >= (prefix | 2u << s);
      c.c += x >= (prefix | 3u << s);
    };
    bool exact = false;
    while (s > 0 && !exact && at - upper > (uint32_t)kList) {
      s -= 2;
      Counts c = {0, 0, 0};
      if (KEYS > 0 && s >= 18) {
        // per half max(min(x + 1 - t, 1), 0): is x >= t?
        const auto less = [&](uint32_t d) { return (1u - ((prefix | d << s) >> 17) & 0xFFFFu) * 0x10001u; };
        const uint32_t ta = less(1), tb = less(2), tc = less(3);
#pragma unroll
        for (int i = 0; i < KEYS / 2; ++i) {
          c.a += __viaddmin_s16x2_relu(high[i], ta, 0x10001u);
          c.b += __viaddmin_s16x2_relu(high[i], tb, 0x10001u);
          c.c += __viaddmin_s16x2_relu(high[i], tc, 0x10001u);
        }
        c = {(c.a & 0xFFFFu) + (c.a >> 16), (c.b & 0xFFFFu) + (c.b >> 16), (c.c & 0xFFFFu) + (c.c >> 16)};
      } else {
        each([&](int, uint32_t x) { count(c, x); });
      }
      exact = narrow(total(warp_sum<kSmall>(c), nullptr));
    }
    if (s > 0 && !exact) {
      // the few keys that share the prefix, in any order: the other rounds look at these
      if (threadIdx.x == 0) s_listed = s_close = 0;
      __syncthreads();
      uint32_t n = 0, to = 0;
      each([&](int, uint32_t x) { n += x >> s == prefix >> s; });
      uint32_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31 && upto) to = atomicAdd(&s_listed, upto);
      to = __shfl_sync(0xffffffffu, to, 31) + upto - n;
      if (n) each([&](int, uint32_t x) {
        if (x >> s == prefix >> s) s_list[to++] = x;
      });
      __syncthreads();
      const int listed = (int)s_listed;
      int few = C > 1 ? kSelWarps : (listed + 127) / 128;        // warps that go on, with up to four keys a lane
      if (warp < few) {
        constexpr int kMine = kList / kSelThreads;
        static_assert(kMine * 32 < 1 << 10 && kList < 1 << 16, "packed counts");
        uint32_t mine[kMine], above = upper;
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine[i] = i * few * 32 + (int)threadIdx.x < listed ? s_list[i * few * 32 + threadIdx.x] : 0u;
        while (s > 0 && !exact) {
          if (C == 1 && few > 1 && at - upper <= 128u) {
            // few enough for one warp, without barriers
            uint32_t n = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) n += mine[i] >> s == prefix >> s;
            if (n) {
              uint32_t to = atomicAdd(&s_close, n);
#pragma unroll
              for (int i = 0; i < kMine; ++i)
                if (mine[i] >> s == prefix >> s) s_list[to++] = mine[i];
            }
            asm volatile("bar.sync 1, %0;" ::"r"(few * 32) : "memory");
            if (warp > 0) break;
            few = 1;
            above = upper;
#pragma unroll
            for (int i = 0; i < kMine; ++i) mine[i] = i * 32 + lane < (int)s_close ? s_list[i * 32 + lane] : 0u;
          }
          s -= 2;
          Counts c = {0, 0, 0};
#pragma unroll
          for (int i = 0; i < kMine; ++i) count(c, mine[i]);
          if (C > 1) {
            c = total(warp_sum<true>(c), nullptr);
          } else {
            const uint32_t sum = __reduce_add_sync(0xffffffffu, c.a | c.b << 10 | c.c << 20);
            c = {sum & 0x3FFu, sum >> 10 & 0x3FFu, sum >> 20};
            if (few > 1) {
              const int t = s >> 1 & 1;                // the other buffer may still be read
              if (lane == 0) s_few[t][warp] = sum;
              asm volatile("bar.sync 1, %0;" ::"r"(few * 32) : "memory");
              const uint32_t y = lane < few ? s_few[t][lane] : 0u;
              c = warp_sum<true>({y & 0x3FFu, y >> 10 & 0x3FFu, y >> 20});
            }
          }
          exact = narrow({c.a + above, c.b + above, c.c + above});
        }
        if (threadIdx.x == 0) {
          s_found[0] = prefix;
          s_found[1] = upper;
          s_found[2] = exact;
        }
      }
      __syncthreads();
      prefix = s_found[0];
      upper = s_found[1];
      exact = s_found[2] != 0;
    }
    // k keys at or above the prefix: all of them; T is not 0, as there are more than k keys above 0
    T = exact ? prefix - 1 : prefix;
    ties = exact ? 0u : (uint32_t)k - upper;
  }
  Counts mine = {0, 0, 0};
  each([&](int, uint32_t x) {
    mine.a += x > T;
    mine.b += x == T;
  });
  mine = warp_sum<kSmall>(mine);
  Counts before;
  total(mine, &before);
  const uint32_t lt = (1u << lane) - 1;
  uint32_t at = before.a + min(before.b, ties), tied = before.b;
  const bool some = ties > 0;
  each([&](int i, uint32_t x) {
    bool keep = x > T;
    if (some) {                                        // the first `ties` of those at T
      const uint32_t eq = __ballot_sync(0xffffffffu, x == T);
      keep = keep || (x == T && tied + __popc(eq & lt) < ties);
      tied += __popc(eq);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, keep);
    if (keep) kept[at + __popc(mask & lt)] = start + i * 32;
    at += __popc(mask);
  });
  if (C > 1) cluster.sync();                           // the others may still read this block's sums
}

// ---------------------------------------------------------------- gathering
constexpr int kWarps = 8;

// Where a kept row lies: its K row's first value, in values from the pool's first one; its codec (-1:
// nowhere); the scale of its unit (8-bit codecs).
struct Place {
  long long at;
  int codec;
  float scale;
};

// ---- rows of any codec: sixteen values at a time
__device__ __forceinline__ void values(const VParams& p, const Place& s, long long at, float (&x)[16]) {
  const PoolRef& pool = p.pool[max(s.codec, 0)];
  if (s.codec < 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  } else if (s.codec <= ARGUS_BF16) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(pool.codes + 2 * at)), b = __ldg(reinterpret_cast<const uint4*>(pool.codes + 2 * at) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = s.codec == ARGUS_BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                                             : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
  } else if (s.codec <= ARGUS_INT8) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(pool.codes + at));
    const float f = s.scale;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
      if (s.codec == ARGUS_FP8_E4M3) fp8_to_16<false>(w[i], h[0], h[1]);
      else int8_to_16<false>(w[i], h[0], h[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        x[4 * i + 2 * j] = y.x * f;
        x[4 * i + 2 * j + 1] = y.y * f;
      }
    }
  } else {
    uint32_t w[2] = {0, 0};
    if (s.codec == ARGUS_INT4_G32) {
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(pool.codes + at / 2));
      w[0] = y.x;
      w[1] = y.y;
    } else if (s.codec == ARGUS_INT2_G32) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(pool.codes + at / 4));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(pool.codes + at / 8));
    }
    const uint32_t m = __ldg(reinterpret_cast<const uint32_t*>(pool.meta) + at / 32);   // scale, zero
    const float2 sz = __half22float2(*reinterpret_cast<const __half2*>(&m));
    const int bits = s.codec == ARGUS_INT4_G32 ? 4 : s.codec == ARGUS_INT2_G32 ? 2 : 1;
    const unsigned long long q = (unsigned long long)w[1] << 32 | w[0];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf((float)((uint32_t)(q >> (bits * i)) & ((1u << bits) - 1)), sz.x, sz.y);   // the product is exact
  }
}

// ---- codes of RN(x / scale).  With y = RN(1 / scale) the quotient is q + r y, rounded once, for q = RN(x y)
// and r = x - q scale, which an FMA gives exactly (P. Markstein, IBM J. Res. Dev. 34, 1990): where it is
// next to a border between codes, a number of few bits, the quotient is no closer to the middle between
// two floats than 2^-24 of their distance over scale's mantissa, and r y is off by less.  r is taken towards -inf, which
// changes nothing in an exact one but makes a difference of equals -0: so a quotient of -0 keeps its sign.
__device__ __forceinline__ void f2_fma_down(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rm.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
template <int DST>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (DST == ARGUS_FP8_E4M3) return f32x4_to_e4m3(a, b, c, d);
  // |y| <= 127, or next to it by a rounding: the adder's low bits are the rounded integer
  constexpr float kRound = 12582912.f;
  f2_add(a, b, a, b, kRound, kRound);
  f2_add(c, d, c, d, kRound, kRound);
  return prmt(prmt(__float_as_uint(a), __float_as_uint(b), 0x0040), prmt(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}
// Sixteen codes of y s / scale; rcp = RN(1 / scale), 0 where the scale is so small or large that a step could leave
// fp32's range.  There an INT8 scale may be a few units of 2^-149, whose rounding takes quotients past 127: they end
// there (e4m3's conversion saturates).
template <int DST>
__device__ __forceinline__ uint4 encode(float (&y)[16], float s, float rcp, float scale) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) f2_mul(y[e], y[e + 1], y[e], y[e + 1], s, s);
  if (rcp != 0.f) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float q[2], r[2];
      f2_mul(q[0], q[1], y[e], y[e + 1], rcp, rcp);
      f2_fma_down(r[0], r[1], q[0], q[1], -scale, -scale, y[e], y[e + 1]);
      f2_fma(y[e], y[e + 1], r[0], r[1], rcp, rcp, q[0], q[1]);
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j == e) {
          const float q = scale > 0.f ? y[j] / scale : 0.f;
          y[j] = DST == ARGUS_INT8 ? fminf(fmaxf(q, -127.f), 127.f) : q;
        }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = encode4<DST>(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ bool moderate(float x) { return x >= 0x1p-60f && x <= 0x1p60f; }

// ---- rows of one codec, 16-bit or 8: sixteen values as pairs of fp16 (or bf16) codes
template <int SRC>
struct Raw {
  uint4 a, b;                          // b: the second half of 16-bit rows
};
template <int SRC>
__device__ __forceinline__ Raw<SRC> fetch(const VParams& p, long long at) {   // at < 0: nowhere
  Raw<SRC> r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  if (at < 0) return r;
  const uint4* x = reinterpret_cast<const uint4*>(p.pool[SRC].codes + (SRC <= ARGUS_BF16 ? 2 * at : at));
  r.a = __ldg(x);
  if (SRC <= ARGUS_BF16) r.b = __ldg(x + 1);
  return r;
}
template <int SRC>
__device__ __forceinline__ void pairs(const Raw<SRC>& r, uint32_t (&h)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if constexpr (SRC <= ARGUS_BF16) {
    h[0] = r.a.x; h[1] = r.a.y; h[2] = r.a.z; h[3] = r.a.w;
    h[4] = r.b.x; h[5] = r.b.y; h[6] = r.b.z; h[7] = r.b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (SRC == ARGUS_FP8_E4M3) fp8_to_16<false>(w[i], h[2 * i], h[2 * i + 1]);
      else int8_to_16<false>(w[i], h[2 * i], h[2 * i + 1]);
    }
  }
}
template <int SRC>
__device__ __forceinline__ float2 pair_values(uint32_t h) {
  if (SRC == ARGUS_BF16) return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The largest magnitude of sixteen values: the largest code's, as a product with the same scale keeps the
// order, and so do the bits of magnitudes.
template <int SRC>
__device__ __forceinline__ float largest(const uint32_t (&h)[8], float s) {
  if constexpr (SRC != ARGUS_BF16) {
    __half2 m = __habs2(*reinterpret_cast<const __half2*>(&h[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&h[i])));
    const float2 y = __half22float2(m);
    return fabsf(fmaxf(y.x, y.y) * s);
  }
  uint32_t m = h[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(h[i] & 0x7FFF7FFFu));
  const float2 y = pair_values<SRC>(m);
  return fabsf(fmaxf(y.x, y.y) * s);
}

// Rows row0 .. row0 + 15 of KV head h of sequence b's new cache, by a warp: the places, a row per lane
// (lanes 16 to 31 hold those of 0 to 15; the scales are K's in lanes 0 to 15, V's in 16 to 31).  `first`: their
// weights are copied, and rows without a place counted.
template <int D>
__device__ __forceinline__ Place find(const VParams& p, int b, int h, int row0, int m, int lane, bool first) {
  Place s = {-1, -1, 1.f};
  const int r = row0 + (lane & 15);
  const long long unit = (long long)b * p.Hkv + h;
  bool lost = false;
  if (r < m) {
    const int pos = p.kept[unit * p.budget + r];
    const int page = page_of(p, pos);
    const size_t e = (size_t)b * p.max_pages + page;
    const int codec = p.page_codec[e];
    const long long slot = p.block_table[e];
    lost = codec > ARGUS_INT1_G32 || slot < 0 || slot >= p.pool[codec > ARGUS_INT1_G32 ? 0 : codec].n_slots;
    if (!lost) {
      const long long u = slot * 2 * p.Hkv + h;
      s.at = (u * p.P + (pos - page * p.P)) * D;
      s.codec = codec;
      if (codec == ARGUS_FP8_E4M3 || codec == ARGUS_INT8) s.scale = __ldg(reinterpret_cast<const float*>(p.pool[codec].meta) + u + (lane < 16 ? 0 : p.Hkv));
    }
    if (first && lane < 16) p.weights_out[unit * p.row_len_out + r] = __ldg(p.weights + unit * p.row_len + pos);
  }
  if (first) {
    const unsigned x = __ballot_sync(0xffffffffu, lost && lane < 16);
    if (x && lane == 0 && p.status) atomicAdd(p.status, __popc(x));
  }
  return s;
}

// DST: the new pages' codec.  T warps share a page (1 where rows need no scale): teams of
// 1, 2, 4 or 8, so that a page of up to 128 tokens has a warp per 16 rows.  Where all rows of a warp are of
// one codec, and a warp has one group of 16 rows, they are read once and stay in registers as codes; the path for
// everything else reads them twice (from the L2, the second time) and is short, so that both
// fit the instruction cache.
template <int D, int DST>
__global__ void __launch_bounds__(32 * kWarps, 4) gather_kernel(const VParams p, int T, int units) {
  constexpr bool kScaled = DST == ARGUS_FP8_E4M3 || DST == ARGUS_INT8;
  constexpr int V = D / 16, RS = 32 / V, STEPS = 16 / RS;   // lanes per row, rows per step
  __shared__ float s_max[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / T, tw = warp % T;
  const int unit = blockIdx.x * (kWarps / T) + team;        // KV heads fastest, then pages (or groups of 16 rows)
  if (unit >= units) return;                                // whole teams
  const int g = unit / p.Hkv, h = unit - g * p.Hkv, b = blockIdx.y, rows = kScaled ? p.P : 16;
  const int m = min(length(p, b), p.budget), row0 = g * rows;
  const int page = kScaled ? g : page_of(p, row0), in_page = row0 - page * p.P;
  if (row0 - in_page >= m) return;                          // a page that holds something is written whole
  const long long slot = p.dst_table[(size_t)b * p.dst_pages + page];
  const int subs = rows / 16, v = lane % V;
  Place s = {-1, -1, 1.f};
  for (int sub = tw; sub < subs; sub += T) s = find<D>(p, b, h, row0 + 16 * sub, m, lane, true);
  if (slot < 0 || slot >= p.dst_slots) {                    // the whole team
    if (p.status && h == 0 && in_page == 0 && tw == 0 && lane == 0) atomicAdd(p.status, 1u);
    return;
  }
  const long long to_v = (long long)p.Hkv * p.P * D;         // from a K row to its V row, in old pages and new
  // this lane's sixteen values in a step's rows: their place, and where they go
  auto row_at = [&](int step) {
    const long long at = __shfl_sync(0xffffffffu, s.at, step * RS + lane / V);
    return at < 0 ? at : at + 16 * v;
  };
  const long long page_at = ((slot * 2 * p.Hkv + h) * p.P + in_page + lane / V) * D + 16 * v;
  auto target = [&](int sub, int kv, int step) { return page_at + (kv ? to_v : 0) + (16 * sub + step * RS) * D; };
  // the page's scale, from every warp's largest magnitude
  auto scale_of = [&](int kv, float top) {
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (T > 1) {
      if (lane == 0) s_max[kv][warp] = top;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * T) : "memory");
      for (int i = 0; i < T; ++i) top = fmaxf(top, s_max[kv][team * T + i]);
    }
    const float scale = top / (DST == ARGUS_FP8_E4M3 ? 448.f : 127.f);
    if (tw == 0 && lane == 0) p.dst_meta[(slot * 2 + kv) * p.Hkv + h] = scale;
    return scale;
  };
  // the codec of all this warp's rows that have a place; -1 where they differ, or a warp has several groups
  const int first = __reduce_max_sync(0xffffffffu, s.codec);
  const int src = subs <= T && __all_sync(0xffffffffu, s.codec == first || s.codec < 0) ? (first < 0 ? DST : first) : -1;
  auto fast = [&](auto codec) {
    constexpr int SRC = decltype(codec)::value;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      float f[STEPS], top = 0.f;
      Raw<SRC> raw[STEPS];
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const long long at = row_at(i);
        raw[i] = fetch<SRC>(p, at < 0 || kv == 0 ? at : at + to_v);
      }
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        f[i] = SRC <= ARGUS_BF16 ? 1.f : __shfl_sync(0xffffffffu, s.scale, 16 * kv + i * RS + lane / V);
        if (kScaled) {
          uint32_t q[8];
          pairs<SRC>(raw[i], q);
          top = fmaxf(top, largest<SRC>(q, f[i]));
          // codes stay in registers, not the pairs, which are twice as many
          if (SRC > ARGUS_BF16) asm volatile("" : "+r"(raw[i].a.x), "+r"(raw[i].a.y), "+r"(raw[i].a.z), "+r"(raw[i].a.w));
        }
      }
      [[maybe_unused]] float scale = 1.f, rcp = 1.f;
      if constexpr (kScaled) {
        scale = scale_of(kv, top);
        rcp = moderate(scale) ? 1.f / scale : 0.f;
      }
      if (tw < subs) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const long long to = target(tw, kv, i);
          uint32_t q[8];
          pairs<SRC>(raw[i], q);
          if constexpr (DST == SRC && !kScaled) {           // as it is
            uint4* d = reinterpret_cast<uint4*>(p.dst_codes + 2 * to);
            d[0] = make_uint4(q[0], q[1], q[2], q[3]);
            d[1] = make_uint4(q[4], q[5], q[6], q[7]);
          } else {
            float y[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 z = pair_values<SRC>(q[e]);
              y[2 * e] = z.x;
              y[2 * e + 1] = z.y;
            }
            if constexpr (kScaled) {
              *reinterpret_cast<uint4*>(p.dst_codes + to) = encode<DST>(y, f[i], rcp, scale);
            } else {
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                o[e] = DST == ARGUS_BF16 ? pack_bf16x2(y[2 * e] * f[i], y[2 * e + 1] * f[i]) : pack_f16x2(y[2 * e] * f[i], y[2 * e + 1] * f[i]);
              uint4* d = reinterpret_cast<uint4*>(p.dst_codes + 2 * to);
              d[0] = make_uint4(o[0], o[1], o[2], o[3]);
              d[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      }
    }
  };
  // of a team, every warp has to take the same number of barriers: one per scale, on either path
  if (src == ARGUS_FP8_E4M3) {
    fast(std::integral_constant<int, ARGUS_FP8_E4M3>{});
  } else if (src == ARGUS_INT8) {
    fast(std::integral_constant<int, ARGUS_INT8>{});
  } else if (src == ARGUS_BF16 && DST != ARGUS_FP16) {
    fast(std::integral_constant<int, ARGUS_BF16>{});
  } else if (src == ARGUS_FP16 && DST != ARGUS_BF16) {
    fast(std::integral_constant<int, ARGUS_FP16>{});
  } else {
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      [[maybe_unused]] float scale = 1.f, rcp = 1.f;
#pragma unroll 1
      for (int pass = kScaled ? 0 : 1; pass < 2; ++pass) {
        float top = 0.f;
#pragma unroll 1
        for (int sub = tw; sub < subs; sub += T) {
          if (subs > T) s = find<D>(p, b, h, row0 + 16 * sub, m, lane, false);
#pragma unroll 1
          for (int i = 0; i < STEPS; ++i) {
            const int r = i * RS + lane / V;
            Place at;
            at.at = row_at(i);
            at.codec = __shfl_sync(0xffffffffu, s.codec, r);
            at.scale = __shfl_sync(0xffffffffu, s.scale, 16 * kv + r);
            float x[16];
            values(p, at, at.at + (kv ? to_v : 0), x);
            if (pass == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
            } else if constexpr (kScaled) {
              *reinterpret_cast<uint4*>(p.dst_codes + target(sub, kv, i)) = encode<DST>(x, 1.f, rcp, scale);
            } else {
              // a 16-bit value of the same type comes back as it was
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = DST == ARGUS_BF16 ? pack_bf16x2(x[2 * e], x[2 * e + 1]) : pack_f16x2(x[2 * e], x[2 * e + 1]);
              uint4* d = reinterpret_cast<uint4*>(p.dst_codes + 2 * target(sub, kv, i));
              d[0] = make_uint4(o[0], o[1], o[2], o[3]);
              d[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
        if (kScaled && pass == 0) {
          scale = scale_of(kv, top);
          rcp = moderate(scale) ? 1.f / scale : 0.f;
        }
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
  const long long units = (long long)p.Hkv * ((p.budget + p.P - 1) / p.P) * (p.P / rows), per = kWarps / T;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + per - 1) / per), p.B);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  switch (p.dst_codec) {
    case ARGUS_FP16: return cudaLaunchKernelEx(&cfg, gather_kernel<D, ARGUS_FP16>, p, T, (int)units);
    case ARGUS_BF16: return cudaLaunchKernelEx(&cfg, gather_kernel<D, ARGUS_BF16>, p, T, (int)units);
    case ARGUS_FP8_E4M3: return cudaLaunchKernelEx(&cfg, gather_kernel<D, ARGUS_FP8_E4M3>, p, T, (int)units);
    default: return cudaLaunchKernelEx(&cfg, gather_kernel<D, ARGUS_INT8>, p, T, (int)units);
  }
}

static argus_status status_of(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_evict_tokens: launch of the %s failed: %s", what, cudaGetErrorString(e));
}

static argus_status launch(const VParams& p, int D, cudaStream_t s) {
  // blocks per row: one holds 32,768 keys; more than 8 times that are read again in every round.  (More
  // blocks than a row needs cost more in the cluster's barriers than they save: a call of 16,384 keys 19 us
  // by one block, 37 by eight; 16 sequences of up to 32,768 keys 90 and 361.)
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
  if (((long long)budget + g->page_tokens - 1) / g->page_tokens * g->page_tokens > 0x7fffffffll - 65536)
    return fail(ARGUS_E_UNSUPPORTED, "evict: new pages of 2^31 tokens per sequence or more");
  if (row_len < positions || row_len_out < budget) return fail(ARGUS_E_INVALID, "evict: rows of weights shorter than the cache, or weights_out than the budget");
  if ((long long)g->n_kv_heads > 0x7fffffffll / std::max(1ll, ((long long)budget + g->page_tokens - 1) / g->page_tokens * (g->page_tokens / 16))) return fail(ARGUS_E_UNSUPPORTED, "evict: 2^31 groups of 16 rows or more");
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
  int bits = 0;
  while ((1ll << bits) < p.P) ++bits;  // P >= 16
  p.p_mul = (uint32_t)(((1ull << (31 + bits)) + p.P - 1) / p.P);
  p.p_shift = bits - 1;
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
