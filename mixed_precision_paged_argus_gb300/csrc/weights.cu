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
//  * Two chunks at a time, copied into a ring of the warp's own some steps ahead: their 32 sums
//    end up in the 32 lanes, one line of weights.
// Many rows per KV head are weights_rows.cu's, but not over group codes, whose scales its products cannot carry.
//
// Measured (GB300): one token of 32 sequences of 8,192 to 32,768 FP8 tokens, 32/8 heads of 128: 133 to 136 us, 5.3 TB/s
// (78 to 80% of a plain copy).  On the way: chunks loaded into registers when they were wanted 238 us, a ring of single
// chunks 168 to 204 (spilled values came back from the L2, as the rings leave the L1 little room), pairs with three
// blocks of 80 registers per SM 171, with two of 127 as it is.  11 sequences of 3,736 to 13,632 tokens, 32/8 heads of 128:
// INT4, one token 24 us, 21 tokens 155 (215 with one tile of rows per pass, 148 with four, in bf16 187 and 190: four
// cost registers, and with them warps); 4 tokens over 16-bit pages 37 (58 with one).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "codes.cuh"
#include "common.cuh"
#include "weights.cuh"

namespace argus {
namespace weights {

// Warps per block, blocks per SM, bytes of a warp's ring (pairs of chunks on their way) for calls with
// pages of every codec, and with 8-bit ones alone.
template <bool ANY>
struct Shape {
  static constexpr int kWarps = ANY ? 12 : 8, kBlocks = ANY ? 1 : 2, kRing = ANY ? 16384 : 12288;
};
constexpr int kBatch = 32;             // chunks looked up at once
constexpr int kMaxSlots = 4;
constexpr int kMany = 16;              // rows from which on the tensor cores' large tiles pay

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// A sequence's chunks, KV heads one after the other; those that another kernel takes have none here.
__device__ __forceinline__ long long chunks_of(const WParams& p, int b) {
  const int rows = rows_of(p, b).rows;
  return rows <= p.few || rows > p.many ? 0 : (long long)p.Hkv * ((length(p, b) + 15) / 16);
}

// How a page's operands are formed, and with it the order of a row's dims in them.
enum Form { kNone = -1, k16 = 0, k8 = 1, kGroup = 2 };
__device__ __forceinline__ int form_of(int codec) { return codec <= ARGUS_BF16 ? k16 : codec <= ARGUS_INT8 ? k8 : kGroup; }

// Sixteen keys as the MMA's A operand (BF: bf16, else fp16): rows lane / 4 and eight further down, dims by
// the lane's place c in its row.  src: the chunk in shared memory.
template <int D, bool BF, bool ANY>
__device__ __forceinline__ void load_keys(uint32_t src, int codec, int lane, uint32_t (&a)[D / 16][4]) {
  const int r = lane >> 2, c = lane & 3;
  if (ANY && codec <= ARGUS_BF16) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 x = lds16(src + r * 2 * D + i * 64 + c * 16), y = lds16(src + (r + 8) * 2 * D + i * 64 + c * 16);
      a[2 * i][0] = x.x;
      a[2 * i][1] = y.x;
      a[2 * i][2] = x.y;
      a[2 * i][3] = y.y;
      a[2 * i + 1][0] = x.z;
      a[2 * i + 1][1] = y.z;
      a[2 * i + 1][2] = x.w;
      a[2 * i + 1][3] = y.w;
    }
  } else if (!ANY || codec <= ARGUS_INT8) {
    uint4 y[2][D / 64];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) y[x][i] = lds16(src + (r + 8 * x) * D + i * 64 + c * 16);
    }
    auto turn = [&](auto fp8) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t w[4] = {y[x][i].x, y[x][i].y, y[x][i].z, y[x][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (decltype(fp8)::value) fp8_to_16<BF>(w[e], a[4 * i + e][x], a[4 * i + e][2 + x]);
            else int8_to_16<BF>(w[e], a[4 * i + e][x], a[4 * i + e][2 + x]);
          }
        }
      }
    };
    if (codec == ARGUS_FP8_E4M3) turn(std::true_type{});
    else turn(std::false_type{});
  } else {
    const int bits = codec == ARGUS_INT4_G32 ? 4 : codec == ARGUS_INT2_G32 ? 2 : 1, row = D * bits / 8;
    const uint32_t mask = ((1u << bits) - 1) * 0x10001u;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t at = src + (r + 8 * x) * row;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // eight codes of group i: elements j and j + 4 in the two halves, j codes up
        uint32_t w;
        if (codec == ARGUS_INT4_G32) {
          w = lds4(at + i * 16 + c * 4);
        } else if (codec == ARGUS_INT2_G32) {
          const uint32_t y = lds4(at + i * 8 + (c & 2) * 2) >> (16 * (c & 1));
          w = (y & 0xFF) | (y >> 8 & 0xFF) << 16;
        } else {
          const uint32_t y = lds4(at + i * 4) >> (8 * c);
          w = (y & 0xF) | (y >> 4 & 0xF) << 16;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {                    // fp16 1024 + code, minus 1024; bf16 128 + code, minus 128
          const uint32_t y = (w >> (bits * j)) & mask;
          a[2 * i + (j >> 1)][2 * (j & 1) + x] = BF ? bf2_sub(y | 0x43004300u, 0x43004300u) : hsub2_u32(y | 0x64006400u, 0x64006400u);
        }
      }
    }
  }
}

// Eight query rows as the MMA's B operand, in the dims' order of a form.
template <int D>
struct Query {
  uint32_t f[D / 16][2];
  float fac[2];                        // of columns 2c, 2c + 1: undoes the fp16 query's power of two
  float sum[D / 32][2];                // kGroup: sums of a group's elements
};

// BF: the query's type.  TURN: a bf16 query becomes fp16 times a power of two per row.
template <int D, bool BF, bool TURN>
__device__ __forceinline__ void load_query(const uint16_t* row, bool real, int form, int lane, Query<D>& out) {
  const int c = lane & 3;
  uint4 v[D / 32];                     // 8 elements each
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    // k8: two vectors next to each other, 16 codes; else every fourth
    const int at = form == k8 ? (i / 2) * 64 + c * 16 + (i & 1) * 8 : i * 32 + c * 8;
    v[i] = real ? __ldg(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0, 0, 0, 0);
  }
  float fac = 1.f;
  if (TURN && form != k16) {
    // the row's largest magnitude comes to [2^14, 2^15): its 8 bits fit fp16
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t a = max_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), b = max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu);
      mx = max_u16x2(mx, max_u16x2(a, b));
    }
    mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const uint32_t ex = max(max(mx >> 16, mx & 0xFFFFu) >> 7, 15u);   // biased; from 15 on 2^(141 - ex) is a normal number
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
        if (BF && !TURN) {
          s += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xFFFF0000u);
        } else {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
          s += y.x + y.y;
        }
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      out.sum[i][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      out.sum[i][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
      // codes come out of their word in pairs (j, j + 4)
      v[i] = make_uint4(prmt(w[0], w[2], 0x5410), prmt(w[0], w[2], 0x7632), prmt(w[1], w[3], 0x5410), prmt(w[1], w[3], 0x7632));
    }
  }
  out.fac[0] = out.fac[1] = 1.f;
  if (TURN) {
    out.fac[0] = __shfl_sync(0xffffffffu, fac, 8 * c);
    out.fac[1] = __shfl_sync(0xffffffffu, fac, 8 * c + 4);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    out.f[2 * i][0] = v[i].x;
    out.f[2 * i][1] = v[i].y;
    out.f[2 * i + 1][0] = v[i].z;
    out.f[2 * i + 1][1] = v[i].w;
  }
}

template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if (BF) mma_bf16(d, a[0], a[1], a[2], a[3], b[0], b[1]);
  else mma_f16(d, a[0], a[1], a[2], a[3], b[0], b[1]);
}

// Scores of 16 keys by 8 rows: d[0], d[1] key lane / 4, columns 2c and 2c + 1; d[2], d[3] eight keys
// further down.  meta: the chunk's scales and zeros in shared memory (kGroup).
template <int D, bool BF>
__device__ __forceinline__ void scores(const uint32_t (&a)[D / 16][4], const Query<D>& q, int form, uint32_t meta, int lane, float (&d)[4]) {
  if (form != kGroup) {
    float e[4] = {0.f, 0.f, 0.f, 0.f};                   // two chains: an MMA does not wait for the one before
    d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      mma<BF>(d, a[i], q.f[i]);
      mma<BF>(e, a[i + 1], q.f[i + 1]);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) d[x] += e[x];
  } else {
    d[0] = d[1] = d[2] = d[3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float g[4] = {0.f, 0.f, 0.f, 0.f};
      mma<BF>(g, a[2 * i], q.f[2 * i]);
      mma<BF>(g, a[2 * i + 1], q.f[2 * i + 1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t sz = lds4(meta + (((lane >> 2) + 8 * x) * (D / 32) + i) * 4);
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&sz));
#pragma unroll
        for (int k = 0; k < 2; ++k) d[2 * x + k] = fmaf(y.x, g[2 * x + k], fmaf(y.y, q.sum[i][k], d[2 * x + k]));
      }
    }
  }
}

// Some chunks of one (sequence, KV head), and its query rows: they are taken in tiles of eight, and
// for one tile, or two, the chunks pass through the ring once (from the L2, behind the first).
struct Batch {
  int b, h, c0, n, len;
  int t0, rows, passes;                // first token; its rows by tokens and heads; at least one pass
};

// Where a chunk lies.
struct __align__(16) Found {
  const uint8_t* src;
  float ks;
  int codec;                           // -1: nothing to read
};
constexpr int kLooked = 2 * kBatch;    // chunks whose places are kept

// Where a warp's range goes on.
struct Walk {
  long long left, at;                  // chunks ahead; the next one within its sequence, KV heads one after the other
  int b;
};

// The next batch, its chunks looked up into the places from `to` on, a lane each.
template <int D, bool ANY, int TILES>
__device__ __forceinline__ Batch next_batch(const WParams& p, Walk& w, Found* found, const uint8_t** metas, uint32_t to, int lane) {
  Batch x;
  x.b = x.h = x.c0 = x.n = x.len = x.t0 = x.rows = x.passes = 0;
  if (w.left <= 0) return x;
  int per;
  for (;;) {                           // there is a chunk ahead: the loop ends at its sequence
    x.len = length(p, w.b);
    per = (x.len + 15) / 16;
    if (w.at < chunks_of(p, w.b)) break;
    w.at = 0;
    ++w.b;
  }
  x.b = w.b;
  x.h = (int)(w.at / per);
  x.c0 = (int)(w.at - (long long)x.h * per);
  x.n = (int)min(w.left, (long long)min(kBatch, per - x.c0));
  w.left -= x.n;
  w.at += x.n;
  const Span r = rows_of(p, x.b);
  x.t0 = r.t0;
  x.rows = r.rows;
  x.passes = max((x.rows + 8 * TILES - 1) / (8 * TILES), 1);
  if (lane < x.n) {
    Found f = {nullptr, 1.f, -1};
    const uint8_t* meta = nullptr;
    const int key = (x.c0 + lane) * 16, page = (int)((uint32_t)key / (uint32_t)p.P), row = key - page * p.P;
    const size_t e = (size_t)x.b * p.max_pages + page;
    const int k = p.page_codec[e];
    const long long slot = p.block_table[e];
    const PoolRef pool = p.pool[k <= ARGUS_INT1_G32 ? k : 0];
    if (k > ARGUS_INT1_G32 || slot < 0 || slot >= pool.n_slots) {
      if (x.h == 0 && row == 0 && p.status) atomicAdd(p.status, 1u);
    } else {
      f.codec = k;
      const long long unit = slot * 2 * p.Hkv + x.h, token = unit * p.P + row;
      f.src = pool.codes + token * (!ANY ? D : k <= ARGUS_BF16 ? 2 * D : k <= ARGUS_INT8 ? D : D >> (k - ARGUS_INT8));
      if (ANY && k >= ARGUS_INT4_G32) meta = pool.meta + token * (D / 32) * 4;
      else if (k >= ARGUS_FP8_E4M3) f.ks = __ldg(reinterpret_cast<const float*>(pool.meta) + unit);
    }
    found[(to + lane) % kLooked] = f;
    if (ANY) metas[(to + lane) % kLooked] = meta;
  }
  __syncwarp();
  return x;
}

// Query row `mine` of a batch: its address (nullptr: there is none), log-sum and last visible key.
template <int D>
__device__ __forceinline__ const uint16_t* row_of(const WParams& p, const Batch& x, int mine, float& L, int& last) {
  const bool real = mine < x.rows;
  const int tok = real ? mine / p.G : 0, g = real ? mine - tok * p.G : 0;
  L = INFINITY;                        // a row that sees nothing gives nothing
  if (real) {
    L = __ldg(p.lse2 + (size_t)(x.t0 + tok) * p.Hq + x.h * p.G + g);
    if (L == -INFINITY) L = INFINITY;
  }
  last = !real ? -1 : p.causal ? min(x.len - x.rows / p.G + tok, x.len - 1) : x.len - 1;
  return real ? p.q + (x.t0 + tok) * p.qs + (long long)(x.h * p.G + g) * D : nullptr;
}
// ... and of a lane's two columns
struct Columns {
  float lse[2];
  int see[2];
};
__device__ __forceinline__ Columns columns(float L, int last, int lane) {
  Columns x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.lse[i] = __shfl_sync(0xffffffffu, L, 8 * (lane & 3) + 4 * i);
    x.see[i] = __shfl_sync(0xffffffffu, last, 8 * (lane & 3) + 4 * i);
  }
  return x;
}
// Weights of the scores d, summed per key over the lane's columns: x key lane / 4, y eight further down.
// Selected, not multiplied: rows behind the end may hold anything.
__device__ __forceinline__ float2 weigh(const float (&d)[4], float f0, float f1, const Columns& x, int key) {
  float2 s;
  s.x = (key <= x.see[0] ? fast_exp2(fmaf(d[0], f0, -x.lse[0])) : 0.f) + (key <= x.see[1] ? fast_exp2(fmaf(d[1], f1, -x.lse[1])) : 0.f);
  s.y = (key + 8 <= x.see[0] ? fast_exp2(fmaf(d[2], f0, -x.lse[0])) : 0.f) + (key + 8 <= x.see[1] ? fast_exp2(fmaf(d[3], f1, -x.lse[1])) : 0.f);
  return s;
}

// BF: the queries' (and 16-bit pages') type.  ANY: pages of every codec, else of 8 bits alone, which need
// fewer registers.  TILES: of eight query rows per pass over the chunks.  slot: bytes of a ring slot, n_slots of them per warp.
template <int D, bool BF, bool ANY, int TILES>
__global__ void __launch_bounds__(32 * Shape<ANY>::kWarps, Shape<ANY>::kBlocks) weights_kernel(const WParams p, int slot, int n_slots) {
  constexpr int kWarps = Shape<ANY>::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Found s_found[kWarps][kLooked];
  __shared__ const uint8_t* s_meta[ANY ? kWarps : 1][kLooked];
  __shared__ uint64_t s_full[kWarps][kMaxSlots];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
  uint64_t* full = s_full[warp];
  Found* found = s_found[warp];
  const uint8_t** metas = s_meta[ANY ? warp : 0];
  uint8_t* ring = smem + (size_t)warp * slot * n_slots;
  if (p.leads) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // this warp's range of chunks
  const int nw = gridDim.x * kWarps, w = blockIdx.x * kWarps + warp;
  const long long first = lane < p.B ? chunks_of(p, lane) : 0;
  long long total = first;
  for (int x = lane + 32; x < p.B; x += 32) total += chunks_of(p, x);
  total = warp_sum(total);
  const long long u0 = total / nw * w + total % nw * w / nw, u1 = total / nw * (w + 1) + total % nw * (w + 1) / nw;
  Walk walk = {u1 - u0, 0, 0};
  if (walk.left <= 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  {
    long long before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const long long mine = b0 == 0 ? first : b0 + lane < p.B ? chunks_of(p, b0 + lane) : 0, incl = warp_scan(mine);
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > u0);
      if (hit) {
        const int src = __ffs(hit) - 1;
        walk.b = b0 + src;
        walk.at = u0 - before - __shfl_sync(0xffffffffu, incl - mine, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane < n_slots) mbar_init(&full[lane], 1);
  fence_mbar_init();
  __syncwarp();
  Batch cur = next_batch<D, ANY, TILES>(p, walk, found, metas, 0, lane), ahead = next_batch<D, ANY, TILES>(p, walk, found, metas, cur.n, lane);
  uint32_t base = 0;                                     // place of cur's first chunk
  // the next copies: chunks feed_i and feed_i + 1 for pass feed_t of cur (feed = 0) or ahead (1); 2: all issued
  int feed = 0, feed_t = 0, feed_i = 0;
  int put = 0, take = 0, flying = 0;                     // next slot to fill and to read, pairs on their way
  uint32_t phase = 0;                                    // of the slots
  auto issue = [&]() {                                   // copies, as far as there are slots
    while (flying < n_slots && feed < 2) {
      const int n = feed ? ahead.n : cur.n, passes = feed ? ahead.passes : cur.passes;
      if (feed_i >= n) {
        feed_i = 0;
        if (++feed_t >= passes) {                        // (no chunks: no passes)
          feed_t = 0;
          ++feed;
        }
        continue;
      }
      // a lane per chunk; a chunk that is not read adds no bytes
      uint32_t bytes = 0, more = 0;
      const uint32_t from = (base + (feed ? cur.n : 0) + feed_i + (lane & 1)) % kLooked;
      if (feed_i + (lane & 1) < n) {
        const int k = found[from].codec;
        if (k >= 0) bytes = ANY ? 16 * (k <= ARGUS_BF16 ? 2 * D : k <= ARGUS_INT8 ? D : D >> (k - ARGUS_INT8)) : 16 * D;
        if (ANY && k > ARGUS_INT8) more = 16 * (D / 32) * 4;
      }
      const uint32_t both = bytes + more + __shfl_xor_sync(0xffffffffu, bytes + more, 1);
      if (lane == 0) mbar_arrive_expect_tx(&full[put], both);
      __syncwarp();
      if (lane < 2 && bytes) {
        uint8_t* to = ring + put * slot + lane * (slot / 2);
        bulk_g2s(to, found[from].src, bytes, &full[put]);
        if (ANY && more) bulk_g2s(to + 8 * D, metas[from], more, &full[put]);   // behind the codes: at most D / 2 bytes a row
      }
      feed_i += 2;
      ++flying;
      if (++put == n_slots) put = 0;
    }
  };
  bool ok = true;
  Query<D> q[TILES];
  Columns col[TILES] = {};
  int have_b = -1, have_h = -1, have_t = -1, have_form = kNone;   // whose rows q and col hold
  while (cur.n > 0 && ok) {
    // the lane's position in a pair of chunks: neighbouring lanes have neighbouring keys' sums
    const int mine = (c >> 1) * 16 + (c & 1) * 8 + (lane >> 2);
    float* out = p.weights + ((size_t)cur.b * p.Hkv + cur.h) * p.row_len;
    for (int t = 0; t < cur.passes && ok; ++t) {
      const int tiles = (cur.rows + 7) / 8 - TILES * t;
      for (int i = 0; i < cur.n; i += 2) {
        issue();
        const int pos = (cur.c0 + i) * 16 + mine;
        const bool writes = pos < cur.len && i + (c >> 1) < cur.n;
        // by t > 0 the sum so far, which this lane wrote
        const float old = writes && (t > 0 || p.decay != 0.f) ? out[pos] : 0.f;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[take], phase >> take & 1));
        if (!ok) break;
        float2 s[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j] = make_float2(0.f, 0.f);
          const Found at = found[(base + i + j) % kLooked];
          const int k = i + j < cur.n ? at.codec : -1;
          if (k < 0) continue;
          const int form = ANY ? form_of(k) : (int)k8;
          const uint32_t src = smem_u32(ring + take * slot + j * (slot / 2));
          if (have_form != form || have_t != t || have_h != cur.h || have_b != cur.b) {
            have_form = form;
            have_t = t;
            have_h = cur.h;
            have_b = cur.b;
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
              if (u > 0 && u >= tiles) break;
              float L;
              int last;
              const uint16_t* row = row_of<D>(p, cur, 8 * (TILES * t + u) + (lane >> 2), L, last);
              load_query<D, BF, BF>(row, row != nullptr, form, lane, q[u]);
              col[u] = columns(L, last, lane);
            }
          }
          uint32_t a[D / 16][4];
          const bool wide = ANY && BF && form == k16;
          if (wide) load_keys<D, BF, ANY>(src, k, lane, a);
          else load_keys<D, false, ANY>(src, k, lane, a);
          const float f = at.ks * p.scale_log2;
#pragma unroll
          for (int u = 0; u < TILES; ++u) {
            if (u > 0 && u >= tiles) break;
            float d[4];
            if (wide) scores<D, BF>(a, q[u], form, src + 8 * D, lane, d);
            else scores<D, false>(a, q[u], form, src + 8 * D, lane, d);
            const float2 x = weigh(d, f * q[u].fac[0], f * q[u].fac[1], col[u], (cur.c0 + i + j) * 16 + (lane >> 2));
            s[j].x += x.x;
            s[j].y += x.y;
          }
        }
        __syncwarp();                                    // the chunks have been read
        phase ^= 1u << take;
        --flying;
        if (++take == n_slots) take = 0;
        // sums over the four lanes of a row, one of the four values each
        const bool odd = c & 1, high = c & 2;
        const float u = (odd ? s[0].y : s[0].x) + __shfl_xor_sync(0xffffffffu, odd ? s[0].x : s[0].y, 1);
        const float v = (odd ? s[1].y : s[1].x) + __shfl_xor_sync(0xffffffffu, odd ? s[1].x : s[1].y, 1);
        const float x = (high ? v : u) + __shfl_xor_sync(0xffffffffu, high ? u : v, 2);
        if (writes) out[pos] = fmaf(t > 0 ? 1.f : p.decay, old, x);
      }
    }
    if (!ok) break;
    issue();                                             // what there is room for: steps behind cur in any case
    base += cur.n;
    --feed;                                              // all of cur was issued
    cur = ahead;
    ahead = next_batch<D, ANY, TILES>(p, walk, found, metas, base + cur.n, lane);
  }
  if (!ok) {
    // a copy did not arrive: the caller is told, and the ones in flight get as long again
    if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeoutBit);
    for (; flying > 0; --flying) {
      mbar_wait(&full[take], phase >> take & 1);
      if (++take == n_slots) take = 0;
    }
  }
  // who waits for this kernel waits for the call's other one too
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// follows: behind another kernel of the call, which has other sequences: it may start while that one runs.
template <int D, bool BF, bool ANY, int TILES>
static argus_status launch(const WParams& p, cudaStream_t s, bool follows) {
  using S = Shape<ANY>;
  // a slot holds two chunks, 16 rows each, of the widest pages
  const bool wide = p.pool[ARGUS_FP16].n_slots > 0 || p.pool[ARGUS_BF16].n_slots > 0;
  const int slot = wide ? 64 * D : 32 * D, n_slots = std::min(kMaxSlots, S::kRing / slot);
  static PerContext configured;
  const argus_status st = configured.ensure([](int) {
    const cudaError_t e = cudaFuncSetAttribute(weights_kernel<D, BF, ANY, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kWarps * S::kRing);
    return e == cudaSuccess ? ARGUS_OK : fail(ARGUS_E_LAUNCH, "weights: smem attribute: %s", cudaGetErrorString(e));
  });
  if (st != ARGUS_OK) return st;
  const long long chunks = (long long)p.B * p.Hkv * (((long long)p.max_pages * p.P + 15) / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(1ll, std::min(chunks, device_sm_count() * (long long)S::kBlocks)));
  cfg.blockDim = dim3(32 * S::kWarps);
  cfg.dynamicSmemBytes = S::kWarps * slot * n_slots;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = follows ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weights_kernel<D, BF, ANY, TILES>, p, slot, n_slots);
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_attn_weights: launch failed: %s", cudaGetErrorString(e));
}

template <int D>
static argus_status launch_d(WParams p, bool bf, cudaStream_t s) {
  bool any = false, group = false;
  for (int k = 0; k < 7; ++k) {
    if (p.pool[k].n_slots <= 0) continue;
    any |= k != ARGUS_FP8_E4M3 && k != ARGUS_INT8;
    group |= k >= ARGUS_INT4_G32;
  }
  const auto go = [&](auto all, auto tiles, bool follows) {
    constexpr bool ANY = decltype(all)::value;
    constexpr int TILES = decltype(tiles)::value;
    return bf ? launch<D, true, ANY, TILES>(p, s, follows) : launch<D, false, ANY, TILES>(p, s, follows);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  // A call of as many tokens as sequences is taken for a decode step, with one token each.  In any other, one sequence may
  // have all the tokens, whatever the average is (idle slots), and the sequences of many rows get a kernel of their own,
  // beside which the other one may run.  Where no sequence has many it is empty: 2 to 4 us beside a small step of 16 us, 0 to 2
  // beside one of 69.  One sequence of 16,384 tokens asks with 32, 63 slots are empty: FP8 25 us (68 without), BF16 26 (85);
  // the 63 hold 2,000 to 8,192 tokens: FP8 108 (691), BF16 169 (1,214), INT4, with 21 tokens, 184 (1,267).
  const long long all_rows = (long long)p.total_q * p.G;
  const bool decode = p.total_q == p.B, more = all_rows > 8ll * p.B;   // more than one tile of rows on average
  p.few = -1;
  p.many = 0x7fffffff;
  if (group && !decode && p.B > 1 && all_rows > 8) {
    // more than a tile of rows: two tiles per pass, as the large tiles know no group codes; apart from the others
    // also because a chunk of many rows is many times their work.  The kernel that likely has the fewer sequences
    // leads: where it has none, batches of 4 to 21 tokens each lose 1 to 3% (a single sequence 6%: one kernel there).
    const auto part = [&](auto tiles, bool follows) {
      p.few = decltype(tiles)::value == 2 ? 8 : -1;
      p.many = decltype(tiles)::value == 2 ? 0x7fffffff : 8;
      p.leads = !follows;
      return go(std::true_type{}, tiles, follows);
    };
    const argus_status st = more ? part(one, false) : part(two, false);
    if (st != ARGUS_OK) return st;
    return more ? part(two, true) : part(one, true);
  }
  bool follows = false;
  if (!group && !decode && all_rows > kMany) {
    p.many = kMany;
    const argus_status st = launch_rows(p, D, bf, any, s);
    if (st != ARGUS_OK) return st;
    follows = true;
  }
  if (!any) return go(std::false_type{}, one, follows);
  // up to kMany rows: two tiles where sequences have more than one on average (one of eight rows: 24 us by one, 26 by two)
  return more ? go(std::true_type{}, two, follows) : go(std::true_type{}, one, follows);
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
    if (pl.codec >= ARGUS_FP8_E4M3 && (reinterpret_cast<uintptr_t>(pl.meta) & (pl.codec >= ARGUS_INT4_G32 ? 15 : 3)))
      return fail(ARGUS_E_INVALID, "weights: meta must be 4-byte aligned, of group codes 16-byte aligned");
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
  return D == 64 ? weights::launch_d<64>(p, bf, s) : weights::launch_d<128>(p, bf, s);
}
