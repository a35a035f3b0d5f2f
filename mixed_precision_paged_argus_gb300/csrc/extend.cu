// argus_paged_extend_attn: several query tokens per sequence attend to the
// paged cache, read in place.
//
// Mathematics: o = sum p_j v_j / sum p_j with p_j = 2^(s_j - m), in one pass over the
// keys with a reference m that only moves when the maximum grows by more than
// 2^8 (the result does not depend on it).  A page's scales are folded in where they
// cost nothing: the K scale, the softmax scale and log2 e are one factor of a score,
// and the V scale w_j enters the exponent, p_j w_j = 2^(s_j + log2 w_j - m), so
// that codes alone are the MMAs' operands; the row sum divides each 16-key chunk's
// part by its w again (where w is far from 1 it sums the weights on their own: relative
// to an m that holds w they could leave fp32's range).  P is stored times 2^7 (fp16: at
// most 2^15 before m moves).
//
// What bounds it: with few query rows per key (drafted tokens) the bytes of the
// pages; with many (prompt chunks) the tensor cores, and beside them the
// conversion of the codes (every tile of 128 query rows converts the pages again) and
// the exponentials.  So the design keeps all three going at once:
//  * 128 query rows (the G heads of a KV head by tokens) by 128 keys per block;
//    S = Q K^T and O += P V by tcgen05.mma (M = N = 128), scores and P in TMEM (two
//    buffers), Q, K, V as 128-byte swizzled tiles in shared memory.
//  * 8-bit codes become fp16 exactly (bf16 in blocks with bf16 pages), on the way from
//    the page to the tile: 16 loader warps (8 K, 8 V) hold a 16-token chunk each in
//    registers (16-byte loads, a block ahead), convert, and store to the tile.
//    Chunks, not blocks, carry a page's codec and scales, so pages of 16 tokens and
//    more, and tiers, mix freely.  A lookup warp reads table and scales batches
//    of four blocks ahead and has the L2 fetch the pages.
//  * Two softmax groups of 4 warps share every block, 64 keys each, with an O and a
//    (m, l) of their own, joined in the epilogue: a row's 64 scores stay in
//    registers between the maximum and the exponentials.
//  * Few rows (<= 32 or <= 64, the drafted tokens) would leave TMEM lanes idle: the
//    tile holds 4 or 2 copies of them, and each copy's lanes take other 16-key chunks
//    (their P is 0 elsewhere); the epilogue adds the copies.
//  * One CTA per SM; the key blocks of all items are dealt out evenly, found on
//    the device (below).  Items that are cut leave pieces; a second kernel joins them.
//    It is launched early, which saves its launch; its blocks find room only on SMs that
//    no CTA of the first kernel holds (64,512 of 65,536 registers) any more.
//
// Measured (GB300; CUDA events, buffers rotated past the L2): FP8 pages of 16 tokens, 32
// sequences of 8,192 to 32,768, 1 to 8 drafted tokens, 32/8 heads of 128: 311 to 313 us, 4.6 TB/s
// of pages (67% of a plain copy; decode reaches 72% on the same pages).  A 1,024-token chunk over
// 131,072 FP8 tokens, 16/2 heads of 128: 1.02 ms, 1.07 PFLOP/s (56% of cuBLAS bf16);
// with neither softmax nor MMAs the loads and conversions alone took 0.71 ms, the
// MMAs alone 0.67 ms.  BF16, FP8 and INT8 pages mixed, 8 sequences of up to 16,384
// with 1 to 256 new tokens: 244 us (the same in FP8 alone 152, INT8 217, BF16 315: a
// 16-bit page is twice the bytes for every query tile, and the second half of its rows
// of 128 dims is read only when it is stored).
// Per-item cost is what bounds short sequences (1,024 of 64 tokens: 263 us): its code
// runs once per item, out of a cold instruction cache, hence the rolled loops in
// load_q and the epilogue (unrolled as far as registers allow, mixed tiers took 259 us and cross
// attention over 1 to 1,500 INT8 states 53; it takes 49).  Sums kept apart for far V
// scales are 1 to 3% of that (mixed tiers 240, cross 48 without them).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace argus {
namespace extend {

using namespace tc;

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
  int n_ctas;
  int last_query[8];                 // (128 (r + 1) - 1) / G: the query of tile r's last row
  uint32_t g_mul, g_shift;           // division by G (group_of)
  float* ws;                         // pieces: o [2 n_ctas][128][D], then lse2 [2 n_ctas][128]; cuts [n_ctas]
};

constexpr int kBM = 128;             // query rows per tile (TMEM lanes)
constexpr int kBN = 128;             // keys per block
constexpr int kGroupWarps = 4;       // one softmax warpgroup: a thread per TMEM lane
constexpr int kSoftmaxWarps = 2 * kGroupWarps;
constexpr int kLoadWarps = 16;       // eight for K, eight for V: a 16-token chunk of every block each
constexpr int kLookWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kMmaWarp = kLookWarp + 1;
constexpr int kQWarp0 = kMmaWarp + 1;
constexpr int kQWarps = 2;
constexpr int kThreads = 32 * (kQWarp0 + kQWarps);
// 28 warps get 72 registers a thread at launch; the loaders' four-warp groups give
// up what the softmax groups take.  Nothing may spill: the tiles leave the
// L1 so little that a spilled value comes back from the L2.
constexpr int kLaunchRegs = 72, kSoftmaxRegs = 104, kLoadRegs = 56;
static_assert(kSoftmaxWarps * kSoftmaxRegs + kLoadWarps * kLoadRegs <= (kSoftmaxWarps + kLoadWarps) * kLaunchRegs, "registers");
constexpr int kHalf = kBM * 64 * 2;  // 128 rows x 64 dims: one 128-byte swizzle column
constexpr int kTmemCols = 512;       // S0 S1 O0 O1, 128 columns each
constexpr float kRescaleThreshold = 8.f;
// |log2| of a V scale beyond which it does not enter the sums' reference: with
// scales within 2^+-32, a P that falls below fp32's range (2^-126) next to the
// row's largest has a weight below 2^-(126 + 7 - 2 * 32) = 2^-69 of it
constexpr float kFarScale = 32.f;
constexpr int kBatch = 4;            // blocks looked up at once: a lane per chunk
constexpr int kBatches = 4;          // batches whose descriptions are kept
constexpr int kSlots = kBatch * kBatches;
constexpr int kMergePad = 20;        // floats per row of the replica merge (16 used; conflict-free vectors)

template <int D>
struct Smem {
  static constexpr int kTile = kBM * D * 2;
  static constexpr int kOffQ = 0;                                        // two items' tiles
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffChunk = kOffV + 2 * kTile;                    // [slot][chunk] uint4: source, state
  static constexpr int kOffScale = kOffChunk + kSlots * 8 * 16;          // [slot][chunk] float4: ks, log2 vs, 1 / vs
  static constexpr int kOffQScale = kOffScale + kSlots * 8 * 16;         // [2][128]
  static constexpr int kOffML = kOffQScale + 2 * kBM * 4;
  static constexpr int kOffMerge = kOffML + 2 * kBM * 8;
  static constexpr int kOffBar = kOffMerge + 2 * 96 * kMergePad * 4;
  // q_first, q_full[2], k_full[2], pv_ready[2], s_full[2], o_done[2], o_free[2], drain, looked[kBatches], used[kBatches]
  static constexpr int kNumBars = 14 + 2 * kBatches;
  static constexpr int kOffItem = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // two items' descriptions
  static constexpr int kOffMisc = kOffItem + 2 * 32;
  static constexpr int kBytes = kOffMisc + 64;
  static_assert(kBytes <= 232448, "shared memory");
};

// ---------------------------------------------------------------- the work list
// An item is (sequence b, KV head h, tile t of 128 query rows); its work is its
// key blocks, plus what every item costs (its first scores, its epilogue), counted as
// kItemCost blocks in front of them: without that, a CTA that got many short
// items ran several times as long as the others.  All units of all items in that
// order are dealt to the CTAs in equal contiguous ranges, so an item's blocks may
// be cut anywhere: the pieces are partial softmaxes, joined by the second
// kernel.  The host knows neither the lengths nor the query counts; every
// CTA finds its range from them.
constexpr int kItemCost = 4;
struct Seq {
  int q0, n, len;
};

// x / G for 0 <= x < 2^31.  With s = ceil(log2 G) and mul = ceil(2^(31 + s) / G), mul G
// is above 2^(31 + s) by less than 2^s, so x mul is above x 2^(31 + s) / G by less
// than 2^(31 + s) / G: the quotient's whole part is the same.  (A division takes some
// twenty instructions, at eight places of the code that every item runs through.)
__device__ __forceinline__ int group_of(const EParams& p, int x) {
  return p.g_mul ? (int)(__umulhi((uint32_t)x, p.g_mul) >> p.g_shift) : x;
}

__device__ __forceinline__ Seq load_seq(const EParams& p, int b) {
  Seq s;
  const int a = min(max(p.q_start[b], 0), p.total_q), e = min(max(p.q_start[b + 1], 0), p.total_q);
  s.q0 = a;
  s.n = max(e - a, 0);
  s.len = (int)min((long long)max(p.seq_lens[b], 0), (long long)p.max_pages * p.P);
  return s;
}

__device__ __forceinline__ int n_tiles(const EParams& p, const Seq& s) { return (int)(((long long)s.n * p.G + kBM - 1) / kBM); }

// key blocks of tile t: up to its last row's last key (at least one, so that
// rows that see nothing are written too)
__device__ __forceinline__ int tile_blocks(const EParams& p, const Seq& s, int t) {
  int keys = s.len;
  if (p.causal) {
    const int last = min(group_of(p, (int)((uint32_t)kBM * (t + 1) - 1)), s.n - 1);   // rows: fewer than 2^31
    keys = max(s.len - s.n, 0) + last + 1;
  }
  return max(1, (keys + kBN - 1) / kBN);
}

// blocks of tiles 0 .. m-1 (m <= T): under the causal mask G tiles further down
// are 128 queries, hence exactly one block more; only the last tile may be cut
// short.  With f = G a + r tiles before it, residue r of the tiles modulo G occurs
// a times, or a + 1 times below the remainder.
__device__ __forceinline__ long long blocks_before(const EParams& p, const Seq& s, int m) {
  if (!p.causal) return (long long)m * tile_blocks(p, s, 0);
  const int T = n_tiles(p, s);
  const int f = min(m, T - 1);
  const uint32_t base = (uint32_t)max(s.len - s.n, 0) + kBN;
  const int a = group_of(p, f), rem = f - a * p.G;
  long long sum = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int cnt = r < p.G ? a + (r < rem) : 0;
    sum += (long long)cnt * ((base + (uint32_t)p.last_query[r]) / kBN) + (long long)cnt * (cnt - 1) / 2;
  }
  if (m == T && T > 0) sum += tile_blocks(p, s, T - 1);
  return sum;
}

// units of one KV head's tiles 0 .. m-1
__device__ __forceinline__ long long units_before(const EParams& p, const Seq& s, int m) {
  return blocks_before(p, s, m) + (long long)kItemCost * m;
}

// a sequence's items, and its blocks
struct Load {
  long long items, blocks;
  __device__ __forceinline__ long long units() const { return blocks + kItemCost * items; }
};
__device__ __forceinline__ Load seq_load(const EParams& p, int b) {
  const Seq s = load_seq(p, b);
  if (s.n == 0) return {0, 0};
  const int T = n_tiles(p, s);
  return {(long long)p.Hkv * T, p.Hkv * blocks_before(p, s, T)};
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

// a / b, both >= 0: in 32 bits where they fit
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ long long range_start(long long total, int cta, int n_ctas) { return divide(total * cta, n_ctas); }

struct Cursor {
  Seq s;
  int b, h, t, T, blk, nb;
  int left;                          // blocks of the range still ahead, this one counted

  // the item that unit `rest` of sequence b lies in, and the block there: the
  // units in front of an item's blocks belong to its first.  By a whole warp:
  // 32 tiles are tried per step.
  __device__ __forceinline__ void start(const EParams& p, int b_, long long rest, int left_) {
    const int lane = threadIdx.x & 31;
    b = b_;
    left = left_;
    s = load_seq(p, b);
    T = n_tiles(p, s);
    const long long per = units_before(p, s, T);
    h = (int)divide(rest, per);
    rest -= h * per;
    t = 0;                           // the last tile with units before it <= rest
    for (int n = T; n > 1;) {
      const int step = (n + 31) / 32, i = lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, i < n && units_before(p, s, t + i) <= rest);
      const int k = 31 - __clz(m);   // lane 0's tile is one
      t += k * step;
      n = min(step, n - k * step);
    }
    blk = (int)max(0ll, rest - units_before(p, s, t) - kItemCost);
    nb = tile_blocks(p, s, t);
  }
  // the first warp finds a CTA's start for all
  __device__ __forceinline__ void store(volatile uint32_t* m) const {
    m[0] = s.q0; m[1] = s.n; m[2] = s.len; m[3] = b; m[4] = h; m[5] = t; m[6] = T; m[7] = blk; m[8] = nb;
  }
  __device__ __forceinline__ void load(const volatile uint32_t* m, int blocks) {
    s.q0 = m[0]; s.n = m[1]; s.len = m[2]; b = m[3]; h = m[4]; t = m[5]; T = m[6]; blk = m[7]; nb = m[8]; left = blocks;
  }
  __device__ __forceinline__ void next_item(const EParams& p) {
    blk = 0;
    if (++t == T) {
      t = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.B) { b = p.B - 1; left = 0; return; }
          s = load_seq(p, b);
        } while (s.n == 0);
        T = n_tiles(p, s);
      }
    }
    nb = tile_blocks(p, s, t);
  }
  // `n` blocks further, which end in this item or at its end
  __device__ __forceinline__ void advance(const EParams& p, int n) {
    blk += n;
    left -= n;
    if (blk == nb && left > 0) next_item(p);
  }
};

// Where the range of a CTA begins: its first unit, the block there (left = 0) and
// the number of blocks in front of it.  Only the first min(units, CTAs) CTAs have
// a range; behind the last one's lies the end.  By a whole warp.
struct Boundary {
  long long total, unit, blocks;     // units of the call
  int n;                             // CTAs with a range
  Cursor at;
};
__device__ __forceinline__ Boundary find_boundary(const EParams& p, int cta) {
  const int lane = threadIdx.x & 31;
  const Load first = lane < p.B ? seq_load(p, lane) : Load{0, 0};
  Load sum = first;
  for (int b = lane + 32; b < p.B; b += 32) {
    const Load x = seq_load(p, b);
    sum.items += x.items;
    sum.blocks += x.blocks;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum.items += __shfl_xor_sync(0xffffffffu, sum.items, o);
    sum.blocks += __shfl_xor_sync(0xffffffffu, sum.blocks, o);
  }
  Boundary r;
  r.total = sum.units();
  r.n = (int)min((long long)p.n_ctas, r.total);
  r.unit = r.total;
  r.blocks = sum.blocks;
  r.at = {};
  if (cta >= r.n) return r;
  r.unit = range_start(r.total, cta, r.n);
  Load before = {0, 0};
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const Load mine = b0 == 0 ? first : b0 + lane < p.B ? seq_load(p, b0 + lane) : Load{0, 0};
    const Load incl = {warp_scan(mine.items), warp_scan(mine.blocks)};
    const unsigned hit = __ballot_sync(0xffffffffu, before.units() + incl.units() > r.unit);
    if (hit) {
      const int src = __ffs(hit) - 1;
      before.items += __shfl_sync(0xffffffffu, incl.items - mine.items, src);
      before.blocks += __shfl_sync(0xffffffffu, incl.blocks - mine.blocks, src);
      r.at.start(p, b0 + src, r.unit - before.units(), 0);
      r.blocks = before.blocks + r.at.h * blocks_before(p, r.at.s, r.at.T) + blocks_before(p, r.at.s, r.at.t) + r.at.blk;
      break;
    }
    before.items += __shfl_sync(0xffffffffu, incl.items, 31);
    before.blocks += __shfl_sync(0xffffffffu, incl.blocks, 31);
  }
  return r;
}

// The pieces of the range [w0, w1): the one that does not begin its item (the
// first piece of a range at most) and the one that does not end it (the last)
// lie in the workspace at 2 cta and 2 cta + 1, four dims by all rows by the next four
// dims (a lane has a row).  The CTA behind the first cut of an item
// describes it for the second kernel.
struct Cut {
  int rows, last;                    // rows of the tile (0: nothing to join); last CTA of the item
  int q0, row0, head0, pad[3];       // first query token of the sequence; first row of the tile; first head
};
__device__ __forceinline__ float* piece_o(const EParams& p, int D, int piece) { return p.ws + (size_t)piece * kBM * D; }
__device__ __forceinline__ float* piece_lse(const EParams& p, int D, int piece) {
  return p.ws + (size_t)2 * p.n_ctas * kBM * D + (size_t)piece * kBM;
}
__device__ __forceinline__ Cut* cuts(const EParams& p, int D) {
  return reinterpret_cast<Cut*>(p.ws + (size_t)2 * p.n_ctas * kBM * (D + 1));
}

// copies of a tile's rows over the 128 TMEM lanes (see the head of the file)
__device__ __forceinline__ int replicas(int rows) { return rows <= 32 ? 4 : rows <= 64 ? 2 : 1; }

// ---------------------------------------------------------------- codes -> 16 bits
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Four codes to four 16-bit values, exactly.
template <bool BF>
__device__ __forceinline__ void fp8_to_16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (!BF) {
    lo = e4m3x2_to_f16x2(w);
    hi = e4m3x2_to_f16x2(w >> 16);
  } else {
    // sign to the top, exponent and fraction to the low exponent bits and the
    // top fraction bits: the value times 2^-120 (e4m3's bias is 7, bf16's 127;
    // subnormals land on subnormals), undone by an exact product with 2^120
    const uint32_t a = prmt(w, 0, 0x1404), b = prmt(w, 0, 0x3424);
    lo = bf2_mul(((a >> 4) & 0x07F007F0u) | (a & 0x80008000u), 0x7B807B80u);
    hi = bf2_mul(((b >> 4) & 0x07F007F0u) | (b & 0x80008000u), 0x7B807B80u);
  }
}

template <bool BF>
__device__ __forceinline__ void int8_to_16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (!BF) {
    const uint32_t u = w ^ 0x80808080u;                      // 1024 + (code + 128), minus 1152
    lo = hsub2_u32(prmt(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_u32(prmt(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    // 128 + the low seven bits, minus 128, or 256 for a negative code: the
    // code's sign bit is the lowest exponent bit of 0x43xx
    const uint32_t a = prmt(w, 0x43434343u, 0x4140), b = prmt(w, 0x43434343u, 0x4342);
    lo = bf2_sub(a & 0xFF7FFF7Fu, a & 0xFF80FF80u);
    hi = bf2_sub(b & 0xFF7FFF7Fu, b & 0xFF80FF80u);
  }
}

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {   // read once: past the L1
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// 16 bytes of which `bytes` (16 or 0) are read, the rest zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void prefetch_l2(const uint8_t* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// mbar_wait (common.cuh) whose every attempt lets the hardware suspend the warp
// for a while (28 warps share the issue slots, and most of them wait), and that
// reads the clock only every 64 attempts.
constexpr uint32_t kSuspendNs = 1000;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return true;
    if ((i & 63u) == 0) {
      const unsigned long long t = global_ns();
      if (t0 == 0) t0 = t;
      if (*abort || t - t0 > kWaitLimitNs) return false;
    }
  }
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void group_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
// group_bar that tells every thread whether any of them said yes
__device__ __forceinline__ bool group_bar_any(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// offset of 16-byte vector c (8 dims) of row r in a tile of 64-dim halves, each
// row 128 bytes, vectors permuted by the row (128-byte swizzle)
__device__ __forceinline__ uint32_t tile_off(int r, int c) { return (uint32_t)((c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)); }

// A loader warp's chunk is 16 rows of K or V, contiguous in its page; a lane
// holds 16-byte vectors of it in registers, step s the 512 bytes from 512 s on.
// Eight neighbouring lanes have to store to eight different 16-byte vectors of
// 128 bytes.  Sixteen codes become two such vectors, so over 128-byte raw rows
// (8-bit pages, 128 dims) they take two rows by four vectors of one 64-dim
// half; everywhere else raw order does it.
template <int D, int VB>             // VB: 16-byte vectors of a raw row
__device__ __forceinline__ int lane_row(int lane) {
  return (VB == 8 && D == 128) ? 2 * (lane >> 4) + ((lane >> 2) & 1) : lane / VB;
}
template <int D, int VB>
__device__ __forceinline__ int lane_vec(int lane) {
  return (VB == 8 && D == 128) ? 4 * ((lane >> 3) & 1) + (lane & 3) : lane % VB;
}

// kSteps steps of a chunk from step s0 on: registers from the chunk at src ...
constexpr int kSteps = 4;
template <int D, int VB>
__device__ __forceinline__ void load_steps(uint4 (&v)[kSteps], const uint8_t* src, int lane, int s0) {
  src += (lane_row<D, VB>(lane) * VB + lane_vec<D, VB>(lane)) * 16 + s0 * 512;
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    if (s < VB / 2) v[s] = ldg16(src + s * 512);
}

// ... and to the tile; `tile`: the place of the chunk's first row.  Rows from
// n_rows on become zeros (P is 0 there, and 0 times what the page holds behind
// the sequence would be NaN if that is).
template <int D, bool BF, int CODEC>
__device__ __forceinline__ void store_steps(uint4 (&v)[kSteps], uint32_t tile, int lane, int n_rows, int s0) {
  constexpr int VB = CODEC <= ARGUS_BF16 ? D / 8 : D / 16;   // vectors per raw row
  constexpr int STEPS = VB / 2 < kSteps ? VB / 2 : kSteps, ROWS = 32 / VB;   // rows per step
  const int r0 = lane_row<D, VB>(lane) + s0 * ROWS, j = lane_vec<D, VB>(lane);
  if (n_rows < 16) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      if (r0 + s * ROWS >= n_rows) v[s] = make_uint4(0, 0, 0, 0);
  }
  // vector c of row r0 is the first that this lane writes; rows further down
  // are 128 bytes apart, and their permutation differs by the row's low bits
  const int c = CODEC <= ARGUS_BF16 ? j : 2 * j;
  const uint32_t base = tile + (c >> 3) * kHalf + r0 * 128;
  const uint32_t off = (uint32_t)(((c & 7) ^ (r0 & 7)) << 4);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    // r0 + s ROWS adds no carry into or out of r0's low bits: xor and sum agree
    const uint32_t at = base + s * ROWS * 128 + (off ^ (uint32_t)(((s * ROWS) & 7) << 4));
    if constexpr (CODEC <= ARGUS_BF16) {
      sts16(at, v[s].x, v[s].y, v[s].z, v[s].w);
    } else {
      uint32_t o[8];
      const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (CODEC == ARGUS_FP8_E4M3) fp8_to_16<BF>(w[e], o[2 * e], o[2 * e + 1]);
        else int8_to_16<BF>(w[e], o[2 * e], o[2 * e + 1]);
      }
      sts16(at, o[0], o[1], o[2], o[3]);
      sts16(at ^ 16u, o[4], o[5], o[6], o[7]);
    }
  }
}

// Q tile of an item, by warps w = 0 .. nw - 1: row l of the tile goes to TMEM lanes
// l, l + per, ....  All rows are on their way at once (asynchronous copies,
// which write zeros where they read nothing); those that become fp16 (TURN: from
// the tile at q_s to the one at q16, which may be the same unless KEEP) are
// turned by the lanes that copied them.  Behind the last row the tile gets zeros
// if `fill`, else keeps what it holds: rows of an item before, whose scores
// nobody uses.
template <int D, bool TURN, bool KEEP>
__device__ __forceinline__ void load_q(const EParams& p, const Cursor& c, uint32_t q_s, uint32_t q16, float* q_scale, int w, int nw, int lane,
                                       bool fill) {
  constexpr int V = D / 8, RW = 32 / V;                  // vectors per row; rows of a warp's step
  const int v = lane % V, r0 = w * RW + lane / V, RS = RW * nw;
  const int lin0 = c.t * kBM, rows = min(kBM, c.s.n * p.G - lin0);
  const int nrep = replicas(rows), per = kBM / nrep, lim = fill ? per : rows;
  const int ncopy = TURN && !KEEP ? 1 : nrep;            // the turned rows are copied below
  const int tok = group_of(p, lin0 + r0), dt = group_of(p, RS), dg = RS - dt * p.G;
  int g = lin0 + r0 - tok * p.G;
  const uint16_t* src = p.q + (long long)(c.s.q0 + tok) * p.qs + (long long)(c.h * p.G + g) * D + v * 8;
  const long long step = dt * p.qs + dg * D, wrap = p.qs - (long long)p.G * D;
#pragma unroll 1
  for (int l = r0; l < lim; l += RS) {
    const bool real = l < rows;
#pragma unroll 1
    for (int r = 0; r < ncopy; ++r) cp_async16(q_s + tile_off(l + r * per, v), real ? src : p.q, real ? 16 : 0);
    src += step;
    g += dg;
    if (g >= p.G) {
      g -= p.G;
      src += wrap;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (TURN) {
    // the row's largest magnitude comes to [2^14, 2^15); its D / 8 lanes are
    // neighbours.  Four rows at once: one after the other, their reads,
    // exchanges and stores would only wait for each other.
    constexpr int R = 4;
    for (int i0 = w * RW; i0 < lim; i0 += R * RS) {      // by whole warps
      const int l0 = i0 + lane / V;
      uint4 q[R];
      uint32_t mx[R];
#pragma unroll
      for (int x = 0; x < R; ++x) q[x] = lds16(q_s + tile_off(min(l0 + x * RS, kBM - 1), v));
#pragma unroll
      for (int x = 0; x < R; ++x)                        // magnitudes of bf16 order like their bits
        mx[x] = max_u16x2(max_u16x2(q[x].x & 0x7FFF7FFFu, q[x].y & 0x7FFF7FFFu), max_u16x2(q[x].z & 0x7FFF7FFFu, q[x].w & 0x7FFF7FFFu));
#pragma unroll
      for (int o = V / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int x = 0; x < R; ++x) mx[x] = max_u16x2(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], o));
      }
      uint32_t ex[R];
#pragma unroll
      for (int x = 0; x < R; ++x) {
        ex[x] = max(max(mx[x] >> 16, mx[x] & 0xFFFFu) >> 7, 15u);   // biased; from 15 on 2^(141 - ex) is a normal number
        const float f = __uint_as_float((268 - ex[x]) << 23);
        uint32_t* w = reinterpret_cast<uint32_t*>(&q[x]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a, b;
          f2_mul(a, b, __uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u), f, f);
          w[e] = pack_f16x2(a, b);
        }
      }
#pragma unroll 1
      for (int r = 0; r < nrep; ++r) {
#pragma unroll
        for (int x = 0; x < R; ++x) {
          const int l = l0 + x * RS;
          if (l < lim) {
            sts16(q16 + tile_off(l + r * per, v), q[x].x, q[x].y, q[x].z, q[x].w);
            if (v == 0) q_scale[l + r * per] = __uint_as_float((ex[x] - 14) << 23);   // 1 / f
          }
        }
      }
    }
  }
  fence_async();
  __syncwarp();
}

// The lookup warp finds the pages of kBatch blocks at once, a lane per chunk
// (lane = 8 * block + chunk): the two dependent reads (table, then scales) are
// paid once per batch, and the batches behind are read meanwhile.
struct Lookup {
  int codec, slot, row, n_rows, h, first;   // first: this chunk counts a page that cannot be read
};
struct Found {
  const uint8_t* src;
  uint32_t state;                    // codec | rows << 8; 0: nothing to read
  float ks, vs;                      // ks < 0: a page that cannot be read
};

// One lane of the warp, the same each time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x;
}
// Shared-memory operands of 128-byte swizzled tiles: the descriptor's high word
// is the same for all (stride 1024 bytes between 8-row groups, layout, version; tc::sdesc).
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) { return (uint32_t)tc::sdesc(saddr, lbo, 1024); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss_lead(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(lead), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lead(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(acc), "r"(lead), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit_lead(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lead)
      : "memory");
}

// BF: q and out are bf16, else fp16.  W16: the call has a 16-bit pool.  The
// operands are bf16 only in blocks that hold bf16 pages: elsewhere a bf16 query
// is taken as fp16 times a power of two per row (its 8 bits fit, down to
// 2^-31 of the row's largest element), because e4m3 codes
// turn into fp16 with one conversion per pair, into bf16 with five operations,
// and fp16 P has three more bits.  A call with both kinds of pages keeps both
// query tiles and chooses per block.
template <int D, bool BF, bool W16>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const EParams p) {
  using SM = Smem<D>;
  constexpr int kTile = SM::kTile;
  constexpr bool MIXED = BF && W16;          // bf16 or fp16 operands, block by block
  constexpr float kPBias = 7.f;              // P is stored as P * 2^7 (fp16: at most 2^15)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {         // the swizzled tiles need it
    if (threadIdx.x == 0) {
      cuts(p, D)[blockIdx.x] = Cut{};
      if (p.status) atomicOr(p.status, kStatusTimeoutBit);
    }
    return;
  }
  uint64_t* q_first = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);  // the first item's Q tile
  uint64_t* q_full = q_first + 1;      // item k >= 1: buffer k & 1
  uint64_t* k_full = q_full + 2;       // block n: buffer n & 1
  uint64_t* pv_ready = k_full + 2;     // V tile and P written
  uint64_t* s_full = pv_ready + 2;     // scores complete; the K tile is free
  uint64_t* o_done = s_full + 2;       // P.V complete; the V tile is free
  uint64_t* o_free = o_done + 2;       // item k: its epilogue is done with O and with its Q buffer
  uint64_t* drain = o_free + 2;
  uint64_t* looked = drain + 1;        // a batch of blocks is looked up
  uint64_t* used = looked + kBatches;  // nobody needs the batch any more
  // [0] TMEM base, [1] error, [2..11] the range's first block (Cursor::store), [12..15] the
  // blocks in front of the range's begin and end
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::kOffMisc);
  volatile long long* misc64 = reinterpret_cast<volatile long long*>(smem + SM::kOffMisc);
  // [2][8]: q0, n, len, h, t, first block, blocks of the piece, blocks of the item
  volatile int* items = reinterpret_cast<volatile int*>(smem + SM::kOffItem);
  float2* ml = reinterpret_cast<float2*>(smem + SM::kOffML);            // [group][lane]: (m, l)
  float* q_scale = reinterpret_cast<float*>(smem + SM::kOffQScale);
  uint4* chunks = reinterpret_cast<uint4*>(smem + SM::kOffChunk);       // [slot][chunk]: K source, state
  float4* scales = reinterpret_cast<float4*>(smem + SM::kOffScale);     // [slot][chunk]: ks (< 0: not to be read), log2 vs, 1 / vs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the second kernel may be put in place; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 2) {
    // the range's begin and end, a warp each
    const Boundary r = find_boundary(p, blockIdx.x + warp);
    if (lane == 0) misc64[6 + warp] = r.blocks;
    if (warp == 0) {
      const Cursor& c = r.at;
      if (lane == 0) c.store(misc + 2);
      Cut cut = {};
      if ((int)blockIdx.x < r.n && c.blk > 0) {
        const long long first = r.unit - c.blk;          // the unit of the item's first block
        // this range begins inside an item's blocks; is it the first to?
        if (range_start(r.total, blockIdx.x - 1, r.n) <= first) {
          cut.rows = min(kBM, c.s.n * p.G - c.t * kBM);
          cut.last = blockIdx.x;
          while (cut.last + 1 < r.n && range_start(r.total, cut.last + 1, r.n) < first + c.nb) ++cut.last;
          cut.q0 = c.s.q0;
          cut.row0 = c.t * kBM;
          cut.head0 = c.h * p.G;
        }
      }
      if (lane == 0) cuts(p, D)[blockIdx.x] = cut;
    }
  }
  if (threadIdx.x == 64) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], kQWarps);
      mbar_init(&k_full[b], kLoadWarps / 2);
      mbar_init(&pv_ready[b], kLoadWarps / 2 + kSoftmaxWarps);
      mbar_init(&s_full[b], 1);
      mbar_init(&o_done[b], 1);
      mbar_init(&o_free[b], kSoftmaxWarps);
    }
    mbar_init(q_first, kSoftmaxWarps);
    mbar_init(drain, 1);
    for (int k = 0; k < kBatches; ++k) {
      mbar_init(&looked[k], 1);
      mbar_init(&used[k], kLoadWarps);
    }
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32((const void*)&misc[0])),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int n_blocks = (int)(misc64[7] - misc64[6]);   // fewer than 2^31 (checked on the host)
  auto describe_item = [&](int k, const Cursor& c, int nb) {
    volatile int* it = items + 8 * (k & 1);
    it[0] = c.s.q0; it[1] = c.s.n; it[2] = c.s.len; it[3] = c.h; it[4] = c.t; it[5] = c.blk; it[6] = nb; it[7] = c.nb;
  };
  // item k's Q tile and description are there
  auto wait_q = [&](int k) {
    return k == 0 ? wait(q_first, 0, &misc[1]) : wait(&q_full[k & 1], (uint32_t)((k - 1) >> 1) & 1, &misc[1]);
  };
  auto tS = [tmem](int b) { return tmem + 128u * (uint32_t)b; };
  auto tO = [tmem](int b) { return tmem + 256u + 128u * (uint32_t)b; };

  if (n_blocks <= 0) {
    // nothing in this CTA's range
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // within an item: S0, S1, then per block i: P.V of i, S of i + 2.  The whole
    // warp runs this, one elected lane issues: descriptors and loop counters
    // stay warp-uniform, where the MMA instruction wants them.
    constexpr uint32_t kBf16Operands = (1u << 7) | (1u << 10);
    constexpr uint32_t idQK = idesc_f16kind(false, false, kBN), idPV = idesc_f16kind(false, true, D);
    static_assert((idQK | kBf16Operands) == idesc_f16kind(true, false, kBN), "operand type bits");
    // whether block n's operands are bf16
    auto is_wide = [&](int n) { return MIXED ? __shfl_sync(0xffffffffu, chunks[(n % kSlots) * 8].w, 0) : 0u; };
    const uint32_t lead = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    // low words of the operand descriptors: address and leading offset in 16-byte units
    const uint32_t q_lo = sdesc_lo(smem_u32(smem + SM::kOffQ), kHalf), k_lo = sdesc_lo(smem_u32(smem + SM::kOffK), kHalf);
    const uint32_t v_lo = sdesc_lo(smem_u32(smem + SM::kOffV), kHalf);
    Cursor c;
    c.load(misc + 2, n_blocks);
    int n0 = 0;                        // blocks before this item's
    bool ok = true;
    auto issue_s = [&](int n, int k) {
      const int b = n & 1;
      if (!__all_sync(0xffffffffu, wait(&k_full[b], (uint32_t)(n >> 1) & 1, &misc[1]))) return false;
      tc_fence_after();
      const uint32_t wide = is_wide(n), id = idQK | (wide ? kBf16Operands : 0u);
      // two items' tiles, or an item's bf16 and fp16 tile
      const uint32_t ql = q_lo + (MIXED ? 1 - wide : (uint32_t)(k & 1)) * (kTile / 16), kl = k_lo + (uint32_t)b * (kTile / 16);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) / 16;
        mma_ss_lead(tm + 128u * b, ql + off, kl + off, id, kk > 0, lead);
      }
      commit_lead(&s_full[b], lead);
      return true;
    };
    auto issue_pv = [&](int n, bool first) {
      const int b = n & 1;
      if (!__all_sync(0xffffffffu, wait(&pv_ready[b], (uint32_t)(n >> 1) & 1, &misc[1]))) return false;
      tc_fence_after();
      const uint32_t vl = v_lo + (uint32_t)b * (kTile / 16), id = idPV | (is_wide(n) ? kBf16Operands : 0u);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)              // group g: keys 64 g ..., its P and its O
        mma_ts_lead(tm + 256u + 128u * (kk >> 2), tm + 128u * b + (kk >> 2) * 64 + (kk & 3) * 8, vl + kk * 128, id,
                    !first || (kk & 3) > 0, lead);
      commit_lead(&o_done[b], lead);
      return true;
    };
    for (int k = 0; ok && n0 < n_blocks; ++k) {
      const int nb = __shfl_sync(0xffffffffu, min(c.nb - c.blk, c.left), 0);
      ok = __all_sync(0xffffffffu, wait_q(k));
      if (ok) ok = issue_s(n0, k);
      if (ok && nb > 1) ok = issue_s(n0 + 1, k);
      // the scores of this item may overtake the epilogue of the one before; its P.V may not
      if (ok && k > 0) ok = __all_sync(0xffffffffu, wait(&o_free[(k - 1) & 1], (uint32_t)((k - 1) >> 1) & 1, &misc[1]));
      for (int i = 0; i < nb && ok; ++i) {
        ok = issue_pv(n0 + i, i == 0);
        if (ok && i + 2 < nb) ok = issue_s(n0 + i + 2, k);
      }
      n0 += nb;
      c.advance(p, nb);
    }
    if (!ok) {
      const volatile uint32_t never = 0;
      misc[1] = 1;
      commit_lead(drain, lead);        // TMEM is freed after the MMAs in flight
      wait(drain, 0, &never);
    }
  } else if (warp >= kQWarp0) {
    // ---------------------------------------------------------- Q tiles
    // From the second item on, an item ahead of the softmax groups (which load the
    // first one's themselves).
    Cursor c;
    c.load(misc + 2, n_blocks);
    c.advance(p, min(c.nb - c.blk, c.left));
    for (int k = 1; c.left > 0; ++k) {
      const int nb = min(c.nb - c.blk, c.left);
      // the buffer's last item is done: two items ago, or with two tiles per item the one before
      const int last = MIXED ? k - 1 : k - 2;
      if (last >= 0 && !__all_sync(0xffffffffu, wait(&o_free[last & 1], (uint32_t)(last >> 1) & 1, &misc[1]))) { misc[1] = 1; break; }
      if (warp == kQWarp0 && lane == 0) describe_item(k, c, nb);
      const uint32_t q_s = smem_u32(smem + SM::kOffQ + (MIXED ? 0 : (k & 1) * kTile));
      load_q<D, BF, MIXED>(p, c, q_s, MIXED ? q_s + kTile : q_s, q_scale + (k & 1) * kBM, warp - kQWarp0, kQWarps, lane, k == 1);
      if (lane == 0) mbar_arrive(&q_full[k & 1]);
      c.advance(p, nb);
    }
  } else if (warp == kLookWarp) {
    // ---------------------------------------------------------- lookup
    Cursor c;
    c.load(misc + 2, n_blocks);
    auto look = [&]() {
      Lookup k;
      k.codec = k.slot = -1;
      k.row = k.n_rows = k.h = k.first = 0;
      int b = 0, key = 0;
#pragma unroll 1
      for (int x = 0; x < kBatch && c.left > 0; ++x) {
        if (lane / 8 == x) {
          b = c.b;
          key = c.blk * kBN + (lane & 7) * 16;
          k.n_rows = min(max(c.s.len - key, 0), 16);
          k.h = c.h;
          k.first = c.h == 0 && c.t == c.T - 1;
        }
        c.advance(p, 1);
      }
      if (k.n_rows > 0) {
        const int page = (int)((uint32_t)key / (uint32_t)p.P);
        k.row = key - page * p.P;
        k.first = k.first && k.row == 0;
        const size_t e = (size_t)b * p.max_pages + page;
        k.codec = p.page_codec[e];
        k.slot = p.block_table[e];
      }
      return k;
    };
    auto resolve = [&](const Lookup& k) {
      Found f;
      f.src = nullptr;
      f.state = 0;
      f.ks = f.vs = 1.f;
      if (k.n_rows > 0) {
        const bool known = k.codec <= ARGUS_INT8 && (W16 || k.codec >= ARGUS_FP8_E4M3);
        const PoolRef r = p.pool[k.codec & 3];
        if (!known || k.slot < 0 || k.slot >= r.n_slots) {
          f.ks = -1.f;
          if (k.first && p.status) atomicAdd(p.status, 1u);
        } else {
          const int rb = k.codec <= ARGUS_BF16 ? 2 * D : D;
          const long long unit = (long long)k.slot * 2 * p.Hkv + k.h;
          f.src = r.codes + (unit * p.P + k.row) * rb;
          f.state = k.codec | k.n_rows << 8;
          if (k.codec >= ARGUS_FP8_E4M3) {
            f.ks = r.meta[unit];
            f.vs = r.meta[unit + p.Hkv];
          }
        }
      }
      return f;
    };
    // toward the L2, some blocks before a loader asks for it: what the loaders have
    // in flight in registers would not cover a DRAM read
    auto ahead = [&](const Found& f) {
      if (!f.state) return;
      const int rb = (W16 && (f.state & 0xFF) <= ARGUS_BF16) ? 2 * D : D;
      prefetch_l2(f.src, 16 * rb);
      prefetch_l2(f.src + (long long)p.Hkv * p.P * rb, 16 * rb);
    };
    // three batches on their way: table entries, scales, and the one handed out
    Lookup table = look();
    Found next = resolve(table);
    table = look();
    for (int k = 0; k * kBatch < n_blocks; ++k) {
      const Found now = next;
      next = resolve(table);
      table = look();
      if (k >= kBatches && !__all_sync(0xffffffffu, wait(&used[k % kBatches], (uint32_t)(k / kBatches - 1) & 1, &misc[1]))) {
        misc[1] = 1;
        break;
      }
      const int at = (k % kBatches) * 32 + lane;
      const unsigned long long addr = reinterpret_cast<unsigned long long>(now.src);
      // does the block (this lane's group of eight) hold a bf16 page?
      const unsigned bf16s = __ballot_sync(0xffffffffu, MIXED && now.state && (now.state & 0xFF) <= ARGUS_BF16);
      const uint32_t wide = (bf16s >> (lane & 24) & 0xFF) != 0;
      chunks[at] = make_uint4((uint32_t)addr, (uint32_t)(addr >> 32), now.state, wide);
      const float lvs = log2f(now.vs);   // 0: -inf
      // a scale far from 1: its chunk's sum is kept apart, and does not enter the others'
      scales[at] = make_float4(now.ks < 0.f ? -1.f : now.ks * p.scale_log2, lvs, fabsf(lvs) > kFarScale ? 0.f : 1.f / now.vs, wide ? 1.f : 0.f);
      __syncwarp();
      if (lane == 0) mbar_arrive(&looked[k % kBatches]);
      ahead(now);
    }
  } else if (warp >= kSoftmaxWarps) {
    // ---------------------------------------------------------- loaders
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    const int lw = warp - kSoftmaxWarps, ch = lw & 7;
    const bool is_v = lw >= kLoadWarps / 2;
    const uint32_t tiles = smem_u32(smem + (is_v ? SM::kOffV : SM::kOffK)) + ch * 2048;
    uint64_t* full = is_v ? pv_ready : k_full;
    uint64_t* empty = is_v ? o_done : s_full;
    const long long v_off = is_v ? (long long)p.Hkv * p.P * D : 0;   // V behind K in an 8-bit page
    bool ok = true;
    uint4 v[kSteps];
    uint32_t state = 0;
    const uint8_t* src = nullptr;
    // the description of the warp's chunk of block i
    auto describe = [&](uint32_t i) {
      if (i >= (uint32_t)n_blocks) return make_uint4(0, 0, 0, 0);
      if (i % kBatch == 0 && ok) ok = wait(&looked[(i / kBatch) % kBatches], (i / kSlots) & 1, &misc[1]);
      return chunks[(i % kSlots) * 8 + ch];
    };
    // the chunk on its way: all of it, or the first half of 16-bit rows of 128 dims
    auto fetch = [&](const uint4& d) {
      state = ok ? d.z | d.w << 16 : 0;                  // codec | rows << 8 | bf16 operands << 16
      if (!(state & 0xFF00)) return;
      src = reinterpret_cast<const uint8_t*>((unsigned long long)d.y << 32 | d.x) + v_off;
      if (W16 && (state & 0xFF) <= ARGUS_BF16) {
        src += v_off;
        load_steps<D, D / 8>(v, src, lane, 0);
      } else {
        load_steps<D, D / 16>(v, src, lane, 0);
      }
    };
    fetch(describe(0));
    uint4 next = describe(1);
    for (uint32_t i = 0; i < (uint32_t)n_blocks; ++i) {
      const uint32_t b = i & 1;
      if (i >= 2 && ok) ok = wait(&empty[b], ((i >> 1) - 1) & 1, &misc[1]);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        const int codec = state & 0xFF, n_rows = (state >> 8) & 0xFF;
        const bool wide = MIXED && (state >> 16);
        const uint32_t to = tiles + b * kTile;
        if (n_rows > 0 || is_v) {                      // a chunk without rows: K is masked, V is set to zero
          if (W16 && codec <= ARGUS_BF16) {
            store_steps<D, MIXED, ARGUS_BF16>(v, to, lane, n_rows, 0);
            if (D == 128) {
              if (n_rows > 0) load_steps<D, D / 8>(v, src, lane, kSteps);
              store_steps<D, MIXED, ARGUS_BF16>(v, to, lane, n_rows, kSteps);
            }
          } else if (MIXED && wide) {
            if (codec == ARGUS_INT8) store_steps<D, true, ARGUS_INT8>(v, to, lane, n_rows, 0);
            else store_steps<D, true, ARGUS_FP8_E4M3>(v, to, lane, n_rows, 0);
          } else if (codec == ARGUS_INT8) {
            store_steps<D, false, ARGUS_INT8>(v, to, lane, n_rows, 0);
          } else {
            store_steps<D, false, ARGUS_FP8_E4M3>(v, to, lane, n_rows, 0);
          }
        }
        fetch(next);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[b]);
          // this block's tile was free, so the softmax of four blocks ago is
          // done: the batch before the last one is not needed any more
          if (i % kBatch == kBatch - 1 && i >= kBatch) mbar_arrive(&used[(i / kBatch - 1) % kBatches]);
        }
        next = describe(i + 2);
      }
    }
    if (!ok) misc[1] = 1;
  } else {
    // ---------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int grp = warp / kGroupWarps, wq = warp % kGroupWarps;
    const int tl = wq * 32 + lane;                     // TMEM lane
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t sO = tO(grp) + lane_off;
    float* merge = reinterpret_cast<float*>(smem + SM::kOffMerge) + grp * 96 * kMergePad;
    int n0 = 0;
    {
      Cursor c;
      c.load(misc + 2, n_blocks);
      if (threadIdx.x == 0) describe_item(0, c, min(c.nb - c.blk, c.left));
      const uint32_t q_s = smem_u32(smem + SM::kOffQ);
      load_q<D, BF, MIXED>(p, c, q_s, MIXED ? q_s + kTile : q_s, q_scale, warp, kSoftmaxWarps, lane, true);
      if (lane == 0) mbar_arrive(q_first);
    }
    for (int k = 0; n0 < n_blocks; ++k) {
      bool alive = wait_q(k);
      if (group_bar_any(1, kSoftmaxWarps * 32, !alive)) { misc[1] = 1; break; }   // all leave, or none
      const volatile int* it = items + 8 * (k & 1);
      const int nb = it[6], k_first = it[5] * kBN;
      const int rows = min(kBM, it[1] * p.G - it[4] * kBM);
      const int nrep = replicas(rows), per = kBM / nrep;
      const float q_fac = BF ? q_scale[(k & 1) * kBM + tl] : 1.f;   // undoes the fp16 query's power of two
      const int l_row = tl & (per - 1);                // row within the tile
      const int rep = tl / per;                        // this lane's replica: chunks c0 ... of the group's four
      const int c0 = 4 * grp + rep * (4 / nrep);
      // rows behind the last one see what the last one sees: they are never written
      const int tok = min(group_of(p, it[4] * kBM + l_row), it[1] - 1);
      const int vis_last = min(p.causal ? it[2] - it[1] + tok : it[2] - 1, it[2] - 1);
      // running reference and sum.  m bounds score + log2 of the V scale, for P's
      // range; a weight's share of the sum knows nothing of the scale, so where scales
      // are far from 1 sums are kept apart, in lz relative to mz, the largest score:
      // of a chunk with a far scale (it may be 0), and from the first one far above 1
      // on of all chunks (relative to an m that it raised they could leave fp32's range).
      float m = -INFINITY, l = 0.f, mz = -INFINITY, lz = 0.f;
      bool apart = false;                              // the same in the whole warp
      auto scale_acc = [&](float r) {                  // rare: few registers, not speed
#pragma unroll 1
        for (int x = 0; x < D / 8; ++x) {
          uint32_t v[8];
          tmem_ld8(sO + x * 8, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * r);
          tmem_st8(sO + x * 8, v);
        }
        tmem_wait_st();
      };
      // One block, N chunks of 16 keys per lane, all scores in registers.
      auto block = [&](auto chunks_of, int n, int k0) {
        constexpr int N = decltype(chunks_of)::value;
        const uint32_t sS = tS(n & 1) + lane_off;
        const float4* sc = scales + (n % kSlots) * 8 + c0;
        const bool wide = MIXED && sc[0].w != 0.f;     // the same for the block's chunks
        const float qf = wide ? 1.f : q_fac;
        float v[N][16];
#pragma unroll
        for (int x = 0; x < N; ++x) tmem_ld16(sS + (c0 + x) * 16, reinterpret_cast<uint32_t(&)[16]>(v[x]));
        // lanes 0 .. N-1 look at their chunk, every lane at its row's last key
        const bool odd = lane < N && (sc[lane].x < 0.f || fabsf(sc[lane].y) > kFarScale);
        const int lim = vis_last - k0 - c0 * 16;       // keys e <= lim of the lane's are visible
        const bool edge = __any_sync(0xffffffffu, odd || lim < N * 16 - 1) || apart;
        tmem_wait_ld();
        if (edge) {
          // the scores scaled and masked here, log2 of the V scale added, sums kept apart
          bool above = false;
#pragma unroll
          for (int x = 0; x < N; ++x) above |= sc[x].y > kFarScale;
          if (above && !apart) {
            apart = true;
            const float ref = m - kPBias, top = fmaxf(mz, ref);
            if (m != -INFINITY) {
              lz = lz * fast_exp2(mz - top) + l * fast_exp2(ref - top);
              mz = top;
            }
          }
#pragma unroll
          for (int x = 0; x < N; ++x) {
            const float kq = sc[x].x * qf, lvc = sc[x].y;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[x][e] = (kq >= 0.f && x * 16 + e <= lim) ? v[x][e] * kq : -INFINITY;
            if (apart || fabsf(lvc) > kFarScale) {
              float top = mz;
#pragma unroll
              for (int e = 0; e < 16; ++e) top = fmaxf(top, v[x][e]);
              if (top != -INFINITY) {
                lz *= fast_exp2(mz - top);
                mz = top;
#pragma unroll
                for (int e = 0; e < 16; ++e) lz += fast_exp2(v[x][e] - top);
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[x][e] += lvc;
          }
        }
        // the maximum of score + log2 of the V scale, so that P times that scale stays in range
        float mj = -INFINITY;
#pragma unroll
        for (int x = 0; x < N; ++x) {
          float a0 = max3(v[x][0], v[x][1], v[x][2]), a1 = max3(v[x][3], v[x][4], v[x][5]);
          a0 = max3(a0, v[x][6], v[x][7]);
          a1 = max3(a1, v[x][8], v[x][9]);
          a0 = max3(a0, v[x][10], v[x][11]);
          a1 = max3(a1, v[x][12], v[x][13]);
          a0 = max3(a0, v[x][14], v[x][15]);
          const float a = fmaxf(a0, a1);
          mj = fmaxf(mj, edge ? a : fmaf(a, sc[x].x * qf, sc[x].y));
        }
        const bool move = mj > m + kRescaleThreshold || (m == -INFINITY && mj != -INFINITY);
        const bool scale_o = move && m != -INFINITY;
        if (__any_sync(0xffffffffu, scale_o)) {
          // the block before (of this item, as m is set) is the last that added to O
          if (!__all_sync(0xffffffffu, wait(&o_done[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1, &misc[1]))) return false;
          tc_fence_after();
          const float r = scale_o ? fast_exp2(m - mj) : 1.f;
          scale_acc(r);
          l *= r;
        }
        if (move) m = mj;
        // P times the V scale over the consumed scores, packed: the group's 64
        // keys in 32 columns, zeros for the other replicas' keys.  The row sum wants P
        // without the scale: a chunk's sum is divided by it once.
        const float mm = (m == -INFINITY) ? 0.f : m - kPBias;
        const uint32_t sP = sS + 64 * grp;
        if (N < 4) {
          const uint32_t z[8] = {};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (x < c0 - 4 * grp || x >= c0 - 4 * grp + N) tmem_st8(sP + x * 8, z);
        }
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const float4 s = sc[x];
          const float kq = edge ? 1.f : s.x * qf, shift = edge ? -mm : s.y - mm;
          float la = 0.f, lb = 0.f;
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float x0, x1, p0, p1;
            f2_fma(x0, x1, v[x][2 * e], v[x][2 * e + 1], kq, kq, shift, shift);
            p0 = fast_exp2(x0);
            p1 = fast_exp2(x1);
            f2_add(la, lb, la, lb, p0, p1);
            o[e] = wide ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
          }
          l = fmaf(la + lb, s.z, l);
          tmem_st8(sP + (c0 - 4 * grp + x) * 8, o);
        }
        tmem_wait_st();
        return true;
      };
      for (int i = 0; i < nb; ++i) {
        const int n = n0 + i, k0 = k_first + i * kBN;
        if (!__all_sync(0xffffffffu, wait(&s_full[n & 1], (uint32_t)(n >> 1) & 1, &misc[1]))) { alive = false; break; }
        tc_fence_after();
        if (nrep == 4) alive = block(std::integral_constant<int, 1>{}, n, k0);
        else if (nrep == 2) alive = block(std::integral_constant<int, 2>{}, n, k0);
        else alive = block(std::integral_constant<int, 4>{}, n, k0);
        if (!alive) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pv_ready[n & 1]);
      }
      if (alive) alive = __all_sync(0xffffffffu, wait(&o_done[(n0 + nb - 1) & 1], (uint32_t)((n0 + nb - 1) >> 1) & 1, &misc[1]));
      if (!alive) misc[1] = 1;
      tc_fence_after();
      // references in the units that l was summed in.  Sums kept apart stay near
      // mz, a score: what the other group and the other copies have does not fall out
      // of range beside them.  O in those units is the result times lz: 2^-32 of
      // it where it could overflow.
      float ref = m == -INFINITY ? -INFINITY : m - kPBias, sum = l;
      if (__any_sync(0xffffffffu, mz != -INFINITY)) {
        float r = 1.f;                                 // its square is what O is scaled by: 2^+-140
        if (mz != -INFINITY) {
          const float top = apart ? (ref - mz > 64.f ? mz + 32.f : mz) : fmaxf(ref, mz);
          r = fast_exp2(0.5f * (ref - top));           // ref = -inf: 0
          // with all sums in lz, l counts for nothing (unless a query that holds NaN made it NaN)
          sum = sum * (apart ? 0.f : r * r) + lz * fast_exp2(mz - top);
          ref = top;
        }
#pragma unroll 1
        for (int x = 0; x < 2; ++x) scale_acc(r);
      }
      ml[grp * kBM + tl] = make_float2(ref, sum);
      tc_fence_before();
      group_bar(1, kSoftmaxWarps * 32);
      tc_fence_after();
      // ---- epilogue: both groups' and all replicas' sums of a row joined; group g takes half the dims
      float M = -INFINITY, l_all = 0.f;
      float2 y[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) y[x] = x < 2 * nrep ? ml[(x & 1) * kBM + (x >> 1) * per + l_row] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int x = 0; x < 8; ++x) M = fmaxf(M, y[x].x);
#pragma unroll
      for (int x = 0; x < 8; ++x) l_all += y[x].x == -INFINITY ? y[x].y : y[x].y * fast_exp2(y[x].x - M);   // the first: 0, or NaN
      const float2 y0 = ml[tl], y1 = ml[kBM + tl];
      const bool have = l_all != 0.f;                  // NaN (from a query that holds one) is not nothing
      const float inv = have ? 1.f / l_all : 0.f;
      const float w0 = (have && y0.x != -INFINITY) ? fast_exp2(y0.x - M) * inv : 0.f;
      const float w1 = (have && y1.x != -INFINITY) ? fast_exp2(y1.x - M) * inv : 0.f;
      const bool whole = it[5] == 0 && nb == it[7];
      const int piece = 2 * blockIdx.x + (it[5] == 0 ? 1 : 0);
      const bool writes = alive && rep == 0 && l_row < rows;
      const int lin = it[4] * kBM + l_row, otok = group_of(p, lin);
      const size_t orow = writes ? (size_t)(it[0] + otok) * p.Hq + it[3] * p.G + (lin - otok * p.G) : 0;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {                 // short code: every item runs through it once, out of a cold cache
        const int col = grp * (D / 2) + x * 16;
        uint32_t v0[16], v1[16];
        float o[16];
        tmem_ld16(tO(0) + lane_off + col, v0);
        tmem_ld16(tO(1) + lane_off + col, v1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(w0, __uint_as_float(v0[e]), w1 * __uint_as_float(v1[e]));
        if (nrep > 1) {
          if (rep > 0) {
            float4* d = reinterpret_cast<float4*>(merge + ((rep - 1) * per + l_row) * kMergePad);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          group_bar(2 + grp, kGroupWarps * 32);
          if (rep == 0) {
#pragma unroll 1
            for (int r = 0; r < nrep - 1; ++r) {
              const float4* d = reinterpret_cast<const float4*>(merge + (r * per + l_row) * kMergePad);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 a = d[e];
                o[4 * e] += a.x;
                o[4 * e + 1] += a.y;
                o[4 * e + 2] += a.z;
                o[4 * e + 3] += a.w;
              }
            }
          }
          if (x + 1 < D / 32) group_bar(2 + grp, kGroupWarps * 32);
        }
        if (x + 1 == D / 32 && nrep == 1) {
          // the last of O, (m, l) and the description is in registers: the next
          // item's P.V need not wait for the stores
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[k & 1]);
        }
        if (!whole) {
          // columns by rows: 32 lanes, 512 bytes
          float4* d = reinterpret_cast<float4*>(piece_o(p, D, piece)) + (col / 4) * kBM + l_row;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (writes) d[e * kBM] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint32_t u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = BF ? pack_bf16x2(o[2 * e], o[2 * e + 1]) : pack_f16x2(o[2 * e], o[2 * e + 1]);
          if (nrep > 1) {
            uint4* d = reinterpret_cast<uint4*>(p.out + orow * D + col);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (writes) d[e] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
          } else {
            // turned over in the (unused) merge area, so that two lanes store a row's 32 bytes
            uint32_t* mine = reinterpret_cast<uint32_t*>(smem + SM::kOffMerge) + warp * 32 * 12;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(mine + lane * 12 + 4 * e) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = e * 16 + lane / 2;
              const uint4 y = *reinterpret_cast<const uint4*>(mine + r * 12 + 4 * (lane & 1));
              const unsigned long long to = __shfl_sync(0xffffffffu, (unsigned long long)(writes ? orow : ~0ull), r);
              if (to != ~0ull) *reinterpret_cast<uint4*>(p.out + to * D + col + 8 * (lane & 1)) = y;
            }
            __syncwarp();
          }
        }
      }
      if (writes && grp == 0) {
        const float lse = have ? M + log2f(l_all) : -INFINITY;
        if (!whole) piece_lse(p, D, piece)[l_row] = lse;
        else if (p.lse2) p.lse2[orow] = lse;
      }
      // O, (m, l), the merge area and the item's description have been read
      tc_fence_before();
      if (group_bar_any(1, kSoftmaxWarps * 32, !alive)) break;   // all leave, or none
      if (lane == 0 && nrep > 1) mbar_arrive(&o_free[k & 1]);
      n0 += nb;
    }
  }

  // ---- teardown: the epilogues waited for every P.V
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && misc[1] && p.status) atomicOr(p.status, kStatusTimeoutBit);
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the pieces of the items that the ranges cut: blocks (x, .) the item that
// range x + 1 is the first to cut; a warp per 32 rows (a row per lane) and four dims.
constexpr int kJoinWarps = 8, kJoinAhead = 8;
template <int D, bool BF>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const EParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, cta = blockIdx.x + 1;
  const Cut cut = cuts(p, D)[cta];
  const int unit = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), col = unit % (D / 4), row = unit / (D / 4) * 32 + lane;
  const int n = cut.last - cta + 2;                      // pieces: 2 (cta - 1) + 1, 2 cta, 2 (cta + 1), ...
  if (row >= cut.rows) return;
  float M = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x0 = 0; x0 < n; x0 += kJoinAhead) {
    float l[kJoinAhead];
    float4 v[kJoinAhead];
    float top = M;
#pragma unroll
    for (int y = 0; y < kJoinAhead; ++y) {
      const int x = x0 + y, piece = x == 0 ? 2 * (cta - 1) + 1 : 2 * (cta - 1 + x);
      l[y] = -INFINITY;
      v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x < n) {
        l[y] = piece_lse(p, D, piece)[row];
        v[y] = reinterpret_cast<const float4*>(piece_o(p, D, piece))[col * kBM + row];
      }
    }
#pragma unroll
    for (int y = 0; y < kJoinAhead; ++y) top = fmaxf(top, l[y]);
    const float ref = top == -INFINITY ? 0.f : top;      // nothing visible so far, or NaN
    const float r = fast_exp2(M - ref);                  // 2^-inf = 0
    M = top;
    sum *= r;
    o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
#pragma unroll
    for (int y = 0; y < kJoinAhead; ++y) {
      const float w = fast_exp2(l[y] - ref);
      sum += w;
      o.x = fmaf(w, v[y].x, o.x);
      o.y = fmaf(w, v[y].y, o.y);
      o.z = fmaf(w, v[y].z, o.z);
      o.w = fmaf(w, v[y].w, o.w);
    }
  }
  const int lin = cut.row0 + row, tok = group_of(p, lin);
  const size_t orow = (size_t)(cut.q0 + tok) * p.Hq + cut.head0 + (lin - tok * p.G);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint2 u;
  u.x = BF ? pack_bf16x2(o.x * inv, o.y * inv) : pack_f16x2(o.x * inv, o.y * inv);
  u.y = BF ? pack_bf16x2(o.z * inv, o.w * inv) : pack_f16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.out + orow * D + 4 * col) = u;
  if (col == 0 && p.lse2) p.lse2[orow] = sum != 0.f ? M + log2f(sum) : -INFINITY;
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

template <int D, bool BF, bool W16>
static argus_status launch(const EParams& p, cudaStream_t s) {
  constexpr int smem = Smem<D>::kBytes;
  static PerContext configured;
  argus_status st = configured.ensure([](int) {
    const cudaError_t e = cudaFuncSetAttribute(extend_kernel<D, BF, W16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e == cudaSuccess ? ARGUS_OK : fail(ARGUS_E_LAUNCH, "extend: smem attribute: %s", cudaGetErrorString(e));
  });
  if (st != ARGUS_OK) return st;
  auto status = [](cudaError_t e, const char* what) {
    if (e == cudaSuccess) return ARGUS_OK;
    cudaGetLastError();                // not left for the next call to find
    return fail(ARGUS_E_LAUNCH, "argus_paged_extend_attn: launch of the %s failed: %s", what, cudaGetErrorString(e));
  };
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  st = status(cudaLaunchKernelEx(&cfg, extend_kernel<D, BF, W16>, p), "attention");
  // without the cuts that the first kernel writes, the join would follow whatever the workspace holds
  if (st != ARGUS_OK || p.n_ctas == 1) return st;
  cfg.gridDim = dim3(p.n_ctas - 1, kBM / 32 * (D / 4) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return status(cudaLaunchKernelEx(&cfg, join_kernel<D, BF>, p), "join");
}

template <int D>
static argus_status launch_d(bool bf, bool w16, const EParams& p, cudaStream_t s) {
  if (bf) return w16 ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
  return w16 ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
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
  // an item that two CTAs share has its queries read while rows of others are written
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(a->q), o0 = reinterpret_cast<uintptr_t>(a->out);
  const uintptr_t token = (uintptr_t)g.n_q_heads * D * 2, q_bytes = (uintptr_t)(a->total_q - 1) * qs * 2 + token;
  if (q0 < o0 + a->total_q * token && o0 < q0 + q_bytes) return fail(ARGUS_E_INVALID, "extend: out overlaps q");
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
  p.n_ctas = extend::grid_size(a);
  int bits = 0;
  while ((1 << bits) < p.G) ++bits;
  if (bits) {
    p.g_mul = (uint32_t)(((1ull << (31 + bits)) + p.G - 1) / p.G);
    p.g_shift = bits - 1;
  }
  for (int r = 0; r < 8; ++r) p.last_query[r] = (extend::kBM * (r + 1) - 1) / p.G;
  if (extend::max_blocks(a) / p.n_ctas >= 0x7fffffffll) return fail(ARGUS_E_UNSUPPORTED, "extend: too many key blocks");
  p.ws = static_cast<float*>(ws);
  const bool bf = a->q_dtype == ARGUS_BF16, w16 = p.pool[a->q_dtype].n_slots > 0;
  return D == 64 ? extend::launch_d<64>(bf, w16, p, s) : extend::launch_d<128>(bf, w16, p, s);
}
