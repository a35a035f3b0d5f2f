// argus_paged_extend_attn: several query tokens per sequence attend to the
// paged cache, read in place.
#include <algorithm>
#include <cmath>

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
  float* ws;                         // pieces: o [2 n_ctas][128][D], then lse2 [2 n_ctas][128]
};

constexpr int kBM = 128;             // query rows per tile (TMEM lanes)
constexpr int kBN = 128;             // keys per block
constexpr int kGroupWarps = 4;       // one softmax warpgroup: a thread per TMEM lane
constexpr int kSoftmaxWarps = 2 * kGroupWarps;
constexpr int kLoadWarps = 8;        // one per 16-token chunk of a block
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kHalf = kBM * 64 * 2;  // 128 rows x 64 dims: one 128-byte swizzle column
constexpr int kTmemCols = 512;       // S0 S1 O0 O1, 128 columns each
constexpr float kRescaleThreshold = 8.f;
constexpr int kScaleSlots = 4;       // blocks whose page scales are kept
constexpr int kMergePad = 20;        // floats per row of the replica merge (16 used; conflict-free vectors)

template <int D, bool W16>
struct Smem {
  static constexpr int kTile = kBM * D * 2;
  // a loader warp's raw ring: kAhead blocks of a K and a V chunk (16 rows each)
  static constexpr int kSlot = 16 * D * (W16 ? 2 : 1);
  static constexpr int kAhead = (128 / D) * (W16 ? 1 : 2);
  static constexpr int kRing = 2 * kAhead * kSlot;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTile;
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffRaw = kOffV + 2 * kTile;
  static constexpr int kOffScale = kOffRaw + kLoadWarps * kRing;
  static constexpr int kOffML = kOffScale + kScaleSlots * 8 * 16;
  static constexpr int kOffBar = kOffML + 2 * kBM * 8;
  // q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], drain
  static constexpr int kNumBars = 16;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 64;
  static_assert(kBytes <= 232448, "shared memory");
};

// ---------------------------------------------------------------- the work list
// An item is (sequence b, KV head h, tile t of 128 query rows); its work is its
// key blocks.  All blocks of all items in that order are dealt to the CTAs in equal
// contiguous ranges, so an item may be cut anywhere: the pieces are
// partial softmaxes, joined by the second kernel.  The host knows neither the lengths
// nor the query counts; every CTA finds its range from them.
struct Seq {
  int q0, n, len;
};

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
    const long long last = min(((long long)kBM * (t + 1) - 1) / p.G, (long long)s.n - 1);
    keys = max(s.len - s.n, 0) + (int)last + 1;
  }
  return max(1, (keys + kBN - 1) / kBN);
}

// blocks of tiles 0 .. m-1 (m <= T): under the causal mask G tiles further down
// are 128 queries, hence exactly one block more; only the last tile may be cut short
__device__ __forceinline__ long long blocks_before(const EParams& p, const Seq& s, int m) {
  if (!p.causal) return (long long)m * tile_blocks(p, s, 0);
  const int T = n_tiles(p, s);
  const int f = min(m, T - 1);
  const int base = max(s.len - s.n, 0);
  long long sum = 0;
  for (int r = 0; r < min(p.G, f); ++r) {
    const long long cnt = (f - r + p.G - 1) / p.G;
    const long long nb0 = (base + (kBM * (r + 1) - 1) / p.G + kBN) / kBN;
    sum += cnt * nb0 + cnt * (cnt - 1) / 2;
  }
  if (m == T && T > 0) sum += tile_blocks(p, s, T - 1);
  return sum;
}

__device__ __forceinline__ long long seq_blocks(const EParams& p, int b) {
  const Seq s = load_seq(p, b);
  return s.n == 0 ? 0 : p.Hkv * blocks_before(p, s, n_tiles(p, s));
}

// by a whole warp: blocks of all sequences
__device__ __forceinline__ long long total_blocks(const EParams& p) {
  const int lane = threadIdx.x & 31;
  long long x = 0;
  for (int b = lane; b < p.B; b += 32) x += seq_blocks(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// by a whole warp: the sequence that block w (< total) belongs to; w becomes its
// number within the sequence
__device__ __forceinline__ int find_seq(const EParams& p, long long& w) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const long long mine = b0 + lane < p.B ? seq_blocks(p, b0 + lane) : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > w);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w -= __shfl_sync(0xffffffffu, incl - mine, src);
      return b0 + src;
    }
    w -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return p.B - 1;
}

struct Cursor {
  Seq s;
  int b, h, t, T, blk, nb;
  long long left;                    // blocks of the range still ahead, this one counted

  // block `rest` of sequence b
  __device__ __forceinline__ void start(const EParams& p, int b_, long long rest, long long left_) {
    b = b_;
    left = left_;
    s = load_seq(p, b);
    T = n_tiles(p, s);
    const long long per = blocks_before(p, s, T);
    h = (int)(rest / per);
    rest -= h * per;
    int lo = 0, hi = T - 1;          // the last tile with blocks_before(t) <= rest
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (blocks_before(p, s, mid) <= rest) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
    blk = (int)(rest - blocks_before(p, s, t));
    nb = tile_blocks(p, s, t);
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

__device__ __forceinline__ long long range_start(long long total, int cta, int n_ctas) { return total * cta / n_ctas; }

// the pieces of the range [w0, w1): the one that does not begin its item (the
// first piece of a range at most) and the one that does not end it (the last)
// lie in the workspace at 2 cta and 2 cta + 1
__device__ __forceinline__ float* piece_o(const EParams& p, int D, int piece) { return p.ws + (size_t)piece * kBM * D; }
__device__ __forceinline__ float* piece_lse(const EParams& p, int D, int piece) {
  return p.ws + (size_t)2 * p.n_ctas * kBM * D + (size_t)piece * kBM;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
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

// One chunk (16 rows of K or V) from the lane's raw vectors to the tile; rows
// from n_rows on become zeros (P is 0 there, and 0 times what the page holds
// behind the sequence would be NaN if that is).
template <int D, bool BF>
__device__ __forceinline__ void convert_chunk(uint32_t raw, uint32_t tile, int chunk, int lane, int codec, int n_rows) {
  if (codec <= ARGUS_BF16) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const int f = s * 32 + lane, r = f / (D / 8), c = f % (D / 8);
      uint4 v = lds16(raw + f * 16);
      if (r >= n_rows) v = make_uint4(0, 0, 0, 0);
      sts16(tile + tile_off(chunk * 16 + r, c), v.x, v.y, v.z, v.w);
    }
  } else {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const int f = s * 32 + lane, r = f / (D / 16), j = f % (D / 16);
      uint4 v = lds16(raw + f * 16);
      if (r >= n_rows) v = make_uint4(0, 0, 0, 0);
      uint32_t o[8];
      if (codec == ARGUS_FP8_E4M3) {
        fp8_to_16<BF>(v.x, o[0], o[1]);
        fp8_to_16<BF>(v.y, o[2], o[3]);
        fp8_to_16<BF>(v.z, o[4], o[5]);
        fp8_to_16<BF>(v.w, o[6], o[7]);
      } else {
        int8_to_16<BF>(v.x, o[0], o[1]);
        int8_to_16<BF>(v.y, o[2], o[3]);
        int8_to_16<BF>(v.z, o[4], o[5]);
        int8_to_16<BF>(v.w, o[6], o[7]);
      }
      // lanes of the second half store their odd vector first: eight lanes then
      // hit eight different 16-byte banks
      const int sw = (D == 128 && j >= 4) ? 1 : 0;
      const uint32_t a0 = tile + tile_off(chunk * 16 + r, 2 * j + sw), a1 = tile + tile_off(chunk * 16 + r, 2 * j + 1 - sw);
      sts16(a0, sw ? o[4] : o[0], sw ? o[5] : o[1], sw ? o[6] : o[2], sw ? o[7] : o[3]);
      sts16(a1, sw ? o[0] : o[4], sw ? o[1] : o[5], sw ? o[2] : o[6], sw ? o[3] : o[7]);
    }
  }
}

// what a loader warp knows of its chunk of a block
struct Chunk {
  int codec, slot, row, n_rows, h, first;   // n_rows 0: nothing to read; first: counts a bad page
};
struct Loaded {
  int codec, n_rows;                        // n_rows 0: an empty chunk, -1: a page that cannot be read
  float ks, vs;
};

template <int D, bool BF, bool W16>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const EParams p) {
  using SM = Smem<D, W16>;
  constexpr int kTile = SM::kTile;
  constexpr float kPBias = BF ? 0.f : 7.f;   // fp16 P is stored as P * 2^7 (at most 2^15)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {         // the swizzled tiles need it, and there is no room to round up
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kStatusTimeoutBit);
    return;
  }
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* drain = o_done + 2;
  // [0] TMEM base, [1] error, [2] first sequence, [4..5] its block, [6..7] blocks of the range
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::kOffMisc);
  volatile long long* misc64 = reinterpret_cast<volatile long long*>(smem + SM::kOffMisc);
  float2* ml = reinterpret_cast<float2*>(smem + SM::kOffML);            // [group][lane]: (m, l)
  float4* scales = reinterpret_cast<float4*>(smem + SM::kOffScale);     // [slot][chunk]: ks, vs, log2 vs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    const long long total = total_blocks(p);
    const long long w0 = range_start(total, blockIdx.x, p.n_ctas), w1 = range_start(total, blockIdx.x + 1, p.n_ctas);
    long long w = w0;
    const int b = w1 > w0 ? find_seq(p, w) : 0;
    if (lane == 0) {
      misc[2] = b;
      misc64[2] = w;
      misc64[3] = w1 - w0;
    }
  }
  if (threadIdx.x == 32) {
    mbar_init(q_full, kSoftmaxWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&k_full[b], kLoadWarps);
      mbar_init(&k_empty[b], 1);
      mbar_init(&v_full[b], kLoadWarps);
      mbar_init(&v_empty[b], 1);
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], kGroupWarps);
      mbar_init(&o_done[b], 1);
    }
    mbar_init(drain, 1);
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
  const long long n_blocks = misc64[3];
  auto tS = [tmem](int b) { return tmem + 128u * (uint32_t)b; };
  auto tO = [tmem](int b) { return tmem + 256u + 128u * (uint32_t)b; };

  if (n_blocks <= 0) {
    // nothing in this CTA's range
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    // within an item: S0, S1, then per block i: P.V of i, S of i + 2
    if (lane == 0) {
      constexpr uint32_t idQK = idesc_f16kind(BF, false, kBN);
      constexpr uint32_t idPV = idesc_f16kind(BF, true, D);
      const uint32_t q_s = smem_u32(smem + SM::kOffQ);
      Cursor c;
      c.start(p, misc[2], misc64[2], n_blocks);
      long long n0 = 0;                // blocks before this item's
      bool ok = true;
      auto issue_s = [&](long long n) {
        const int b = (int)(n & 1);
        if (!mbar_wait(&k_full[b], (uint32_t)(n >> 1) & 1, &misc[1])) return false;
        tc_fence_after();
        const uint32_t k_s = smem_u32(smem + SM::kOffK + b * kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
          mma_ss(tS(b), sdesc(q_s + off, kHalf, 1024), sdesc(k_s + off, kHalf, 1024), idQK, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[b]);
        mma_commit(&k_empty[b]);
        return true;
      };
      auto issue_pv = [&](long long n, bool first) {
        const int b = (int)(n & 1);
        if (!mbar_wait(&v_full[b], (uint32_t)(n >> 1) & 1, &misc[1])) return false;
        if (!mbar_wait(&p_full[b], (uint32_t)(n >> 1) & 1, &misc[1])) return false;
        tc_fence_after();
        const uint32_t v_s = smem_u32(smem + SM::kOffV + b * kTile);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          mma_ts(tO(b), tS(b) + kk * 16, sdesc(v_s + kk * 2048, kHalf, 1024), idPV, (!first || kk > 0) ? 1u : 0u);
        mma_commit(&o_done[b]);
        mma_commit(&v_empty[b]);
        return true;
      };
      for (uint32_t item = 0; ok && c.left > 0; ++item) {
        const int nb = (int)min((long long)(c.nb - c.blk), c.left);
        ok = mbar_wait(q_full, item & 1, &misc[1]);
        if (ok) ok = issue_s(n0);
        if (ok && nb > 1) ok = issue_s(n0 + 1);
        for (int i = 0; i < nb && ok; ++i) {
          ok = issue_pv(n0 + i, i < 2);
          if (ok && i + 2 < nb) ok = issue_s(n0 + i + 2);
        }
        n0 += nb;
        c.advance(p, nb);
      }
      if (!ok) {
        misc[1] = 1;
        mma_commit(drain);             // TMEM is freed after the MMAs in flight
        mbar_wait(drain, 0);
      }
    }
  } else if (warp >= kSoftmaxWarps) {
    // ---------------------------------------------------------- loaders
    const int ch = warp - kSoftmaxWarps;
    constexpr int A = SM::kAhead;
    const uint32_t ring = smem_u32(smem + SM::kOffRaw + ch * SM::kRing);
    Cursor c;
    c.start(p, misc[2], misc64[2], n_blocks);
    auto look = [&]() {
      Chunk k;
      k.codec = -1;
      k.slot = -1;
      k.row = 0;
      k.h = c.h;
      k.first = 0;
      k.n_rows = 0;
      if (c.left <= 0) return k;
      const int key = c.blk * kBN + ch * 16;
      k.n_rows = min(max(c.s.len - key, 0), 16);
      if (k.n_rows > 0) {
        const int page = key / p.P;
        k.row = key - page * p.P;
        const size_t e = (size_t)c.b * p.max_pages + page;
        k.codec = p.page_codec[e];
        k.slot = p.block_table[e];
        k.first = c.h == 0 && c.t == c.T - 1 && k.row == 0;
      }
      c.advance(p, 1);
      return k;
    };
    const uint8_t* src = nullptr;      // K chunk of the block being issued
    long long v_off = 0;
    auto copy = [&](const Loaded& l, const uint8_t* from, uint32_t to) {
      if (l.n_rows > 0) {
        if (W16 && l.codec <= ARGUS_BF16) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) cp_async16(to + (s * 32 + lane) * 16, from + (s * 32 + lane) * 16);
        } else {
#pragma unroll
          for (int s = 0; s < D / 32; ++s) cp_async16(to + (s * 32 + lane) * 16, from + (s * 32 + lane) * 16);
        }
      }
      cp_async_commit();
    };
    auto resolve = [&](const Chunk& k) {
      Loaded l;
      l.codec = k.codec;
      l.n_rows = k.n_rows;
      l.ks = l.vs = 1.f;
      if (k.n_rows > 0) {
        const bool known = k.codec <= ARGUS_INT8 && (W16 || k.codec >= ARGUS_FP8_E4M3);
        if (!known || k.slot < 0 || k.slot >= p.pool[k.codec & 3].n_slots) {
          l.n_rows = -1;
          if (k.first && lane == 0 && p.status) atomicAdd(p.status, 1u);
        } else {
          const PoolRef& r = p.pool[k.codec & 3];
          const int rb = k.codec <= ARGUS_BF16 ? 2 * D : D;
          const long long unit = (long long)k.slot * 2 * p.Hkv + k.h;
          src = r.codes + (unit * p.P + k.row) * rb;
          v_off = (long long)p.Hkv * p.P * rb;
          if (k.codec >= ARGUS_FP8_E4M3) {
            l.ks = r.meta[unit];
            l.vs = r.meta[unit + p.Hkv];
          }
        }
      }
      return l;
    };
    Loaded queue[A];
    Chunk next = look();
#pragma unroll
    for (int f = 0; f < A; ++f) {
      queue[f] = resolve(next);
      next = look();
      copy(queue[f], src, ring + 2 * f * SM::kSlot);
      copy(queue[f], src + v_off, ring + (2 * f + 1) * SM::kSlot);
    }
    for (long long i = 0; i < n_blocks; ++i) {
      const int b = (int)(i & 1), at = (int)(i % A);
      const uint32_t raw_k = ring + 2 * at * SM::kSlot, raw_v = raw_k + SM::kSlot;
      const Loaded cur = queue[0];
      const Loaded ahead = resolve(next);
      next = look();
      const uint32_t par = (uint32_t)((i >> 1) - 1) & 1;
      cp_async_wait<2 * A - 1>();
      if (i >= 2 && !__all_sync(0xffffffffu, mbar_wait(&k_empty[b], par, &misc[1]))) { misc[1] = 1; break; }
      convert_chunk<D, BF>(raw_k, smem_u32(smem + SM::kOffK + b * kTile), ch, lane, W16 ? cur.codec : max(cur.codec, 2), max(cur.n_rows, 0));
      if (lane == 0) {
        const float lvs = log2f(fminf(fmaxf(cur.vs, 0x1p-64f), 0x1p64f));
        scales[(int)(i % kScaleSlots) * 8 + ch] = make_float4(cur.n_rows < 0 ? -1.f : cur.ks * p.scale_log2, cur.vs, lvs, 0.f);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[b]);
      copy(ahead, src, raw_k);
      cp_async_wait<2 * A - 1>();
      if (i >= 2 && !__all_sync(0xffffffffu, mbar_wait(&v_empty[b], par, &misc[1]))) { misc[1] = 1; break; }
      convert_chunk<D, BF>(raw_v, smem_u32(smem + SM::kOffV + b * kTile), ch, lane, W16 ? cur.codec : max(cur.codec, 2), max(cur.n_rows, 0));
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[b]);
      copy(ahead, src + v_off, raw_v);
#pragma unroll
      for (int f = 0; f + 1 < A; ++f) queue[f] = queue[f + 1];
      queue[A - 1] = ahead;
    }
    cp_async_wait<0>();
  } else {
    // ---------------------------------------------------------- softmax
    const int grp = warp / kGroupWarps, wq = warp % kGroupWarps;
    const int lane_row = wq * 32 + lane;               // TMEM lane
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t sS = tS(grp) + lane_off, sO = tO(grp) + lane_off;
    const uint32_t q_s = smem_u32(smem + SM::kOffQ);
    float* merge = reinterpret_cast<float*>(smem + SM::kOffQ) + grp * 96 * kMergePad;
    Cursor c;
    c.start(p, misc[2], misc64[2], n_blocks);
    long long n0 = 0;
    bool alive = true;
    while (c.left > 0) {
      const int nb = (int)min((long long)(c.nb - c.blk), c.left);
      const long long R = (long long)c.s.n * p.G, lin0 = (long long)c.t * kBM;
      const int rows = (int)min((long long)kBM, R - lin0);
      const int nrep = replicas(rows), per = kBM / nrep;
      // ---- Q tile: row l of the tile in lanes l, l + per, ...; zeros behind the last row
      for (int f = threadIdx.x; f < kBM * (D / 8); f += kSoftmaxWarps * 32) {
        const int pr = f / (D / 8), v = f % (D / 8), l = pr & (per - 1);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (l < rows) {
          const int lin = (int)lin0 + l, tok = lin / p.G, g = lin - tok * p.G;
          x = *reinterpret_cast<const uint4*>(p.q + (long long)(c.s.q0 + tok) * p.qs + (c.h * p.G + g) * D + v * 8);
        }
        sts16(q_s + tile_off(pr, v), x.x, x.y, x.z, x.w);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      const int l_row = lane_row & (per - 1);          // row within the tile
      const int rep = lane_row / per;                  // this lane's replica: keys of chunks [c0, c1)
      const int c0 = rep * (8 / nrep), c1 = c0 + 8 / nrep;
      // rows behind the last one (zero queries) see what the last one sees: they are never written
      const int tok = min((int)((lin0 + l_row) / p.G), c.s.n - 1);
      const int vis_last = min(p.causal ? c.s.len - c.s.n + tok : c.s.len - 1, c.s.len - 1);
      float m = -INFINITY, la = 0.f, lb = 0.f;
      int last = -1;                                   // this group's last block (local)
      for (int i = (int)((grp - n0) & 1); i < nb; i += 2) {
        const long long n = n0 + i;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[grp], (uint32_t)(n >> 1) & 1, &misc[1]))) { alive = false; misc[1] = 1; break; }
        tc_fence_after();
        last = i;
        const int k0 = (c.blk + i) * kBN;
        const float4* sc = scales + (int)(n % kScaleSlots) * 8;
        bool flagged = false;
        for (int cc = c0; cc < c1; ++cc) flagged |= sc[cc].x < 0.f;
        const bool edge = __any_sync(0xffffffffu, k0 + c1 * 16 - 1 > vis_last) || flagged;   // uniform
        const int lim = vis_last - k0;                 // keys e <= lim of the block are visible
        // pass 1: maximum of score + log2 of the V scale, so that P times that scale stays in range
        float mj = -INFINITY;
        for (int cc = c0; cc < c1; cc += 2) {
          uint32_t v[32];
          tmem_ld32(sS + cc * 16, v);
          const float4 s0 = sc[cc], s1 = sc[cc + 1];
          tmem_wait_ld();
          if (!edge) {
            float a0 = -INFINITY, a1 = -INFINITY, b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              a0 = max3(a0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              a1 = max3(a1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
              b0 = max3(b0, __uint_as_float(v[16 + e]), __uint_as_float(v[16 + e + 1]));
              b1 = max3(b1, __uint_as_float(v[16 + e + 2]), __uint_as_float(v[16 + e + 3]));
            }
            mj = max3(mj, fmaf(fmaxf(a0, a1), s0.x, s0.z), fmaf(fmaxf(b0, b1), s1.x, s1.z));
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float4 s = e < 16 ? s0 : s1;
              if (cc * 16 + e <= lim && s.x >= 0.f) mj = fmaxf(mj, fmaf(__uint_as_float(v[e]), s.x, s.z));
            }
          }
        }
        const bool move = mj > m + kRescaleThreshold || (m == -INFINITY && mj != -INFINITY);
        const bool scale_o = move && m != -INFINITY;
        if (__any_sync(0xffffffffu, scale_o)) {
          // this block's scores are complete, hence also the group's P.V before them
          const float r = scale_o ? fast_exp2(m - mj) : 1.f;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t v[32];
            tmem_ld32(sO + x * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * r);
            tmem_st32(sO + x * 32, v);
          }
          tmem_wait_st();
          la *= r;
          lb *= r;
        }
        if (move) m = mj;
        // pass 2: P over the consumed scores; the keys of the other replicas are zeros
        const float mm = (m == -INFINITY) ? 0.f : m - kPBias;
        if (nrep > 1) {
          const uint32_t z[8] = {};
          for (int cc = 0; cc < 8; ++cc)
            if (cc < c0 || cc >= c1) tmem_st8(sS + cc * 16, z);
        }
#pragma unroll 2
        for (int cc = c0; cc < c1; ++cc) {
          uint32_t v[16], o[8];
          tmem_ld16(sS + cc * 16, v);
          const float4 s = sc[cc];
          tmem_wait_ld();
          if (!edge) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float x0, x1, p0, p1;
              f2_fma(x0, x1, __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), s.x, s.x, -mm, -mm);
              p0 = fast_exp2(x0);
              p1 = fast_exp2(x1);
              f2_add(la, lb, la, lb, p0, p1);
              f2_mul(p0, p1, p0, p1, s.y, s.y);
              o[e] = BF ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
            }
          } else {
            const bool see = m != -INFINITY && s.x >= 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float p0 = (see && cc * 16 + 2 * e <= lim) ? fast_exp2(fmaf(__uint_as_float(v[2 * e]), s.x, -mm)) : 0.f;
              const float p1 = (see && cc * 16 + 2 * e + 1 <= lim) ? fast_exp2(fmaf(__uint_as_float(v[2 * e + 1]), s.x, -mm)) : 0.f;
              f2_add(la, lb, la, lb, p0, p1);
              o[e] = BF ? pack_bf16x2(p0 * s.y, p1 * s.y) : pack_f16x2(p0 * s.y, p1 * s.y);
            }
          }
          tmem_st8(sS + cc * 16, o);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      }
      if (alive && last >= 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_done[grp], (uint32_t)((n0 + last) >> 1) & 1, &misc[1]))) { alive = false; misc[1] = 1; }
        tc_fence_after();
      }
      // references in the units that l was summed in
      ml[grp * kBM + lane_row] = make_float2(m == -INFINITY ? -INFINITY : m - kPBias, la + lb);
      tc_fence_before();
      group_bar(1, kSoftmaxWarps * 32);
      tc_fence_after();
      // ---- epilogue: both groups' and all replicas' sums of a row joined; group g takes half the dims
      const bool has0 = nb > 1 || (n0 & 1) == 0, has1 = nb > 1 || (n0 & 1) == 1;   // which groups had a block
      float M = -INFINITY;
      for (int x = 0; x < 2 * nrep; ++x) M = fmaxf(M, ml[(x & 1) * kBM + (x >> 1) * per + l_row].x);
      float l_all = 0.f;
      for (int x = 0; x < 2 * nrep; ++x) {
        const float2 y = ml[(x & 1) * kBM + (x >> 1) * per + l_row];
        if (y.x != -INFINITY) l_all += y.y * fast_exp2(y.x - M);
      }
      const float2 y0 = ml[lane_row], y1 = ml[kBM + lane_row];
      const bool have = l_all > 0.f;
      const float inv = have ? 1.f / l_all : 0.f;
      const float w0 = (have && y0.x != -INFINITY) ? fast_exp2(y0.x - M) * inv : 0.f;
      const float w1 = (have && y1.x != -INFINITY) ? fast_exp2(y1.x - M) * inv : 0.f;
      const bool whole = c.blk == 0 && nb == c.nb;
      const int piece = 2 * blockIdx.x + (c.blk == 0 ? 1 : 0);
      const bool writes = alive && rep == 0 && l_row < rows;
      const long long lin = lin0 + l_row;
      const int otok = (int)(lin / p.G);
      const size_t orow = writes ? (size_t)(c.s.q0 + otok) * p.Hq + c.h * p.G + (int)(lin - (long long)otok * p.G) : 0;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        const int col = grp * (D / 2) + x * 16;
        uint32_t v0[16], v1[16];
        float o[16];
        if (has0) tmem_ld16(tO(0) + lane_off + col, v0);
        if (has1) tmem_ld16(tO(1) + lane_off + col, v1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a = 0.f;
          if (has0 && w0 != 0.f) a = w0 * __uint_as_float(v0[e]);
          if (has1 && w1 != 0.f) a += w1 * __uint_as_float(v1[e]);
          o[e] = a;
        }
        if (nrep > 1) {
          if (rep > 0) {
            float4* d = reinterpret_cast<float4*>(merge + ((rep - 1) * per + l_row) * kMergePad);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          group_bar(2 + grp, kGroupWarps * 32);
          if (rep == 0) {
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
          group_bar(2 + grp, kGroupWarps * 32);
        }
        if (writes) {
          if (whole) {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = BF ? pack_bf16x2(o[2 * e], o[2 * e + 1]) : pack_f16x2(o[2 * e], o[2 * e + 1]);
            uint4* d = reinterpret_cast<uint4*>(p.out + orow * D + col);
            d[0] = make_uint4(u[0], u[1], u[2], u[3]);
            d[1] = make_uint4(u[4], u[5], u[6], u[7]);
          } else {
            float4* d = reinterpret_cast<float4*>(piece_o(p, D, piece) + (size_t)l_row * D + col);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      if (writes && grp == 0) {
        const float lse = have ? M + log2f(l_all) : -INFINITY;
        if (!whole) piece_lse(p, D, piece)[l_row] = lse;
        else if (p.lse2) p.lse2[orow] = lse;
      }
      // O, (m, l) and the merge area (the Q tile) are read before the next item's
      tc_fence_before();
      if (group_bar_any(1, kSoftmaxWarps * 32, !alive)) break;   // all leave, or none
      n0 += nb;
      c.advance(p, nb);
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

// Joins the pieces of items that the ranges cut: block x looks at the boundary
// before CTA x + 1 and joins the item that it is the first to cut; a warp per row.
constexpr int kJoinWarps = 8;
template <int D, bool BF>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const EParams p) {
  __shared__ long long s_w[2];
  __shared__ int s_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x + 1;
  if (warp == 0) {
    const long long total = total_blocks(p);
    const long long at = range_start(total, cta, p.n_ctas);
    long long w = at;
    const int b = at < total ? find_seq(p, w) : 0;
    if (lane == 0) {
      s_w[0] = total;
      s_w[1] = w;
      s_b = b;
    }
  }
  __syncthreads();
  const long long total = s_w[0], at = range_start(total, cta, p.n_ctas);
  if (at >= total) return;
  Cursor c;
  c.start(p, s_b, s_w[1], 1);
  const long long begin = at - c.blk, end = begin + c.nb;
  const long long prev = range_start(total, cta - 1, p.n_ctas);
  if (c.blk == 0 || prev > begin || prev == at) return;   // not cut here, cut before, or an empty range
  const long long lin0 = (long long)c.t * kBM;
  const int rows = (int)min((long long)kBM, (long long)c.s.n * p.G - lin0);
  const int row = blockIdx.y * kJoinWarps + warp;
  if (row >= rows) return;
  const long long lin = lin0 + row;
  const int tok = (int)(lin / p.G);
  const size_t orow = (size_t)(c.s.q0 + tok) * p.Hq + c.h * p.G + (int)(lin - (long long)tok * p.G);
  auto each = [&](auto&& f) {
    f(2 * (cta - 1) + 1);
    for (int x = cta; x < p.n_ctas && range_start(total, x, p.n_ctas) < end; ++x)
      if (range_start(total, x + 1, p.n_ctas) > range_start(total, x, p.n_ctas)) f(2 * x);
  };
  float M = -INFINITY;
  each([&](int piece) { M = fmaxf(M, piece_lse(p, D, piece)[row]); });
  float sum = 0.f;
  float o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  if (M != -INFINITY) {
    each([&](int piece) {
      const float l = piece_lse(p, D, piece)[row];
      if (l == -INFINITY) return;
      const float w = fast_exp2(l - M);
      sum += w;
      const float* src = piece_o(p, D, piece) + (size_t)row * D + lane * (D / 32);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = fmaf(w, src[e], o[e]);
    });
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint32_t u[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    u[e] = BF ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : pack_f16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  uint32_t* d = reinterpret_cast<uint32_t*>(p.out + orow * D) + lane * (D / 64);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) d[e] = u[e];
  if (lane == 0 && p.lse2) p.lse2[orow] = sum > 0.f ? M + log2f(sum) : -INFINITY;
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

// One CTA per SM, and no more than there can be key blocks: every query tile
// has at most all its sequence's blocks.
static int grid_size(const argus_extend_args* a) {
  const long long G = a->g.n_q_heads / a->g.n_kv_heads;
  const long long tiles = ((long long)a->total_q * G + kBM - 1) / kBM + a->batch;
  const long long blocks = std::max(1ll, ((long long)a->max_pages * a->g.page_tokens + kBN - 1) / kBN);
  const long long sms = device_sm_count();
  const long long most = tiles * a->g.n_kv_heads;      // items; the product below cannot overflow
  return (int)std::min(sms, most >= sms ? sms : most * blocks);
}

static size_t workspace(const argus_extend_args* a) {
  return (size_t)2 * std::max(1, grid_size(a)) * kBM * (a->g.head_dim + 1) * sizeof(float);
}

template <int D, bool BF, bool W16>
static argus_status launch(const EParams& p, cudaStream_t s) {
  constexpr int smem = Smem<D, W16>::kBytes;
  static PerContext configured;
  argus_status st = configured.ensure([](int) {
    const cudaError_t e = cudaFuncSetAttribute(extend_kernel<D, BF, W16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e == cudaSuccess ? ARGUS_OK : fail(ARGUS_E_LAUNCH, "extend: smem attribute: %s", cudaGetErrorString(e));
  });
  if (st != ARGUS_OK) return st;
  extend_kernel<D, BF, W16><<<p.n_ctas, kThreads, smem, s>>>(p);
  if (p.n_ctas > 1) join_kernel<D, BF><<<dim3(p.n_ctas - 1, kBM / kJoinWarps), 32 * kJoinWarps, 0, s>>>(p);
  return launch_status("argus_paged_extend_attn");
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
  p.ws = static_cast<float*>(ws);
  const bool bf = a->q_dtype == ARGUS_BF16, w16 = p.pool[a->q_dtype].n_slots > 0;
  return D == 64 ? extend::launch_d<64>(bf, w16, p, s) : extend::launch_d<128>(bf, w16, p, s);
}
