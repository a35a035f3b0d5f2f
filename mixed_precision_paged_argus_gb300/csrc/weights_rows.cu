// argus_attn_weights for many query rows per KV head (prompt chunks, the last tokens of a
// prompt): sums of 2^(score - L) over the rows, on the 5th-generation tensor cores.
//
// Mathematics as in weights.cu.  With R rows a key costs 2 R D operations and R
// exponentials; the scores S^T = K Q^T are taken with the keys as the tile's rows:
//  * 128 keys by 128 query rows by tcgen05.mma, keys on the TMEM lanes: a key's sum over the rows is a
//    thread's own, without exchange between lanes, and its page's scale is one factor of that
//    thread.  A row's log-sum is the same for all lanes: a broadcast from shared memory.
//  * K tiles are converted into the query's type on their way to shared memory (the loader warps are
//    extend.cuh's), up to four tiles of 128 rows of Q stay there; more rows take another pass
//    over the keys, by the same block, whose threads add to the weights that they wrote.
//  * Four groups of four warps sum 32 columns each of every tile; four score tiles in TMEM let the
//    MMAs run ahead.  Exponentials (32 per cycle) and MMAs take 512 cycles per tile each.
// One block per SM; key blocks, weighted by their tiles, are dealt in equal ranges.
//
// Measured (GB300): the last 32 tokens of 4 sequences of 4,096 to 32,768 BF16 tokens, 32/8 heads of 128 (one tile of 128 rows
// per KV head): 45 us, 3.2 TB/s (48% of a plain copy), tensor pipe 20%.  What bounds it: loader warps hold one block of 32 KB per
// SM in registers (a block every 2,200 cycles), and a group's wait, TMEM loads, exponentials and sums in a row
// take 700.  Tried: two groups of 64 columns 55 us (1,100 to 1,800 cycles of sums), two sets of loaders
// beside them 56 to 62, pages prefetched toward the L2 52 to 64.  By weights.cu's path the same call takes 380 us.
#include <algorithm>

#include "extend.cuh"
#include "weights.cuh"

namespace argus {
namespace weights {

using namespace tc;
using extend::kHalf;

namespace rowwise {

constexpr int kBM = 128;               // keys per block: TMEM lanes
constexpr int kBN = 128;               // query rows per tile: TMEM columns
constexpr int kTiles = 4;              // of Q in shared memory, and of scores in TMEM
constexpr int kSumWarps = 16, kLoadWarps = 8, kMmaWarp = kSumWarps + kLoadWarps;
constexpr int kGroups = kSumWarps / 4, kCols = kBN / kGroups;   // of warps that see all lanes; columns each
constexpr int kWarps = kMmaWarp + 1;
constexpr int kThreads = 32 * kWarps;
constexpr int kScales = 8;             // blocks whose scales are kept: loaders are two ahead of the MMAs, these four tiles of the sums

template <int D>
struct Smem {
  static constexpr int kTile = kBM * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTiles * kTile;
  static constexpr int kOffL = kOffK + 2 * kTile;                  // [kTiles * kBN] minus the rows' log-sums
  static constexpr int kOffScale = kOffL + kTiles * kBN * 4;       // [kScales][8]
  static constexpr int kOffHalf = kOffScale + kScales * 8 * 4;     // [2][kGroups - 1][kBM]: the other groups' sums
  static constexpr int kOffBar = kOffHalf + 2 * (kGroups - 1) * kBM * 4;           // k_full[2], k_empty[2], s_full[4], s_free[4], drain
  static constexpr int kOffMisc = kOffBar + 13 * 8 + 8;
  static constexpr int kOffPass = kOffMisc + 32;
  static constexpr int kOffWalk = kOffPass + 48;
  static constexpr int kBytes = kOffWalk + 32;
  static_assert(kBytes <= 232448, "shared memory");
};

// Blocks of a sequence's KV head by tiles of rows: what is dealt out.
struct Seq {
  int t0, rows, len, blocks, tiles;
  __device__ __forceinline__ long long units() const { return (long long)blocks * tiles; }
};
__device__ __forceinline__ Seq load_seq(const WParams& p, int b) {
  Seq s;
  const Span r = rows_of(p, b);
  s.t0 = r.t0;
  s.rows = r.rows;
  s.len = length(p, b);
  s.blocks = r.rows > p.many ? (s.len + kBM - 1) / kBM : 0;
  s.tiles = (int)(((long long)r.rows + kBN - 1) / kBN);
  return s;
}

// What a block does between two barriers of all its warps: blocks blk0 .. of a sequence's KV head, up to kTiles tiles
// of rows from tile0 on; n0 blocks and i0 score tiles before it.  n_blk = 0: its range is done.
struct Pass {
  int t0, rows, len, b, h, blk0, n_blk, tile0, tiles;
  uint32_t n0, i0;
};
// Where its range goes on: units ahead, the next one within its sequence.
struct Walk {
  long long left, at;
  int b;
};
// By one thread: the pass behind x, in x.
__device__ __noinline__ void next_pass(const WParams& p, Walk& w, Pass& x) {
  x.n0 += x.n_blk;
  x.i0 += x.n_blk * x.tiles;
  x.tile0 += kTiles;
  if (x.n_blk == 0 || (long long)x.tile0 * kBN >= x.rows) {   // the first, or the last of its blocks' passes
    x.n_blk = 0;
    x.tile0 = 0;
    while (w.left > 0 && x.n_blk == 0) {
      const Seq s = load_seq(p, w.b);
      const long long per = s.units();
      if (w.at >= p.Hkv * per) {                         // the next sequence that has any
        w.at = 0;
        ++w.b;
        continue;
      }
      x.h = (int)(w.at / per);
      const long long in = w.at - x.h * per, take = min(w.left, per - in);
      x.t0 = s.t0;
      x.rows = s.rows;
      x.len = s.len;
      x.b = w.b;
      x.blk0 = (int)(in / s.tiles);
      x.n_blk = (int)((in + take) / s.tiles) - x.blk0;
      w.at += take;
      w.left -= take;
    }
  }
  x.tiles = min(kTiles, (int)(((long long)x.rows + kBN - 1) / kBN) - x.tile0);
}

// BF: queries and operands are bf16, else fp16; W16: there are 16-bit pages.
template <int D, bool BF, bool W16>
__global__ void __launch_bounds__(kThreads, 1) weights_rows_kernel(const WParams p) {
  using SM = Smem<D>;
  constexpr int kTile = SM::kTile, V = D / 8;            // 16-byte vectors of a 16-bit row
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {                           // the swizzled tiles need it
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kStatusTimeoutBit);
    return;
  }
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* k_empty = k_full + 2;
  uint64_t* s_full = k_empty + 2;
  uint64_t* s_free = s_full + kTiles;
  uint64_t* drain = s_free + kTiles;
  // [0] TMEM base, [1] error
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + SM::kOffMisc);
  Pass& pass = *reinterpret_cast<Pass*>(smem + SM::kOffPass);
  Walk& range = *reinterpret_cast<Walk*>(smem + SM::kOffWalk);
  float* neg_lse = reinterpret_cast<float*>(smem + SM::kOffL);
  float* scales = reinterpret_cast<float*>(smem + SM::kOffScale);
  float* half = reinterpret_cast<float*>(smem + SM::kOffHalf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the other sequences' kernel shares nothing with this one but the caller's status
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    long long total = 0;
    for (int b = lane; b < p.B; b += 32) total += p.Hkv * load_seq(p, b).units();
    total = warp_sum(total);
    const long long n = gridDim.x, i = blockIdx.x;
    const long long u0 = total / n * i + total % n * i / n, u1 = total / n * (i + 1) + total % n * (i + 1) / n;
    long long before = 0;
    int first = 0;
    for (int b0 = 0; b0 < p.B && u0 < u1; b0 += 32) {
      const long long mine = b0 + lane < p.B ? p.Hkv * load_seq(p, b0 + lane).units() : 0, incl = warp_scan(mine);
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > u0);
      if (hit) {
        const int src = __ffs(hit) - 1;
        first = b0 + src;
        before += __shfl_sync(0xffffffffu, incl - mine, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      range = {u1 - u0, u0 - before, first};
      pass = {};
    }
  }
  if (threadIdx.x == 64) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&k_full[b], kLoadWarps);
      mbar_init(&k_empty[b], 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], kSumWarps);
    }
    mbar_init(drain, 1);
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32((const void*)&misc[0])), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  // every role goes through the same passes
  auto walk = [&](auto role) {
    for (;;) {
      tc_fence_before();
      __syncthreads();                                   // the tiles, scores and halves have been used
      tc_fence_after();
      if (misc[1]) return;
      if (threadIdx.x == 0) next_pass(p, range, pass);
      __syncthreads();
      const Pass x = pass;
      if (x.n_blk == 0) return;
      // Q tiles and log-sums
      const int row0 = x.tile0 * kBN;
#pragma unroll 1
      for (int y = threadIdx.x; y < x.tiles * kBN * V; y += kThreads) {
        const int l = y / V, v = y % V, r = row0 + l;
        const bool real = r < x.rows;
        const int tok = real ? r / p.G : 0, g = real ? r - tok * p.G : 0;
        const uint16_t* src = p.q + (x.t0 + tok) * p.qs + (long long)(x.h * p.G + g) * D + v * 8;
        extend::cp_async16(smem_u32(smem + SM::kOffQ) + (l / kBN) * kTile + extend::tile_off(l % kBN, v), real ? src : p.q, real ? 16 : 0);
      }
#pragma unroll 1
      for (int l = threadIdx.x; l < x.tiles * kBN; l += kThreads) {
        const int r = row0 + l, tok = r / p.G;
        float L = INFINITY;                              // a row that is not there, or sees nothing, gives nothing
        if (r < x.rows) {
          L = p.lse2[(size_t)(x.t0 + tok) * p.Hq + x.h * p.G + (r - tok * p.G)];
          if (L == -INFINITY) L = INFINITY;
        }
        neg_lse[l] = -L;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      extend::fence_async();
      __syncthreads();
      role(x);
    }
  };
  if (warp >= kMmaWarp) {
    walk([&](const Pass& x) {
        // -------------------------------------------------------- MMAs
        constexpr uint32_t id = idesc_f16kind(BF, false, kBN);
        const uint32_t lead = extend::elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t q_lo = extend::sdesc_lo(smem_u32(smem + SM::kOffQ), kHalf), k_lo = extend::sdesc_lo(smem_u32(smem + SM::kOffK), kHalf);
        bool ok = true;
        for (uint32_t n = x.n0; n < x.n0 + x.n_blk && ok; ++n) {
          const uint32_t kb = n & 1;
          ok = __all_sync(0xffffffffu, extend::wait(&k_full[kb], n >> 1 & 1, &misc[1]));
          for (int t = 0; t < x.tiles && ok; ++t) {
            const uint32_t i = x.i0 + (n - x.n0) * x.tiles + t, sb = i % kTiles;
            if (i >= kTiles) ok = __all_sync(0xffffffffu, extend::wait(&s_free[sb], (i / kTiles - 1) & 1, &misc[1]));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) / 16;
              extend::mma_ss_lead(tm + kBN * sb, k_lo + kb * (kTile / 16) + off, q_lo + t * (kTile / 16) + off, id, kk > 0, lead);
            }
            extend::commit_lead(&s_full[sb], lead);
          }
          if (ok) extend::commit_lead(&k_empty[kb], lead);
        }
        if (!ok) {
          const volatile uint32_t never = 0;
          misc[1] = 1;
          extend::commit_lead(drain, lead);              // TMEM is freed after the MMAs in flight
          extend::wait(drain, 0, &never);
        }
    });
  } else if (warp >= kSumWarps) {
    walk([&](const Pass& x) {
        // -------------------------------------------------------- K tiles: 16 keys of every block per warp
        const int ch = warp - kSumWarps;
        const uint32_t tile = smem_u32(smem + SM::kOffK) + ch * 2048;
        bool ok = true;
        constexpr bool kTwice = W16 && D == 128;         // 16-bit rows of 128 dims: a chunk is twice as many vectors
        uint4 v[extend::kSteps], v2[kTwice ? extend::kSteps : 1];
        const uint8_t* src = nullptr;
        int codec = -1, rows = 0;
        float ks = 0.f;
        // the places of 32 blocks' chunks, a lane each; a chunk that cannot be read has ks < 0
        unsigned long long f_src = 0;
        int f_state = -1;
        float f_ks = 0.f;
        auto look = [&](uint32_t n) {
          f_src = 0;
          f_state = -1;
          f_ks = -1.f;
          const int blk = x.blk0 + (int)(n - x.n0) + lane, key = blk * kBM + ch * 16;
          if (blk < x.blk0 + x.n_blk && key < x.len) {
            const int page = (int)((uint32_t)key / (uint32_t)p.P), row = key - page * p.P;
            const size_t e = (size_t)x.b * p.max_pages + page;
            const int k = p.page_codec[e];
            const long long slot = p.block_table[e];
            if (k > ARGUS_INT8 || slot < 0 || slot >= p.pool[k & 3].n_slots) {
              if (x.h == 0 && x.tile0 == 0 && row == 0 && p.status) atomicAdd(p.status, 1u);
            } else {
              const PoolRef& r = p.pool[k];
              const long long unit = slot * 2 * p.Hkv + x.h;
              f_src = reinterpret_cast<unsigned long long>(r.codes + (unit * p.P + row) * (k <= ARGUS_BF16 ? 2 * D : D));
              f_state = k;
              f_ks = k <= ARGUS_BF16 ? 1.f : __ldg(reinterpret_cast<const float*>(r.meta) + unit);
            }
          }
        };
        // block n's chunk on its way
        auto fetch = [&](uint32_t n) {
          codec = -1;
          if (n >= x.n0 + x.n_blk) return;
          const int from = (int)((n - x.n0) % 32);
          if (from == 0) look(n);
          codec = __shfl_sync(0xffffffffu, f_state, from);
          src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, f_src, from));
          ks = __shfl_sync(0xffffffffu, f_ks, from);
          rows = 16;                                     // a chunk's page is whole
          if (codec < 0) return;
          if (W16 && codec <= ARGUS_BF16) {
            extend::load_steps<D, D / 8>(v, src, lane, 0);
            if constexpr (kTwice) extend::load_steps<D, D / 8>(v2, src, lane, extend::kSteps);
          } else {
            extend::load_steps<D, D / 16>(v, src, lane, 0);
          }
        };
        fetch(x.n0);
        for (uint32_t n = x.n0; n < x.n0 + x.n_blk; ++n) {
          const uint32_t kb = n & 1;
          if (n >= 2 && ok) ok = extend::wait(&k_empty[kb], ((n >> 1) - 1) & 1, &misc[1]);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t to = tile + kb * kTile;
          if (codec >= 0) {
            if (W16 && codec <= ARGUS_BF16) {
              extend::store_steps<D, BF, ARGUS_BF16>(v, to, lane, rows, 0);
              if constexpr (kTwice) extend::store_steps<D, BF, ARGUS_BF16>(v2, to, lane, rows, extend::kSteps);
            } else if (codec == ARGUS_INT8) {
              extend::store_steps<D, BF, ARGUS_INT8>(v, to, lane, rows, 0);
            } else {
              extend::store_steps<D, BF, ARGUS_FP8_E4M3>(v, to, lane, rows, 0);
            }
          }
          if (lane == 0) scales[n % kScales * 8 + ch] = ks;
          fetch(n + 1);
          extend::fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[kb]);
        }
        if (!ok) misc[1] = 1;
    });
  } else {
    walk([&](const Pass& x) {
        // -------------------------------------------------------- sums
        const int grp = warp / 4, tl = threadIdx.x & 127;   // its share of the columns; key within the block
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const int shift = x.len - x.rows / p.G;          // causal: token i sees keys <= shift + i
        float* out = p.weights + ((size_t)x.b * p.Hkv + x.h) * p.row_len;
        bool ok = true;
        for (uint32_t n = x.n0; n < x.n0 + x.n_blk; ++n) {
          const int key = (x.blk0 + (int)(n - x.n0)) * kBM + tl;
          // by a later pass the sum so far, which this thread wrote
          const bool writes = grp == 0 && key < x.len;
          const float old = writes && (x.tile0 > 0 || p.decay != 0.f) ? out[key] : 0.f;
          // the first row that sees the key: a token for each key behind the first token's
          const int need = p.causal ? min(max(key - shift, 0), x.rows / p.G) * p.G : 0;
          float sum = 0.f, f = 0.f;
          for (int t = 0; t < x.tiles; ++t) {
            const uint32_t i = x.i0 + (n - x.n0) * x.tiles + t, sb = i % kTiles;
            ok = __all_sync(0xffffffffu, extend::wait(&s_full[sb], i / kTiles & 1, &misc[1]));
            if (!ok) break;
            tc_fence_after();
            uint32_t u[kCols / 16][16];
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) tmem_ld16(tmem + lanes + kBN * sb + kCols * grp + 16 * c, u[c]);
            if (t == 0) f = scales[n % kScales * 8 + tl / 16];   // the block's K tile was full
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[sb]);
            const float m = f * p.scale_log2;
            const int col = x.tile0 * kBN + t * kBN + kCols * grp;
            const float4* L = reinterpret_cast<const float4*>(neg_lse + t * kBN + kCols * grp);
            const bool edge = __any_sync(0xffffffffu, need > col);
            const int hidden = need - col;   // columns in front of the first that sees the key
            // sixteen columns at a time: a chain of sums through all of them would be waited for
            auto run = [&](auto masked) {
#pragma unroll
              for (int c = 0; c < kCols / 16; ++c) {
                float q[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 l4 = L[4 * c + e];
                  const float* y = reinterpret_cast<const float*>(&u[c][4 * e]);
                  q[4 * e] = fmaf(y[0], m, l4.x);
                  q[4 * e + 1] = fmaf(y[1], m, l4.y);
                  q[4 * e + 2] = fmaf(y[2], m, l4.z);
                  q[4 * e + 3] = fmaf(y[3], m, l4.w);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  q[e] = fast_exp2(q[e]);
                  if (decltype(masked)::value) q[e] = 16 * c + e >= hidden ? q[e] : 0.f;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
                  for (int e = 0; e < o; ++e) q[e] += q[e + o];
                }
                sum += q[0];
              }
            };
            if (edge) run(std::true_type{});
            else run(std::false_type{});
          }
          float* mine = half + (n & 1) * (kGroups - 1) * kBM + tl;
          if (grp > 0) mine[(grp - 1) * kBM] = sum;
          if (extend::group_bar_any(1, kSumWarps * 32, !ok)) {   // all leave, or none
            ok = false;
            break;
          }
          // a chunk that cannot be read adds nothing, whatever its tile held
          if (writes) {
#pragma unroll
            for (int g = 0; g < kGroups - 1; ++g) sum += mine[g * kBM];
            out[key] = fmaf(x.tile0 > 0 ? 1.f : p.decay, old, f < 0.f ? 0.f : sum);
          }
        }
        if (!ok) misc[1] = 1;
    });
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && misc[1] && p.status) atomicOr(p.status, kStatusTimeoutBit);
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int D, bool BF, bool W16>
static argus_status launch(const WParams& p, cudaStream_t s) {
  constexpr int smem = Smem<D>::kBytes;
  static PerContext configured;
  const argus_status st = configured.ensure([](int) {
    const cudaError_t e = cudaFuncSetAttribute(weights_rows_kernel<D, BF, W16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e == cudaSuccess ? ARGUS_OK : fail(ARGUS_E_LAUNCH, "weights: smem attribute: %s", cudaGetErrorString(e));
  });
  if (st != ARGUS_OK) return st;
  // no more blocks than there can be key blocks
  const long long blocks = (long long)p.B * p.Hkv * (((long long)p.max_pages * p.P + kBM - 1) / kBM);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(1ll, std::min<long long>(blocks, device_sm_count())));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weights_rows_kernel<D, BF, W16>, p);
  if (e == cudaSuccess) return ARGUS_OK;
  cudaGetLastError();                  // not left for the next call to find
  return fail(ARGUS_E_LAUNCH, "argus_attn_weights: launch failed: %s", cudaGetErrorString(e));
}

}  // namespace rowwise

argus_status launch_rows(const WParams& p, int D, bool bf, bool w16, cudaStream_t s) {
  using namespace rowwise;
  if (D == 64) {
    if (bf) return w16 ? launch<64, true, true>(p, s) : launch<64, true, false>(p, s);
    return w16 ? launch<64, false, true>(p, s) : launch<64, false, false>(p, s);
  }
  if (bf) return w16 ? launch<128, true, true>(p, s) : launch<128, true, false>(p, s);
  return w16 ? launch<128, false, true>(p, s) : launch<128, false, false>(p, s);
}

}  // namespace weights
}  // namespace argus
