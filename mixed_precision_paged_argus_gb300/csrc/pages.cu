// argus_fork_pages and argus_compact_pages: the page table of a paged cache on
// the device -- forking, freeing, copying and allocating pages, and moving the
// live pages of a pool together.
//
// Both are pure functions of the old table and counts into new arrays, so the
// result does not depend on the order of work: reference counts change by
// integer atomics (order-free), and every rank (the k-th free slot, the k-th
// request, the k-th live slot) is a prefix count in slot or row order.
//
// What bounds them: the bytes of the table and the counts, and of the pages that
// are copied; for small calls the chain of dependent steps.  So each call is ONE
// cooperative launch with a grid barrier between its steps (as a launch per step, the
// small cases spent most of their time between launches).  A prefix count over
// a pool takes two steps over tiles of 1,024 slots: a count per tile, then every
// tile sums the counts before its own (a pool of a million slots has 1,024 tiles).
// Which of the rows that are about to write a page keeps it is found row against
// row, batch^2 reads of 32 bytes, which bound the call from a few thousand rows on: a step
// in which every row writes took 27 us with 512 rows, 88 us with 4,096, 0.57 ms with
// 16,384 and 4.5 ms with 65,535.
//
// Measured (GB300, CUDA events, buffers rotated past the L2): compaction of 16,384 pages of 64 KB,
// half of them live: 96 us, 5.6 TB/s read and written (82% of a plain copy).  In a graph,
// where the host's share does not count: a fork step of 512 rows 32 us and of 8 rows
// 18 us, compaction of 96 pages 11 us; each grid barrier with the step's dependent
// reads is 2 to 5 us of that.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"

namespace argus {
namespace pages {

constexpr int kMaxPools = 7;         // one per codec
constexpr int kTile = 1024;          // slots per tile: one per thread
constexpr int kPart = 32 * 8 * 16;   // bytes a warp copies per step: eight 16-byte vectors per lane

namespace cg = cooperative_groups;

struct PoolRef {
  uint8_t* codes;
  uint8_t* meta;
  long long page_bytes, meta_bytes;  // per slot
  int codec, n_slots, tile0, n_tiles;
  const int32_t* ref_in;
  int32_t* ref_out;
  int32_t* free_list;                // fork: the free slots in order
};

// what a row of the new table asks for (fork workspace)
struct RowInfo {
  int src;       // slot of the partial last page that the row is about to write, or -1
  int pool;      // its pool
  int tail;      // its page
  int pages;     // pages the row has
  int grow;      // new pages
  int copy;      // 1: the row gets a copy of src
  int copy_at;   // rank of the copy among the requests to its pool
  int grow_at;   // rank of the first new page among the requests to its pool
};

struct FParams {
  PoolRef pool[kMaxPools];
  int n_pools, new_pool, new_codec, B, P, max_pages, n_tiles;
  const int32_t *parents, *n_new, *seq_in;
  const uint8_t* codec_in;
  const int32_t* table_in;
  uint8_t* codec_out;
  int32_t *table_out, *seq_out;
  RowInfo* rows;
  int32_t* tile_free;                // free slots per tile
  int32_t* copies;                   // rows with a copy, in order; their number behind them
  uint32_t* status;
};

__device__ __forceinline__ void count(uint32_t* status, int n) {
  if (status && n > 0) atomicAdd(status, (uint32_t)n);
}

// index of the pool that entry (codec, slot) names a slot of, or -1
__device__ __forceinline__ int pool_of(const FParams& p, int codec, int slot) {
  for (int i = 0; i < p.n_pools; ++i)
    if (p.pool[i].codec == codec) return (slot >= 0 && slot < p.pool[i].n_slots) ? i : -1;
  return -1;
}

__device__ __forceinline__ int clamped_len(const FParams& p, int b) {
  const long long cap = (long long)p.max_pages * p.P;
  return (int)min(max((long long)p.seq_in[b], 0ll), min(cap, 0x7fffffffll));
}

__device__ __forceinline__ int n_pages_of(const FParams& p, int len) { return (int)(((long long)len + p.P - 1) / p.P); }

// block-wide sum (any multiple of 32 threads up to 1024); sh: 33 ints
__device__ __forceinline__ int block_sum(int x, int* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) sh[w] = x;
  __syncthreads();
  if (w == 0) {
    int y = lane < nw ? sh[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) sh[32] = y;
  }
  __syncthreads();
  return sh[32];
}

// rank of this thread's flag among the block's flags before it
__device__ __forceinline__ int block_rank(bool flag, int* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) sh[w] = __popc(m);
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w && i < nw; ++i) before += sh[i];
  return before + __popc(m & ((1u << lane) - 1));
}

// sum of counts[0 .. n) by the whole block
__device__ __forceinline__ int block_total(const int32_t* counts, int n, int* sh) {
  int x = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) x += counts[i];
  return block_sum(x, sh);
}

// bytes [part * kPart, ...) of a page, by a warp, eight vectors in flight per
// lane; part 0 with the meta.  Warps copy on their own: one waits for its
// loads while another stores.
__device__ __forceinline__ void copy_part(const PoolRef& r, long long dst, long long src, int part) {
  const int lane = threadIdx.x & 31;
  const uint8_t* s = r.codes + src * r.page_bytes;
  uint8_t* d = r.codes + dst * r.page_bytes;
  const long long base = (long long)part * kPart + lane * 16;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (base + i * 512 < r.page_bytes) v[i] = *reinterpret_cast<const uint4*>(s + base + i * 512);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (base + i * 512 < r.page_bytes) *reinterpret_cast<uint4*>(d + base + i * 512) = v[i];
  if (part == 0 && r.meta_bytes) {
    const uint32_t* ms = reinterpret_cast<const uint32_t*>(r.meta + src * r.meta_bytes);
    uint32_t* md = reinterpret_cast<uint32_t*>(r.meta + dst * r.meta_bytes);
    for (int i = lane; i < r.meta_bytes / 4; i += 32) md[i] = ms[i];
  }
}

// exclusive prefix sum over the block; *total: the sum
__device__ __forceinline__ int block_prefix(int x, int* sh, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = incl;
  __syncthreads();
  if (w == 0) {
    int y = sh[lane];                // kTile threads: 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    sh[lane] = y;
  }
  __syncthreads();
  *total = sh[31];
  return incl - x + (w > 0 ? sh[w - 1] : 0);
}

// ---------------------------------------------------------------- fork
// the pool that tile `tile` belongs to
__device__ __forceinline__ int pool_of_tile(const FParams& p, int tile) {
  int i = 0;
  while (i + 1 < p.n_pools && tile >= p.pool[i + 1].tile0) ++i;
  return i;
}

// what a row becomes: its parent, pages and length
struct RowPlan {
  int par, len, np, ends, end, bad;
};
__device__ __forceinline__ RowPlan plan_row(const FParams& p, int b) {
  RowPlan r;
  r.bad = 0;
  r.par = p.parents[b];
  if (r.par < -1 || r.par >= p.B) { r.par = -1; ++r.bad; }
  r.len = r.par < 0 ? 0 : clamped_len(p, r.par);
  r.np = n_pages_of(p, r.len);
  int add = (r.par >= 0 && p.n_new) ? p.n_new[b] : 0;
  if (add < 0) { add = 0; ++r.bad; }
  const long long cap = min((long long)p.max_pages * p.P, 0x7fffffffll);
  long long end = (long long)r.len + add;
  if (end > cap) { end = cap; ++r.bad; }
  if (p.seq_in[b] < 0 || p.seq_in[b] > cap) ++r.bad;
  r.end = (int)end;
  r.ends = n_pages_of(p, r.end);
  return r;
}

// what row i asks of pool k
__device__ __forceinline__ int asks(const FParams& p, const RowInfo& r, int k) {
  return (r.copy && r.pool == k) + (k == p.new_pool ? r.grow : 0);
}

__global__ void __launch_bounds__(kTile, 1) fork_kernel(const FParams p) {
  __shared__ int sh[33];
  cg::grid_group grid = cg::this_grid();
  const int tid = threadIdx.x;

  // 1. the counts carried over, the new rows, and what each row is about to write
  for (int i = 0; i < p.n_pools; ++i) {
    const PoolRef& r = p.pool[i];
    for (long long s = (long long)blockIdx.x * kTile + tid; s < r.n_slots; s += (long long)gridDim.x * kTile) r.ref_out[s] = r.ref_in[s];
  }
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const RowPlan r = plan_row(p, b);
    const size_t rb = (size_t)b * p.max_pages, rp = (size_t)(r.par < 0 ? 0 : r.par) * p.max_pages;
    int bad = 0;
    for (int page = tid; page < p.max_pages; page += kTile) {
      int slot = -1, codec = 0;
      if (page < r.np) {
        slot = p.table_in[rp + page];
        codec = p.codec_in[rp + page];
        bad += pool_of(p, codec, slot) < 0;
      } else if (page < r.ends) {
        codec = p.new_codec;         // its slot comes last
      }
      p.table_out[rb + page] = slot;
      p.codec_out[rb + page] = (uint8_t)codec;
    }
    count(p.status, bad);
    if (tid == 0) {
      count(p.status, r.bad);
      p.seq_out[b] = r.end;
      RowInfo w = {-1, -1, r.np - 1, r.np, r.ends - r.np, 0, 0, 0};
      if (r.end > r.len && r.len % p.P) {
        const int slot = p.table_in[rp + r.np - 1];
        w.pool = pool_of(p, p.codec_in[rp + r.np - 1], slot);
        if (w.pool >= 0) w.src = slot;
      }
      p.rows[b] = w;
    }
  }
  grid.sync();

  // 2. references given up and taken
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int raw = p.parents[b], par = (raw < -1 || raw >= p.B) ? -1 : raw;
    if (par == b) continue;
    const int old = n_pages_of(p, clamped_len(p, b)), np = par < 0 ? 0 : n_pages_of(p, clamped_len(p, par));
    const size_t rb = (size_t)b * p.max_pages, rp = (size_t)(par < 0 ? 0 : par) * p.max_pages;
    for (int page = tid; page < max(old, np); page += kTile) {
      if (page < old) {
        const int s = p.table_in[rb + page], i = pool_of(p, p.codec_in[rb + page], s);
        if (i >= 0) atomicAdd(p.pool[i].ref_out + s, -1);
      }
      if (page < np) {
        const int s = p.table_in[rp + page], i = pool_of(p, p.codec_in[rp + page], s);
        if (i >= 0) atomicAdd(p.pool[i].ref_out + s, 1);
      }
    }
  }
  grid.sync();

  // 3. free slots per tile; a warp per row: does it get a copy of its partial page?
  for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
    const PoolRef& r = p.pool[pool_of_tile(p, tile)];
    const long long s = (long long)(tile - r.tile0) * kTile + tid;
    const int n = block_sum(s < r.n_slots && r.ref_out[s] == 0, sh);
    if (tid == 0) p.tile_free[tile] = n;
  }
  for (int b = blockIdx.x * (kTile / 32) + (tid >> 5); b < p.B; b += gridDim.x * (kTile / 32)) {
    const int lane = tid & 31, src = p.rows[b].src, pool = p.rows[b].pool;
    if (src < 0) continue;
    int writers = 0, lowest = p.B;
    for (int i = lane; i < p.B; i += 32)
      if (p.rows[i].src == src && p.rows[i].pool == pool) {
        ++writers;
        lowest = min(lowest, i);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      writers += __shfl_xor_sync(0xffffffffu, writers, o);
      lowest = min(lowest, __shfl_xor_sync(0xffffffffu, lowest, o));
    }
    if (lane == 0) p.rows[b].copy = !(p.pool[pool].ref_out[src] == writers && lowest == b);
  }
  grid.sync();

  // 4. the first free slots of each pool, as many as are asked for, in order, held
  // from here on; a block per pool ranks the requests, one more lists the copies
  for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
    const int k = pool_of_tile(p, tile);
    const PoolRef& r = p.pool[k];
    int x = 0;
    for (int b = tid; b < p.B; b += kTile) x += asks(p, p.rows[b], k);
    const int wanted = block_sum(x, sh);
    const int before = wanted == 0 ? 0 : block_total(p.tile_free + r.tile0, tile - r.tile0, sh);
    if (before >= wanted) continue;
    const long long s = (long long)(tile - r.tile0) * kTile + tid;
    const bool is_free = s < r.n_slots && r.ref_out[s] == 0;
    const int rank = before + block_rank(is_free, sh);
    if (is_free && rank < wanted) {
      r.free_list[rank] = (int)s;
      r.ref_out[s] = 1;
    }
  }
  for (int k = gridDim.x - 1 - blockIdx.x; k <= p.n_pools; k += gridDim.x) {
    int at = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTile) {
      const int b = b0 + tid;
      const RowInfo r = b < p.B ? p.rows[b] : RowInfo{};
      int total;
      if (k < p.n_pools) {
        const int rank = at + block_prefix(b < p.B ? asks(p, r, k) : 0, sh, &total);
        const bool mine = b < p.B && r.copy && r.pool == k;
        if (mine) p.rows[b].copy_at = rank;
        if (b < p.B && k == p.new_pool) p.rows[b].grow_at = rank + mine;
      } else {
        const int rank = at + block_prefix(b < p.B && r.copy, sh, &total);
        if (b < p.B && r.copy) p.copies[rank] = b;
      }
      at += total;
    }
    if (k == p.n_pools && tid == 0) p.copies[p.B] = at;
  }
  grid.sync();

  // 5. every row takes its slots; the pages are copied
  auto taken = [&](int k, int rank, int have) { return rank < have ? p.pool[k].free_list[rank] : -1; };
  const int n_copies = p.copies[p.B];
  for (int k = 0; k < p.n_pools && n_copies > 0; ++k) {
    const PoolRef& r = p.pool[k];
    const int have = block_total(p.tile_free + r.tile0, r.n_tiles, sh);
    const int parts = (int)((r.page_bytes + kPart - 1) / kPart);
    for (long long u = (long long)blockIdx.x * 32 + (tid >> 5); u < (long long)n_copies * parts; u += (long long)gridDim.x * 32) {
      const int b = p.copies[u / parts], part = (int)(u % parts);
      const RowInfo w = p.rows[b];
      if (w.pool != k) continue;
      const int dst = taken(k, w.copy_at, have);
      if (part == 0 && (tid & 31) == 0) {
        p.table_out[(size_t)b * p.max_pages + w.tail] = dst;
        atomicAdd(r.ref_out + w.src, -1);
        count(p.status, dst < 0);
      }
      if (dst >= 0) copy_part(r, dst, w.src, part);
    }
  }
  {
    const PoolRef& r = p.pool[p.new_pool];
    const int have = block_total(p.tile_free + r.tile0, r.n_tiles, sh);
    for (int b = blockIdx.x * (kTile / 32) + (tid >> 5); b < p.B; b += gridDim.x * (kTile / 32)) {
      const RowInfo w = p.rows[b];
      int missing = 0;
      for (int j = tid & 31; j < w.grow; j += 32) {
        const int slot = taken(p.new_pool, w.grow_at + j, have);
        p.table_out[(size_t)b * p.max_pages + w.pages + j] = slot;
        missing += slot < 0;
      }
      count(p.status, missing);
    }
  }
}

// ---------------------------------------------------------------- compact
struct CParams {
  PoolRef pool;
  int B, P, max_pages, n_tiles;
  const int32_t *seq, *table_in;
  const uint8_t* codec_in;
  int32_t *table_out, *n_live;
  int32_t *tile_live, *src, *dst, *rank;
  uint32_t* status;
};

__global__ void __launch_bounds__(kTile, 1) compact_kernel(const CParams p) {
  __shared__ int sh[33];
  cg::grid_group grid = cg::this_grid();
  const int tid = threadIdx.x, n = p.pool.n_slots;

  // 1. live slots per tile
  for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
    const long long s = (long long)tile * kTile + tid;
    const int x = block_sum(s < n && p.pool.ref_in[s] > 0, sh);
    if (tid == 0) p.tile_live[tile] = x;
  }
  grid.sync();

  // 2. the free slots below the number of live ones, the live slots above, in order
  const int live_total = block_total(p.tile_live, p.n_tiles, sh);
  // live slots below slot live_total: whole tiles, and part of the one it lies in
  const int lt = live_total / kTile;
  const long long ls = (long long)lt * kTile + tid;
  const int below = block_total(p.tile_live, min(lt, p.n_tiles), sh) + block_sum(ls < live_total && ls < n && p.pool.ref_in[ls] > 0, sh);
  const int moves = live_total - below;
  for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
    const int before = block_total(p.tile_live, tile, sh);
    const long long s = (long long)tile * kTile + tid;
    const int ref = s < n ? p.pool.ref_in[s] : 0;
    const bool live = ref > 0;
    const int rank = before + block_rank(live, sh);
    if (s < n) {
      if (s < live_total) {
        if (live) p.pool.ref_out[s] = ref;       // a free one gets its count with its page
        else p.dst[s - rank] = (int)s;
      } else {
        p.pool.ref_out[s] = 0;
        if (live) {
          p.src[rank - below] = (int)s;
          p.rank[s] = rank - below;
        }
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) *p.n_live = live_total;
  grid.sync();

  // 3. the pages move, the table follows
  const int parts = (int)((p.pool.page_bytes + kPart - 1) / kPart);
  for (long long w = (long long)blockIdx.x * 32 + (tid >> 5); w < (long long)moves * parts; w += (long long)gridDim.x * 32) {
    const int k = (int)(w / parts), part = (int)(w - (long long)k * parts);
    const int src = p.src[k], dst = p.dst[k];
    copy_part(p.pool, dst, src, part);
    if (part == 0 && (tid & 31) == 0) p.pool.ref_out[dst] = p.pool.ref_in[src];
  }
  const long long entries = (long long)p.B * p.max_pages;
  int bad = 0;
  for (long long e = (long long)blockIdx.x * kTile + tid; e < entries; e += (long long)gridDim.x * kTile) {
    const int b = (int)(e / p.max_pages), page = (int)(e - (long long)b * p.max_pages);
    int slot = p.table_in[e];
    if (p.codec_in[e] == p.pool.codec && (long long)page * p.P < p.seq[b]) {
      if (slot < 0 || slot >= n) ++bad;
      else if (slot >= live_total && p.pool.ref_in[slot] > 0) slot = p.dst[p.rank[slot]];
    }
    p.table_out[e] = slot;
  }
  count(p.status, bad);
}

// ---------------------------------------------------------------- host
static long long row_bytes(int codec, int D) {
  switch (codec) {
    case ARGUS_FP16:
    case ARGUS_BF16: return 2 * D;
    case ARGUS_FP8_E4M3:
    case ARGUS_INT8: return D;
    case ARGUS_INT4_G32: return D / 2;
    case ARGUS_INT2_G32: return D / 4;
    default: return D / 8;
  }
}

static long long meta_bytes(int codec, const argus_geom& g) {
  if (codec == ARGUS_FP16 || codec == ARGUS_BF16) return 0;
  if (codec == ARGUS_FP8_E4M3 || codec == ARGUS_INT8) return 2ll * g.n_kv_heads * 4;
  return 2ll * g.n_kv_heads * g.page_tokens * (g.head_dim / 32) * 4;
}

static argus_status check_geom(const char* what, const argus_geom* g) {
  if (!g) return fail(ARGUS_E_INVALID, "%s: geometry is NULL", what);
  if (g->n_kv_heads <= 0 || g->page_tokens <= 0) return fail(ARGUS_E_INVALID, "%s: geometry fields must be positive", what);
  if (g->head_dim != 64 && g->head_dim != 128)
    return fail(ARGUS_E_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", what, g->head_dim);
  if (g->page_tokens % 16) return fail(ARGUS_E_UNSUPPORTED, "%s: page_tokens %d not a multiple of 16", what, g->page_tokens);
  return ARGUS_OK;
}

static argus_status check_pool(const char* what, const argus_pool& pool) {
  if (pool.codec < 0 || pool.codec > ARGUS_INT1_G32) return fail(ARGUS_E_INVALID, "%s: bad codec %d", what, pool.codec);
  if (pool.n_slots < 0) return fail(ARGUS_E_INVALID, "%s: negative n_slots", what);
  if (pool.n_slots > 0x7fffffffll - kTile) return fail(ARGUS_E_UNSUPPORTED, "%s: 2^31 slots or more", what);
  if (pool.placement != ARGUS_PLACE_DEVICE) return fail(ARGUS_E_UNSUPPORTED, "%s: pools must lie in device memory", what);
  return ARGUS_OK;
}

static argus_status fill_pool(const char* what, const argus_geom& g, const argus_pool& pool, const int32_t* ref_in,
                              int32_t* ref_out, PoolRef* r) {
  argus_status st = check_pool(what, pool);
  if (st != ARGUS_OK) return st;
  r->codec = pool.codec;
  r->n_slots = (int)pool.n_slots;
  r->codes = static_cast<uint8_t*>(pool.codes);
  r->meta = static_cast<uint8_t*>(pool.meta);
  r->page_bytes = 2ll * g.n_kv_heads * g.page_tokens * row_bytes(pool.codec, g.head_dim);
  r->meta_bytes = meta_bytes(pool.codec, g);
  r->n_tiles = (int)((pool.n_slots + kTile - 1) / kTile);
  r->ref_in = ref_in;
  r->ref_out = ref_out;
  if (pool.n_slots == 0) return ARGUS_OK;
  if (!pool.codes || (r->meta_bytes && !pool.meta)) return fail(ARGUS_E_INVALID, "%s: NULL codes or meta (codec %d)", what, pool.codec);
  if (reinterpret_cast<uintptr_t>(pool.codes) & 15) return fail(ARGUS_E_INVALID, "%s: codes must be 16-byte aligned", what);
  if (r->meta_bytes && (reinterpret_cast<uintptr_t>(pool.meta) & 3)) return fail(ARGUS_E_INVALID, "%s: meta must be 4-byte aligned", what);
  if (!ref_in || !ref_out) return fail(ARGUS_E_INVALID, "%s: NULL reference counts", what);
  if (ref_in == ref_out) return fail(ARGUS_E_INVALID, "%s: the new counts need an array of their own", what);
  return ARGUS_OK;
}

// One block of kTile threads per SM at most (the kernels' launch bounds let each
// SM hold one): all are resident, as the grid barrier needs.
template <class K, class P>
static argus_status launch_cooperative(const char* what, K kernel, P& p, long long work, cudaStream_t s) {
  const int blocks = (int)std::max<long long>(1, std::min<long long>(work, device_sm_count()));
  void* args[] = {&p};
  const cudaError_t e = cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3(blocks), dim3(kTile), args, 0, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(ARGUS_E_LAUNCH, "%s: launch failed: %s", what, cudaGetErrorString(e));
  }
  return ARGUS_OK;
}

static size_t up16(size_t x) { return (x + 15) / 16 * 16; }

// An array of a call.  What a call writes overlaps neither what it reads nor what
// else it writes: every step reads the old table and counts while others write.
struct Span {
  const void* at;
  size_t bytes;
};
static bool overlap(const Span* out, int n_out, const Span* in, int n_in) {
  const auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
  };
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
  }
  return false;
}

// fork workspace: RowInfo [B], the rows with copies, free slots per tile, the free lists
static size_t fork_bytes(int B, const argus_pool* pools, int n_pools) {
  size_t n = up16((size_t)B * sizeof(RowInfo)) + up16((size_t)(B + 1) * 4);
  for (int i = 0; i < n_pools; ++i)
    n += up16((size_t)((pools[i].n_slots + kTile - 1) / kTile) * 4) + up16((size_t)pools[i].n_slots * 4);
  return n + 16 * kMaxPools;
}

static argus_status check_fork(int32_t batch, const argus_pool* pools, int32_t n_pools) {
  if (batch < 0 || n_pools < 0) return fail(ARGUS_E_INVALID, "fork: negative size");
  if (batch > 65535) return fail(ARGUS_E_UNSUPPORTED, "fork: batch %d above 65535", batch);
  if (n_pools > 0 && !pools) return fail(ARGUS_E_INVALID, "fork: pools is NULL");
  if (n_pools > kMaxPools) return fail(ARGUS_E_INVALID, "fork: more than one pool per codec");
  for (int i = 0; i < n_pools; ++i) {
    argus_status st = check_pool("fork", pools[i]);
    if (st != ARGUS_OK) return st;
    for (int j = 0; j < i; ++j)
      if (pools[j].codec == pools[i].codec) return fail(ARGUS_E_INVALID, "fork: more than one pool of codec %d", pools[i].codec);
  }
  return ARGUS_OK;
}

}  // namespace pages
}  // namespace argus

using namespace argus;
using namespace argus::pages;

extern "C" argus_status argus_fork_workspace_bytes(int32_t batch, const argus_pool* pools, int32_t n_pools, size_t* bytes) {
  if (!bytes) return fail(ARGUS_E_INVALID, "fork: bytes is NULL");
  argus_status st = check_fork(batch, pools, n_pools);
  if (st != ARGUS_OK) return st;
  *bytes = fork_bytes(batch, pools, n_pools);
  return ARGUS_OK;
}

extern "C" argus_status argus_fork_pages(const argus_geom* g, int32_t batch, const int32_t* parents, const int32_t* n_new,
                                         int32_t new_codec, const argus_pool* pools, int32_t n_pools,
                                         const int32_t* const* ref_in, int32_t* const* ref_out, const uint8_t* page_codec,
                                         const int32_t* block_table, const int32_t* seq_lens, uint8_t* page_codec_out,
                                         int32_t* block_table_out, int32_t* seq_lens_out, int32_t max_pages, void* ws,
                                         size_t ws_bytes, uint32_t* status, void* stream) {
  argus_status st = check_geom("fork", g);
  if (st == ARGUS_OK) st = check_fork(batch, pools, n_pools);
  if (st != ARGUS_OK) return st;
  if (n_pools < 1) return fail(ARGUS_E_INVALID, "fork: no pool");
  if (max_pages <= 0) return fail(ARGUS_E_INVALID, "fork: max_pages must be positive");
  if (!ref_in || !ref_out) return fail(ARGUS_E_INVALID, "fork: NULL reference counts");
  FParams p{};
  p.new_pool = -1;
  int tiles = 0;
  for (int i = 0; i < n_pools; ++i) {
    st = fill_pool("fork", *g, pools[i], ref_in[i], ref_out[i], &p.pool[i]);
    if (st != ARGUS_OK) return st;
    p.pool[i].tile0 = tiles;
    tiles += p.pool[i].n_tiles;
    if (pools[i].codec == new_codec) p.new_pool = i;
  }
  if (p.new_pool < 0) return fail(ARGUS_E_INVALID, "fork: no pool of the new pages' codec %d", new_codec);
  if (batch == 0 && tiles == 0) return ARGUS_OK;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15)) return fail(ARGUS_E_INVALID, "fork: ws must be a 16-byte aligned device pointer");
  if (ws_bytes < fork_bytes(batch, pools, n_pools))
    return fail(ARGUS_E_WORKSPACE, "fork: workspace of %zu bytes, %zu needed", ws_bytes, fork_bytes(batch, pools, n_pools));
  if (batch > 0) {
    if (!parents || !page_codec || !block_table || !seq_lens || !page_codec_out || !block_table_out || !seq_lens_out)
      return fail(ARGUS_E_INVALID, "fork: NULL pointer");
    if (page_codec == page_codec_out || block_table == block_table_out || seq_lens == seq_lens_out)
      return fail(ARGUS_E_INVALID, "fork: the new table needs arrays of its own");
  }
  const size_t rows = (size_t)batch * 4, entries = (size_t)batch * max_pages;
  Span out[4 + kMaxPools] = {{page_codec_out, entries}, {block_table_out, 4 * entries}, {seq_lens_out, rows}, {ws, fork_bytes(batch, pools, n_pools)}};
  Span in[5 + kMaxPools] = {{parents, rows}, {n_new, rows}, {page_codec, entries}, {block_table, 4 * entries}, {seq_lens, rows}};
  for (int i = 0; i < n_pools; ++i) {
    out[4 + i] = {ref_out[i], (size_t)pools[i].n_slots * 4};
    in[5 + i] = {ref_in[i], (size_t)pools[i].n_slots * 4};
  }
  if (overlap(out, 4 + n_pools, in, 5 + n_pools)) return fail(ARGUS_E_INVALID, "fork: the new table, counts and ws need memory of their own");
  p.n_pools = n_pools;
  p.new_codec = new_codec;
  p.B = batch;
  p.P = g->page_tokens;
  p.max_pages = max_pages;
  p.n_tiles = tiles;
  p.parents = parents;
  p.n_new = n_new;
  p.seq_in = seq_lens;
  p.codec_in = page_codec;
  p.table_in = block_table;
  p.codec_out = page_codec_out;
  p.table_out = block_table_out;
  p.seq_out = seq_lens_out;
  p.status = status;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.rows = reinterpret_cast<RowInfo*>(w);
  w += up16((size_t)batch * sizeof(RowInfo));
  p.copies = reinterpret_cast<int32_t*>(w);
  w += up16((size_t)(batch + 1) * 4);
  p.tile_free = reinterpret_cast<int32_t*>(w);
  w += up16((size_t)tiles * 4);
  long long part_max = 1;
  for (int i = 0; i < n_pools; ++i) {
    p.pool[i].free_list = reinterpret_cast<int32_t*>(w);
    w += up16((size_t)p.pool[i].n_slots * 4);
    part_max = std::max(part_max, (p.pool[i].page_bytes + kPart - 1) / kPart);
  }
  // a block per row, tile or 32 copied parts that there can be, one per SM at most
  const long long work = std::max<long long>(std::max(tiles, batch), ((long long)batch * part_max + 31) / 32);
  return launch_cooperative("argus_fork_pages", fork_kernel, p, work, static_cast<cudaStream_t>(stream));
}

static size_t compact_bytes(const argus_pool& pool) {
  return up16((size_t)((pool.n_slots + kTile - 1) / kTile) * 4) + 3 * up16((size_t)pool.n_slots * 4) + 16;
}

extern "C" argus_status argus_compact_workspace_bytes(const argus_pool* pool, size_t* bytes) {
  if (!pool || !bytes) return fail(ARGUS_E_INVALID, "compact: NULL pointer");
  argus_status st = check_pool("compact", *pool);
  if (st != ARGUS_OK) return st;
  *bytes = compact_bytes(*pool);
  return ARGUS_OK;
}

extern "C" argus_status argus_compact_pages(const argus_geom* g, int32_t batch, const argus_pool* pool, const int32_t* ref_in,
                                            int32_t* ref_out, const uint8_t* page_codec, const int32_t* block_table,
                                            const int32_t* seq_lens, int32_t* block_table_out, int32_t max_pages,
                                            int32_t* n_live, void* ws, size_t ws_bytes, uint32_t* status, void* stream) {
  argus_status st = check_geom("compact", g);
  if (st != ARGUS_OK) return st;
  if (!pool || !n_live) return fail(ARGUS_E_INVALID, "compact: NULL pointer");
  if (batch < 0 || max_pages < 0) return fail(ARGUS_E_INVALID, "compact: negative size");
  CParams p{};
  st = fill_pool("compact", *g, *pool, ref_in, ref_out, &p.pool);
  if (st != ARGUS_OK) return st;
  if ((long long)batch * max_pages > 0) {
    if (!page_codec || !block_table || !seq_lens || !block_table_out) return fail(ARGUS_E_INVALID, "compact: NULL pointer");
    if (block_table == block_table_out) return fail(ARGUS_E_INVALID, "compact: the new table needs an array of its own");
  }
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15)) return fail(ARGUS_E_INVALID, "compact: ws must be a 16-byte aligned device pointer");
  if (ws_bytes < compact_bytes(*pool))
    return fail(ARGUS_E_WORKSPACE, "compact: workspace of %zu bytes, %zu needed", ws_bytes, compact_bytes(*pool));
  const size_t entries = (size_t)batch * max_pages, slots = (size_t)pool->n_slots * 4;
  const Span out[] = {{ref_out, slots}, {block_table_out, 4 * entries}, {n_live, 4}, {ws, compact_bytes(*pool)}};
  const Span in[] = {{ref_in, slots}, {page_codec, entries}, {block_table, 4 * entries}, {seq_lens, (size_t)batch * 4}};
  if (overlap(out, 4, in, 4)) return fail(ARGUS_E_INVALID, "compact: the new table, counts, n_live and ws need memory of their own");
  p.B = batch;
  p.P = g->page_tokens;
  p.max_pages = max_pages;
  p.n_tiles = p.pool.n_tiles;
  p.seq = seq_lens;
  p.table_in = block_table;
  p.codec_in = page_codec;
  p.table_out = block_table_out;
  p.n_live = n_live;
  p.status = status;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.tile_live = reinterpret_cast<int32_t*>(w);
  w += up16((size_t)p.n_tiles * 4);
  const size_t per = up16((size_t)pool->n_slots * 4);
  p.src = reinterpret_cast<int32_t*>(w);
  p.dst = reinterpret_cast<int32_t*>(w + per);
  p.rank = reinterpret_cast<int32_t*>(w + 2 * per);
  const long long parts = (p.pool.page_bytes + kPart - 1) / kPart;
  const long long work = std::max(((long long)pool->n_slots / 2 * parts + 31) / 32, ((long long)batch * max_pages + kTile - 1) / kTile);
  return launch_cooperative("argus_compact_pages", compact_kernel, p, work, static_cast<cudaStream_t>(stream));
}
