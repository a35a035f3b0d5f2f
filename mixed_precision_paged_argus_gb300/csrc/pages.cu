// argus_fork_pages and argus_compact_pages: the page table of a paged cache on
// the device -- forking, freeing, copying and allocating pages, and moving the
// live pages of a pool together.
//
// Both are pure functions of the old table and counts into new arrays, so the
// result does not depend on the order of work: reference counts change by
// integer atomics (order-free), and every rank (the k-th free slot, the k-th
// request, the k-th live slot) is a prefix count in slot or row order.
//
// What bounds them: the bytes of the table and the counts, and of the pages
// that are copied; for small calls the chain of dependent launches.  A prefix
// count over a pool takes two passes over tiles of 1,024 slots: a count per
// tile, then every tile sums the counts before its own (the sum is short: a
// pool of a million slots has 1,024 tiles), which saves a launch for a scan.
#include <algorithm>

#include "common.cuh"

namespace argus {
namespace pages {

constexpr int kMaxPools = 7;         // one per codec
constexpr int kTile = 1024;          // slots per tile: one per thread
constexpr int kRowThreads = 256;
constexpr int kCopyThreads = 256;
constexpr int kPart = kCopyThreads * 4 * 16;   // bytes a CTA copies per step: four 16-byte vectors per thread

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

// bytes [part * kPart, ...) of a page, four vectors in flight per thread
__device__ __forceinline__ void copy_part(uint8_t* dst, const uint8_t* src, long long bytes, int part) {
  const long long base = (long long)part * kPart;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long o = base + (i * kCopyThreads + threadIdx.x) * 16ll;
    if (o < bytes) v[i] = *reinterpret_cast<const uint4*>(src + o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long o = base + (i * kCopyThreads + threadIdx.x) * 16ll;
    if (o < bytes) *reinterpret_cast<uint4*>(dst + o) = v[i];
  }
}

__device__ __forceinline__ void copy_meta(const PoolRef& r, long long dst, long long src) {
  const uint32_t* s = reinterpret_cast<const uint32_t*>(r.meta + src * r.meta_bytes);
  uint32_t* d = reinterpret_cast<uint32_t*>(r.meta + dst * r.meta_bytes);
  for (int i = threadIdx.x; i < r.meta_bytes / 4; i += blockDim.x) d[i] = s[i];
}

// ---------------------------------------------------------------- fork
__global__ void __launch_bounds__(kTile) fork_counts_kernel(const FParams p) {
  for (int i = 0; i < p.n_pools; ++i) {
    const PoolRef& r = p.pool[i];
    for (long long s = (long long)blockIdx.x * kTile + threadIdx.x; s < r.n_slots; s += (long long)gridDim.x * kTile)
      r.ref_out[s] = r.ref_in[s];
  }
}

// the new rows, the references given up and taken, and what each row asks for
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const FParams p) {
  const int b = blockIdx.x;
  int bad = 0;
  int par = p.parents[b];
  if (par < -1 || par >= p.B) { par = -1; bad = 1; }
  const int old_len = clamped_len(p, b), old_pages = n_pages_of(p, old_len);
  const int len = par < 0 ? 0 : clamped_len(p, par), np = n_pages_of(p, len);
  int add = (par >= 0 && p.n_new) ? p.n_new[b] : 0;
  if (add < 0) { add = 0; bad = bad + 1; }
  const long long cap = min((long long)p.max_pages * p.P, 0x7fffffffll);
  long long end = (long long)len + add;
  if (end > cap) { end = cap; ++bad; }
  const int ends = n_pages_of(p, (int)end);
  const size_t rb = (size_t)b * p.max_pages, rp = (size_t)(par < 0 ? 0 : par) * p.max_pages;
  const bool moves = par != b;
  const int page0 = blockIdx.y * kRowThreads + threadIdx.x;
  int bad_entries = 0;
  for (int page = page0; page < p.max_pages; page += gridDim.y * kRowThreads) {
    int slot = -1, codec = 0;
    if (page < np) {
      slot = p.table_in[rp + page];
      codec = p.codec_in[rp + page];
      const int pi = pool_of(p, codec, slot);
      if (pi < 0) ++bad_entries;
      else if (moves) atomicAdd(p.pool[pi].ref_out + slot, 1);
    } else if (page < ends) {
      codec = p.new_codec;           // its slot is filled in below
    }
    p.table_out[rb + page] = slot;
    p.codec_out[rb + page] = (uint8_t)codec;
    if (moves && page < old_pages) {
      const int s = p.table_in[rb + page];
      const int pi = pool_of(p, p.codec_in[rb + page], s);
      if (pi >= 0) atomicAdd(p.pool[pi].ref_out + s, -1);
    }
  }
  count(p.status, bad_entries);
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    const int raw = p.seq_in[b];
    if (raw < 0 || raw > cap) ++bad;
    count(p.status, bad);
    p.seq_out[b] = (int)end;
    RowInfo r;
    r.src = -1;
    r.pool = -1;
    r.tail = np - 1;
    r.pages = np;
    r.grow = ends - np;
    r.copy = 0;
    if (end > len && len % p.P) {
      const int slot = p.table_in[rp + np - 1];
      r.pool = pool_of(p, p.codec_in[rp + np - 1], slot);
      if (r.pool >= 0) r.src = slot;
    }
    p.rows[b] = r;
  }
}

// blocks [0, n_tiles): free slots per tile.  The blocks behind them, a warp per
// row: does the row get a copy of its partial page?
__global__ void __launch_bounds__(kTile) fork_decide_kernel(const FParams p) {
  __shared__ int sh[33];
  if ((int)blockIdx.x < p.n_tiles) {
    int i = 0;
    while (i + 1 < p.n_pools && (int)blockIdx.x >= p.pool[i + 1].tile0) ++i;
    const PoolRef& r = p.pool[i];
    const long long s = (long long)(blockIdx.x - r.tile0) * kTile + threadIdx.x;
    const int n = block_sum(s < r.n_slots && r.ref_out[s] == 0, sh);
    if (threadIdx.x == 0) p.tile_free[blockIdx.x] = n;
    return;
  }
  const int b = (blockIdx.x - p.n_tiles) * (kTile / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.B) return;
  const int src = p.rows[b].src, pool = p.rows[b].pool;
  if (src < 0) return;
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

// what row i asks of pool k
__device__ __forceinline__ int asks(const FParams& p, int i, int k) {
  const RowInfo& r = p.rows[i];
  return (r.copy && r.pool == k) + (k == p.new_pool ? r.grow : 0);
}

// the first free slots of each pool, as many as are asked for, in order; they
// are held from here on
__global__ void __launch_bounds__(kTile) fork_list_kernel(const FParams p) {
  __shared__ int sh[33];
  int i = 0;
  while (i + 1 < p.n_pools && (int)blockIdx.x >= p.pool[i + 1].tile0) ++i;
  const PoolRef& r = p.pool[i];
  int x = 0;
  for (int b = threadIdx.x; b < p.B; b += kTile) x += asks(p, b, i);
  const int wanted = block_sum(x, sh);
  if (wanted == 0) return;
  const int before = block_total(p.tile_free + r.tile0, blockIdx.x - r.tile0, sh);
  if (before >= wanted) return;
  const long long s = (long long)(blockIdx.x - r.tile0) * kTile + threadIdx.x;
  const bool is_free = s < r.n_slots && r.ref_out[s] == 0;
  const int rank = before + block_rank(is_free, sh);
  if (is_free && rank < wanted) {
    r.free_list[rank] = (int)s;
    r.ref_out[s] = 1;
  }
}

// every row takes its slots and copies its page; blockIdx.y: a part of the page
__global__ void __launch_bounds__(kCopyThreads) fork_fill_kernel(const FParams p) {
  __shared__ int sh[33];
  const int b = blockIdx.x;
  const RowInfo r = p.rows[b];
  if (!r.copy && (blockIdx.y > 0 || r.grow == 0)) return;
  const size_t rb = (size_t)b * p.max_pages;
  int missing = 0;
  // requests of pool k before this row's, and that pool's free slots
  auto before = [&](int k) {
    int x = 0;
    for (int i = threadIdx.x; i < b; i += kCopyThreads) x += asks(p, i, k);
    return block_sum(x, sh);
  };
  auto n_free = [&](int k) { return block_total(p.tile_free + p.pool[k].tile0, p.pool[k].n_tiles, sh); };
  if (r.copy) {
    const PoolRef& pr = p.pool[r.pool];
    const int at = before(r.pool), have = n_free(r.pool);
    const int dst = at < have ? pr.free_list[at] : -1;
    if (blockIdx.y == 0 && threadIdx.x == 0) {
      p.table_out[rb + r.tail] = dst;
      atomicAdd(pr.ref_out + r.src, -1);
      missing += dst < 0;
    }
    if (dst >= 0) {
      const uint8_t* s = pr.codes + (long long)r.src * pr.page_bytes;
      uint8_t* d = pr.codes + (long long)dst * pr.page_bytes;
      const int parts = (int)((pr.page_bytes + kPart - 1) / kPart);
      for (int part = blockIdx.y; part < parts; part += gridDim.y) copy_part(d, s, pr.page_bytes, part);
      if (blockIdx.y == 0 && pr.meta_bytes) copy_meta(pr, dst, r.src);
    }
  }
  if (blockIdx.y == 0 && r.grow) {
    const PoolRef& pr = p.pool[p.new_pool];
    const int at = before(p.new_pool) + (r.copy && r.pool == p.new_pool), have = n_free(p.new_pool);
    for (int j = threadIdx.x; j < r.grow; j += kCopyThreads) {
      const int slot = at + j < have ? pr.free_list[at + j] : -1;
      p.table_out[rb + r.pages + j] = slot;
      missing += slot < 0;
    }
  }
  count(p.status, missing);
}

// ---------------------------------------------------------------- compact
struct CParams {
  PoolRef pool;
  int B, P, max_pages, n_tiles;
  const int32_t *seq, *table_in;
  const uint8_t* codec_in;
  int32_t *table_out, *n_live;
  int32_t *tile_live, *src, *dst, *rank, *n_moves;
  uint32_t* status;
};

__global__ void __launch_bounds__(kTile) compact_count_kernel(const CParams p) {
  __shared__ int sh[33];
  const long long s = (long long)blockIdx.x * kTile + threadIdx.x;
  const int n = block_sum(s < p.pool.n_slots && p.pool.ref_in[s] > 0, sh);
  if (threadIdx.x == 0) p.tile_live[blockIdx.x] = n;
}

__global__ void __launch_bounds__(kTile) compact_list_kernel(const CParams p) {
  __shared__ int sh[33];
  const int n = p.pool.n_slots;
  const int live_total = block_total(p.tile_live, p.n_tiles, sh);
  const int before = block_total(p.tile_live, blockIdx.x, sh);
  // live slots below slot live_total: whole tiles, and part of the one it lies in
  const int lt = live_total / kTile;
  const long long ls = (long long)lt * kTile + threadIdx.x;
  const int below = block_total(p.tile_live, min(lt, p.n_tiles), sh) + block_sum(ls < live_total && ls < n && p.pool.ref_in[ls] > 0, sh);
  const long long s = (long long)blockIdx.x * kTile + threadIdx.x;
  const int ref = s < n ? p.pool.ref_in[s] : 0;
  const bool live = ref > 0;
  const int rank = before + block_rank(live, sh);
  if (s < n) {
    if (s < live_total) {
      if (live) p.pool.ref_out[s] = ref;         // a free one gets its count with its page
      else p.dst[s - rank] = (int)s;
    } else {
      p.pool.ref_out[s] = 0;
      if (live) {
        p.src[rank - below] = (int)s;
        p.rank[s] = rank - below;
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.n_moves = live_total - below;
    *p.n_live = live_total;
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const CParams p) {
  const int live = *p.n_live, moves = *p.n_moves;
  const int parts = (int)((p.pool.page_bytes + kPart - 1) / kPart);
  for (long long w = blockIdx.x; w < (long long)moves * parts; w += gridDim.x) {
    const int k = (int)(w / parts), part = (int)(w - (long long)k * parts);
    const int src = p.src[k], dst = p.dst[k];
    copy_part(p.pool.codes + dst * p.pool.page_bytes, p.pool.codes + src * p.pool.page_bytes, p.pool.page_bytes, part);
    if (part == 0) {
      if (p.pool.meta_bytes) copy_meta(p.pool, dst, src);
      if (threadIdx.x == 0) p.pool.ref_out[dst] = p.pool.ref_in[src];
    }
  }
  const long long entries = (long long)p.B * p.max_pages;
  int bad = 0;
  for (long long e = (long long)blockIdx.x * kCopyThreads + threadIdx.x; e < entries; e += (long long)gridDim.x * kCopyThreads) {
    const int b = (int)(e / p.max_pages), page = (int)(e - (long long)b * p.max_pages);
    int slot = p.table_in[e];
    if (p.codec_in[e] == p.pool.codec && (long long)page * p.P < p.seq[b]) {
      if (slot < 0 || slot >= p.pool.n_slots) ++bad;
      else if (slot >= live && p.pool.ref_in[slot] > 0) slot = p.dst[p.rank[slot]];
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

static size_t up16(size_t x) { return (x + 15) / 16 * 16; }

// fork workspace: RowInfo [B], free slots per tile, the free lists
static size_t fork_bytes(int B, const argus_pool* pools, int n_pools) {
  size_t n = up16((size_t)B * sizeof(RowInfo));
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
  if (batch > 0) {
    if (!parents || !page_codec || !block_table || !seq_lens || !page_codec_out || !block_table_out || !seq_lens_out)
      return fail(ARGUS_E_INVALID, "fork: NULL pointer");
    if (page_codec == page_codec_out || block_table == block_table_out || seq_lens == seq_lens_out)
      return fail(ARGUS_E_INVALID, "fork: the new table needs arrays of its own");
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15)) return fail(ARGUS_E_INVALID, "fork: ws must be a 16-byte aligned device pointer");
    if (ws_bytes < fork_bytes(batch, pools, n_pools))
      return fail(ARGUS_E_WORKSPACE, "fork: workspace of %zu bytes, %zu needed", ws_bytes, fork_bytes(batch, pools, n_pools));
  }
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
  p.tile_free = reinterpret_cast<int32_t*>(w);
  w += up16((size_t)tiles * 4);
  long long part_max = 1;
  for (int i = 0; i < n_pools; ++i) {
    p.pool[i].free_list = reinterpret_cast<int32_t*>(w);
    w += up16((size_t)p.pool[i].n_slots * 4);
    part_max = std::max(part_max, (p.pool[i].page_bytes + kPart - 1) / kPart);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  if (tiles > 0) fork_counts_kernel<<<std::min(tiles, 2 * sms), kTile, 0, s>>>(p);
  if (batch > 0) {
    const int ychunks = std::max(1, std::min((max_pages + kRowThreads * 4 - 1) / (kRowThreads * 4), std::max(1, 8 * sms / batch)));
    fork_rows_kernel<<<dim3(batch, ychunks), kRowThreads, 0, s>>>(p);
    fork_decide_kernel<<<tiles + (batch + kTile / 32 - 1) / (kTile / 32), kTile, 0, s>>>(p);
    if (tiles > 0) fork_list_kernel<<<tiles, kTile, 0, s>>>(p);
    fork_fill_kernel<<<dim3(batch, (unsigned)std::min<long long>(part_max, 64)), kCopyThreads, 0, s>>>(p);
  }
  return launch_status("argus_fork_pages");
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
  p.n_moves = reinterpret_cast<int32_t*>(w);
  w += 16;
  p.tile_live = reinterpret_cast<int32_t*>(w);
  w += up16((size_t)p.n_tiles * 4);
  const size_t per = up16((size_t)pool->n_slots * 4);
  p.src = reinterpret_cast<int32_t*>(w);
  p.dst = reinterpret_cast<int32_t*>(w + per);
  p.rank = reinterpret_cast<int32_t*>(w + 2 * per);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = device_sm_count();
  if (p.n_tiles > 0) compact_count_kernel<<<p.n_tiles, kTile, 0, s>>>(p);
  compact_list_kernel<<<std::max(1, p.n_tiles), kTile, 0, s>>>(p);   // with no slot: n_live = 0
  const long long parts = (p.pool.page_bytes + kPart - 1) / kPart;
  const long long work = std::max((long long)pool->n_slots / 2 * parts, ((long long)batch * max_pages + kCopyThreads - 1) / kCopyThreads);
  compact_move_kernel<<<(int)std::max<long long>(1, std::min<long long>(work, 8ll * sms)), kCopyThreads, 0, s>>>(p);
  return launch_status("argus_compact_pages");
}
