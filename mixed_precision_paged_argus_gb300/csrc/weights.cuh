// What the kernels of argus_attn_weights share.
#pragma once

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
  int few, many;                       // a kernel takes the sequences of more than `few` query rows per KV head and up to `many`;
                                       // weights_rows.cu's takes those of more than `many`
  bool leads;                          // another kernel of this call follows, which may be put in place at once
  uint32_t* status;
};

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
struct Span {
  int t0, rows;                        // first query token; rows per KV head: tokens by heads, fewer than 2^31
};
__device__ __forceinline__ Span rows_of(const WParams& p, int b) {
  const int t0 = min(max(p.q_start[b], 0), p.total_q), t1 = min(max(p.q_start[b + 1], 0), p.total_q);
  return {t0, max(t1 - t0, 0) * p.G};
}

// weights_rows.cu: the sequences of more than p.many rows, 16-bit pages (w16) and 8-bit ones.
argus_status launch_rows(const WParams& p, int D, bool bf, bool w16, cudaStream_t s);

}  // namespace weights
}  // namespace argus
