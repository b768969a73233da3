// What the two grouped-attention kernels over the 4-bit cache share: a call's parameters and the way
// from a tile number to its request.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace rocs {

struct KaParams {
  const __nv_bfloat16* Q;
  long long ldq;
  const uint8_t* cache;
  const int32_t* table;
  int max_blocks;
  const int32_t *kv_len, *offsets;
  int B_R;
  long long rows;
  int Hkv, share, P_log2, n_pages;
  float sl2;            // |scale| * log2(e), at least the smallest normal number
  uint32_t q_flip;      // sign bits to flip in a query pair (a negative scale)
  int causal;
  __nv_bfloat16* O;
  long long ldo;
  int n_split;
  int per_item;         // warps a (tile, head) of the kernel for few rows
  float* part;          // [tile][head][split][row][D] sums, then [tile][head][split][row] (max, sum) pairs
  float2* part_ml;
  int* status;
};

// The request of tile t: request r's tiles start at floor(offsets[r] * share / T) + r, which leaves
// room for ceil(n_r * share / T) of them without another pass over the counts.  Every lane of the
// calling warp gets the answer (32 probes a step).
__device__ __forceinline__ long long ka_tile_start(const KaParams& p, int r, int T) {
  long long o = p.offsets[r];
  o = o < 0 ? 0 : o > p.rows ? p.rows : o;
  return o * p.share / T + r;
}
__device__ __forceinline__ int ka_request(const KaParams& p, long long t, int T) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B_R;   // start(lo) <= t; the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int r = lo + lane * step;
    const bool le = r < hi && (lane == 0 || ka_tile_start(p, r, T) <= t);
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m == 0xffffffffu ? 31 : __ffs((int)~m) - 2;   // lanes 0..k hold
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Every request's lengths are looked at once, whether a tile reads them or not; the grid's x extent is
// at least B_R.
__device__ __forceinline__ void ka_check_lengths(const KaParams& p) {
  const long long r = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= p.B_R) return;
  const long long q0 = p.offsets[r], q1 = p.offsets[r + 1], len = p.kv_len[r];
  if (q0 < 0 || q1 < q0 || q1 > p.rows) set_status(p.status, ROCS_ERR_INDEX);
  if (len < 0 || len > ((long long)p.max_blocks << p.P_log2)) set_status(p.status, ROCS_ERR_COUNTS);
}

struct KaTile {
  int r, n, first;       // request, its packed rows (n_r * share), the tile's first packed row
  long long q0;          // the request's first query row
  int len, n_r;          // keys, query rows
};

// Geometry of tile t; false where there is nothing to do.
__device__ __forceinline__ bool ka_tile(const KaParams& p, long long t, int T, KaTile& a) {
  a.r = ka_request(p, t, T);
  const long long q0 = p.offsets[a.r], q1 = p.offsets[a.r + 1];
  a.len = p.kv_len[a.r];
  if (q0 < 0 || q1 < q0 || q1 > p.rows || a.len < 0 || a.len > ((long long)p.max_blocks << p.P_log2)) return false;
  const long long ti = t - ka_tile_start(p, a.r, T), n = (q1 - q0) * p.share;
  if (ti < 0 || ti * T >= n) return false;
  a.q0 = q0;
  a.n_r = (int)(q1 - q0);
  a.n = (int)n;
  a.first = (int)(ti * T);
  return true;
}

// The same for a whole block of 256 threads, in one round of loads up to 1024 requests (the start of a
// tile is a chain of latencies: 3300 cycles with the warp's search, of some 20000 a tile): each
// thread looks at up to four requests, and whoever finds the tile's publishes all there is to it.
__device__ __forceinline__ bool ka_tile_block(const KaParams& p, long long t, int T, KaTile& a) {
  __shared__ KaTile s_tile;
  __shared__ int s_found;
  if (p.B_R > 1024) return ka_tile(p, t, T, a);
  if (threadIdx.x == 0) s_found = 0;
  long long o[5];
  int len[4];
  const int r0 = threadIdx.x * 4;
#pragma unroll
  for (int i = 0; i < 5; ++i) o[i] = r0 + i <= p.B_R ? p.offsets[r0 + i] : -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) len[i] = r0 + i < p.B_R ? p.kv_len[r0 + i] : -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i;
    if (r >= p.B_R || o[i] < 0 || o[i + 1] < o[i] || o[i + 1] > p.rows || len[i] < 0 ||
        len[i] > ((long long)p.max_blocks << p.P_log2))
      continue;
    const long long ti = t - (o[i] * p.share / T + r), n = (o[i + 1] - o[i]) * p.share;
    if (ti < 0 || ti * T >= n) continue;
    // with offsets in order no other request has this tile; otherwise any of them will do
    if (atomicExch(&s_found, 1) == 0) {
      s_tile.r = r;
      s_tile.q0 = o[i];
      s_tile.n_r = (int)(o[i + 1] - o[i]);
      s_tile.n = (int)n;
      s_tile.first = (int)(ti * T);
      s_tile.len = len[i];
    }
  }
  __syncthreads();
  a = s_tile;
  return s_found != 0;
}

// Keys that packed row m of the tile's request sees: [0, limit).
__device__ __forceinline__ int ka_limit(const KaParams& p, const KaTile& a, int m) {
  return p.causal ? max(0, a.len - a.n_r + m / p.share + 1) : a.len;
}

// Many query rows per request (attn_kv4_tc.cu): tiles of 128 packed rows, p.n_split splits of the keys.
rocs_status launch_attn_kv4_tc(rocs_context* ctx, int d_h, const KaParams& p, long long tiles, cudaStream_t s);

}  // namespace rocs
