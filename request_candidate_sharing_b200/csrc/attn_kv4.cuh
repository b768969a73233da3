// What the two grouped-attention kernels over the 4-bit cache share: a call's parameters and the way
// from a tile number to its request.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace rocs {

// A row's reference (raw score, unscaled) moves when a weight would exceed 2^kKaLazyLog2.  A weight is 2 to
// s * sl2 - ref * sl2 in one fused step while the second product is below kKaFarLog2, where its rounding is below
// 2^-14; beyond, the difference is taken first, or the largest weight itself would round to nothing or infinity.
constexpr float kKaLazyLog2 = 8.0f, kKaFarLog2 = 1024.0f;

// A block's work: tile `first` .. (packed rows) of request r, whose n_r query rows begin at q0 and whose
// keys are len; key units [c_lo, c_hi) of `unit` keys; the partial result's place, or -1 where the block
// has all of the tile's keys and writes its output.
struct __align__(16) KaItem {
  int r, first, n_r, len;
  int q0, c_lo, c_hi, part;
};
// A tile whose keys were split: its `parts` partial results from `part` on.
struct __align__(16) KaJoin {
  int first, n_r, q0, part;
  int parts, pad[3];
};

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
  float sl2;            // |scale| * log2(e), above zero (a masked score times it is an infinity)
  float lazy;           // how far a score may exceed its row's reference: kKaLazyLog2 / sl2
  uint32_t q_flip;      // sign bits to flip in a query pair (a negative scale)
  int causal;
  __nv_bfloat16* O;
  long long ldo;
  int per_item;         // warps a (tile, head) of the kernel for few rows
  int groups;           // blocks a tile: its heads, or groups of them
  // the list of blocks' work, heaviest first, made by ka_list_kernel; null: block = tile * groups + group,
  // in the order of the requests
  int* counts;          // items, joins
  KaItem* items;
  KaJoin* joins;
  float* part;          // [part][head][row][D] sums, and [part][head][row] (reference, sum) pairs
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

// Every request's lengths are looked at once, whether a tile reads them or not, by the blocks that work
// without a list (there are at least B_R of them, and each looks at 32).
__device__ __forceinline__ void ka_check_lengths(const KaParams& p) {
  const long long r = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
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

// Keys that packed row m of the tile's request sees: [0, limit).
__device__ __forceinline__ int ka_limit(const KaParams& p, const KaTile& a, int m) {
  return p.causal ? max(0, a.len - a.n_r + m / p.share + 1) : a.len;
}

// What this block does: its tile, its key units and its partial's place (-1: none), and its head or group of
// heads; false where there is nothing to do.  For a whole warp.
__device__ __forceinline__ bool ka_work(const KaParams& p, int T, int unit_log2, KaTile& a, int& c_lo, int& c_hi, int& part, int& group) {
  const unsigned b = blockIdx.x, t = b / (unsigned)p.groups;
  group = (int)(b - t * (unsigned)p.groups);
  if (p.items != nullptr) {
    grid_dependency_wait();
    if ((int)t >= p.counts[0]) return false;
    const int4 x = *reinterpret_cast<const int4*>(&p.items[t]), y = *(reinterpret_cast<const int4*>(&p.items[t]) + 1);
    a.r = x.x; a.first = x.y; a.n_r = x.z; a.len = x.w;
    a.q0 = y.x; c_lo = y.y; c_hi = y.z; part = y.w;
    a.n = a.n_r * p.share;
    return true;
  }
  ka_check_lengths(p);
  if (!ka_tile(p, t, T, a)) return false;
  c_lo = 0;
  c_hi = (ka_limit(p, a, min(a.first + T, a.n) - 1) + (1 << unit_log2) - 1) >> unit_log2;
  part = -1;
  return true;
}

// Many query rows per request (attn_kv4_tc.cu): tiles of 128 packed rows, units of 64 keys.
rocs_status launch_attn_kv4_tc(rocs_context* ctx, int d_h, const KaParams& p, long long blocks, cudaStream_t s);

}  // namespace rocs
