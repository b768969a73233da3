// Writing keys and values into the 4-bit history cache, and reading them back as bf16.
//
// Per group of 32 elements of one token and head: a = max |x|, scale = the smallest number of four
// significant bits that is no less than a / 7 (kept in [2^-120, 2^120]), code = 8 + sign(x) *
// min(7, floor(|x| / scale + 1/2)).  Borders are exact: x and (k + 1/2) * scale are both bf16 numbers,
// so an x that is not a tie is at least 2^-8 away from it, relatively, and the product with the
// rounded reciprocal, raised by 2^-16, falls on the right side of every border and rounds ties away
// from zero.  Likewise a / 7 is either a four-bit number (then the division is exact) or well away
// from one.
//
// Bound by memory (4 bytes read and 9/8 written per key and value element when appending, the same
// back).  A lane takes eight elements: one 16-byte load, one 4-byte word of codes; a head's row is
// d / 8 lanes, and a warp takes consecutive rows of one head, whose codes lie side by side in a page;
// kRows row sets are in flight per warp.  Neighbouring warps take the row set's other heads, so
// that whole rows of the input pass through the cache lines together.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace rocs {
namespace {

constexpr int kSets = 4;   // row sets of 256 / d rows in flight per warp

struct Kv4Params {
  const void *K, *V;       // append: the source
  void *Ko, *Vo;           // gather: the destination
  long long ldk, ldv;
  const int64_t* slots;
  long long rows;
  int H, P_log2;
  long long n_slots;
  uint8_t* cache;
  int* status;
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Where row i's element block (head h, this lane's eight elements) lies: the code word and its scale.
template <int D>
__device__ __forceinline__ uint8_t* kv4_codes_at(const Kv4Params& p, long long slot, int h, int v) {
  const int P = 1 << p.P_log2;
  const long long page = slot >> p.P_log2;
  return p.cache + (page * p.H + h) * kv4_record_bytes(P, D) + v * kv4_half_bytes(P, D);
}

template <int D, bool APPEND>
__global__ void __launch_bounds__(256) kv4_rows_kernel(const Kv4Params p) {
  constexpr int T = D / 8;              // lanes of one head's row
  constexpr int ROWS = 32 / T;          // rows of a set
  const int lane = threadIdx.x & 31, sub = lane % T, rr = lane / T;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int per = 2 * p.H;              // (keys, values) x heads
  const long long tile = w / per;
  const int hv = (int)(w - tile * per);
  const int v = hv >= p.H, h = v ? hv - p.H : hv;
  const long long row0 = tile * (ROWS * kSets) + rr;
  if (tile * (ROWS * kSets) >= p.rows) return;
  const int P = 1 << p.P_log2;
  const long long ld = v ? p.ldv : p.ldk;
  long long slot[kSets];
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    const long long row = row0 + k * ROWS;
    slot[k] = row < p.rows ? p.slots[row] : -1;
    if (slot[k] < -1 || slot[k] >= p.n_slots) {
      set_status(p.status, ROCS_ERR_INDEX);
      slot[k] = -1;
    }
  }
  if (APPEND) {
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(v ? p.V : p.K) + (long long)h * D + sub * 8;
    uint4 x[kSets];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      x[k] = make_uint4(0, 0, 0, 0);
      if (slot[k] >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(src + (row0 + k * ROWS) * ld));
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max2(m, wd[i] & 0x7FFF7FFFu);
      uint32_t a = max(m & 0xFFFFu, m >> 16);
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const bool bad = a >= 0x7F80u;      // an infinity or NaN in the group: it is stored as zeros
      const float top = bad ? 0.f : __uint_as_float(a << 16);
      const uint32_t seventh = __float_as_uint(__fdiv_rn(top, 7.0f));
      const float scale = fminf(fmaxf(__uint_as_float((seventh + 0xFFFFFu) & 0xFFF00000u), 0x1p-120f), 0x1p+120f);
      const float inv = __fdiv_rn(1.0f, scale) * (1.0f + 0x1p-16f);
      uint32_t code = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xi = (i & 1) ? bf16_hi(wd[i >> 1]) : bf16_lo(wd[i >> 1]);
        const int q = bad ? 0 : min(7, (int)fmaf(fabsf(xi), inv, 0.5f));
        code |= (uint32_t)(xi < 0.f ? 8 - q : 8 + q) << (4 * i);
      }
      if (slot[k] >= 0) {
        uint8_t* at = kv4_codes_at<D>(p, slot[k], h, v);
        const int o = (int)(slot[k] & (P - 1));
        *reinterpret_cast<uint32_t*>(at + o * (D / 2) + sub * 4) = code;
        if ((sub & 3) == 0) {
          uint16_t* sc = reinterpret_cast<uint16_t*>(at + kv4_codes_bytes(P, D));
          sc[o * (D / KV4_GROUP) + (sub >> 2)] = (uint16_t)(__float_as_uint(scale) >> 16);
          if (bad) set_status(p.status, ROCS_ERR_VALUE);
        }
      }
    }
  } else {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(v ? p.Vo : p.Ko) + (long long)h * D + sub * 8;
    uint32_t code[kSets], sc[kSets];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      code[k] = sc[k] = 0;
      if (slot[k] >= 0) {
        const uint8_t* at = kv4_codes_at<D>(p, slot[k], h, v);
        const int o = (int)(slot[k] & (P - 1));
        code[k] = __ldcs(reinterpret_cast<const uint32_t*>(at + o * (D / 2) + sub * 4));
        sc[k] = __ldg(reinterpret_cast<const uint16_t*>(at + kv4_codes_bytes(P, D)) + o * (D / KV4_GROUP) + (sub >> 2));
      }
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      if (slot[k] < 0) continue;
      const uint32_t s2 = sc[k] | (sc[k] << 16), c2 = kv4_offset(s2);
      uint32_t e[4];   // nibbles (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = kv4_fma2(kv4_pair(code[k] >> (4 * i)), s2, c2);
      const uint4 out = make_uint4(__byte_perm(e[0], e[1], 0x5410), __byte_perm(e[2], e[3], 0x5410),
                                   __byte_perm(e[0], e[1], 0x7632), __byte_perm(e[2], e[3], 0x7632));
      __stcs(reinterpret_cast<uint4*>(dst + (row0 + k * ROWS) * ld), out);
    }
  }
}

template <bool APPEND>
rocs_status kv4_rows_launch(rocs_context* ctx, Kv4Params& p, const rocs_kv4_desc& d, cudaStream_t s) {
  if (p.rows == 0) return ROCS_OK;
  p.H = d.H_kv;
  p.P_log2 = 31 - __builtin_clz((unsigned)d.page_size);
  p.n_slots = (long long)d.n_pages * d.page_size;
  p.status = ctx->d_status;
  const int set_rows = 256 / d.d_h * kSets;
  const long long warps = (p.rows + set_rows - 1) / set_rows * 2 * d.H_kv;
  const long long grid = (warps + 7) / 8;
  if (grid > 2147483647LL) {
    set_error("kv4 rows: rows=%lld too many", p.rows);
    return ROCS_ERR_INVALID_ARG;
  }
  LaunchTimer lt_(APPEND ? "kv4_append" : "kv4_gather", s);
  switch (d.d_h) {
    case 32: kv4_rows_kernel<32, APPEND><<<(unsigned)grid, 256, 0, s>>>(p); break;
    case 64: kv4_rows_kernel<64, APPEND><<<(unsigned)grid, 256, 0, s>>>(p); break;
    default: kv4_rows_kernel<128, APPEND><<<(unsigned)grid, 256, 0, s>>>(p); break;
  }
  return cuda_check(cudaGetLastError(), "kv4_rows_kernel");
}

}  // namespace

rocs_status launch_kv4_append(rocs_context* ctx, const rocs_kv4_desc& d, const void* K, long long ldk, const void* V,
                              long long ldv, const int64_t* slots, long long rows, void* cache, cudaStream_t s) {
  Kv4Params p = {};
  p.K = K; p.V = V; p.ldk = ldk; p.ldv = ldv; p.slots = slots; p.rows = rows; p.cache = (uint8_t*)cache;
  return kv4_rows_launch<true>(ctx, p, d, s);
}

rocs_status launch_kv4_gather(rocs_context* ctx, const rocs_kv4_desc& d, const void* cache, const int64_t* slots,
                              long long rows, void* K, long long ldk, void* V, long long ldv, cudaStream_t s) {
  Kv4Params p = {};
  p.Ko = K; p.Vo = V; p.ldk = ldk; p.ldv = ldv; p.slots = slots; p.rows = rows;
  p.cache = (uint8_t*)const_cast<void*>(cache);
  return kv4_rows_launch<false>(ctx, p, d, s);
}

}  // namespace rocs
