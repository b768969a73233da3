// Writing keys and values into the 4-bit history cache, and reading them back as bf16.
//
// Per group of 32 elements of one token and head: a = max |x|, scale = the smallest number of four
// significant bits that is no less than a / 7 (kept in [2^-120, 2^120]), code = 8 + sign(x) *
// min(7, floor(|x| / scale + 1/2)).  Borders are exact:
//   scale: a is a bf16 number, so it is either 7 times a four-bit number or relatively 2^-8 away from one;
//     the product with 1/7 rounded down is at most 2^-23 too small, and is then rounded up;
//   codes: x and (k + 1/2) * scale are both bf16 numbers, so an x that is not a tie is 2^-8 away from
//     it; the product with the rounded reciprocal, raised by 2^-16, falls on the right side of every
//     border and rounds ties away from zero.  Added to 1.5 * 2^23 + 8 in one fused step it leaves the code
//     in the sum's lowest bits, and eight such sums shifted and added are the word of codes plus a
//     constant.
//
// Bound by memory (2 bytes read and 9/16 written per element when appending, the same back) only if an element costs few instructions: an SM has about 14 issue slots' worth of lanes per
// element at full bandwidth.  A lane takes eight elements: one 16-byte load, one 4-byte word of codes; a
// head's row is d / 8 lanes, and a warp takes the keys and values (which share their place in the
// record) of a few consecutive rows of one head, whose codes lie side by side in a page.  Neighbouring
// warps take the rows' other heads, so that whole rows of the input pass through the cache together.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace rocs {
namespace {

struct Kv4Params {
  const void *K, *V;       // append: the source
  void *Ko, *Vo;           // gather: the destination
  long long ldk, ldv;
  const int64_t* slots;
  long long rows;
  int H, P_log2;
  unsigned long long inv_H;   // 2^64 / H, rounded up (H > 1)
  long long n_slots;
  uint8_t* cache;
  int* status;
};

// Eight bf16 of a group's 32 (the other 24 are in the neighbouring three lanes) to a word of codes and
// the group's scale (bf16 bits).  Returns whether the group holds an infinity or NaN (codes of zeros then).
__device__ __forceinline__ bool kv4_quantize8(const uint4& x, uint32_t& word, uint32_t& scale_bits) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  uint32_t a = max(m & 0xFFFFu, m >> 16);
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const bool bad = a >= 0x7F80u;
  if (bad) {
    a = 0;
    w[0] = w[1] = w[2] = w[3] = 0;
  }
  const float top = __uint_as_float(a << 16);
  const uint32_t seventh = __float_as_uint(top * 0x1.249248p-3f);
  const float scale = fminf(fmaxf(__uint_as_float((seventh + 0xFFFFFu) & 0xFFF00000u), 0x1p-120f), 0x1p+120f);
  const float inv = rcp_approx(scale) * (1.0f + 0x1p-16f);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
  if (top > 7.0f * 0x1p+120f) {           // beyond the largest scale: magnitudes saturate
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -7.0f * 0x1p+120f), 7.0f * 0x1p+120f);
  }
  word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) word = (word << 4) + __float_as_uint(fmaf(v[i], inv, 12582920.0f));   // 1.5 * 2^23 + 8
  // less the sums' other bits: 0x4B400000 shifted by 0, 4 and 8 (further shifts leave the word)
  word -= 0x4B400000u + 0xB4000000u + 0x40000000u;
  scale_bits = __float_as_uint(scale) >> 16;
  return bad;
}

// kSets: row sets of 256 / d rows a warp takes.
template <int D, bool APPEND, int kSets>
__global__ void __launch_bounds__(256) kv4_rows_kernel(const Kv4Params p) {
  constexpr int T = D / 8;              // lanes of one head's row
  constexpr int ROWS = 32 / T;          // rows of a set
  const int lane = threadIdx.x & 31, sub = lane % T, rr = lane / T;
  const unsigned long long w = ((unsigned long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  // warp = tile * H + head; the quotient by the rounded-up reciprocal is exact below 2^53
  const long long tile = p.H == 1 ? (long long)w : (long long)__umul64hi(w, p.inv_H);
  const int h = (int)(w - tile * p.H);
  const long long row0 = tile * (ROWS * kSets) + rr;
  if (tile * (ROWS * kSets) >= p.rows) return;
  const int P = 1 << p.P_log2;
  const uint32_t record = kv4_record_bytes(P, D), half = kv4_half_bytes(P, D), scales = kv4_codes_bytes(P, D);
  uint8_t* head = p.cache + (size_t)h * record;
  const uint32_t page_bytes = (uint32_t)p.H * record;        // below 2^32: at most 1024 heads of 18 KB
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
  // a row's record, and its place in it
  auto at = [&](long long s) { return head + (size_t)(uint32_t)(s >> p.P_log2) * page_bytes; };
  auto row_of = [&](long long s) { return (uint32_t)s & (uint32_t)(P - 1); };
  if (APPEND) {
    const __nv_bfloat16* k_src = reinterpret_cast<const __nv_bfloat16*>(p.K) + row0 * p.ldk + h * D + sub * 8;
    const __nv_bfloat16* v_src = reinterpret_cast<const __nv_bfloat16*>(p.V) + row0 * p.ldv + h * D + sub * 8;
    uint4 x[kSets][2];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
      if (slot[k] >= 0) {
        x[k][0] = __ldcs(reinterpret_cast<const uint4*>(k_src + k * ROWS * p.ldk));
        x[k][1] = __ldcs(reinterpret_cast<const uint4*>(v_src + k * ROWS * p.ldv));
      }
    }
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      uint32_t word[2], scale[2];
      const bool bad0 = kv4_quantize8(x[k][0], word[0], scale[0]);
      const bool bad1 = kv4_quantize8(x[k][1], word[1], scale[1]);
      if (slot[k] >= 0) {
        uint8_t* rec = at(slot[k]);
        const uint32_t o = row_of(slot[k]);
        uint8_t* code = rec + o * (D / 2) + sub * 4;
        *reinterpret_cast<uint32_t*>(code) = word[0];
        *reinterpret_cast<uint32_t*>(code + half) = word[1];
        if ((sub & 3) == 0) {
          uint8_t* sc = rec + scales + (o * (D / KV4_GROUP) + (sub >> 2)) * 2;
          *reinterpret_cast<uint16_t*>(sc) = (uint16_t)scale[0];
          *reinterpret_cast<uint16_t*>(sc + half) = (uint16_t)scale[1];
          if (bad0 || bad1) set_status(p.status, ROCS_ERR_VALUE);
        }
      }
    }
  } else {
    uint32_t code[kSets][2], sc[kSets][2];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      if (slot[k] >= 0) {
        const uint8_t* rec = at(slot[k]);
        const uint32_t o = row_of(slot[k]);
        const uint8_t* c = rec + o * (D / 2) + sub * 4;
        const uint8_t* s = rec + scales + (o * (D / KV4_GROUP) + (sub >> 2)) * 2;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          code[k][v] = __ldcs(reinterpret_cast<const uint32_t*>(c + v * half));
          sc[k][v] = __ldg(reinterpret_cast<const uint16_t*>(s + v * half));
        }
      }
    }
    __nv_bfloat16* k_dst = reinterpret_cast<__nv_bfloat16*>(p.Ko) + row0 * p.ldk + h * D + sub * 8;
    __nv_bfloat16* v_dst = reinterpret_cast<__nv_bfloat16*>(p.Vo) + row0 * p.ldv + h * D + sub * 8;
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      if (slot[k] < 0) continue;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t s2 = __byte_perm(sc[k][v], sc[k][v], 0x1010), c2 = kv4_offset(s2);
        uint32_t e[4];   // nibbles (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = kv4_fma2(kv4_pair(code[k][v] >> (4 * i)), s2, c2);
        const uint4 out = make_uint4(__byte_perm(e[0], e[1], 0x5410), __byte_perm(e[2], e[3], 0x5410),
                                     __byte_perm(e[0], e[1], 0x7632), __byte_perm(e[2], e[3], 0x7632));
        __stcs(reinterpret_cast<uint4*>(v ? v_dst + k * ROWS * p.ldv : k_dst + k * ROWS * p.ldk), out);
      }
    }
  }
}

template <int D, bool APPEND>
void kv4_rows_sets(const Kv4Params& p, int sets, unsigned grid, cudaStream_t s) {
  if (sets == 1) kv4_rows_kernel<D, APPEND, 1><<<grid, 256, 0, s>>>(p);
  else kv4_rows_kernel<D, APPEND, 2><<<grid, 256, 0, s>>>(p);
}

template <bool APPEND>
rocs_status kv4_rows_launch(rocs_context* ctx, Kv4Params& p, const rocs_kv4_desc& d, cudaStream_t s) {
  if (p.rows == 0) return ROCS_OK;
  p.H = d.H_kv;
  p.P_log2 = 31 - __builtin_clz((unsigned)d.page_size);
  p.n_slots = (long long)d.n_pages * d.page_size;
  p.status = ctx->d_status;
  // one row set a warp until the warps fill the GPU, then two: append and gather of 512 rows of 8 heads of
  // 32 take 3.4 instead of 4.2 us, of 262147 rows 113 instead of 125 us
  p.inv_H = d.H_kv > 1 ? ~0ULL / d.H_kv + 1 : 0;
  const int set_rows = 256 / d.d_h;
  const int sets = (p.rows + set_rows - 1) / set_rows * d.H_kv < 96LL * ctx->num_sms ? 1 : 2;
  const long long warps = (p.rows + set_rows * sets - 1) / (set_rows * sets) * d.H_kv;
  const long long grid = (warps + 7) / 8;
  if (grid > 2147483647LL) {
    set_error("kv4 rows: rows=%lld too many", p.rows);
    return ROCS_ERR_INVALID_ARG;
  }
  LaunchTimer lt_(APPEND ? "kv4_append" : "kv4_gather", s);
  switch (d.d_h) {
    case 32: kv4_rows_sets<32, APPEND>(p, sets, (unsigned)grid, s); break;
    case 64: kv4_rows_sets<64, APPEND>(p, sets, (unsigned)grid, s); break;
    default: kv4_rows_sets<128, APPEND>(p, sets, (unsigned)grid, s); break;
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
