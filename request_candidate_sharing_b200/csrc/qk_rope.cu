// RMS norm of every query and key head with the position rotation in the same pass.
//
// Per row i, head h and element e of a head of d: y_e = x_e / sqrt(mean_e(x_e^2) + eps) * gamma_e, then
// for the first d_rot elements and pair t < d_rot / 2, with (c, s) the table's row of the row's
// position: (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s), where (a, b) = (t, t + d_rot / 2), or
// (2 t, 2 t + 1) when pairs are neighbours.  fp32 inside, one rounding at the end.
//
// Bound by memory: every element is read and written once; but only if an element costs few
// instructions (at 6.5 TB/s there are about 177 issue slots of a lane per eight bf16 elements, and about 127
// are taken).  So a lane keeps
// four whole pairs of a head: with half-split pairs elements 4 l .. 4 l + 3 and their partners d_rot / 2
// further on, no shuffles; else (neighbouring pairs, or past d_rot) eight neighbours.  A head is d / 8
// lanes of one warp, the mean a few shuffles, a warp covers 32 / lanes heads of a row at a time; the
// arithmetic is on packed fp32 pairs, and lanes past d_rot turn by nothing.
// A warp takes a few (row, unit of heads) items of the queries or of the keys, and asks for their
// elements, positions and then angles before it works on the first; nothing loops, so that the registers
// allow many warps.  For 524288 rows of 8 + 8 heads of 32: 193 us (85% of the measured copy bandwidth);
// 295 us where warps walked over many rows with the next elements in flight, 253 us where each item
// chose its side.  fp32, 30011 rows of 16 + 2 heads of 128: 92 us (94%).
#include "common.cuh"
#include "internal.h"

namespace rocs {
namespace {

struct QkSide {
  const void* x;
  void* y;
  long long ldx, ldy;
  int H, units;            // heads, units of 32 / T of them
  unsigned long long inv_units;   // 2^64 / units, rounded up (units > 1)
  const float* gamma;
};

struct QkParams {
  QkSide side[2];          // queries, keys
  long long rows;
  int d, d_rot;
  const float* table;
  const int32_t* pos;
  int max_pos;
  float eps, inv_d;
  unsigned blocks_q;       // blocks of the queries; the keys' follow
  int items;               // of a warp
  bool full;               // the head fills its lanes and turns as a whole
  int* status;
};

// A lane's eight elements as they lie in memory: two runs of four.
template <typename E> struct QkRaw;
template <> struct QkRaw<__nv_bfloat16> {
  static constexpr int ITEMS = 3, ITEMS_PARTIAL = 4;      // of a warp, where there are many; without FULL
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int oa, int ob) {
    a = __ldcs(reinterpret_cast<const uint2*>(p + oa));
    b = __ldcs(reinterpret_cast<const uint2*>(p + ob));
  }
  __device__ __forceinline__ void zero() { a = b = make_uint2(0, 0); }
  // the four pairs (x, y): of the two runs, or of neighbours
  template <bool HALVES>
  __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (HALVES) {
        x[i] = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        y[i] = (i & 1) ? bf16_hi(w[2 + (i >> 1)]) : bf16_lo(w[2 + (i >> 1)]);
      } else {
        x[i] = bf16_lo(w[i]);
        y[i] = bf16_hi(w[i]);
      }
    }
  }
  template <bool HALVES>
  static __device__ __forceinline__ void put(__nv_bfloat16* p, int oa, int ob, const float (&x)[4], const float (&y)[4]) {
    const uint2 ra = HALVES ? make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]))
                            : make_uint2(pack_bf16x2(x[0], y[0]), pack_bf16x2(x[1], y[1]));
    const uint2 rb = HALVES ? make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]))
                            : make_uint2(pack_bf16x2(x[2], y[2]), pack_bf16x2(x[3], y[3]));
    *reinterpret_cast<uint2*>(p + oa) = ra;
    *reinterpret_cast<uint2*>(p + ob) = rb;
  }
};
template <> struct QkRaw<float> {
  static constexpr int ITEMS = 2, ITEMS_PARTIAL = 2;
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int oa, int ob) {
    a = __ldcs(reinterpret_cast<const float4*>(p + oa));
    b = __ldcs(reinterpret_cast<const float4*>(p + ob));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <bool HALVES>
  __device__ __forceinline__ void get(float (&x)[4], float (&y)[4]) const {
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = HALVES ? w[i] : w[2 * i];
      y[i] = HALVES ? w[4 + i] : w[2 * i + 1];
    }
  }
  template <bool HALVES>
  static __device__ __forceinline__ void put(float* p, int oa, int ob, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<float4*>(p + oa) = HALVES ? make_float4(x[0], x[1], x[2], x[3]) : make_float4(x[0], y[0], x[1], y[1]);
    *reinterpret_cast<float4*>(p + ob) = HALVES ? make_float4(y[0], y[1], y[2], y[3]) : make_float4(x[2], y[2], x[3], y[3]);
  }
};

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t qk_pk(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void qk_un(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t qk_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t qk_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Means of squares that fp32 holds as exactly as any; heads beyond are scaled by a power of two, which changes
// nothing else of y.
constexpr float kQkSmall = 0x1p-100f, kQkLarge = 0x1p+120f;

// T lanes a head (a power of two, T * 8 >= d).  HALVES: pairs are (t, t + d_rot / 2).  FULL: d = 8 T and
// all of it turns, the usual case, without predicates.  N items a warp.
template <typename E, int T, bool HALVES, bool FULL, int N>
__global__ void __launch_bounds__(256, N == 1 ? 6 : N == 4 ? 3 : 4) qk_norm_rope_kernel(const QkParams p) {
  constexpr int HEADS = 32 / T;
  const int lane = threadIdx.x & 31, sub = lane & (T - 1), hw = lane / T;
  const bool key = blockIdx.x >= p.blocks_q;
  const QkSide& sd = p.side[key ? 1 : 0];
  const long long item0 = ((long long)(blockIdx.x - (key ? p.blocks_q : 0)) * 8 + (threadIdx.x >> 5)) * N;
  const int d = FULL ? 8 * T : p.d, d_rot = FULL ? 8 * T : p.d_rot;
  const bool in = FULL || sub * 8 < d;
  const bool turns = FULL || sub * 8 < d_rot;
  const int half = d_rot >> 1;
  const int oa = HALVES && turns ? 4 * sub : 8 * sub, ob = HALVES && turns ? half + 4 * sub : 8 * sub + 4;

  // item = row * units + unit; the quotient by the rounded-up reciprocal is exact below 2^51
  long long row = sd.units == 1 ? item0 : (long long)__umul64hi((unsigned long long)item0, sd.inv_units);
  int u = (int)(item0 - row * sd.units);
  const E* src = reinterpret_cast<const E*>(sd.x) + row * sd.ldx + (u * HEADS + hw) * d + oa;
  E* dst = reinterpret_cast<E*>(sd.y) + row * sd.ldy + (u * HEADS + hw) * d + oa;
  QkRaw<E> raw[N];
  E* out[N];
  int ps[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool has = row < p.rows && in && u * HEADS + hw < sd.H;
    raw[i].zero();
    if (has) raw[i].load(src, 0, ob - oa);
    out[i] = has ? dst : nullptr;
    ps[i] = row < p.rows ? p.pos[row] : -1;
    if (++u == sd.units) {
      u = 0;
      ++row;
      src += sd.ldx - (long long)(sd.units - 1) * HEADS * d;
      dst += sd.ldy - (long long)(sd.units - 1) * HEADS * d;
    } else {
      src += HEADS * d;
      dst += HEADS * d;
    }
  }
  // gammas of the pairs' first and second elements
  uint64_t gx[2], gy[2];
  {
    float ga[4] = {1.f, 1.f, 1.f, 1.f}, gb[4] = {1.f, 1.f, 1.f, 1.f};
    if (sd.gamma != nullptr && in) {
      QkRaw<float> g;
      g.a = __ldg(reinterpret_cast<const float4*>(sd.gamma + oa));
      g.b = __ldg(reinterpret_cast<const float4*>(sd.gamma + ob));
      g.get<HALVES>(ga, gb);
    }
    gx[0] = qk_pk(ga[0], ga[1]); gx[1] = qk_pk(ga[2], ga[3]);
    gy[0] = qk_pk(gb[0], gb[1]); gy[1] = qk_pk(gb[2], gb[3]);
  }
  float4 cv[N], sv[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    cv[i] = make_float4(1.f, 1.f, 1.f, 1.f);
    sv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ps[i] < 0 || ps[i] >= p.max_pos) {        // -1 marks a padded row; anything else is an error
      if (ps[i] != -1 && lane == 0) set_status(p.status, ROCS_ERR_INDEX);
      out[i] = nullptr;
    } else if (turns) {
      const float* t = p.table + (long long)ps[i] * d_rot + 4 * sub;
      cv[i] = __ldg(reinterpret_cast<const float4*>(t));
      sv[i] = __ldg(reinterpret_cast<const float4*>(t + half));
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x[4], y[4];
    raw[i].template get<HALVES>(x, y);
    uint64_t xp[2] = {qk_pk(x[0], x[1]), qk_pk(x[2], x[3])}, yp[2] = {qk_pk(y[0], y[1]), qk_pk(y[2], y[3])};
    auto squares = [&]() {               // of the head
      float s0, s1;
      qk_un(qk_fma(yp[1], yp[1], qk_fma(yp[0], yp[0], qk_fma(xp[1], xp[1], qk_mul(xp[0], xp[0])))), s0, s1);
      float ss = s0 + s1;
#pragma unroll
      for (int o = 1; o < T; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      return ss;
    };
    float mean = fmaf(squares(), p.inv_d, p.eps);
    if (__any_sync(0xffffffffu, !(mean > kQkSmall && mean < kQkLarge))) {
      const float k = mean <= kQkSmall ? 0x1p+100f : mean < kQkLarge ? 1.0f : 0x1p-70f;
      const uint64_t kp = qk_pk(k, k);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        xp[j] = qk_mul(xp[j], kp);
        yp[j] = qk_mul(yp[j], kp);
      }
      mean = fmaf(squares(), p.inv_d, p.eps * k * k);
    }
    const float rn = rsqrtf(mean);
    const uint64_t rp = qk_pk(rn, rn);
    const float c[4] = {cv[i].x, cv[i].y, cv[i].z, cv[i].w}, s[4] = {sv[i].x, sv[i].y, sv[i].z, sv[i].w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t cp = qk_pk(c[2 * k], c[2 * k + 1]), sp = qk_pk(s[2 * k], s[2 * k + 1]), np = qk_pk(-s[2 * k], -s[2 * k + 1]);
      const uint64_t a = qk_mul(qk_mul(xp[k], rp), gx[k]), b = qk_mul(qk_mul(yp[k], rp), gy[k]);
      qk_un(qk_fma(b, np, qk_mul(a, cp)), x[2 * k], x[2 * k + 1]);
      qk_un(qk_fma(a, sp, qk_mul(b, cp)), y[2 * k], y[2 * k + 1]);
    }
    if (out[i] != nullptr) QkRaw<E>::template put<HALVES>(out[i], 0, ob - oa, x, y);
  }
}

template <typename E, int T, bool FULL, int N>
void qk_launch_n(const QkParams& p, bool halves, unsigned grid, cudaStream_t s) {
  if (halves) qk_norm_rope_kernel<E, T, true, FULL, N><<<grid, 256, 0, s>>>(p);
  else qk_norm_rope_kernel<E, T, false, FULL, N><<<grid, 256, 0, s>>>(p);
}

template <typename E, int T>
void qk_launch(const QkParams& p, bool halves, unsigned grid, cudaStream_t s) {
  if (p.full && p.items == 1) qk_launch_n<E, T, true, 1>(p, halves, grid, s);
  else if (p.full) qk_launch_n<E, T, true, QkRaw<E>::ITEMS>(p, halves, grid, s);
  else if (p.items == 1) qk_launch_n<E, T, false, 1>(p, halves, grid, s);
  else qk_launch_n<E, T, false, QkRaw<E>::ITEMS_PARTIAL>(p, halves, grid, s);
}

template <typename E>
void qk_launch_t(const QkParams& p, int T, bool halves, unsigned grid, cudaStream_t s) {
  switch (T) {
    case 2: return qk_launch<E, 2>(p, halves, grid, s);
    case 4: return qk_launch<E, 4>(p, halves, grid, s);
    case 8: return qk_launch<E, 8>(p, halves, grid, s);
    case 16: return qk_launch<E, 16>(p, halves, grid, s);
    default: return qk_launch<E, 32>(p, halves, grid, s);
  }
}

}  // namespace

rocs_status launch_qk_norm_rope(rocs_context* ctx, const rocs_qk_desc& d, const void* Q, long long ldq, const void* K,
                                long long ldk, const float* gq, const float* gk, const float* table,
                                const int32_t* pos, void* Qo, long long ldqo, void* Ko, long long ldko,
                                cudaStream_t s) {
  if (d.rows == 0) return ROCS_OK;
  QkParams p;
  p.side[0] = {Q, Qo, ldq, ldqo, d.H_q, 0, 0, gq};
  p.side[1] = {K, Ko, ldk, ldko, d.H_k, 0, 0, gk};
  p.rows = d.rows; p.d = d.d_h; p.d_rot = d.d_rot;
  p.table = table; p.pos = pos; p.max_pos = d.max_pos;
  p.eps = d.eps; p.inv_d = 1.0f / (float)d.d_h;
  p.status = ctx->d_status;
  int T = 2;
  while (T * 8 < d.d_h) T <<= 1;
  const int heads = 32 / T;
  long long blocks[2];
  for (QkSide& sd : p.side) sd.units = (sd.H + heads - 1) / heads;
  p.full = d.d_h == 8 * T && d.d_rot == d.d_h;
  // One item a warp until the warps fill the GPU (1.7 instead of 2.2 us on 512 rows), then several: bf16 three
  // and four blocks an SM where the head is full (193 us on 524288 rows of 16 heads of 32, four and three
  // 11 more), else four and three (131072 rows of 20 heads of 128 of which 64 turn: 286 us, three and three 297).
  const long long all = d.rows * (p.side[0].units + p.side[1].units);
  p.items = all < 48LL * ctx->num_sms ? 1
            : d.io != ROCS_BF16       ? (p.full ? QkRaw<float>::ITEMS : QkRaw<float>::ITEMS_PARTIAL)
                                      : (p.full ? QkRaw<__nv_bfloat16>::ITEMS : QkRaw<__nv_bfloat16>::ITEMS_PARTIAL);
  const int items = 8 * p.items;      // of a block
  for (int i = 0; i < 2; ++i) {
    QkSide& sd = p.side[i];
    sd.inv_units = sd.units > 1 ? ~0ULL / sd.units + 1 : 0;
    blocks[i] = (d.rows * sd.units + items - 1) / items;
  }
  p.blocks_q = (unsigned)blocks[0];
  const long long grid = blocks[0] + blocks[1];
  if (grid > 2147483647LL) {
    set_error("rocs_qk_norm_rope: rows=%lld too many", (long long)d.rows);
    return ROCS_ERR_INVALID_ARG;
  }
  LaunchTimer lt_("qk_norm_rope", s);
  if (d.io == ROCS_BF16) qk_launch_t<__nv_bfloat16>(p, T, d.interleaved == 0, (unsigned)grid, s);
  else qk_launch_t<float>(p, T, d.interleaved == 0, (unsigned)grid, s);
  return cuda_check(cudaGetLastError(), "qk_norm_rope_kernel");
}

}  // namespace rocs
