// RMS norm of every query and key head with the position rotation in the same pass.
//
// Per row i, head h and element e of a head of d: y_e = x_e / sqrt(mean_e(x_e^2) + eps) * gamma_e, then
// for the first d_rot elements and pair t < d_rot / 2, with (c, s) the table's row of the row's
// position: (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s), where (a, b) = (t, t + d_rot / 2), or
// (2 t, 2 t + 1) when pairs are neighbours.  fp32 inside, one rounding at the end.
//
// Bound by memory: every element is read and written once.  A lane keeps eight elements of a head
// (16 or 32 bytes), so a head is d / 8 lanes of one warp and a warp covers 32 / lanes heads of a row at
// a time: contiguous in memory, the mean by shuffles within the head's lanes, and with half-split
// pairs the partner's eight elements from the lane d_rot / 16 away.  A warp walks over the heads of
// its row with gamma and the row's angles in registers; where rows are few, it takes one unit of heads
// only, so that they spread over the GPU.
#include "common.cuh"
#include "internal.h"

namespace rocs {
namespace {

struct QkParams {
  const void *Q, *K;
  long long ldq, ldk, ldqo, ldko;
  void *Qo, *Ko;
  long long rows;
  int Hq, Hk, d, d_rot;
  const float *gq, *gk, *table;
  const int32_t* pos;
  int max_pos;
  float eps, inv_d;
  int units_q, units;      // units of 32 / T heads: of the queries, of both
  int per_warp;            // units a warp walks over
  int* status;
};

__device__ __forceinline__ void qk_load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void qk_load8(const float* p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void qk_store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                            pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void qk_store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void qk_angles8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// T lanes a head (a power of two, T * 8 >= d).  HALVES: pairs are (t, t + d_rot / 2).
template <typename E, int T, bool HALVES>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkParams p) {
  constexpr int HEADS = 32 / T;
  const int lane = threadIdx.x & 31, sub = lane & (T - 1), hw = lane / T;
  const int parts = (p.units + p.per_warp - 1) / p.per_warp;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const long long row = w / parts;
  if (row >= p.rows) return;
  const int u0 = (int)(w - row * parts) * p.per_warp;
  const int u1 = min(u0 + p.per_warp, p.units);

  const int at = p.pos[row];
  if (at < 0 || at >= p.max_pos) {        // -1 marks a padded row; anything else is an error
    if (at != -1 && lane == 0) set_status(p.status, ROCS_ERR_INDEX);
    return;
  }
  const int e0 = sub * 8;
  const bool in = e0 < p.d;
  const bool turns = e0 < p.d_rot;
  const int half = p.d_rot >> 1;
  // the angles of this lane's elements; sg is -1 for the first of a half-split pair, 1 for the second
  float c[8], s[8];
  int partner = lane;
  float sg = 1.f;
  if (turns) {
    const float* t = p.table + (long long)at * p.d_rot;
    if (HALVES) {
      const bool second = e0 >= half;
      partner = second ? lane - (half >> 3) : lane + (half >> 3);
      sg = second ? 1.f : -1.f;
      qk_angles8(t + (second ? e0 - half : e0), c);
      qk_angles8(t + half + (second ? e0 - half : e0), s);
    } else {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(t + (e0 >> 1)));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(t + half + (e0 >> 1)));
      c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
      s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
    }
  }
  float g[8];
  int g_of = -1;   // whose gamma g holds: 0 the queries', 1 the keys'
  for (int u = u0; u < u1; ++u) {
    const bool key = u >= p.units_q;
    const int h = (key ? u - p.units_q : u) * HEADS + hw;
    const bool live = in && h < (key ? p.Hk : p.Hq);
    const E* src = reinterpret_cast<const E*>(key ? p.K : p.Q) + row * (key ? p.ldk : p.ldq) + (long long)h * p.d + e0;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (live) qk_load8(src, x);
    if (g_of != (int)key) {
      g_of = (int)key;
      const float* gm = key ? p.gk : p.gq;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
      if (gm != nullptr && in) qk_angles8(gm + e0, g);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 1; o < T; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
    if (HALVES) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], sg * y[i] * s[i]);
      }
    } else if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[i] - b * s[i];
        x[2 * i + 1] = b * c[i] + a * s[i];
      }
    }
    if (live)
      qk_store8(reinterpret_cast<E*>(key ? p.Ko : p.Qo) + row * (key ? p.ldko : p.ldqo) + (long long)h * p.d + e0, x);
  }
}

template <typename E, int T>
void qk_launch(const QkParams& p, bool halves, unsigned grid, cudaStream_t s) {
  if (halves) qk_norm_rope_kernel<E, T, true><<<grid, 256, 0, s>>>(p);
  else qk_norm_rope_kernel<E, T, false><<<grid, 256, 0, s>>>(p);
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
  p.Q = Q; p.K = K; p.ldq = ldq; p.ldk = ldk; p.Qo = Qo; p.Ko = Ko; p.ldqo = ldqo; p.ldko = ldko;
  p.rows = d.rows; p.Hq = d.H_q; p.Hk = d.H_k; p.d = d.d_h; p.d_rot = d.d_rot;
  p.gq = gq; p.gk = gk; p.table = table; p.pos = pos; p.max_pos = d.max_pos;
  p.eps = d.eps; p.inv_d = 1.0f / (float)d.d_h;
  p.status = ctx->d_status;
  int T = 2;
  while (T * 8 < d.d_h) T <<= 1;
  const int heads = 32 / T;
  p.units_q = (d.H_q + heads - 1) / heads;
  p.units = p.units_q + (d.H_k + heads - 1) / heads;
  // a warp per row once that fills the GPU's resident warps, else a warp per unit
  p.per_warp = d.rows >= 32LL * ctx->num_sms ? p.units : 1;
  const long long warps = d.rows * ((p.units + p.per_warp - 1) / p.per_warp);
  const long long grid = (warps + 7) / 8;
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
