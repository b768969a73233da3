// Grouped attention over the 4-bit paged history cache, for many query rows per request, on the
// 5th-generation tensor cores.
//
// One CTA takes 128 packed rows (query row x shared head) of one request against one key head, in
// blocks of 64 keys; three CTAs share an SM (two with d = 64 or 128), so that one's waits, start and end
// hide behind the others.
//   warps 0-3  softmax, one thread per row (TMEM lane): S is read from tensor memory, its maximum and
//              exponentials are taken in registers, and P is written back over S as bf16 pairs, the A
//              operand of P V.  The row's reference maximum moves only when a block exceeds it by more
//              than 2^8.
//   warps 4-6  (and 8-10 with d = 64 or 128) producers: a thread takes one group (16 bytes of codes and
//              their scale) of a key or a value at a time, a block ahead in registers, dequantises it
//              (exactly) and writes it as bf16 into the operand's swizzled tile in shared memory.  The
//              conversion is paid once per 128 rows.  (Codes by bulk copies several blocks ahead, as the
//              kernel for few rows has them, are not tried here.)
//   warp 7     issues the MMAs: S_j = Q K_j^T into one of two buffers, O += P_j V_j.  They execute in
//              order, so S_{j+1} is there when the softmax is done with S_j, and the P in a buffer is
//              consumed before the S two blocks later lands on it: one wait and one arrival a block.
// Codes come out of a word as the pairs (0, 4), (1, 5), (2, 6), (3, 7); keys and queries keep that
// order (a contraction index may be permuted), and the output's columns are put right as they are
// stored.  All waits are bounded (ROCS_ERR_DEVICE_TIMEOUT), after which the CTA drains its MMAs, releases
// tensor memory and returns.
//
// Weights enter the product as bf16, and their sum is of those: a value that all keys share comes out as it
// is.  Two bf16 numbers a weight would leave the output's rounding alone (1.65e-3 of the result instead of
// 2.2e-3) for 142 and 120 us below.
// No unit is full: 41388 candidates of 96 requests (8 heads of 32, 675 keys a request on average) take 129 us
// with the exponential unit 43% and the issue slots 55% busy, and the exponentials alone would take 39 and the
// products 17.  A third is the CTAs' start and end, the rest latency between the roles; without exponentials it
// took 6 us less, without the conversion 2, without both 14.  7601 causal rows of 48 requests (4 heads of
// 64 shared by two query heads, 2200 keys) 109 us, of 22 and 19.
// Tried and slower, when these took 123 and 106: exponentials by polynomial for 1/8 to 3/8 of the elements (1 to 5%), loads two
// blocks ahead (145 and 122 us), blocks of 32 keys with four CTAs an SM (124 and 138), three CTAs of one S
// buffer with d = 64 (146 against 139 then), heads outside tiles in the order of blocks (135 and 133),
// keys split where blocks are about as many as slots (no gain).
#include "attn_kv4.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "softmax_math.cuh"
#include "tc_attn.cuh"

namespace rocs {
namespace {

constexpr int KT_ROWS = 128;
constexpr int KT_KEYS = 64;
// pauses between polls of the roles off the critical path, whose polls take issue slots from the softmax
constexpr unsigned kKtProducerSleepNs = 200, kKtIssuerSleepNs = 32;

template <int D>
struct KtCfg {
  static constexpr int PANELS = D == 128 ? 2 : 1;          // swizzled panels of at most 64 elements
  static constexpr int ROWB = D == 32 ? 64 : 128;          // bytes of a panel's row
  static constexpr uint32_t SW = D == 32 ? 4u : 2u;        // 64- or 128-byte swizzle
  static constexpr uint32_t SBO = 8 * ROWB;
  static constexpr int Q_PANEL = KT_ROWS * ROWB, KV_PANEL = KT_KEYS * ROWB;
  static constexpr int Q_BYTES = PANELS * Q_PANEL, KV_BYTES = PANELS * KV_PANEL;   // of K, and of V
  static constexpr int STAGES = D == 32 ? 4 : D == 64 ? 3 : 2;
  // tensor memory: two S buffers (64 columns each, P written over the first half as bf16 pairs) and O
  // (D).  With d = 32 in two pieces, so that three CTAs fit the SM's 512 columns.
  static constexpr int CTAS = D == 32 ? 3 : 2;
  static constexpr int COLS = D == 32 ? 128 : 256, MORE_COLS = D == 32 ? 32 : 0;
  // three producer warps (of a warpgroup with the MMA issuer), or six: with d = 64, three took longer
  // over a block than the softmax does
  static constexpr int TEAMS = D == 32 ? 1 : 2, THREADS = 128 + 128 * TEAMS, PRODUCERS = 96 * TEAMS;
  // registers a thread after the split: the launch gives every thread LAUNCH
  static constexpr int LAUNCH = 80, CONTROL = 56, SOFTMAX = D == 32 ? 104 : 128;
  static_assert(128 * (TEAMS * CONTROL + SOFTMAX) <= THREADS * LAUNCH, "register split");
  static constexpr int USED = Q_BYTES + 2 * STAGES * KV_BYTES + 1024;
  // no more CTAs an SM than tensor memory has room for
  static constexpr int LEAST = 227 * 1024 / (CTAS + 1) / 1024 * 1024;
  static constexpr int SMEM = USED > LEAST ? USED : LEAST;
  static constexpr int ALL = KT_KEYS * (D / KV4_GROUP) * 2;             // groups of a block
  static constexpr int UNITS = (ALL + PRODUCERS - 1) / PRODUCERS;   // ... per producer thread
};

// Byte offset of 16-byte unit c (of the whole row of D elements) of row r in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t kt_unit(int r, int c, int panel_bytes) {
  if constexpr (D == 32) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)((c >> 3) * panel_bytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// One arrival for the whole warp (32 arrivals at one barrier would queue up).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Eight elements of a row in the codes' order (0, 4, 1, 5, 2, 6, 3, 7).
__device__ __forceinline__ uint4 kt_order(uint4 x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                    __byte_perm(x.y, x.w, 0x7632));
}

template <int D>
__global__ void __launch_bounds__(KtCfg<D>::THREADS, KtCfg<D>::CTAS) attn_kv4_tc_kernel(const KaParams p) {
  using C = KtCfg<D>;
  constexpr uint32_t IDESC_S = idesc_bf16(KT_ROWS, KT_KEYS, false);
  constexpr uint32_t IDESC_O = idesc_bf16(KT_ROWS, D == 128 ? 64 : D, true);
  extern __shared__ uint8_t kt_raw[];
  __shared__ uint64_t kv_full[C::STAGES], kv_empty[C::STAGES], q_full, s_full[2], p_full[2], pv_done[2], drain;
  __shared__ uint32_t s_bad[8];            // per block (mod 8): 16-key pieces whose page does not exist
  __shared__ uint32_t tmem_slot[2];
  __shared__ KaTile s_tile;
  __shared__ int4 s_range;                 // first block, blocks, partial's place, head
  __shared__ volatile int abort_flag;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(kt_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sKV = base + C::Q_BYTES;        // [STAGES][K | V]
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x < 8) s_bad[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&kv_full[i], C::PRODUCERS / 32);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 7) {
    tmem_alloc(&tmem_slot[0], C::COLS);
    if (C::MORE_COLS > 0) tmem_alloc(&tmem_slot[1], C::MORE_COLS);
    tmem_relinquish();
  }
  // looked up while thread 0 and warp 7 set up (with a list it may still be in the making); without any work
  // every role has zero blocks and nothing is written
  if (warp == 4) {
    KaTile w;
    int lo = 0, hi = 0, place = -1, group = 0;
    if (!ka_work(p, KT_ROWS, 6, w, lo, hi, place, group)) {
      w = KaTile{};
      hi = lo;
    }
    s_tile = w;
    s_range = make_int4(lo, hi - lo, place, group);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const KaTile a = s_tile;
  const int b_lo = s_range.x, n = s_range.y, part = s_range.z, h = s_range.w;
  const int sees_all = ka_limit(p, a, a.first);     // keys that every row sees
  const uint32_t s_tmem = tmem_slot[0], o_tmem = C::MORE_COLS > 0 ? tmem_slot[1] : s_tmem + 2 * KT_KEYS;
  if (warp < 4) {
    // ---------------- softmax: thread = row = TMEM lane ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX));
    const int row = threadIdx.x;
    const int m = a.first + row;
    const bool live = m < a.n;
    const long long qrow = a.q0 + m / p.share;
    const long long col = ((long long)h * p.share + m % p.share) * D;
    {
      const __nv_bfloat16* q = p.Q + qrow * p.ldq + col;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live) x = kt_order(*reinterpret_cast<const uint4*>(q + 8 * c));
        x.x ^= p.q_flip; x.y ^= p.q_flip; x.z ^= p.q_flip; x.w ^= p.q_flip;
        *reinterpret_cast<uint4*>(sQ + kt_unit<D>(row, c, C::Q_PANEL)) = x;
      }
      fence_proxy_async_smem();
      warp_arrive(&q_full);
    }
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t oaddr = o_tmem + lanes;
    const bool warp_live = a.first + warp * 32 < a.n;      // rows past the request's end are not computed
    const int limit = live ? ka_limit(p, a, m) : 0;
    const float sl2 = p.sl2, lazy = p.lazy;
    float m_cur = -INFINITY, l = 0.f;
    bool ok = true, far = false;
    for (int j = 0; j < n; ++j) {
      const int b = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[b], (j >> 1) & 1, p.status, &abort_flag))) { ok = false; break; }
      tc_fence_after();
      if (warp_live) {
        const uint32_t saddr = s_tmem + lanes + b * KT_KEYS;
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(saddr, v[0]);
        tmem_ld_32x32b_x32(saddr + 32, v[1]);
        const uint32_t bad = *(volatile uint32_t*)&s_bad[j & 7];
        tmem_ld_wait();
        const int k0 = (b_lo + j) * KT_KEYS;
        const bool masked = bad != 0 || k0 + KT_KEYS > sees_all;
        if (masked) {
          const int valid = limit - k0;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= valid || ((bad >> (e >> 4)) & 1u)) v[e >> 5][e & 31] = __float_as_uint(-INFINITY);
        }
        float mt[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) mt[t] = fmaxf(__uint_as_float(v[0][t]), __uint_as_float(v[0][t + 8]));
#pragma unroll
        for (int e = 16; e < 64; e += 16)
#pragma unroll
          for (int t = 0; t < 8; ++t)
            mt[t] = fmax3(mt[t], __uint_as_float(v[(e + t) >> 5][(e + t) & 31]), __uint_as_float(v[(e + 8 + t) >> 5][(e + 8 + t) & 31]));
        const float mx = fmax3(fmax3(mt[0], mt[1], mt[2]), fmax3(mt[3], mt[4], mt[5]), fmaxf(mt[6], mt[7]));
        // the reference: the first block's maximum, then moved (for the whole warp, whose O it rescales in
        // tensor memory) when a row would produce weights above 2^8
        if (j == 0 || __any_sync(0xffffffffu, mx > m_cur + lazy)) {
          const float m_new = j == 0 ? mx : fmaxf(m_cur, mx);
          if (j > 0) {
            const float corr = m_new == -INFINITY ? 1.f : ex2_approx((m_cur - m_new) * sl2);
            if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[b ^ 1], ((j - 1) >> 1) & 1, p.status, &abort_flag))) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t w[16];
              tmem_ld_32x32b_x16(oaddr + c * 16, w);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * corr);
              tmem_st_32x32b_x16(oaddr + c * 16, w);
            }
            l *= corr;
          }
          m_cur = m_new;
          far = __any_sync(0xffffffffu, m_new != -INFINITY && !(fabsf(m_new * sl2) < kKaFarLog2));
        }
        // a row that has seen nothing yet weighs nothing; one with an infinite score is undefined (NaN)
        const float ref = m_cur == -INFINITY ? 0.f : m_cur;
        float neg = -ref * sl2;
        if (far) {
          neg = 0.f;
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e >> 5][e & 31] = __float_as_uint(__uint_as_float(v[e >> 5][e & 31]) - ref);
        }
        // the sum is of the weights as they enter the product, rounded: then numerator and denominator
        // weigh alike
        float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1, p0, p1;
            ffma2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]), sl2, neg, x0, x1);
            p0 = ex2_approx(x0);
            p1 = ex2_approx(x1);
            const uint32_t w = pack_bf16x2(p0, p1);
            rs0 = add_lo(w, rs0);
            rs1 = add_hi(w, rs1);
            pk[e >> 1] = w;
          }
          tmem_st_32x32b_x16(saddr + c * 16, pk);
        }
        l += rs0 + rs1;
        tmem_st_wait();
      }
      // no softmax warp is more than a block ahead of another, and the producers reach block j + 4, the
      // next to use this slot, only after P_j V_j, which waits for this arrival
      if (threadIdx.x == 0) s_bad[(j + 4) & 7] = 0;
      tc_fence_before();
      warp_arrive(&p_full[b]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, p.status, &abort_flag));
    if (ok && warp_live) {
      tc_fence_after();
      const long long item = ((long long)part * p.Hkv + h) * KT_ROWS + row;
      const float inv = part >= 0 ? 1.f : l == 0.f ? 0.f : 1.0f / l;    // a row that sees nothing is zero
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t w[16];
        if (n > 0) {
          tmem_ld_32x32b_x16(oaddr + c * 16, w);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0;
        }
        float o[16];   // columns back in order
#pragma unroll
        for (int e = 0; e < 16; ++e) o[(e & 8) + ((e & 7) >> 1) + 4 * (e & 1)] = __uint_as_float(w[e]) * inv;
        if (live && part < 0) {
          __nv_bfloat16* out = p.O + qrow * p.ldo + col + 16 * c;
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(out + e) = make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                                            pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
        } else if (live) {
          float* out = p.part + item * D + 16 * c;
#pragma unroll
          for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(out + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (live && part >= 0) p.part_ml[item] = make_float2(m_cur, l);
    }
  } else {
    // (one instruction for all warps of the warpgroup, in front of the roles)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CONTROL));
    if (warp != 7) {
      // ---------------- producers ----------------
      const int t = threadIdx.x - (warp < 8 ? 128 : 160);     // (warp 11 has nothing to do)
      constexpr int G = D / KV4_GROUP;
      const int P = 1 << p.P_log2;
      const int32_t* table = p.table + (long long)a.r * p.max_blocks;
      // unit u of this thread: group i = u * PRODUCERS + t of [K: key, group | V: key, group].  A block starts on
      // a page's or (128 tokens) half page's edge, so a unit's place in its record stays the same.
      uint4 wd[C::UNITS];
      uint32_t sc[C::UNITS];
      int next[C::UNITS], key_in[C::UNITS];
      uint32_t code_at[C::UNITS], scale_at[C::UNITS];
      uint32_t piece_bad = 0;
#pragma unroll
      for (int u = 0; u < C::UNITS; ++u) {
        const int i = u * C::PRODUCERS + t, v = i >= KT_KEYS * G;
        const bool has = i < C::ALL;
        key_in[u] = has ? (i / G) % KT_KEYS : 0x7FFFFFFF;   // a unit too many lies past every key
        const int o = key_in[u] & (P - 1);
        code_at[u] = v * kv4_half_bytes(P, D) + o * (D / 2) + (i % G) * 16;
        scale_at[u] = v * kv4_half_bytes(P, D) + kv4_codes_bytes(P, D) + (o * G + i % G) * 2;
      }
      auto pages = [&](int j) {                       // of block j's units; -1 where there is none
        const int left = j < n ? a.len - (b_lo + j) * KT_KEYS : 0;
        const int32_t* at = table + (((long long)(b_lo + j) * KT_KEYS) >> p.P_log2);
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) next[u] = key_in[u] < left ? at[key_in[u] >> p.P_log2] : -1;
      };
      auto load = [&](int j) {
        piece_bad = 0;
        const int left = j < n ? a.len - (b_lo + j) * KT_KEYS : 0;
        const int odd = P > KT_KEYS ? (b_lo + j) & 1 : 0;
        const uint8_t* head = p.cache + (long long)h * kv4_record_bytes(P, D);
        const long long stride = (long long)p.Hkv * kv4_record_bytes(P, D);
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) {
          wd[u] = make_uint4(0, 0, 0, 0);
          sc[u] = 0;
          if (key_in[u] < left) {
            if (next[u] >= 0 && next[u] < p.n_pages) {
              const uint8_t* at = head + next[u] * stride;
              wd[u] = *reinterpret_cast<const uint4*>(at + code_at[u] + odd * kv4_codes_bytes(KT_KEYS, D));
              sc[u] = *reinterpret_cast<const uint16_t*>(at + scale_at[u] + odd * kv4_scales_bytes(KT_KEYS, D));
            } else {
              piece_bad |= 1u << (key_in[u] >> 4);
            }
          }
        }
      };
      if (t < C::PRODUCERS) {
        pages(0);
        load(0);
        pages(1);
        for (int j = 0; j < n; ++j) {
          const int st = j % C::STAGES;
          if (j >= C::STAGES && !__all_sync(0xffffffffu, mbar_wait_sleep(&kv_empty[st], ((j / C::STAGES) - 1) & 1, p.status, &abort_flag, kKtProducerSleepNs)))
            break;
          uint8_t* kv = sKV + st * 2 * C::KV_BYTES;
#pragma unroll
          for (int u = 0; u < C::UNITS; ++u) {
            const int i = u * C::PRODUCERS + t, v = i >= KT_KEYS * G;
            const int g = i % G;
            const uint32_t s2 = sc[u] | (sc[u] << 16), c2 = kv4_offset(s2);
            const uint32_t w[4] = {wd[u].x, wd[u].y, wd[u].z, wd[u].w};
            if (key_in[u] < KT_KEYS) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 e = make_uint4(kv4_fma2(kv4_pair(w[k]), s2, c2), kv4_fma2(kv4_pair(w[k] >> 4), s2, c2),
                                           kv4_fma2(kv4_pair(w[k] >> 8), s2, c2), kv4_fma2(kv4_pair(w[k] >> 12), s2, c2));
                *reinterpret_cast<uint4*>(kv + v * C::KV_BYTES + kt_unit<D>(key_in[u], g * 4 + k, C::KV_PANEL)) = e;
              }
            }
          }
          if (piece_bad != 0) {
            atomicOr(&s_bad[j & 7], piece_bad);
            set_status(p.status, ROCS_ERR_INDEX);
          }
          fence_proxy_async_smem();
          warp_arrive(&kv_full[st]);
          // after the fence, which would wait for loads in front of it
          load(j + 1);
          pages(j + 2);
        }
      }
    } else {
      // ---------------- MMA issuer: the whole warp, so that its operands stay uniform ----------------
      const uint64_t qd = sdesc(smem_u32(sQ), C::SBO, C::SW), kd = sdesc(smem_u32(sKV), C::SBO, C::SW);
      const bool one = elect_one();
      auto issue_s = [&](int j) -> bool {
        const int st = j % C::STAGES;
        if (!__all_sync(0xffffffffu, mbar_wait_sleep(&kv_full[st], (j / C::STAGES) & 1, p.status, &abort_flag, kKtIssuerSleepNs))) return false;
        tc_fence_after();
        if (one) {
          const uint64_t k = kd + st * (2 * C::KV_BYTES >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma_ss(s_tmem + (j & 1) * KT_KEYS, qd + (((ks >> 2) * C::Q_PANEL + (ks & 3) * 32) >> 4),
                      k + (((ks >> 2) * C::KV_PANEL + (ks & 3) * 32) >> 4), IDESC_S, ks > 0 ? 1u : 0u);
          tc_commit(&s_full[j & 1]);
        }
        return true;
      };
      auto issue_pv = [&](int j) -> bool {
        const int st = j % C::STAGES;
        if (!__all_sync(0xffffffffu, mbar_wait_sleep(&p_full[j & 1], (j >> 1) & 1, p.status, &abort_flag, kKtIssuerSleepNs))) return false;
        tc_fence_after();
        if (one) {
          const uint64_t v = kd + st * (2 * C::KV_BYTES >> 4) + (C::KV_BYTES >> 4);
          const uint32_t acc = j > 0 ? 1u : 0u;
#pragma unroll
          for (int pn = 0; pn < C::PANELS; ++pn)
#pragma unroll
            for (int ks = 0; ks < KT_KEYS / 16; ++ks)
              tc_mma_ts(o_tmem + pn * 64, s_tmem + (j & 1) * KT_KEYS + ks * 8,
                        v + ((pn * C::KV_PANEL + ks * 16 * C::ROWB) >> 4), IDESC_O, ks > 0 ? 1u : acc);
          tc_commit(&kv_empty[st]);
          tc_commit(&pv_done[j & 1]);
        }
        return true;
      };
      bool ok = n == 0 || __all_sync(0xffffffffu, mbar_wait_sleep(&q_full, 0, p.status, &abort_flag, kKtIssuerSleepNs));
      if (ok && n > 0) ok = issue_s(0) && (n < 2 || issue_s(1));
      for (int j = 0; ok && j < n; ++j) ok = issue_pv(j) && (j + 2 >= n || issue_s(j + 2));
      __syncwarp();
      if (one) {
        tc_commit(&drain);
        mbar_wait(&drain, 0, p.status, nullptr);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 7) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(s_tmem, C::COLS);
    if (C::MORE_COLS > 0) tmem_dealloc(o_tmem, C::MORE_COLS);
  }
}

template <int D>
rocs_status kt_launch(rocs_context* ctx, const KaParams& p, long long blocks, cudaStream_t s) {
  using C = KtCfg<D>;
  static bool attr[64] = {false};
  if (ctx->device >= 64 || !attr[ctx->device]) {
    rocs_status st = cuda_check(cudaFuncSetAttribute(attn_kv4_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM),
                                "cudaFuncSetAttribute(attn_kv4_tc)");
    if (st != ROCS_OK) return st;
    // the softmax warps raise their register limit out of the launch's allocation; refuse to launch if
    // the compiled kernel was given fewer registers than that split needs
    cudaFuncAttributes fa;
    st = cuda_check(cudaFuncGetAttributes(&fa, attn_kv4_tc_kernel<D>), "cudaFuncGetAttributes(attn_kv4_tc)");
    if (st != ROCS_OK) return st;
    if (fa.numRegs < C::LAUNCH) {
      set_error("attn_kv4_tc: kernel compiled with %d registers per thread, below the warpgroup split", fa.numRegs);
      return ROCS_ERR_UNSUPPORTED;
    }
    if (ctx->device < 64) attr[ctx->device] = true;
  }
  LaunchTimer lt_("attn_kv4_tc", s);
  if (p.items != nullptr)
    return launch_dependent(attn_kv4_tc_kernel<D>, dim3((unsigned)blocks), dim3(C::THREADS), C::SMEM, s, "attn_kv4_tc_kernel", p);
  attn_kv4_tc_kernel<D><<<(unsigned)blocks, C::THREADS, C::SMEM, s>>>(p);
  return cuda_check(cudaGetLastError(), "attn_kv4_tc_kernel");
}

}  // namespace

rocs_status launch_attn_kv4_tc(rocs_context* ctx, int d_h, const KaParams& p, long long blocks, cudaStream_t s) {
  switch (d_h) {
    case 32: return kt_launch<32>(ctx, p, blocks, s);
    case 64: return kt_launch<64>(ctx, p, blocks, s);
    default: return kt_launch<128>(ctx, p, blocks, s);
  }
}

}  // namespace rocs
