// Grouped attention over the 4-bit paged history cache, for few query rows per request.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j   over the keys j that row i sees,
// with k_j, v_j = (code - 8) * scale dequantised in registers (exactly: see kv4.cuh).
//
// The share query heads of a key head are packed with the request's query rows into tiles of 8 NT
// rows, and the products are taken transposed on m16n8k16 MMAs (S^T = K Q^T, O^T = V^T P^T): the
// cache is the 16-row operand, which comes straight from the packed words, and one to eight query
// rows waste no more than an 8-wide tile.  The contraction index of either product may be permuted
// at will as long as both operands agree, so
//   S^T: a lane takes whole words of a key's row (d / 32 neighbouring ones), whose nibbles (0, 4),
//        (1, 5), (2, 6), (3, 7) are the bf16 pairs; the queries are loaded in that order once;
//   O^T: a lane takes the word of its eight output elements from four keys, and pairs equal nibbles
//        of two keys (ka_key says which rows of a score tile are which keys).
// P^T moves from the accumulator's layout to the operand's by an 8x8 transpose in registers.
//
// A block of four warps has the keys of one (tile, head, split); each warp streams its own keys through
// a ring of bulk copies and keeps its own running maximum, sum and output, joined through shared memory
// at the end, so the loop has no block-wide wait.  Short histories of many requests give each warp a head
// of its own instead.  Where the (tile, head) items are too few to fill the GPU the keys are split over
// blocks, whose partial results another launch joins in a fixed order; where they are more than it holds,
// a list made on the device starts the longest first.
//
// The cache's bytes would be the bound, but turning codes into operands takes as many issue slots: for
// three histories of 351531 tokens together (8 heads of 128, shared by four query heads) 104 us, of which 62 us are
// the bytes at the measured copy rate, with the integer pipe 58% busy and 2.3 instructions a cycle; for
// 512 single queries against histories of 567 keys on average (8 heads of 32) 36 us, of which 13 us are the
// bytes, 3 the list and the rest the start, the longest histories and the end.  The same calls on the
// 128-row kernel took three to four times as long.
// Weights enter the product as bf16 (two bf16 numbers a weight would take 113 and 39 us), and their sum is of those.
#include <float.h>

#include <type_traits>

#include "attn_kv4.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "mma_frag.cuh"
#include "tc_attn.cuh"

namespace rocs {
namespace {

constexpr int KA_WARPS = 4;
constexpr int kTcRows = 32;     // packed rows a request above which the 128-row tensor-core tiles pay

template <int D>
struct KaCfg {
  static constexpr int KEYS_LOG2 = D == 32 ? 7 : 6;          // keys per stage of a warp's ring
  static constexpr int KEYS = 1 << KEYS_LOG2;
  static constexpr int CHUNK = 64;                           // keys scored at a time
  static constexpr int STAGE = KEYS * D * 9 / 8;
  static constexpr int STAGES = D == 64 ? 3 : 2;
  static constexpr int RING = STAGE * STAGES;
  static constexpr int SMEM = KA_WARPS * RING;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void ka_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
}

// The key, of 16 neighbouring ones, that row rho of a score tile stands for.  d = 32: 0, 2, 4, .. and 1, 3,
// 5, .., which gives a lane pairs and fours of neighbouring keys, whose scales are one load.  Wider heads:
// in each half 0, 4, 1, 5, 2, 6, 3, 7, so that the words that the lanes read of their values lie in
// different banks.
template <int D>
__device__ __forceinline__ int ka_key(int rho) {
  if constexpr (D == 32) return 2 * (rho & 7) + (rho >> 3);
  return (rho & 8) + ((rho & 7) >> 1) + 4 * (rho & 1);
}

// BIG: pages of at least 64 tokens, so that a chunk lies in one page's record.
template <int D, int NT, bool BIG>
__global__ void __launch_bounds__(KA_WARPS * 32) attn_kv4_kernel(const KaParams p) {
  using C = KaCfg<D>;
  constexpr int T = 8 * NT;
  constexpr int KW = D / 32;                  // words of a key row per lane (scores)
  constexpr int VW = D >= 64 ? D / 64 : 1;    // words of a key row per lane (values)
  constexpr int VN = D >= 64 ? 4 : 2;         // 16-row output tiles per word
  constexpr int MT = VW * VN;                 // = D / 16
  extern __shared__ __align__(128) uint8_t ka_smem[];
  __shared__ uint64_t bars[KA_WARPS][C::STAGES];
  __shared__ float s_m[KA_WARPS][T], s_l[KA_WARPS][T];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3;
  // p.per_item warps (1, 2 or 4) share a (tile, head); the block has 4 / per_item neighbouring heads
  const int heads = KA_WARPS / p.per_item, part = warp & (p.per_item - 1);
  KaTile a;
  int c_lo, c_hi, place, group;
  if (!ka_work(p, T, C::KEYS_LOG2, a, c_lo, c_hi, place, group)) return;
  const int h = group * heads + warp / p.per_item;
  const int last = min(a.first + T, a.n) - 1;       // last packed row of the tile
  const int seen = ka_limit(p, a, last);            // keys that any row of the tile sees
  const int sees_all = ka_limit(p, a, a.first);     // keys that every row sees
  if (h >= p.Hkv) c_hi = c_lo;

  uint8_t* ring = ka_smem + warp * C::RING;
  if (lane == 0)
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&bars[warp][i], 1);
  fence_barrier_init();
  fence_proxy_async_smem();
  __syncwarp();

  // a stage's pages: pieces of PE = min(page, KEYS) keys, each a record of PE keys in the stage
  const int PE_log2 = min(p.P_log2, C::KEYS_LOG2), PE = 1 << PE_log2;
  const int pieces = C::KEYS >> PE_log2;
  const int rec = kv4_record_bytes(PE, D);
  const int32_t* table = p.table + (long long)a.r * p.max_blocks;
  const uint8_t* head = p.cache + (long long)h * kv4_record_bytes(1 << p.P_log2, D);
  const long long page_bytes = (long long)p.Hkv * kv4_record_bytes(1 << p.P_log2, D);
  auto page_of = [&](int c) -> int {      // lane i < pieces: the page of piece i of stage c (-2: none is needed)
    const long long key = (long long)c * C::KEYS + ((long long)lane << PE_log2);
    return lane < pieces && c < c_hi && key < a.len ? table[key >> p.P_log2] : -2;
  };
  uint32_t bad_of = 0;                    // 8 bits per stage: pieces whose page does not exist
  auto issue = [&](int c, int st, int page) {
    const bool ok = page >= 0 && page < p.n_pages;
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    const uint32_t bad = __ballot_sync(0xffffffffu, !ok && page != -2);
    bad_of = (bad_of & ~(255u << (8 * st))) | (bad << (8 * st));
    if (bad != 0 && lane == 0) set_status(p.status, ROCS_ERR_INDEX);
    uint64_t* bar = &bars[warp][st];
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(__popc(mask) * rec));
    __syncwarp();
    if (ok) {
      uint8_t* dst = ring + st * C::STAGE + lane * rec;
      const uint8_t* src = head + page * page_bytes;
      if (p.P_log2 <= C::KEYS_LOG2) {
        bulk_load(dst, src, rec, bar);
      } else {                            // part of a page: codes and scales of keys and values one by one
        const int P = 1 << p.P_log2, o = (c * C::KEYS) & (P - 1);
        constexpr int CB = kv4_codes_bytes(C::KEYS, D), SB = kv4_scales_bytes(C::KEYS, D);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint8_t* half = src + v * kv4_half_bytes(P, D);
          bulk_load(dst + v * (CB + SB), half + kv4_codes_bytes(o, D), CB, bar);
          bulk_load(dst + v * (CB + SB) + CB, half + kv4_codes_bytes(P, D) + kv4_scales_bytes(o, D), SB, bar);
        }
      }
    }
  };

  // the queries, in the order of the keys' nibble pairs
  uint32_t qf[NT][KW][4];
  int limit[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int m = a.first + nt * 8 + g;
    const bool live = m < a.n && h < p.Hkv;
    const __nv_bfloat16* q = p.Q + (a.q0 + m / p.share) * p.ldq + ((long long)h * p.share + m % p.share) * D;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live) x = *reinterpret_cast<const uint4*>(q + (tq * KW + w) * 8);
      qf[nt][w][0] = __byte_perm(x.x, x.z, 0x5410) ^ p.q_flip;   // (0, 4)
      qf[nt][w][1] = __byte_perm(x.x, x.z, 0x7632) ^ p.q_flip;   // (1, 5)
      qf[nt][w][2] = __byte_perm(x.y, x.w, 0x5410) ^ p.q_flip;   // (2, 6)
      qf[nt][w][3] = __byte_perm(x.y, x.w, 0x7632) ^ p.q_flip;   // (3, 7)
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) limit[nt][e] = ka_limit(p, a, min(a.first + nt * 8 + 2 * tq + e, a.n - 1));
  }

  float o[MT][NT][4];
  // sums of the weights as they enter the product, rounded (numerator and denominator weigh alike): a further
  // row tile of that product, of ones, whose rows are all the sum
  float m_run[NT][2], l_run[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = l_run[nt][2] = l_run[nt][3] = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
  }

  // the warp's stages: c_lo + part, then every per_item-th; the ring is filled ahead, page numbers one
  // stage further ahead still
  int c_issue = c_lo + part;
  int st_issue = 0;
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (c_issue < c_hi) {
      issue(c_issue, st_issue, page_of(c_issue));
      c_issue += p.per_item;
      ++st_issue;
    }
  }
  int next_page = page_of(c_issue);
  int st = 0;
  uint32_t phase = 0;
  bool alive = true;
  for (int c = c_lo + part; c < c_hi; c += p.per_item) {
    if (c_issue < c_hi) {     // into the stage read in the last turn
      __syncwarp();
      issue(c_issue, st_issue, next_page);
      if (++st_issue == C::STAGES) st_issue = 0;
      c_issue += p.per_item;
      next_page = page_of(c_issue);
    }
    // after a wait that ran out, what is in flight is still waited for, then the warp leaves
    alive = __all_sync(0xffffffffu, mbar_wait(&bars[warp][st], phase, p.status, nullptr)) && alive;
    const uint8_t* stage = ring + st * C::STAGE;
    const uint32_t bad = (bad_of >> (8 * st)) & 255u;
    // one chunk; WHOLE: every row sees every key of it
    auto chunk = [&](auto whole_c, int sub) {
      constexpr bool WHOLE = decltype(whole_c)::value;
      const int k0 = c * C::KEYS + sub * C::CHUNK;
      // the record and the row in it of the 16 keys of score tile t
      const uint8_t* base0 = stage;
      int in0 = 0;
      if (BIG) {
        base0 = stage + ((sub * C::CHUNK) >> PE_log2) * rec;
        in0 = (sub * C::CHUNK) & (PE - 1);
      }
      auto base_of = [&](int t) { return BIG ? base0 : stage + ((sub * C::CHUNK + 16 * t) >> PE_log2) * rec; };
      auto in_of = [&](int t) { return BIG ? in0 + 16 * t : (sub * C::CHUNK + 16 * t) & (PE - 1); };
      auto lost_of = [&](int t) { return ((bad >> ((sub * C::CHUNK + 16 * t) >> PE_log2)) & 1u) != 0; };
      constexpr int ST = C::CHUNK / 16;      // score tiles
      float s[ST][NT][4];
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const uint8_t* base = base_of(t);
        const int in = in_of(t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[t][nt][0] = s[t][nt][1] = s[t][nt][2] = s[t][nt][3] = 0.f;
        uint32_t w0[KW], w1[KW], s0, s1;
        const int r0 = in + ka_key<D>(g), r1 = in + ka_key<D>(g + 8);
        ka_words<KW>(base + r0 * (D / 2) + tq * (4 * KW), w0);
        ka_words<KW>(base + r1 * (D / 2) + tq * (4 * KW), w1);
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(base + kv4_codes_bytes(PE, D));
        if (D == 32) {           // keys 2g and 2g + 1: their scales are one word
          const uint32_t x = *reinterpret_cast<const uint32_t*>(sc + r0);
          s0 = __byte_perm(x, x, 0x1010);
          s1 = __byte_perm(x, x, 0x3232);
        } else {
          const int grp = (tq * KW) >> 2;
          s0 = sc[r0 * (D / 32) + grp];
          s1 = sc[r1 * (D / 32) + grp];
          s0 = __byte_perm(s0, s0, 0x1010);
          s1 = __byte_perm(s1, s1, 0x1010);
        }
        const uint32_t f0 = kv4_offset(s0), f1 = kv4_offset(s1);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t e0[4], e1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e0[i] = kv4_fma2(kv4_pair(w0[w] >> (4 * i)), s0, f0);
            e1[i] = kv4_fma2(kv4_pair(w1[w] >> (4 * i)), s1, f1);
          }
          const uint32_t a0[4] = {e0[0], e1[0], e0[1], e1[1]}, a1[4] = {e0[2], e1[2], e0[3], e1[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(s[t][nt], a0, qf[nt][w][0], qf[nt][w][1]);
            mma_bf16_16816(s[t][nt], a1, qf[nt][w][2], qf[nt][w][3]);
          }
        }
      }
      if (!WHOLE) {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          const bool lost = lost_of(t);
          const int j = k0 + 16 * t;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (lost || j + ka_key<D>(g + 8 * (e >> 1)) >= limit[nt][e & 1]) s[t][nt][e] = -INFINITY;
        }
      }
      // each query column's maximum; the reference moves, and what was summed against it is rescaled,
      // where a weight would exceed 2^8
      bool moves = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
          for (int t = 1; t < ST; ++t) m = fmax3(m, s[t][nt][e], s[t][nt][e + 2]);
          mx[nt][e] = m;
          moves = moves || m > m_run[nt][e] + p.lazy;
        }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], x));
            const float m_new = fmaxf(m_run[nt][e], mx[nt][e]);
            corr[e] = m_new == -INFINITY ? 1.f : ex2_approx((m_run[nt][e] - m_new) * p.sl2);
            m_run[nt][e] = m_new;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) l_run[nt][e] *= corr[e & 1];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] *= corr[e & 1];
        }
      }
      float neg[NT][2];
      bool far = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          neg[nt][e] = m_run[nt][e] == -INFINITY ? 0.f : -m_run[nt][e] * p.sl2;   // nothing seen yet: weights of 0
          far = far || !(fabsf(neg[nt][e]) < kKaFarLog2);
        }
      if (__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ref = m_run[nt][e & 1] == -INFINITY ? 0.f : m_run[nt][e & 1];
#pragma unroll
            for (int t = 0; t < ST; ++t) s[t][nt][e] -= ref;
            neg[nt][e & 1] = 0.f;
          }
      }
      // weights and their sums; P^T in the operand's layout
      uint32_t pf[ST][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4[e] = ex2_approx(fmaf(s[t][nt][e], p.sl2, neg[nt][e & 1]));
          pf[t][nt][0] = transpose8x8(pack_bf16x2(e4[0], e4[1]));
          pf[t][nt][1] = transpose8x8(pack_bf16x2(e4[2], e4[3]));
          constexpr uint32_t ONES[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
          mma_bf16_16816(l_run[nt], ONES, pf[t][nt][0], pf[t][nt][1]);
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const uint8_t* base = base_of(t) + kv4_half_bytes(PE, D);
        const int in = in_of(t);
        const int word = D >= 64 ? g * VW : (g & 3), grp = word >> 2;
        // the lane's keys: operand columns 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
        const int col[4] = {2 * tq, 2 * tq + 1, 2 * tq + 8, 2 * tq + 9};
        uint32_t vw[4][VW], sa, sb;
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(base + kv4_codes_bytes(PE, D));
#pragma unroll
        for (int i = 0; i < 4; ++i) ka_words<VW>(base + (in + ka_key<D>(col[i])) * (D / 2) + word * 4, vw[i]);
        if (D == 32) {           // keys 4 tq .. 4 tq + 3, in the order 0, 2, 1, 3
          const uint2 x = *reinterpret_cast<const uint2*>(sc + in + 4 * tq);
          sa = __byte_perm(x.x, x.y, 0x5410);
          sb = __byte_perm(x.x, x.y, 0x7632);
        } else {
          uint32_t vs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) vs[i] = sc[(in + ka_key<D>(col[i])) * (D / 32) + grp];
          sa = __byte_perm(vs[0], vs[1], 0x5410);
          sb = __byte_perm(vs[2], vs[3], 0x5410);
        }
        if (!WHOLE) {
          // a key that does not exist has a weight of zero, but what lies in its place may be
          // anything: its value is made zero too
          const int left = lost_of(t) ? 0 : a.len - (k0 + 16 * t);
          sa &= (ka_key<D>(col[0]) < left ? 0xffffu : 0u) | (ka_key<D>(col[1]) < left ? 0xffff0000u : 0u);
          sb &= (ka_key<D>(col[2]) < left ? 0xffffu : 0u) | (ka_key<D>(col[3]) < left ? 0xffff0000u : 0u);
        }
        const uint32_t fa = kv4_offset(sa), fb = kv4_offset(sb);
        // nibbles i (lo) and 4 + i (hi) of two keys' words as pairs; with d = 32 lanes 4 apart share a
        // word and take nibbles 0, 1 and 4, 5 or 2, 3 and 6, 7 of it
        const uint32_t lo = D >= 64 ? 0x5410u : g < 4 ? 0x0400u : 0x0501u, hi = D >= 64 ? 0x7632u : g < 4 ? 0x0602u : 0x0703u;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t la = __byte_perm(vw[0][w], vw[1][w], lo), ha = __byte_perm(vw[0][w], vw[1][w], hi);
          const uint32_t lb = __byte_perm(vw[2][w], vw[3][w], lo), hb = __byte_perm(vw[2][w], vw[3][w], hi);
#pragma unroll
          for (int i = 0; i < VN; ++i) {
            const uint32_t av[4] = {kv4_fma2(kv4_pair(la >> (4 * i)), sa, fa), kv4_fma2(kv4_pair(ha >> (4 * i)), sa, fa),
                                    kv4_fma2(kv4_pair(lb >> (4 * i)), sb, fb), kv4_fma2(kv4_pair(hb >> (4 * i)), sb, fb)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[w * VN + i][nt], av, pf[t][nt][0], pf[t][nt][1]);
          }
        }
      }
    };
#pragma unroll 1
    for (int sub = 0; sub < C::KEYS / C::CHUNK; ++sub) {
      const int k0 = c * C::KEYS + sub * C::CHUNK;
      if (!alive || k0 >= seen) break;
      if (bad == 0 && k0 + C::CHUNK <= sees_all && k0 + C::CHUNK <= a.len) chunk(std::true_type{}, sub);
      else chunk(std::false_type{}, sub);
    }
    if (++st == C::STAGES) {
      st = 0;
      phase ^= 1;
    }
  }

  // join an item's warps: outputs through the ring's memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (g == 0) {
        s_m[warp][nt * 8 + 2 * tq + e] = m_run[nt][e];
        s_l[warp][nt * 8 + 2 * tq + e] = l_run[nt][e];
      }
  __syncthreads();
  float* so = reinterpret_cast<float*>(ka_smem);        // [warp][row][D]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int w = mt / VN, i = mt % VN;
    const int d0 = D >= 64 ? 8 * (g * VW + w) + i : 8 * (g & 3) + 2 * (g >> 2) + i;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        so[(warp * T + nt * 8 + 2 * tq + (e & 1)) * D + d0 + 4 * (e >> 1)] = o[mt][nt][e];
  }
  __syncthreads();
  const int live = min(T, a.n - a.first);
  for (int i = threadIdx.x; i < heads * live * (D / 2); i += KA_WARPS * 32) {
    const int d = 2 * (i % (D / 2)), hr = i / (D / 2), hi = hr / live, row = hr - hi * live;
    const int hh = group * heads + hi, w0 = hi * p.per_item;
    if (hh >= p.Hkv) break;
    float top = s_m[w0][row];
    for (int w = 1; w < p.per_item; ++w) top = fmaxf(top, s_m[w0 + w][row]);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, x = 0.f, y = 0.f;
    for (int w = 0; w < p.per_item; ++w) {
      const float f = ex2_approx((s_m[w0 + w][row] - ref) * p.sl2);
      const float2 v = *reinterpret_cast<const float2*>(so + ((w0 + w) * T + row) * D + d);
      l = fmaf(f, s_l[w0 + w][row], l);
      x = fmaf(f, v.x, x);
      y = fmaf(f, v.y, y);
    }
    const int m = a.first + row;
    if (place < 0) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;      // a row that sees nothing is zero
      __nv_bfloat16* out = p.O + (a.q0 + m / p.share) * p.ldo + ((long long)hh * p.share + m % p.share) * D + d;
      *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(x * inv, y * inv);
    } else {
      const long long at = ((long long)place * p.Hkv + hh) * T + row;
      *reinterpret_cast<float2*>(p.part + at * D + d) = make_float2(x, y);
      if (d == 0) p.part_ml[at] = make_float2(top, l);
    }
  }
}

// Joins the splits of each (tile, head), in a fixed order.  D / 2 threads take a row (a pair of
// columns each); the block's 256 / D groups of them take a row each where splits are few, else they
// share one row's splits among them, with four splits' loads in flight a thread.
constexpr int KJ_SPLITS = 8;      // splits above which the groups share a row
template <int D, int T>
__global__ void __launch_bounds__(128) attn_kv4_join_kernel(const KaParams p, int rows_per_block) {
  constexpr int GROUPS = 256 / D;
  __shared__ float s_part[GROUPS][D + 2];
  grid_dependency_wait();
  if ((int)blockIdx.x >= p.counts[1]) return;
  const KaJoin a = p.joins[blockIdx.x];
  const int n = a.n_r * p.share;
  const int h = blockIdx.y, grp = threadIdx.x / (D / 2), d = 2 * (threadIdx.x % (D / 2));
  const bool shared_row = a.parts > KJ_SPLITS;
  const int row_step = shared_row ? 1 : GROUPS, split_step = shared_row ? GROUPS : 1;
  const long long stride = (long long)p.Hkv * T, at0 = (long long)a.part * stride + h * T;     // of the parts' rows
  const int row_end = min((int)(blockIdx.z + 1) * rows_per_block, n - a.first);
  for (int row0 = blockIdx.z * rows_per_block; row0 < row_end; row0 += row_step) {
    const int row = row0 + (shared_row ? 0 : grp);
    float top = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
    if (row < row_end) {
      for (int s0 = shared_row ? grp : 0; s0 < a.parts; s0 += 4 * split_step) {
        float2 ml[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int sp = s0 + i * split_step;
          ml[i] = make_float2(-INFINITY, 0.f);
          v[i] = make_float2(0.f, 0.f);
          if (sp < a.parts) {
            ml[i] = p.part_ml[at0 + sp * stride + row];
            v[i] = *reinterpret_cast<const float2*>(p.part + (at0 + sp * stride + row) * D + d);
          }
        }
        float m = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, ml[i].x);
        const float ref = m == -INFINITY ? 0.f : m, f = ex2_approx((top - ref) * p.sl2);
        l *= f; x *= f; y *= f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = ex2_approx((ml[i].x - ref) * p.sl2);
          l = fmaf(e, ml[i].y, l);
          x = fmaf(e, v[i].x, x);
          y = fmaf(e, v[i].y, y);
        }
        top = m;
      }
    }
    if (shared_row) {
      s_part[grp][d] = x;
      s_part[grp][d + 1] = y;
      if (d == 0) {
        s_part[grp][D] = top;
        s_part[grp][D + 1] = l;
      }
      __syncthreads();
      if (grp == 0) {
        float m = top;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) m = fmaxf(m, s_part[g][D]);
        const float ref = m == -INFINITY ? 0.f : m, f = ex2_approx((top - ref) * p.sl2);
        l *= f; x *= f; y *= f;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) {
          const float e = ex2_approx((s_part[g][D] - ref) * p.sl2);
          l = fmaf(e, s_part[g][D + 1], l);
          x = fmaf(e, s_part[g][d], x);
          y = fmaf(e, s_part[g][d + 1], y);
        }
      }
      __syncthreads();
    }
    if (row < row_end && (!shared_row || grp == 0)) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int m = a.first + row;
      __nv_bfloat16* out = p.O + ((long long)a.q0 + m / p.share) * p.ldo + ((long long)h * p.share + m % p.share) * D + d;
      *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(x * inv, y * inv);
    }
  }
}

// The list of blocks' work, by one block, up to KL_MAX requests.  Tiles come in the order of their key
// units, most first (a counting sort; the order of equal ones does not matter to any result): a request's
// blocks take as long as its keys are many, and started last they would leave most of the GPU idle.
// Where tiles are few, their keys are split so that each block gets about 1.1 times the mean of a
// block per slot, but no less than min_units.
// One block's straight run through code that nothing has run before it is mostly instruction fetches, so
// the code is short: loops are not unrolled, and a request is read again (from L1) in each of the passes.
constexpr int KL_THREADS = 512, KL_MAX = 8192, KL_OWN = 8;
struct KaListParams {
  int T, unit_log2, split, slots, min_units, weight_shift;
};
struct KlReq {
  int q0, n_r, len, tiles, units;
};
__device__ __forceinline__ KlReq kl_request(const KaParams& p, const KaListParams& l, int r, bool tell) {
  KlReq q = {0, 0, 0, 0, 0};
  const int a = p.offsets[r], b = p.offsets[r + 1], len = p.kv_len[r];
  if (a < 0 || b < a || b > p.rows) {
    if (tell) set_status(p.status, ROCS_ERR_INDEX);
  } else if (len < 0 || len > ((long long)p.max_blocks << p.P_log2)) {
    if (tell) set_status(p.status, ROCS_ERR_COUNTS);
  } else {
    q.q0 = a;
    q.n_r = b - a;
    q.len = len;
    q.tiles = (q.n_r * p.share + l.T - 1) / l.T;
    q.units = (len + (1 << l.unit_log2) - 1) >> l.unit_log2;
  }
  return q;
}

// The warps' sums first: 64-bit additions to one shared word by every thread took 8 us of a call.
__device__ __forceinline__ void kl_add(unsigned long long* to, unsigned long long x, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0 && x > 0) atomicAdd(to, x);
}

__global__ void __launch_bounds__(KL_THREADS) ka_list_kernel(const KaParams p, const KaListParams l) {
  __shared__ unsigned s_at[KL_THREADS], s_warp[KL_THREADS / 32];
  __shared__ unsigned long long s_units, s_rows;
  __shared__ int s_joins, s_parts;
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31;
  s_at[tid] = 0;
  if (tid == 0) {
    s_units = s_rows = 0;
    s_joins = s_parts = 0;
  }
  __syncthreads();
  int most = 1 << 30;
  if (l.split) {
    unsigned long long sum = 0;
#pragma unroll 1
    for (int r = tid; r < p.B_R; r += KL_THREADS) {
      const KlReq q = kl_request(p, l, r, false);
      sum += (unsigned long long)q.tiles * q.units * p.groups;
    }
    kl_add(&s_units, sum, lane);
    __syncthreads();
    const unsigned mean = (unsigned)(s_units / (unsigned)l.slots);      // (far below 2^32: see ka_plan)
    most = max(l.min_units, (int)(mean + mean / 10 + 1));
  }
  // the bucket of a request's blocks, by their key units, most first
  auto bucket = [&](int units, int splits) {
    return KL_THREADS - 1 - min((units + splits - 1) / splits >> l.weight_shift, KL_THREADS - 1);
  };
  unsigned long long rows = 0;
#pragma unroll 1
  for (int r = tid; r < p.B_R; r += KL_THREADS) {
    const KlReq q = kl_request(p, l, r, true);
    const int splits = q.units > most ? (q.units + most - 1) / most : 1;
    rows += q.n_r;
    if (q.tiles > 0) atomicAdd(&s_at[bucket(q.units, splits)], (unsigned)(q.tiles * splits));
  }
  kl_add(&s_rows, rows, lane);
  __syncthreads();
  // Offsets that go back and forth give requests more rows than there are, and the list more entries than
  // it has room for: nothing is done then (the status says so already).
  if (s_rows > (unsigned long long)p.rows) {
    if (tid == 0) p.counts[0] = p.counts[1] = 0;
    return;
  }
  // exclusive running total over the buckets
  const unsigned v = s_at[tid];
  unsigned incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_warp[tid >> 5] = incl;
  __syncthreads();
  unsigned before = 0;
#pragma unroll 1
  for (int w = 0; w < (tid >> 5); ++w) before += s_warp[w];
  s_at[tid] = before + incl - v;
  if (tid == KL_THREADS - 1) p.counts[0] = (int)(before + incl);
  __syncthreads();
#pragma unroll 1
  for (int r0 = tid - lane; r0 < p.B_R; r0 += KL_THREADS) {
    const int r = r0 + lane;
    KlReq q = {0, 0, 0, 0, 0};
    if (r < p.B_R) q = kl_request(p, l, r, false);
    const int splits = q.units > most ? (q.units + most - 1) / most : 1, n = q.tiles * splits;
    unsigned at = 0;
    int part = 0, join = 0;
    if (n > 0) {
      at = atomicAdd(&s_at[bucket(q.units, splits)], (unsigned)n);
      if (splits > 1) {
        part = atomicAdd(&s_parts, n);
        join = atomicAdd(&s_joins, q.tiles);
      }
    }
    // a request's entries by its own thread, or by the warp where they are many
    const uint32_t many = __ballot_sync(0xffffffffu, n > KL_OWN);
    const int turns = 1 + __popc(many);
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn) {
      const int w = turn == 0 ? lane : (int)__fns(many, 0, turn);
      KlReq x;
      x.q0 = __shfl_sync(0xffffffffu, q.q0, w);
      x.n_r = __shfl_sync(0xffffffffu, q.n_r, w);
      x.len = __shfl_sync(0xffffffffu, q.len, w);
      const int sp = __shfl_sync(0xffffffffu, splits, w), xn = __shfl_sync(0xffffffffu, n, w);
      const int xp = __shfl_sync(0xffffffffu, part, w), xj = __shfl_sync(0xffffffffu, join, w);
      const unsigned xa = __shfl_sync(0xffffffffu, at, w);
      const int end = turn == 0 && xn > KL_OWN ? 0 : xn, step = turn == 0 ? 1 : 32;
#pragma unroll 1
      for (int i = turn == 0 ? 0 : lane; i < end; i += step) {
        const int t = i / sp, s = i - t * sp, first = t * l.T;
        const int last = min(first + l.T, x.n_r * p.share) - 1;
        const int seen = p.causal ? max(0, x.len - x.n_r + last / p.share + 1) : x.len;
        const int chunks = (seen + (1 << l.unit_log2) - 1) >> l.unit_log2, each = chunks / sp, more = chunks - each * sp;
        int4* to = reinterpret_cast<int4*>(&p.items[xa + i]);
        const int c_lo = each * s + min(s, more);
        to[0] = make_int4(r0 + w, first, x.n_r, x.len);
        to[1] = make_int4(x.q0, c_lo, c_lo + each + (s < more ? 1 : 0), sp > 1 ? xp + i : -1);
        if (sp > 1 && s == 0) p.joins[xj + t] = KaJoin{first, x.n_r, x.q0, xp + i, sp, {0, 0, 0}};
      }
    }
  }
  __syncthreads();
  if (tid == 0) p.counts[1] = s_joins;
}

// How a call is laid out: rows per tile, upper bounds of its tiles and blocks, whether the work is listed
// and the keys may be split.
struct KaPlan {
  int NT = 1, T = 8;                // NT = 0: the tcgen05 kernel
  int per_item = KA_WARPS;          // warps a (tile, head)
  int groups = 1;                   // blocks a tile
  bool list = false, split = false;
  int slots = 0;                    // blocks that the GPU holds at once
  long long tiles = 0;              // without a list; with one, the list's length at most
  long long joins = 0, parts = 0;
  size_t items_at = 0, joins_at = 0, part_at = 0, ml_at = 0, bytes = 0;
};

KaPlan ka_plan(const rocs_context* ctx, const rocs_kv4_desc& d, int H_q, int B_R, long long rows, int max_blocks) {
  KaPlan k;
  if (rows == 0) return k;
  const int share = H_q / d.H_kv;
  const long long packed = rows * share;
  // as many packed rows per tile as a request has on average (all that the host knows): right for requests that
  // are alike.  480 single rows with 32 bursts of 500 take 167 us in one call and 82 in two.
  const double avg = (double)packed / B_R;
  k.NT = avg <= 8 ? 1 : avg <= 16 ? 2 : avg <= kTcRows ? (d.d_h == 128 ? 2 : 4) : 0;
  k.T = k.NT > 0 ? 8 * k.NT : 128;
  // about as many tiles as will have rows: a request's rows begin a tile of their own
  const long long full = packed / k.T, own = rows < B_R ? rows : B_R;
  const long long busy = full > own ? full : own;
  const long long items = (busy < 1 ? 1 : busy) * d.H_kv;
  // one warp an item where items fill the GPU's warps (16 an SM) more than once, two where they nearly do:
  // 41 instead of 57 us on 4096 items of 500 keys (d = 32), 42 instead of 46 us on 1200 with four warps (d = 64)
  if (k.NT > 0) k.per_item = items >= 24LL * ctx->num_sms ? 1 : items >= 12LL * ctx->num_sms ? 2 : 4;
  const int heads = k.NT > 0 ? KA_WARPS / k.per_item : 1;
  k.groups = (d.H_kv + heads - 1) / heads;
  const int an_sm = k.NT == 0 ? (d.d_h == 32 ? 3 : 2) : k.NT > 1 ? 2 : d.d_h == 32 ? 5 : d.d_h == 64 ? 4 : 3;
  k.slots = an_sm * ctx->num_sms;
  const long long blocks = (busy < 1 ? 1 : busy) * k.groups;
  const long long longest = (long long)max_blocks * d.page_size;
  k.split = blocks <= k.slots / 2 && longest >= (k.NT > 0 ? 2048 : 1024) && B_R <= KL_MAX;
  // the list costs a launch of its own (3 us): where blocks outnumber the slots, for its order; where they
  // are few, for the splits; and always in front of the tcgen05 kernel, whose set-up hides it
  k.list = B_R <= KL_MAX && (k.split || k.NT == 0 || blocks > k.slots);
  k.tiles = packed / k.T + B_R;
  if (k.list) {
    if (k.tiles > packed) k.tiles = packed;
    // With u units in all and m = 1.1 u / slots a block, a tile of x units becomes ceil(x / m) <= 1 + x / m
    // blocks, and one with x > m at most 2 x / m.  (Splits are for at most 2 * busy tiles, so u is below
    // slots * 2^27.)
    k.joins = k.split ? k.tiles : 0;
    k.parts = k.split ? 2LL * k.slots / k.groups + 2 : 0;
    if (k.split) k.tiles += k.slots / k.groups + 1;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    k.items_at = 256;
    k.joins_at = up(k.items_at + (size_t)k.tiles * sizeof(KaItem));
    k.part_at = up(k.joins_at + (size_t)k.joins * sizeof(KaJoin));
    k.ml_at = up(k.part_at + (size_t)k.parts * d.H_kv * k.T * d.d_h * 4);
    k.bytes = k.ml_at + (size_t)k.parts * d.H_kv * k.T * 8;
  }
  return k;
}

rocs_status ka_list(const KaParams& p, const KaPlan& k, int unit_log2, cudaStream_t s) {
  KaListParams l;
  l.T = k.T;
  l.unit_log2 = unit_log2;
  l.split = k.split ? 1 : 0;
  l.slots = k.slots;
  l.min_units = (k.NT > 0 ? 1024 : 512) >> unit_log2;
  l.weight_shift = 0;
  while ((((long long)p.max_blocks << p.P_log2) >> unit_log2 >> l.weight_shift) >= KL_THREADS) ++l.weight_shift;
  LaunchTimer lt_("attn_kv4_list", s);
  ka_list_kernel<<<1, KL_THREADS, 0, s>>>(p, l);
  return cuda_check(cudaGetLastError(), "ka_list_kernel");
}

template <int D, int T>
rocs_status ka_join(const KaParams& p, const KaPlan& k, cudaStream_t s) {
  LaunchTimer lt_("attn_kv4_join", s);
  // a block takes one row, or 16 of a 128-row tile
  const int rows = T < 128 ? 1 : 16;
  return launch_dependent(attn_kv4_join_kernel<D, T>, dim3((unsigned)k.joins, p.Hkv, T / rows), dim3(128), 0, s, "attn_kv4_join_kernel",
                          p, rows);
}

template <int D, int NT, bool BIG>
rocs_status ka_launch(rocs_context* ctx, const KaParams& p, const KaPlan& k, cudaStream_t s) {
  using C = KaCfg<D>;
  static_assert(C::SMEM >= KA_WARPS * 8 * NT * D * 4, "the join's outputs fit the ring");
  static bool attr[64] = {false};
  if (C::SMEM > 48 * 1024 && (ctx->device >= 64 || !attr[ctx->device])) {
    rocs_status st = cuda_check(cudaFuncSetAttribute(attn_kv4_kernel<D, NT, BIG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     C::SMEM), "cudaFuncSetAttribute(attn_kv4)");
    if (st != ROCS_OK) return st;
    if (ctx->device < 64) attr[ctx->device] = true;
  }
  rocs_status st;
  {
    LaunchTimer lt_("attn_kv4", s);
    const dim3 grid((unsigned)(k.tiles * k.groups)), block(KA_WARPS * 32);
    if (k.list) {
      st = launch_dependent(attn_kv4_kernel<D, NT, BIG>, grid, block, C::SMEM, s, "attn_kv4_kernel", p);
    } else {
      attn_kv4_kernel<D, NT, BIG><<<grid, block, C::SMEM, s>>>(p);
      st = cuda_check(cudaGetLastError(), "attn_kv4_kernel");
    }
  }
  return st != ROCS_OK || !k.split ? st : ka_join<D, 8 * NT>(p, k, s);
}

template <int D, int NT>
rocs_status ka_launch(rocs_context* ctx, const KaParams& p, const KaPlan& k, cudaStream_t s) {
  return p.P_log2 >= 6 ? ka_launch<D, NT, true>(ctx, p, k, s) : ka_launch<D, NT, false>(ctx, p, k, s);
}

template <int D>
rocs_status ka_dispatch(rocs_context* ctx, const KaParams& p, const KaPlan& k, cudaStream_t s) {
  if (k.list) {
    rocs_status st = ka_list(p, k, k.NT == 0 ? 6 : KaCfg<D>::KEYS_LOG2, s);
    if (st != ROCS_OK) return st;
  }
  if (k.NT == 0) {
    rocs_status st = launch_attn_kv4_tc(ctx, D, p, k.tiles * k.groups, s);
    if (st != ROCS_OK || !k.split) return st;
    return ka_join<D, 128>(p, k, s);
  }
  if (k.NT == 1) return ka_launch<D, 1>(ctx, p, k, s);
  if (k.NT == 2) return ka_launch<D, 2>(ctx, p, k, s);
  if constexpr (D < 128) return ka_launch<D, 4>(ctx, p, k, s);
  return ROCS_ERR_UNSUPPORTED;
}

}  // namespace

size_t attn_kv4_scratch(const rocs_context* ctx, const rocs_kv4_desc& d, int H_q, int B_R, long long rows, int max_blocks) {
  return ka_plan(ctx, d, H_q, B_R, rows, max_blocks).bytes;
}

rocs_status launch_attn_kv4(rocs_context* ctx, const rocs_kv4_desc& d, const void* Q, long long ldq, int H_q,
                            const void* cache, const int32_t* table, int max_blocks, const int32_t* kv_len,
                            const int32_t* offsets, int B_R, long long rows, float scale, int causal, void* O,
                            long long ldo, void* scratch, cudaStream_t s) {
  if (rows == 0) return ROCS_OK;
  const KaPlan k = ka_plan(ctx, d, H_q, B_R, rows, max_blocks);
  KaParams p;
  p.Q = (const __nv_bfloat16*)Q;
  p.ldq = ldq;
  p.cache = (const uint8_t*)cache;
  p.table = table;
  p.max_blocks = max_blocks;
  p.kv_len = kv_len;
  p.offsets = offsets;
  p.B_R = B_R;
  p.rows = rows;
  p.Hkv = d.H_kv;
  p.share = H_q / d.H_kv;
  p.P_log2 = 31 - __builtin_clz((unsigned)d.page_size);
  p.n_pages = d.n_pages;
  // a negative scale turns the queries round, so that the largest product is the largest score
  p.sl2 = fmaxf(fabsf(scale) * 1.4426950408889634f, FLT_TRUE_MIN);
  p.lazy = fminf(kKaLazyLog2 / p.sl2, FLT_MAX);
  p.q_flip = scale < 0.f ? 0x80008000u : 0u;
  p.causal = causal;
  p.O = (__nv_bfloat16*)O;
  p.ldo = ldo;
  p.per_item = k.per_item;
  p.groups = k.groups;
  char* ws = (char*)scratch;
  p.counts = k.list ? (int*)ws : nullptr;
  p.items = k.list ? (KaItem*)(ws + k.items_at) : nullptr;
  p.joins = k.list ? (KaJoin*)(ws + k.joins_at) : nullptr;
  p.part = k.list ? (float*)(ws + k.part_at) : nullptr;
  p.part_ml = k.list ? (float2*)(ws + k.ml_at) : nullptr;
  p.status = ctx->d_status;
  switch (d.d_h) {
    case 32: return ka_dispatch<32>(ctx, p, k, s);
    case 64: return ka_dispatch<64>(ctx, p, k, s);
    default: return ka_dispatch<128>(ctx, p, k, s);
  }
}

}  // namespace rocs
