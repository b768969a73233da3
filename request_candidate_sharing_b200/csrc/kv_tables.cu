// Block tables and slot maps of the paged history cache, from request lengths.
//
// Request r has past_r tokens in the cache and new_r to come.  With P tokens a page it holds
// ceil(past_r / P) pages and needs ceil((past_r + new_r) / P); the difference is taken from the free
// list in request order, so two exclusive running totals place everything: of new_r (the request's
// first row) and of the pages taken (its first free-list entry).  Row off_r + j is token past_r + j;
// its page is either fresh (a free-list entry, known from the totals) or the partly filled page the
// table already names, so rows and table entries can be written in the same launch.
//
// Up to kTabInline requests every block computes both totals by itself in shared memory (two reads of
// 4 B a request from L2, one block-wide scan): one launch instead of three, and the decode step (512
// requests, 512 rows) is all launch latency.  Beyond, a block per kTabInline requests totals its
// part, a second launch scans and writes the totals, a third expands.  Expansion is by output row,
// four neighbouring rows a thread (16-byte stores), each thread finding its first row's request by
// binary search and walking on; so one request with a million rows spreads over the whole GPU.
// Bound by the 12 bytes written per row.
#include "common.cuh"
#include "internal.h"

namespace rocs {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabItems = 8;                              // requests per thread of a scan
constexpr int kTabInline = kTabThreads * kTabItems;       // 4096

struct TabParams {
  const int32_t *past, *fresh_len;   // past may be null: nothing is cached
  int B_R;
  int P_log2;
  const int32_t* free_pages;
  int n_free, n_pages;
  int32_t* table;
  int max_blocks;
  int32_t *kv_len, *row_off;
  int64_t* slots;
  int32_t* positions;
  long long rows;
  int32_t* pages_used;
  long long* part;        // [2 * chunks]: rows and pages of each chunk of kTabInline requests
  long long* page_off;    // [B_R + 1]
  int* status;
};

struct TabReq {
  int past, rows, need, before;   // tokens cached, rows owned, pages wanted, pages held
  bool bad;
};

// A request whose lengths are not usable (negative, or longer than its table) owns its rows all the
// same, so that the others keep their places, but takes no page.
__device__ __forceinline__ TabReq tab_request(const TabParams& p, int r) {
  TabReq q;
  const int past = p.past != nullptr ? p.past[r] : 0, fresh = p.fresh_len[r];
  const long long total = (long long)past + fresh;
  const long long room = (long long)p.max_blocks << p.P_log2;
  q.bad = past < 0 || fresh < 0 || total > room;
  q.rows = fresh > 0 ? fresh : 0;
  q.past = past < 0 || past > room ? 0 : past;
  const int mask = (1 << p.P_log2) - 1;
  q.before = (int)(((long long)q.past + mask) >> p.P_log2);
  q.need = q.bad ? 0 : (int)((total + mask) >> p.P_log2) - q.before;
  return q;
}

// Exclusive running totals of (a, b) over the block's threads; the block's totals in *ta, *tb.
__device__ __forceinline__ void tab_scan(long long& a, long long& b, long long* ta, long long* tb) {
  __shared__ long long wa[kTabThreads / 32], wb[kTabThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) { ia += xa; ib += xb; }
  }
  if (lane == 31) { wa[warp] = ia; wb[warp] = ib; }
  __syncthreads();
  long long pa = 0, pb = 0, sa = 0, sb = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w == warp) { pa = sa; pb = sb; }
    sa += wa[w];
    sb += wb[w];
  }
  *ta = sa;
  *tb = sb;
  a = pa + ia - a;
  b = pb + ib - b;
  __syncthreads();
}

__device__ __forceinline__ int32_t clip32(long long v) { return (int32_t)(v < 2147483647LL ? v : 2147483647LL); }

// Largest r in [lo, hi) with off[r] <= i (off nondecreasing, off[lo] <= i): the owner of row or page
// i once empty owners in front of it are passed over.
template <typename T>
__device__ __forceinline__ int tab_owner(const T* off, int lo, int hi, long long i) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Rows [4 i, 4 i + 4) and free-list entries of this block, given the running totals of requests
// [0, B_R): row(r) and page(r) (with their ends at r = B_R).
template <typename RowT, typename PageT>
__device__ __forceinline__ void tab_expand(const TabParams& p, const RowT* row_off, const PageT* page_off,
                                           long long n_rows, long long n_fresh) {
  const int mask = (1 << p.P_log2) - 1;
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  // fresh pages into the table
  const long long usable = n_fresh < p.n_free ? n_fresh : (long long)p.n_free;
  for (long long i = first; i < usable; i += stride) {
    const int r = tab_owner(page_off, 0, p.B_R, i);
    if ((long long)page_off[r + 1] > p.n_free) continue;   // the free list ran out inside this request
    const TabReq q = tab_request(p, r);
    const int page = p.free_pages[i];
    if (page < 0 || page >= p.n_pages) {
      set_status(p.status, ROCS_ERR_INDEX);
      continue;
    }
    p.table[(long long)r * p.max_blocks + q.before + (int)(i - (long long)page_off[r])] = page;
  }
  // rows
  for (long long i0 = 4 * first; i0 < p.rows; i0 += 4 * stride) {
    int64_t sl[4];
    int32_t po[4];
    int r = -1;
    TabReq q;
    long long row0 = 0, row1 = 0, page0 = 0;
    bool dead = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long i = i0 + e;
      sl[e] = -1;
      po[e] = -1;
      if (i >= p.rows || i >= n_rows) continue;   // a padded batch's rows have no slot
      if (r < 0 || i >= row1) {
        r = tab_owner(row_off, r < 0 ? 0 : r, p.B_R, i);
        q = tab_request(p, r);
        row0 = row_off[r];
        row1 = row_off[r + 1];
        page0 = page_off[r];
        dead = q.bad || (q.need > 0 && page0 + q.need > p.n_free);
      }
      if (dead) continue;
      const int pos = q.past + (int)(i - row0);
      const int blk = pos >> p.P_log2;
      const int page = blk < q.before ? p.table[(long long)r * p.max_blocks + blk] : p.free_pages[page0 + blk - q.before];
      if (page < 0 || page >= p.n_pages) {
        set_status(p.status, ROCS_ERR_INDEX);
        continue;
      }
      sl[e] = ((int64_t)page << p.P_log2) + (pos & mask);
      po[e] = pos;
    }
    if (i0 + 4 <= p.rows) {
      *reinterpret_cast<longlong2*>(p.slots + i0) = make_longlong2(sl[0], sl[1]);
      *reinterpret_cast<longlong2*>(p.slots + i0 + 2) = make_longlong2(sl[2], sl[3]);
      *reinterpret_cast<int4*>(p.positions + i0) = make_int4(po[0], po[1], po[2], po[3]);
    } else {
      for (int e = 0; e < 4 && i0 + e < p.rows; ++e) {
        p.slots[i0 + e] = sl[e];
        p.positions[i0 + e] = po[e];
      }
    }
  }
}

// What the owner of request r writes once its totals are known; returns the end of its pages if it
// got all it wanted.
__device__ __forceinline__ long long tab_owner_writes(const TabParams& p, int r, const TabReq& q, long long row,
                                                      long long page) {
  const bool starved = q.need > 0 && page + q.need > p.n_free;
  p.row_off[r] = clip32(row);
  p.kv_len[r] = q.bad || starved ? q.past : q.past + q.rows;
  if (q.bad || starved) set_status(p.status, ROCS_ERR_COUNTS);
  return starved || q.need == 0 ? 0 : page + q.need;
}

// A thread's kTabItems consecutive requests of chunk `base`: their sums.
__device__ __forceinline__ void tab_items(const TabParams& p, int base, long long& a, long long& b) {
  a = b = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = base + threadIdx.x * kTabItems + k;
    if (r < p.B_R) {
      const TabReq q = tab_request(p, r);
      a += q.rows;
      b += q.need;
    }
  }
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_inline_kernel(const TabParams p) {
  __shared__ int32_t s_row[kTabInline + 1];
  __shared__ int32_t s_page[kTabInline + 1];
  __shared__ int s_used;
  if (threadIdx.x == 0) s_used = 0;
  long long a, b, ta, tb;
  tab_items(p, 0, a, b);
  tab_scan(a, b, &ta, &tb);
  const bool writer = blockIdx.x == 0;
  long long used = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = threadIdx.x * kTabItems + k;
    if (r < p.B_R) {
      const TabReq q = tab_request(p, r);
      // totals past 2^31 are clipped: such rows and pages lie behind every output
      s_row[r] = clip32(a);
      s_page[r] = clip32(b);
      if (writer) {
        const long long end = tab_owner_writes(p, r, q, a, b);
        used = end > used ? end : used;
      }
      a += q.rows;
      b += q.need;
    }
  }
  if (threadIdx.x == 0) {
    s_row[p.B_R] = clip32(ta);
    s_page[p.B_R] = clip32(tb);
  }
  if (writer) {
    if (used > 0) atomicMax(&s_used, (int)used);   // at most n_free
    if (threadIdx.x == 0) {
      p.row_off[p.B_R] = clip32(ta);
      if (ta > p.rows) set_status(p.status, ROCS_ERR_COUNTS);
    }
  }
  __syncthreads();
  if (writer && threadIdx.x == 0) *p.pages_used = s_used;
  tab_expand(p, s_row, s_page, ta, tb);
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_sum_kernel(const TabParams p) {
  long long a, b, ta, tb;
  tab_items(p, blockIdx.x * kTabInline, a, b);
  tab_scan(a, b, &ta, &tb);
  if (threadIdx.x == 0) {
    p.part[2 * blockIdx.x] = ta;
    p.part[2 * blockIdx.x + 1] = tb;
    if (blockIdx.x == 0) *p.pages_used = 0;
  }
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_scan_kernel(const TabParams p) {
  __shared__ int s_used;
  if (threadIdx.x == 0) s_used = 0;
  // the chunks in front of this one
  long long fa = 0, fb = 0, xa, xb;
  for (int c = threadIdx.x; c < (int)blockIdx.x; c += kTabThreads) {
    fa += p.part[2 * c];
    fb += p.part[2 * c + 1];
  }
  tab_scan(fa, fb, &xa, &xb);
  long long a, b, ta, tb;
  tab_items(p, blockIdx.x * kTabInline, a, b);
  tab_scan(a, b, &ta, &tb);
  a += xa;
  b += xb;
  long long used = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = blockIdx.x * kTabInline + threadIdx.x * kTabItems + k;
    if (r < p.B_R) {
      const TabReq q = tab_request(p, r);
      p.page_off[r] = b;
      const long long end = tab_owner_writes(p, r, q, a, b);
      used = end > used ? end : used;
      a += q.rows;
      b += q.need;
      if (r == p.B_R - 1) {
        p.row_off[p.B_R] = clip32(a);
        p.page_off[p.B_R] = b;
        if (a > p.rows) set_status(p.status, ROCS_ERR_COUNTS);
      }
    }
  }
  if (used > 0) atomicMax(&s_used, (int)used);
  __syncthreads();
  if (threadIdx.x == 0 && s_used > 0) atomicMax(p.pages_used, s_used);   // a maximum: any order
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_expand_kernel(const TabParams p) {
  tab_expand(p, p.row_off, p.page_off, (long long)p.row_off[p.B_R], p.page_off[p.B_R]);
}

int tab_chunks(int B_R) { return (B_R + kTabInline - 1) / kTabInline; }

}  // namespace

size_t kv_tables_scratch(int B_R) {
  if (B_R <= kTabInline) return 0;
  return ((size_t)2 * tab_chunks(B_R) + (size_t)B_R + 1) * sizeof(long long);
}

rocs_status launch_kv_tables(rocs_context* ctx, const int32_t* past, const int32_t* fresh_len, int B_R, int page_log2,
                             const int32_t* free_pages, int n_free, int n_pages, int32_t* table, int max_blocks,
                             int32_t* kv_len, int32_t* row_off, int64_t* slots, int32_t* positions, long long rows,
                             int32_t* pages_used, void* scratch, cudaStream_t s) {
  TabParams p;
  p.past = past;
  p.fresh_len = fresh_len;
  p.B_R = B_R;
  p.P_log2 = page_log2;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.n_pages = n_pages;
  p.table = table;
  p.max_blocks = max_blocks;
  p.kv_len = kv_len;
  p.row_off = row_off;
  p.slots = slots;
  p.positions = positions;
  p.rows = rows;
  p.pages_used = pages_used;
  p.part = (long long*)scratch;
  p.page_off = p.part + 2 * tab_chunks(B_R);
  p.status = ctx->d_status;
  const long long blocks = (rows + 4LL * kTabThreads - 1) / (4LL * kTabThreads);
  const long long cap = 4LL * ctx->num_sms;
  const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
  if (B_R <= kTabInline) {
    LaunchTimer lt_("kv_tables", s);
    kv_tables_inline_kernel<<<grid, kTabThreads, 0, s>>>(p);
    return cuda_check(cudaGetLastError(), "kv_tables_inline_kernel");
  }
  {
    LaunchTimer lt_("kv_tables_sum", s);
    kv_tables_sum_kernel<<<tab_chunks(B_R), kTabThreads, 0, s>>>(p);
  }
  {
    LaunchTimer lt_("kv_tables_scan", s);
    kv_tables_scan_kernel<<<tab_chunks(B_R), kTabThreads, 0, s>>>(p);
  }
  LaunchTimer lt_("kv_tables_expand", s);
  kv_tables_expand_kernel<<<grid, kTabThreads, 0, s>>>(p);
  return cuda_check(cudaGetLastError(), "kv_tables_expand_kernel");
}

}  // namespace rocs
