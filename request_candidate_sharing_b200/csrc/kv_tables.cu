// Block tables and slot maps of the paged history cache, from request lengths.
//
// Request r has past_r tokens in the cache and new_r to come.  With P tokens a page it holds
// ceil(past_r / P) pages and needs ceil((past_r + new_r) / P); the difference is taken from the free
// list in request order, so two exclusive running totals place everything: of new_r (the request's
// first row) and of the pages taken (its first free-list entry).  Row off_r + j is token past_r + j;
// its page is either fresh (a free-list entry, known from the totals) or the partly filled page the
// table already names, so rows and table entries can be written in the same launch.
// Where the free list is too short for all, a request that does not fit takes nothing and those behind it
// go on from the same entry: then the total of the pages follows from the decisions before it, and is taken
// request by request (tab_place), which only such calls pay for.
//
// Up to kTabInline requests every block computes both totals by itself in shared memory (two reads of
// 4 B a request from L2, one block-wide scan): one launch instead of three.  A decode step (512 requests,
// 512 rows) is all latency: with at most four rows a request on average one block does it all without a
// search, 3.7 us, where the form below takes 9.7 us.
// Beyond, a block per kTabThreads requests totals its part, a second launch scans and writes the totals,
// a third expands.  Expansion is by output row, so that one request with a million rows spreads over the
// whole GPU.  A block takes a tile of neighbouring rows, finds its first request by two block-wide probes,
// and brings the requests from there on, the pages that their cached tokens end in and the free list's
// entries of the tile into shared memory, so that nothing waits for memory once rows are written.  A warp
// goes through its rows request by request; where requests have under 16 rows on average each lane finds
// its first row's request by binary search and walks on.  For 7.2 M rows of 40000 requests 32 us (5 of
// them the sums, 3 a tile's start): 13.8 us' worth of bytes.  Page numbers read from L2 as they were needed:
// 40 us; lanes on their own everywhere: 44 us; a search per row in L2: 90 us; four neighbouring rows a lane
// with wide stores, which diverge in every warp: 64 us.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace rocs {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabItems = 4;                              // requests per thread of a scan
constexpr int kTabInline = kTabThreads * kTabItems;       // 2048
constexpr int kTabFree = 2048;                            // entries of the free list that a tile has at hand
constexpr int kTabRows = 4;                               // rows a thread of a tile, scanned by every block

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
  long long* part;        // [2 * chunks]: rows and pages of each chunk of kTabThreads requests
  long long* page_off;    // [B_R]; n_free where a request's pages are not there
  int tile_rows;          // rows a thread of a tile, otherwise
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

// Pages for 32 requests in order, one a lane, by one warp, where the free list may run out: returns the first
// entry that the lane's request takes, or n_free where what is left is too little for it.  `taken`: entries
// taken so far.  A turn accepts all up to the first that does not fit, and drops for good those that want
// more than is left (needs are below 2^27, so 32 of them add up below 2^32).
__device__ __forceinline__ int tab_place(unsigned need, unsigned& taken, unsigned n_free) {
  const int lane = threadIdx.x & 31;
  int mine = (int)n_free;
  uint32_t open = 0xffffffffu;
  while (true) {
    const unsigned left = n_free - taken;
    open &= __ballot_sync(0xffffffffu, need <= left);
    const unsigned x = (open >> lane) & 1u ? need : 0;
    unsigned incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, incl > left) & open;
    const uint32_t now = over != 0 ? open & ((over & (0u - over)) - 1) : open;   // those in front of the first that does not fit
    if ((now >> lane) & 1u) mine = (int)(taken + incl - x);
    if (over == 0) {
      taken += __shfl_sync(0xffffffffu, incl, 31);
      return mine;
    }
    const int first = __ffs((int)over) - 1;
    taken += __shfl_sync(0xffffffffu, incl - x, first);
    open = first == 31 ? 0 : open & (0xffffffffu << (first + 1));
  }
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

// Requests [first, first + n) in shared memory: running totals of rows and pages (one more of the rows,
// the end), and the tokens each holds (-1: it gets no slots).
struct TabWindow {
  const int32_t *row, *page, *past;
  int first, n;
  // where rows are taken request by request: the page that each one's cached tokens end in, and the free
  // list's entries [free0, free0 + n_free)
  const int32_t *open, *free_pages;
  int free0, n_free;
};

// Where a request's rows go on for a while: the warp takes its request's rows [i0, i1) together.  Only the page
// that the cached tokens end in is not a fresh one.
__device__ __forceinline__ void tab_run(const TabParams& p, const TabWindow& w, int r, int i0, int i1) {
  constexpr int BATCH = 2;
  const int lane = threadIdx.x & 31, past = w.past[r], to_pos = past - w.row[r], log2 = p.P_log2, mask = (1 << log2) - 1;
  int64_t* slots = p.slots + i0 + lane;
  int32_t* positions = p.positions + i0 + lane;
  int left = i1 - i0 - lane;             // rows of this lane and those behind it
  if (past < 0) {
    for (; left > 0; left -= 32, slots += 32, positions += 32) {
      *slots = -1;
      *positions = -1;
    }
    return;
  }
  const int before = (int)(((unsigned)past + mask) >> log2), pos0 = i0 + to_pos;
  const unsigned n_pages = (unsigned)p.n_pages;
  const int last = (i1 - 1 + to_pos) >> log2, to_free = w.page[r] - before;
  // the free list's part that the tile's rows need is at hand, unless it is an uncommonly long one
  const int first_free = to_free + max(before, pos0 >> log2) - w.free0, last_free = to_free + last - w.free0;
  const int32_t* fresh = first_free >= 0 && last_free < w.n_free ? w.free_pages + (to_free - w.free0) : p.free_pages + to_free;
  int32_t* entries = p.table + (long long)(w.first + r) * p.max_blocks;
  const int open = w.open[r];
  for (int b = max(before, (pos0 + mask) >> log2) + lane; b <= last; b += 32) {     // the fresh pages that begin here
    const int page = fresh[b];
    if ((unsigned)page < n_pages) entries[b] = page;
  }
  bool bad = false;
  auto batch = [&](auto all, int pos) {
    int page[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      page[k] = open;
      const int blk = (pos + 32 * k) >> log2;
      if ((decltype(all)::value || left > 32 * k) && blk >= before) page[k] = fresh[blk];
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const bool ok = (unsigned)page[k] < n_pages;
      if (decltype(all)::value || left > 32 * k) {
        slots[32 * k] = ok ? ((int64_t)page[k] << log2) + ((pos + 32 * k) & mask) : -1;
        positions[32 * k] = ok ? pos + 32 * k : -1;
        bad = bad || !ok;
      }
    }
  };
  int pos = pos0 + lane;
  int whole = (i1 - i0) / (32 * BATCH);          // batches that every lane has all of
  for (; whole > 0; --whole, left -= 32 * BATCH, pos += 32 * BATCH, slots += 32 * BATCH, positions += 32 * BATCH)
    batch(std::true_type{}, pos);
  batch(std::false_type{}, pos);
  if (bad) set_status(p.status, ROCS_ERR_INDEX);
}

// Rows [base, base + 32 count) by one warp.  Request by request where each has 16 rows or more on average;
// else row base + lane, base + lane + 32, ..: a lane finds its first row's request by binary search and
// walks on from there.
template <bool RUNS>
__device__ __forceinline__ void tab_rows(const TabParams& p, const TabWindow& w, long long base, int count, long long n_rows) {
  const int mask = (1 << p.P_log2) - 1;
  const long long stop = base + 32LL * count;
  if (RUNS && stop <= n_rows && stop <= p.rows && stop <= w.row[w.n]) {
    const int r0 = tab_owner(w.row, 0, w.n, base), r1 = tab_owner(w.row, r0, w.n, stop - 1);
    if (r1 - r0 < 2 * count) {
      for (int r = r0; r <= r1; ++r) tab_run(p, w, r, max(w.row[r], (int)base), min(w.row[r + 1], (int)stop));
      return;
    }
  }
  int r = -1;                       // the row's request, counted from the window's first
  for (int k = 0; k < count; ++k) {
    const long long i = base + (threadIdx.x & 31) + 32 * k;
    if (i >= p.rows) return;
    int64_t slot = -1;
    int pos = -1;
    if (i < n_rows) {               // a padded batch's rows have no slot
      long long row0, page0;
      int past, q = w.n;
      if (i < w.row[w.n]) {
        if (r < 0) r = tab_owner(w.row, 0, w.n, i);
        while (i >= w.row[r + 1]) ++r;
        q = r;
        row0 = w.row[r];
        page0 = w.page[r];
        past = w.past[r];
      } else {                      // past the window: thousands of tiny requests in one tile
        q = tab_owner(p.row_off, w.first + w.n, p.B_R, i) - w.first;
        const TabReq t = tab_request(p, w.first + q);
        row0 = p.row_off[w.first + q];
        page0 = p.page_off[w.first + q];
        past = t.bad || (t.need > 0 && page0 + t.need > p.n_free) ? -1 : t.past;
      }
      if (past >= 0) {
        pos = past + (int)(i - row0);
        const int blk = pos >> p.P_log2, before = (int)(((unsigned)past + mask) >> p.P_log2);
        int32_t* entry = p.table + (long long)(w.first + q) * p.max_blocks + blk;
        const int page = blk >= before ? p.free_pages[page0 + (blk - before)] : *entry;
        if (page >= 0 && page < p.n_pages) {
          if (blk >= before && (pos & mask) == 0) *entry = page;
          slot = ((int64_t)page << p.P_log2) + (pos & mask);
        } else {
          set_status(p.status, ROCS_ERR_INDEX);
          pos = -1;
        }
      }
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
}

// What the owner of request r writes once its first page is known; returns the end of its pages if it
// got all it wanted.
__device__ __forceinline__ long long tab_owner_writes(const TabParams& p, int r, const TabReq& q, long long page) {
  const bool starved = q.need > 0 && page + q.need > p.n_free;
  p.kv_len[r] = q.bad || starved ? q.past : q.past + q.rows;
  if (q.bad || starved) set_status(p.status, ROCS_ERR_COUNTS);
  return starved || q.need == 0 ? 0 : page + q.need;
}

// A thread's `per` (at most kTabItems) consecutive requests from `base` on: their sums.
__device__ __forceinline__ void tab_items(const TabParams& p, int base, int per, TabReq (&q)[kTabItems], long long& a,
                                          long long& b) {
  a = b = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = base + threadIdx.x * per + k;
    if (k < per && r < p.B_R) {
      q[k] = tab_request(p, r);
      a += q[k].rows;
      b += q[k].need;
    }
  }
}

// The same requests' first pages where the free list is too short for all, in s_page.  For the whole block.
__device__ __forceinline__ void tab_place_items(const TabParams& p, int per, const TabReq (&q)[kTabItems], int32_t* s_page) {
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = threadIdx.x * per + k;
    if (k < per && r < p.B_R) s_page[r] = q[k].need;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    unsigned taken = 0;
    for (int r0 = 0; r0 < p.B_R; r0 += 32) {
      const int r = r0 + threadIdx.x;
      const int at = tab_place(r < p.B_R ? s_page[r] : 0, taken, p.n_free);
      if (r < p.B_R) s_page[r] = at;
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_inline_kernel(const TabParams p) {
  __shared__ int32_t s_row[kTabInline + 1], s_page[kTabInline], s_past[kTabInline];
  __shared__ int s_used;
  if (threadIdx.x == 0) s_used = 0;
  const int per = (p.B_R + kTabThreads - 1) / kTabThreads;
  TabReq q[kTabItems];
  long long a, b, ta, tb;
  tab_items(p, 0, per, q, a, b);
  tab_scan(a, b, &ta, &tb);
  const bool writer = blockIdx.x == 0, runs_out = tb > p.n_free;
  if (runs_out) tab_place_items(p, per, q, s_page);
  long long used = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = threadIdx.x * per + k;
    if (k < per && r < p.B_R) {
      // a total past 2^31 is clipped: such rows lie behind every output
      s_row[r] = clip32(a);
      const long long page = runs_out ? s_page[r] : b;
      s_page[r] = (int32_t)page;
      s_past[r] = q[k].bad || (q[k].need > 0 && page + q[k].need > p.n_free) ? -1 : q[k].past;
      if (writer) {
        p.row_off[r] = clip32(a);
        const long long end = tab_owner_writes(p, r, q[k], page);
        used = end > used ? end : used;
      }
      a += q[k].rows;
      b += q[k].need;
    }
  }
  if (threadIdx.x == 0) {
    s_row[p.B_R] = clip32(ta);
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
  const TabWindow w = {s_row, s_page, s_past, 0, p.B_R, nullptr, nullptr, 0, 0};
  const long long tile = (long long)kTabThreads * kTabRows;
  for (long long t0 = blockIdx.x * tile; t0 < p.rows; t0 += gridDim.x * tile)
    tab_rows<false>(p, w, t0 + (threadIdx.x >> 5) * (32 * kTabRows), kTabRows, ta);
}

// Few rows (at most four a request on average): one block, each request's rows written by its own thread,
// or by its warp where it has many, without a search; the page that its tokens already end in is asked for
// before the totals are known.
constexpr int kTabOwnRows = 4;
__global__ void __launch_bounds__(kTabThreads) kv_tables_few_kernel(const TabParams p) {
  __shared__ int32_t s_page[kTabInline];
  __shared__ int s_used;
  if (threadIdx.x == 0) s_used = 0;
  const int per = (p.B_R + kTabThreads - 1) / kTabThreads, mask = (1 << p.P_log2) - 1;
  TabReq q[kTabItems];
  long long a, b, ta, tb;
  tab_items(p, 0, per, q, a, b);
  int32_t open_page[kTabItems];      // the partly filled page, if any
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = threadIdx.x * per + k;
    open_page[k] = -1;
    if (k < per && r < p.B_R && !q[k].bad && q[k].rows > 0 && (q[k].past & mask) != 0)
      open_page[k] = p.table[(long long)r * p.max_blocks + (q[k].past >> p.P_log2)];
  }
  tab_scan(a, b, &ta, &tb);
  const bool runs_out = tb > p.n_free;
  if (runs_out) tab_place_items(p, per, q, s_page);
  // row j of a request whose rows start at `row` and whose fresh pages start at `page0`
  auto put = [&](int r, int past, int before, int open, long long page0, long long row, int j) {
    if (row + j >= p.rows) return;
    const int pos = past + j, blk = pos >> p.P_log2;
    const int page = blk >= before ? p.free_pages[page0 + blk - before] : open;
    const bool ok = page >= 0 && page < p.n_pages;
    if (!ok) set_status(p.status, ROCS_ERR_INDEX);
    if (ok && blk >= before && (pos & mask) == 0) p.table[(long long)r * p.max_blocks + blk] = page;
    p.slots[row + j] = ok ? ((int64_t)page << p.P_log2) + (pos & mask) : -1;
    p.positions[row + j] = ok ? pos : -1;
  };
  long long used = 0;
#pragma unroll
  for (int k = 0; k < kTabItems; ++k) {
    const int r = threadIdx.x * per + k;
    const bool mine = k < per && r < p.B_R;
    bool dead = true;
    int n = 0;
    long long page = b;
    if (mine) {
      if (runs_out) page = s_page[r];
      p.row_off[r] = clip32(a);
      const long long end = tab_owner_writes(p, r, q[k], page);
      used = end > used ? end : used;
      dead = q[k].bad || (q[k].need > 0 && page + q[k].need > p.n_free);
      n = q[k].rows;
      if (n <= kTabOwnRows) {
        for (int j = 0; j < n; ++j) {
          if (!dead) {
            put(r, q[k].past, q[k].before, open_page[k], page, a, j);
          } else if (a + j < p.rows) {
            p.slots[a + j] = -1;
            p.positions[a + j] = -1;
          }
        }
      }
    }
    for (uint32_t many = __ballot_sync(0xffffffffu, n > kTabOwnRows); many != 0; many &= many - 1) {
      const int l = __ffs((int)many) - 1;
      const int wr = __shfl_sync(0xffffffffu, r, l), wn = __shfl_sync(0xffffffffu, n, l);
      const int wpast = __shfl_sync(0xffffffffu, mine ? q[k].past : 0, l), wbefore = __shfl_sync(0xffffffffu, mine ? q[k].before : 0, l);
      const int wopen = __shfl_sync(0xffffffffu, open_page[k], l), wdead = __shfl_sync(0xffffffffu, (int)dead, l);
      const long long wa = __shfl_sync(0xffffffffu, a, l), wb = __shfl_sync(0xffffffffu, page, l);
      for (long long j = threadIdx.x & 31; j < wn && wa + j < p.rows; j += 32) {
        if (!wdead) {
          put(wr, wpast, wbefore, wopen, wb, wa, (int)j);
        } else {
          p.slots[wa + j] = -1;
          p.positions[wa + j] = -1;
        }
      }
    }
    if (mine) {
      a += q[k].rows;
      b += q[k].need;
    }
  }
  // a padded batch's rows have no slot
  for (long long i = ta + threadIdx.x; i < p.rows; i += kTabThreads) {
    p.slots[i] = -1;
    p.positions[i] = -1;
  }
  if (used > 0) atomicMax(&s_used, (int)used);   // at most n_free
  if (threadIdx.x == 0) {
    p.row_off[p.B_R] = clip32(ta);
    if (ta > p.rows) set_status(p.status, ROCS_ERR_COUNTS);
  }
  __syncthreads();
  if (threadIdx.x == 0) *p.pages_used = s_used;
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_sum_kernel(const TabParams p) {
  TabReq q[kTabItems];
  long long a, b, ta, tb;
  tab_items(p, blockIdx.x * kTabThreads, 1, q, a, b);
  tab_scan(a, b, &ta, &tb);
  if (threadIdx.x == 0) {
    p.part[2 * blockIdx.x] = ta;
    p.part[2 * blockIdx.x + 1] = tb;
    if (blockIdx.x == 0) *p.pages_used = 0;
  }
}

// Places the pages of the requests from the first chunk on in which the free list runs out, chunk after chunk,
// and writes for those requests what tab_owner_writes does; returns the entries taken.  For one whole block.
// 5 us a chunk: 40000 requests that all get nothing take 0.37 ms, where 40000 that fit take 26 us.
__device__ __forceinline__ long long tab_place_chunks(const TabParams& p) {
  __shared__ int32_t s_need[kTabThreads], s_at[kTabThreads];
  __shared__ unsigned s_taken;
  const int chunks = gridDim.x;
  long long before = 0;               // pages of the chunks that all fit
  int c = 0;                          // how many chunks those are
  while (c < chunks) {
    long long none = 0, x = c + (int)threadIdx.x < chunks ? p.part[2 * (c + threadIdx.x) + 1] : 0, tn, tx;
    const long long mine = x;
    tab_scan(none, x, &tn, &tx);      // x: the total in front of this thread's chunk
    const int n = __syncthreads_count(c + (int)threadIdx.x < chunks && before + x + mine <= p.n_free);
    if (threadIdx.x == 0) s_taken = 0;
    __syncthreads();
    if (n < kTabThreads) {
      if ((int)threadIdx.x == n) s_taken = (unsigned)(before + x);
      __syncthreads();
      c += n;
      break;
    }
    before += tx;
    c += n;
  }
  unsigned taken = s_taken;
  for (; c < chunks; ++c) {
    const int r = c * kTabThreads + threadIdx.x;
    TabReq q = {0, 0, 0, 0, false};
    if (r < p.B_R) q = tab_request(p, r);
    s_need[threadIdx.x] = q.need;
    __syncthreads();
    if (threadIdx.x < 32) {
      for (int i = threadIdx.x; i < kTabThreads; i += 32) s_at[i] = tab_place(s_need[i], taken, p.n_free);
      if (threadIdx.x == 0) s_taken = taken;
    }
    __syncthreads();
    taken = s_taken;
    if (r < p.B_R) {
      p.page_off[r] = s_at[threadIdx.x];
      tab_owner_writes(p, r, q, s_at[threadIdx.x]);
    }
    __syncthreads();
  }
  return taken;
}

__global__ void __launch_bounds__(kTabThreads) kv_tables_scan_kernel(const TabParams p) {
  __shared__ int s_used;
  if (threadIdx.x == 0) s_used = 0;
  grid_dependency_wait();
  // the chunks in front of this one
  long long fa = 0, fb = 0, xa, xb;
  for (int c = threadIdx.x; c < (int)blockIdx.x; c += kTabThreads) {
    fa += p.part[2 * c];
    fb += p.part[2 * c + 1];
  }
  tab_scan(fa, fb, &xa, &xb);
  TabReq q[kTabItems];
  long long a, b, ta, tb;
  tab_items(p, blockIdx.x * kTabThreads, 1, q, a, b);
  tab_scan(a, b, &ta, &tb);
  a += xa;
  b += xb;
  const bool runs_out = xb + tb > p.n_free;
  long long used = 0;
  const int r = blockIdx.x * kTabThreads + threadIdx.x;
  if (r < p.B_R) {
    p.row_off[r] = clip32(a);
    if (!runs_out) {
      p.page_off[r] = b;
      used = tab_owner_writes(p, r, q[0], b);
    }
    if (r == p.B_R - 1) {
      a += q[0].rows;
      p.row_off[p.B_R] = clip32(a);
      if (a > p.rows) set_status(p.status, ROCS_ERR_COUNTS);
    }
  }
  // the chunks that the free list does not reach to the end of: all of them by the last block
  if (runs_out && blockIdx.x == gridDim.x - 1) used = tab_place_chunks(p);
  if (used > 0) atomicMax(&s_used, (int)used);
  __syncthreads();
  if (threadIdx.x == 0 && s_used > 0) atomicMax(p.pages_used, s_used);   // a maximum: any order
}

__global__ void __launch_bounds__(kTabThreads, 4) kv_tables_expand_kernel(const TabParams p) {
  __shared__ int32_t s_row[kTabThreads + 1], s_page[kTabThreads], s_past[kTabThreads], s_open[kTabThreads], s_free[kTabFree];
  __shared__ int s_free0;
  grid_dependency_wait();
  const long long n_rows = p.row_off[p.B_R], tile = (long long)p.tile_rows * kTabThreads;
  for (long long t0 = blockIdx.x * tile; t0 < p.rows; t0 += gridDim.x * tile) {
    __syncthreads();            // the window of the tile before is no longer read
    // the request of the tile's first row: the largest with row_off <= t0, narrowed 512-fold a probe
    int lo = 0, hi = p.B_R;
    while (hi - lo > 1) {
      const int step = (hi - lo + kTabThreads - 1) / kTabThreads;
      const int r = lo + (int)threadIdx.x * step;
      const int k = __syncthreads_count(r < hi && (threadIdx.x == 0 || (long long)p.row_off[r] <= t0)) - 1;
      lo += k * step;
      hi = min(hi, lo + step);
    }
    const int n = min(kTabThreads, p.B_R - lo);
    if ((int)threadIdx.x < n) {
      const int r = lo + threadIdx.x;
      const TabReq q = tab_request(p, r);
      s_row[threadIdx.x] = p.row_off[r];
      s_page[threadIdx.x] = clip32(p.page_off[r]);
      const bool dead = q.bad || (q.need > 0 && p.page_off[r] + q.need > p.n_free);
      s_past[threadIdx.x] = dead ? -1 : q.past;
      if ((int)threadIdx.x == n - 1) s_row[n] = p.row_off[r + 1];
      const int mask = (1 << p.P_log2) - 1;
      s_open[threadIdx.x] = !dead && q.rows > 0 && (q.past & mask) != 0 ? p.table[(long long)r * p.max_blocks + (q.past >> p.P_log2)] : -1;
      // the free list's entry of the tile's first row, or of the first after it
      if (threadIdx.x == 0)
        s_free0 = s_page[0] + (dead ? 0 : max(0, (int)((q.past + (t0 - s_row[0])) >> p.P_log2) - q.before));
    }
    __syncthreads();
    const int free0 = s_free0, n_free = (int)min((long long)kTabFree, min((tile >> p.P_log2) + n + 1, (long long)p.n_free - free0));
    for (int i = threadIdx.x; i < n_free; i += kTabThreads) s_free[i] = p.free_pages[free0 + i];
    __syncthreads();
    const TabWindow w = {s_row, s_page, s_past, lo, n, s_open, s_free, free0, n_free};
    tab_rows<true>(p, w, t0 + (threadIdx.x >> 5) * (32 * p.tile_rows), p.tile_rows, n_rows);
  }
}

int tab_chunks(int B_R) { return (B_R + kTabThreads - 1) / kTabThreads; }

}  // namespace

size_t kv_tables_scratch(int B_R) {
  if (B_R <= kTabInline) return 0;
  return ((size_t)2 * tab_chunks(B_R) + (size_t)B_R) * sizeof(long long);
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
  const bool one = B_R <= kTabInline;
  const long long cap = 4LL * ctx->num_sms;         // resident blocks
  // enough rows a thread that the tiles are one wave, for the search of a tile's first request is a chain
  // of latencies
  const long long per = (rows + kTabThreads * cap - 1) / (kTabThreads * cap);
  p.tile_rows = (int)(per < kTabRows ? kTabRows : per > 64 ? 64 : per);
  const long long tile = (long long)kTabThreads * (one ? kTabRows : p.tile_rows);
  const long long blocks = (rows + tile - 1) / tile;
  const unsigned grid = (unsigned)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
  if (one && rows <= 4LL * B_R) {
    LaunchTimer lt_("kv_tables", s);
    kv_tables_few_kernel<<<1, kTabThreads, 0, s>>>(p);
    return cuda_check(cudaGetLastError(), "kv_tables_few_kernel");
  }
  if (one) {
    LaunchTimer lt_("kv_tables", s);
    kv_tables_inline_kernel<<<grid, kTabThreads, 0, s>>>(p);
    return cuda_check(cudaGetLastError(), "kv_tables_inline_kernel");
  }
  {
    LaunchTimer lt_("kv_tables_sum", s);
    kv_tables_sum_kernel<<<tab_chunks(B_R), kTabThreads, 0, s>>>(p);
  }
  rocs_status st;
  {
    LaunchTimer lt_("kv_tables_scan", s);
    st = launch_dependent(kv_tables_scan_kernel, dim3(tab_chunks(B_R)), dim3(kTabThreads), 0, s, "kv_tables_scan_kernel", p);
    if (st != ROCS_OK) return st;
  }
  LaunchTimer lt_("kv_tables_expand", s);
  return launch_dependent(kv_tables_expand_kernel, dim3(grid), dim3(kTabThreads), 0, s, "kv_tables_expand_kernel", p);
}

}  // namespace rocs
