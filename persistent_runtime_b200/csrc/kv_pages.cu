// Pages of a cache: sharing them between sequences, giving them out and taking
// them back, moving them together, copying them.
//
// Every call is one bookkeeping launch over the page table and the counts (a
// few KB to a few MB) and, where contents move, one copy launch behind it.
// Bookkeeping needs several passes with everything before a pass visible to
// it, so it runs as ONE cluster (1 to 8 CTAs, by the number of entries) whose
// passes are separated by cluster barriers: a grid of independent CTAs would
// need a launch per pass.  All orders that show in the results come from scans
// over contiguous runs of entries or pages (thread i of CTA r takes run
// r * 1024 + i); atomics count, take minima or maxima, or give out room in the
// copy list, whose order does not matter.
//
// The copy is bound by HBM: every moved byte is read and written once, or, where
// one page is copied for several sequences, read once: their copies lie next to
// each other in the list and the later reads hit L2.  About 100 pages of
// an 8B decoder's 8-bit pools (4.7 MB each) move in 143 us (6.5 TB/s); 32 pages
// copied three times each take 119 us with the bookkeeping, where one read and
// three writes at the copy's rate would be 89: the repeated reads go through L2.
// The grid is the CTAs that are resident (a call that moves nothing should cost a
// launch, not thousands of empty CTAs: 64 CTAs per SM cost 9 us more) and takes
// steps as it goes: SMs differ in their distance to memory, and equal shares took
// 7 % longer.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv8.cuh"

namespace cg = cooperative_groups;

namespace mk {
namespace {

constexpr int kTeamThreads = 1024;
constexpr int kMaxTeam = 8;             // CTAs of a cluster (the portable limit)
constexpr int kScans = 8;               // exchanges of one call
constexpr int kCopyBytes = 16 * 1024;   // a CTA's step of the copy
constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 5;            // CTAs per SM of the copy: those that are resident
constexpr int kNear = 4096;             // sequences, free pages kept in shared memory

// Workspace: the header, then the lists.
struct Header {
  int copies;  // entries of the copy list
  int next;    // steps of the copy that have been given out, besides every CTA's first
  int pad[14];
  int slots[kScans][kMaxTeam];
};

struct PageArgs {
  mk_pages p;
  Header *head;
  int2 *list;     // [max(n, n_pages)] source page, destination page (~page: not copied)
  int *free_list; // [n_pages]
  int *mark;      // [n_pages]
  int *last;      // [n_pages]
  int *place;     // [n_pages]
  int *seq;       // [n_seqs + 1]
  int n;
  const int32_t *a, *b;  // the call's two lists
};

// The cluster that does the bookkeeping.
struct Team {
  int rank, size;
  Header *head;
  int *warps;  // 33 ints of shared memory
  int used = 0;

  __device__ __forceinline__ int index() const { return rank * kTeamThreads + (int)threadIdx.x; }
  __device__ __forceinline__ int threads() const { return size * kTeamThreads; }
  __device__ __forceinline__ void sync() const {
    if (size > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  // This thread's contiguous run [i0, i1) of n items, in thread order.
  __device__ __forceinline__ void run(int n, int &i0, int &i1) const {
    const int64_t per = ((int64_t)n + threads() - 1) / threads();
    i0 = (int)min((int64_t)n, per * index());
    i1 = (int)min((int64_t)n, (int64_t)i0 + per);
  }
  // Sum of v over the threads of the CTA before this one; `total` over all.
  __device__ __forceinline__ int cta_scan(int v, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    __syncthreads();  // the last use of `warps` is over
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    if (warp == 0) {
      int x = warps[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      warps[lane] = x;
    }
    __syncthreads();
    total = warps[31];
    return upto - v + (warp ? warps[warp - 1] : 0);
  }
  // The same over the team.  Orders everything before it before everything
  // after it, in the whole team.
  __device__ __forceinline__ int scan(int v, int &total) {
    int before = cta_scan(v, total);
    if (size > 1) {
      int *slot = head->slots[used++];
      if (threadIdx.x == 0) __stcg(slot + rank, total);
      cg::this_cluster().sync();
      total = 0;
      for (int r = 0; r < size; ++r) {
        const int x = __ldcg(slot + r);
        if (r < rank) before += x;
        total += x;
      }
    }
    return before;
  }
  // Whether any thread of the team says so; a barrier like scan().
  __device__ __forceinline__ bool any(bool v) { return any_bits(v ? 1 : 0) != 0; }
  // The same for two flags.
  __device__ __forceinline__ int any_bits(int bits) {
    const int mine = (__syncthreads_or(bits & 1) ? 1 : 0) | (__syncthreads_or(bits & 2) ? 2 : 0);
    if (size == 1) return mine;
    int *slot = head->slots[used++];
    if (threadIdx.x == 0) __stcg(slot + rank, mine);
    cg::this_cluster().sync();
    int all = 0;
    for (int r = 0; r < size; ++r) all |= __ldcg(slot + r);
    return all;
  }
};

__device__ __forceinline__ Team make_team(const PageArgs &a, int *warps) {
  Team t{0, 1, a.head, warps};
  t.size = (int)cg::this_cluster().num_blocks();
  t.rank = (int)cg::this_cluster().block_rank();
  return t;
}

__device__ __forceinline__ bool bad_seq(const PageArgs &a, const int32_t *list, int i) {
  const int s = list[i];
  if (s >= 0 && s < a.p.n_seqs) return false;
  record_status(a.p.d_status, MK_ERR_DEVICE, i, s, MK_CHECK_SEQ);
  return true;
}

// An entry is -1 (no page) or a page of the pools that is counted: one that names a
// free page would share it with whoever is given the page next.
__device__ __forceinline__ bool bad_entry(const PageArgs &a, int s, int page) {
  if (page == -1 || (page >= 0 && page < a.p.n_pages && a.p.d_ref[page] >= 1)) return false;
  record_status(a.p.d_status, MK_ERR_DEVICE, s, page, MK_CHECK_PAGE);
  return true;
}

// --- fork: a = sources, b = destinations -----------------------------------------
__global__ void __launch_bounds__(kTeamThreads) fork_kernel(const __grid_constant__ PageArgs a) {
  __shared__ int warps[32];
  pdl_trigger();
  pdl_wait();
  Team t = make_team(a, warps);
  const int mp = a.p.max_pages;
  bool bad = false;
  for (int i = t.index(); i < a.n; i += t.threads()) {
    const bool b0 = bad_seq(a, a.a, i), b1 = bad_seq(a, a.b, i);
    if (!b0) __stcg(a.seq + a.a[i], 0);
    if (!b1) __stcg(a.seq + a.b[i], 0);
    bad |= b0 || b1;
  }
  if (t.any(bad)) return;
  for (int i = t.index(); i < a.n; i += t.threads()) atomicAdd(a.seq + a.b[i], 1);
  t.sync();
  for (int i = t.index(); i < a.n; i += t.threads())
    if (__ldcg(a.seq + a.b[i]) != 1 || __ldcg(a.seq + a.a[i]) != 0) {
      bad = true;
      record_status(a.p.d_status, MK_ERR_DEVICE, i, a.b[i], MK_CHECK_SEQ);
    }
  const int64_t total = (int64_t)a.n * mp;
  for (int64_t e = t.index(); e < total; e += t.threads()) {
    const int i = (int)(e / mp), j = (int)(e - (int64_t)i * mp);
    const int s = a.a[i], d = a.b[i];
    if (bad_entry(a, s, a.p.d_page_table[(int64_t)s * mp + j])) bad = true;
    if (a.p.d_page_table[(int64_t)d * mp + j] != -1) {
      bad = true;
      record_status(a.p.d_status, MK_ERR_DEVICE, d, j, MK_CHECK_IN_USE);
    }
  }
  if (t.any(bad)) return;
  for (int64_t e = t.index(); e < total; e += t.threads()) {
    const int i = (int)(e / mp), j = (int)(e - (int64_t)i * mp);
    const int page = a.p.d_page_table[(int64_t)a.a[i] * mp + j];
    if (page < 0) continue;
    a.p.d_page_table[(int64_t)a.b[i] * mp + j] = page;
    atomicAdd(a.p.d_ref + page, 1);
  }
}

// --- free: a = sequences -------------------------------------------------------------
__global__ void __launch_bounds__(kTeamThreads) free_kernel(const __grid_constant__ PageArgs a) {
  __shared__ int warps[32];
  pdl_trigger();
  pdl_wait();
  Team t = make_team(a, warps);
  const int mp = a.p.max_pages;
  bool bad = false;
  for (int i = t.index(); i < a.n; i += t.threads()) {
    if (bad_seq(a, a.a, i)) bad = true;
    else __stcg(a.seq + a.a[i], a.n);
  }
  if (t.any(bad)) return;
  // a sequence that is named twice goes by its first place in the list
  for (int i = t.index(); i < a.n; i += t.threads()) atomicMin(a.seq + a.a[i], i);
  const int64_t total = (int64_t)a.n * mp;
  for (int64_t e = t.index(); e < total; e += t.threads()) {
    const int i = (int)(e / mp), j = (int)(e - (int64_t)i * mp);
    if (bad_entry(a, a.a[i], a.p.d_page_table[(int64_t)a.a[i] * mp + j])) bad = true;
  }
  if (t.any(bad)) return;
  for (int64_t e = t.index(); e < total; e += t.threads()) {
    const int i = (int)(e / mp), j = (int)(e - (int64_t)i * mp);
    if (__ldcg(a.seq + a.a[i]) != i) continue;
    int32_t *at = a.p.d_page_table + (int64_t)a.a[i] * mp + j;
    const int page = *at;
    if (page < 0) continue;
    *at = -1;
    atomicSub(a.p.d_ref + page, 1);
  }
}

// --- reserve: a = kv_len, b = n_new ------------------------------------------------------
// The entries that a call looks at: those whose positions overlap
// [c, c + n) of some sequence, in the order of sequence and entry.
struct Walk {
  int s, j, end;  // current sequence, entry, entries of it below `end`
  __device__ __forceinline__ static int first(const PageArgs &a, int s) { return a.a[s] / a.p.page_size; }
  __device__ __forceinline__ static int count(const PageArgs &a, int s) {
    const int n = a.b[s];
    if (n <= 0) return 0;
    return (int)(((int64_t)a.a[s] + n + a.p.page_size - 1) / a.p.page_size) - first(a, s);
  }
  // the e-th entry of the call: before[s] counts the entries before sequence s
  __device__ __forceinline__ void start(const PageArgs &a, const int *before, int e) {
    int lo = 0, hi = a.p.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= e) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    j = first(a, s) + e - before[s];
    end = first(a, s) + count(a, s);
  }
  __device__ __forceinline__ int32_t *at(const PageArgs &a) const {
    return a.p.d_page_table + (int64_t)s * a.p.max_pages + j;
  }
  __device__ __forceinline__ void next(const PageArgs &a, int e, int e1) {  // to entry e, if there is one
    if (e >= e1) return;
    if (++j < end) return;
    do ++s; while (count(a, s) == 0);
    j = first(a, s);
    end = j + count(a, s);
  }
};

__global__ void __launch_bounds__(kTeamThreads) reserve_kernel(const __grid_constant__ PageArgs a) {
  __shared__ int warps[32];
  __shared__ int near_seq[kNear], near_free[kNear];
  pdl_trigger();
  pdl_wait();
  Team t = make_team(a, warps);
  if (t.index() == 0) a.head->copies = a.head->next = 0;
  const int P = a.p.page_size, mp = a.p.max_pages;
  // free pages of this thread's run (the counts change only at the end)
  int p0, p1;
  t.run(a.p.n_pages, p0, p1);
  int n_free = 0;
  for (int p = p0; p < p1; ++p) n_free += a.p.d_ref[p] == 0;
  // lengths, and the number of entries before every sequence: every CTA for itself
  int *before = a.p.n_seqs <= kNear ? near_seq : a.seq;
  const int per = (a.p.n_seqs + kTeamThreads - 1) / kTeamThreads;
  const int s0 = min(a.p.n_seqs, (int)threadIdx.x * per), s1 = min(a.p.n_seqs, s0 + per);
  bool bad = false;
  int mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = a.b[s], c = a.a[s];
    if (n > 0 && (c < 0 || (int64_t)c + n > (int64_t)mp * P)) {
      bad = true;
      record_status(a.p.d_status, MK_ERR_DEVICE, s, c, MK_CHECK_LENGTH);
    } else {
      mine += Walk::count(a, s);
    }
  }
  int entries;
  int upto = t.cta_scan(mine, entries);
  for (int s = s0; s < s1; ++s) {
    before[s] = upto;
    upto += bad ? 0 : Walk::count(a, s);
  }
  if (__syncthreads_or(bad)) return;  // all CTAs have seen the same lengths
  int e0, e1;
  t.run(entries, e0, e1);
  Walk from{0, 0, 0};
  if (e0 < e1) from.start(a, before, e0);
  // a shared page: how many of its holders write it, and the last of them
  bool shared = false;
  Walk w = from;
  for (int e = e0; e < e1; w.next(a, ++e, e1)) {
    const int page = *w.at(a);
    if (bad_entry(a, w.s, page)) bad = true;
    else if (page >= 0 && a.p.d_ref[page] > 1) {
      shared = true;
      __stcg(a.mark + page, 0);
      __stcg(a.last + page, -1);
    }
  }
  const int seen = t.any_bits((bad ? 1 : 0) | (shared ? 2 : 0));
  if (seen & 1) return;
  if (seen & 2) {
    w = from;
    for (int e = e0; e < e1; w.next(a, ++e, e1)) {
      const int page = *w.at(a);
      if (page >= 0 && a.p.d_ref[page] > 1) {
        atomicAdd(a.mark + page, 1);
        atomicMax(a.last + page, e);
      }
    }
    t.sync();
  }
  // an entry gets a free page if it has none, or if its page is shared and it
  // is not the last writer of a page that all its holders write
  auto shared_write = [&](int page, int e) {
    const int refs = a.p.d_ref[page];
    return refs > 1 && !(__ldcg(a.mark + page) == refs && __ldcg(a.last + page) == e);
  };
  int need = 0;
  w = from;
  for (int e = e0; e < e1; w.next(a, ++e, e1)) {
    const int page = *w.at(a);
    if (page < 0 || shared_write(page, e)) ++need;
    if (page >= 0 && a.p.d_ref[page] > 1 && __ldcg(a.last + page) == e) {
      // one writer takes room in the copy list for all of the page's, so that
      // copies of one page are made at the same time and it is read once
      const int writers = __ldcg(a.mark + page);
      __stcg(a.place + page, atomicAdd(&a.head->copies, writers - (writers == a.p.d_ref[page])));
    }
  }
  int all_need, all_free;
  int at = t.scan(need, all_need);
  int k = t.scan(n_free, all_free);
  if (all_free < all_need) {
    if (t.index() == 0) {
      a.head->copies = 0;  // room was given out, but nothing is listed
      record_status(a.p.d_status, MK_ERR_OOM, a.p.n_pages, all_need - all_free, MK_CHECK_FREE);
    }
    return;
  }
  if (all_need == 0) return;
  int *free_list = t.size == 1 && all_need <= kNear ? near_free : a.free_list;
  for (int p = p0; p < p1 && k < all_need; ++p)
    if (a.p.d_ref[p] == 0) free_list[k++] = p;
  t.sync();
  w = from;
  for (int e = e0; e < e1; w.next(a, ++e, e1)) {
    const int page = *w.at(a);
    if (page >= 0 && !shared_write(page, e)) continue;
    const int fresh = free_list == near_free ? near_free[at++] : __ldcg(a.free_list + at++);
    *w.at(a) = fresh;
    if (page >= 0) {
      // contents matter if the page holds positions before the new ones
      const bool copy = (int64_t)w.j * P < a.a[w.s];
      a.list[atomicAdd(a.place + page, 1)] = make_int2(page, copy ? fresh : ~fresh);
    }
  }
  t.sync();
  for (int i = t.index(); i < all_need; i += t.threads())
    a.p.d_ref[free_list == near_free ? near_free[i] : __ldcg(a.free_list + i)] = 1;
  if (seen & 2) {
    const int given_up = __ldcg(&a.head->copies);
    for (int i = t.index(); i < given_up; i += t.threads()) atomicSub(a.p.d_ref + __ldcg(&a.list[i].x), 1);
  }
}

// --- compact --------------------------------------------------------------------------------
__global__ void __launch_bounds__(kTeamThreads) compact_kernel(const __grid_constant__ PageArgs a) {
  __shared__ int warps[32];
  pdl_trigger();
  pdl_wait();
  Team t = make_team(a, warps);
  if (t.index() == 0) a.head->copies = a.head->next = 0;
  const int64_t entries = (int64_t)a.p.n_seqs * a.p.max_pages;
  bool bad = false;
  for (int64_t e = t.index(); e < entries; e += t.threads()) {
    const int page = a.p.d_page_table[e], s = (int)(e / a.p.max_pages);
    if (bad_entry(a, s, page)) bad = true;
  }
  if (t.any(bad)) return;
  int p0, p1;
  t.run(a.p.n_pages, p0, p1);
  int used = 0, n_used;
  for (int p = p0; p < p1; ++p) used += a.p.d_ref[p] != 0;
  int rank = t.scan(used, n_used);  // pages in use before p0
  // of the pages below U, those not in use are filled in order; as many lie in
  // use above U, and the i-th of these goes to the i-th of those
  int holes = 0;
  for (int p = p0; p < p1 && p < n_used; ++p) holes += a.p.d_ref[p] == 0;
  int n_moves;
  int hole = t.scan(holes, n_moves);
  int move = max(0, rank - (n_used - n_moves));  // pages in use in [U, p0), where p0 >= U
  if (p0 < n_used && p1 > n_used) move = 0;
  for (int p = p0; p < p1; ++p) {
    const bool in_use = a.p.d_ref[p] != 0;
    if (p < n_used) {
      if (!in_use) __stcg(&a.list[hole++].y, p);
    } else if (in_use) {
      __stcg(&a.list[move].x, p);
      __stcg(a.mark + p, move++);
    }
  }
  t.sync();
  for (int i = t.index(); i < n_moves; i += t.threads()) {
    const int from = __ldcg(&a.list[i].x), to = __ldcg(&a.list[i].y);
    a.p.d_ref[to] = a.p.d_ref[from];
    a.p.d_ref[from] = 0;
  }
  for (int64_t e = t.index(); e < entries; e += t.threads()) {
    const int page = a.p.d_page_table[e];
    if (page >= n_used) a.p.d_page_table[e] = __ldcg(&a.list[__ldcg(a.mark + page)].y);
  }
  if (t.index() == 0) a.head->copies = n_moves;
}

// --- copy: a = sources, b = destinations ------------------------------------------------------
__global__ void __launch_bounds__(kTeamThreads) copy_list_kernel(const __grid_constant__ PageArgs a) {
  __shared__ int warps[32];
  pdl_trigger();
  pdl_wait();
  Team t = make_team(a, warps);
  if (t.index() == 0) a.head->copies = a.head->next = 0;
  bool bad = false;
  for (int i = t.index(); i < a.n; i += t.threads()) {
    const int from = a.a[i], to = a.b[i];
    const int wrong = from < 0 || from >= a.p.n_pages ? from : to;
    if (wrong < 0 || wrong >= a.p.n_pages) {
      bad = true;
      record_status(a.p.d_status, MK_ERR_DEVICE, i, wrong, MK_CHECK_SEQ);
    } else {
      __stcg(a.mark + from, 0);
      __stcg(a.mark + to, 0);
    }
  }
  if (t.any(bad)) return;
  for (int i = t.index(); i < a.n; i += t.threads()) atomicAdd(a.mark + a.b[i], 1);
  t.sync();
  for (int i = t.index(); i < a.n; i += t.threads()) {
    if (__ldcg(a.mark + a.b[i]) != 1 || __ldcg(a.mark + a.a[i]) != 0) {
      bad = true;
      record_status(a.p.d_status, MK_ERR_DEVICE, i, a.b[i], MK_CHECK_SEQ);
    }
    a.list[i] = make_int2(a.a[i], a.b[i]);
  }
  if (t.any(bad)) return;
  if (t.index() == 0) a.head->copies = a.n;
}

// --- contents ------------------------------------------------------------------------------------
struct CopyArgs {
  int n_pools, steps;                  // steps: of kCopyBytes, of one page over all pools
  char *pool[MK_MAX_POOLS];
  int64_t bytes[MK_MAX_POOLS];
  Header *head;
  const int2 *list;
};

template <typename V>
__device__ __forceinline__ void copy_piece(char *to, const char *from, int bytes) {
  constexpr int kUnroll = kCopyBytes / (kCopyThreads * (int)sizeof(V)) > 8
                              ? 8 : kCopyBytes / (kCopyThreads * (int)sizeof(V));
  V *d = reinterpret_cast<V *>(to);
  const V *s = reinterpret_cast<const V *>(from);
  const int n = bytes / (int)sizeof(V);
  int i = threadIdx.x;
  for (; i + (kUnroll - 1) * kCopyThreads < n; i += kUnroll * kCopyThreads) {
    V v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(s + i + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) d[i + u * kCopyThreads] = v[u];
  }
  for (; i < n; i += kCopyThreads) d[i] = s[i];
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t items = (int64_t)a.head->copies * a.steps;
  __shared__ int upcoming;
  for (int64_t item = blockIdx.x; item < items;) {
    // SMs are not equally fast: a CTA takes the next step that is left
    if (threadIdx.x == 0) upcoming = atomicAdd(&a.head->next, 1);
    const int i = (int)(item / a.steps);
    int step = (int)(item - (int64_t)i * a.steps);
    const int2 pair = a.list[i];
    if (pair.y >= 0) {  // else a page that is replaced without its contents
      int pool = 0;
      for (;; ++pool) {
        const int n = (int)((a.bytes[pool] + kCopyBytes - 1) / kCopyBytes);
        if (step < n) break;
        step -= n;
      }
      const int64_t size = a.bytes[pool], off = (int64_t)step * kCopyBytes;
      const int bytes = (int)min((int64_t)kCopyBytes, size - off);
      char *to = a.pool[pool] + pair.y * size + off;
      const char *from = a.pool[pool] + pair.x * size + off;
      if ((size & 15) == 0 && (reinterpret_cast<uintptr_t>(a.pool[pool]) & 15) == 0)
        copy_piece<uint4>(to, from, bytes);
      else
        copy_piece<uint32_t>(to, from, bytes);
    }
    __syncthreads();
    item = (int64_t)gridDim.x + upcoming;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

struct Places {
  int64_t list, free_list, mark, last, place, seq, total;
};
Places places(const mk_pages &p, int n) {
  Places w{};
  int64_t off = up16(sizeof(Header));
  w.list = off;
  off += up16(8ll * std::max(n, p.n_pages));
  w.free_list = off;
  off += up16(4ll * p.n_pages);
  w.mark = off;
  off += up16(4ll * p.n_pages);
  w.last = off;
  off += up16(4ll * p.n_pages);
  w.place = off;
  off += up16(4ll * p.n_pages);
  w.seq = off;
  off += up16(4ll * (p.n_seqs + 1));
  w.total = off;
  return w;
}

const char *check_pages(const mk_pages *p) {
  if (!p) return "null pages";
  if (p->device < 0) return "bad device";
  if (p->n_pages < 1 || p->n_seqs < 1 || p->max_pages < 1 || p->page_size < 1)
    return "n_pages, n_seqs, max_pages and page_size must be at least 1";
  if ((int64_t)p->n_seqs * p->max_pages >= (1ll << 31) || (int64_t)p->max_pages * p->page_size >= (1ll << 31))
    return "page tables of 2^31 entries or positions and more are not supported";
  if (p->n_pools < 0 || p->n_pools > MK_MAX_POOLS) return "n_pools must be 0 .. MK_MAX_POOLS";
  int64_t bytes = 0, steps = 0;  // steps of the copy of one page
  for (int i = 0; i < p->n_pools; ++i) {
    if (!p->d_pool[i] || (reinterpret_cast<uintptr_t>(p->d_pool[i]) & 3)) return "a pool is null or not 4-byte aligned";
    if (p->page_bytes[i] < 4 || (p->page_bytes[i] & 3)) return "page_bytes must be a positive multiple of 4";
    if (p->page_bytes[i] >= (1ll << 40)) return "page_bytes out of range";  // before they are added
    bytes += p->page_bytes[i];
    steps += (p->page_bytes[i] + kCopyBytes - 1) / kCopyBytes;
  }
  if (bytes >= (1ll << 40)) return "page_bytes out of range";
  // they are counted in 32 bits; the margin is what the CTAs count beyond the last
  if (steps * p->n_pages >= (1ll << 31) - (1 << 20)) return "pools of 2^31 pages and more are not supported";
  if (!p->d_page_table || !p->d_ref) return "null page table or counts";
  return nullptr;
}

const char *check_list(const mk_pages *p, int n, const void *a, const void *b) {
  if (n < 0) return "negative list length";
  if ((int64_t)n * p->max_pages >= (1ll << 31)) return "list too long";
  if (n > 0 && (!a || !b)) return "null list";
  return nullptr;
}

// CTAs of the cluster: one up to 4096 items, then one for every 4096.
int team_size(int64_t items) {
  int size = 1;
  while (size < kMaxTeam && items > 4096ll * size) size *= 2;
  return size;
}

using Kernel = void (*)(const PageArgs);

mk_status run_call(const char *name, Kernel kernel, const mk_pages *p, int n, const void *list_a,
                   const void *list_b, int64_t items, bool copies, void *workspace, int64_t bytes,
                   void *stream) {
  const Places w = places(*p, n);
  const mk_status ws = ops_workspace(name, workspace, bytes, w.total);
  if (ws != MK_OK) return ws;
  DeviceGuard guard(p->device);
  if (guard.error() != cudaSuccess) return ops_cuda_fail(guard.error(), name);
  char *base = static_cast<char *>(workspace);
  PageArgs a{};
  a.p = *p;
  a.head = reinterpret_cast<Header *>(base);
  a.list = reinterpret_cast<int2 *>(base + w.list);
  a.free_list = reinterpret_cast<int *>(base + w.free_list);
  a.mark = reinterpret_cast<int *>(base + w.mark);
  a.last = reinterpret_cast<int *>(base + w.last);
  a.place = reinterpret_cast<int *>(base + w.place);
  a.seq = reinterpret_cast<int *>(base + w.seq);
  a.n = n;
  a.a = static_cast<const int32_t *>(list_a);
  a.b = static_cast<const int32_t *>(list_b);
  const int team = team_size(items);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(team);
  cfg.blockDim = dim3(kTeamThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = team;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return ops_cuda_fail(e, name);
  if (!copies || p->n_pools == 0) return MK_OK;
  CopyArgs c{};
  c.n_pools = p->n_pools;
  int64_t steps = 0;
  for (int i = 0; i < p->n_pools; ++i) {
    c.pool[i] = static_cast<char *>(p->d_pool[i]);
    c.bytes[i] = p->page_bytes[i];
    steps += (p->page_bytes[i] + kCopyBytes - 1) / kCopyBytes;
  }
  c.steps = (int)steps;
  c.head = a.head;
  c.list = a.list;
  const int64_t most = steps * std::max(n, p->n_pages);
  const dim3 grid((unsigned)std::min<int64_t>(most, (int64_t)kCopyCtas * sm_count(p->device)));
  e = pdl_launch(copy_pages_kernel, grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream), c);
  if (e != cudaSuccess) return ops_cuda_fail(e, name);
  return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status mk_pages_workspace(const mk_pages *pages, int n, int64_t *bytes) {
  const char *why = check_pages(pages);
  if (!why) why = check_list(pages, n, pages, pages);
  if (!why && !bytes) why = "null result";
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_workspace", why);
  *bytes = places(*pages, n).total;
  return MK_OK;
}

extern "C" mk_status mk_pages_fork(const mk_pages *pages, int n, const int32_t *d_src,
                                   const int32_t *d_dst, void *d_workspace, int64_t workspace_bytes,
                                   void *stream) {
  const char *why = check_pages(pages);
  if (!why) why = check_list(pages, n, d_src, d_dst);
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_fork", why);
  if (n == 0) return MK_OK;
  return run_call("mk_pages_fork", fork_kernel, pages, n, d_src, d_dst, (int64_t)n * pages->max_pages,
                  false, d_workspace, workspace_bytes, stream);
}

extern "C" mk_status mk_pages_free(const mk_pages *pages, int n, const int32_t *d_seqs,
                                   void *d_workspace, int64_t workspace_bytes, void *stream) {
  const char *why = check_pages(pages);
  if (!why) why = check_list(pages, n, d_seqs, d_seqs);
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_free", why);
  if (n == 0) return MK_OK;
  return run_call("mk_pages_free", free_kernel, pages, n, d_seqs, nullptr, (int64_t)n * pages->max_pages,
                  false, d_workspace, workspace_bytes, stream);
}

extern "C" mk_status mk_pages_reserve(const mk_pages *pages, const int32_t *d_kv_len,
                                      const int32_t *d_n_new, void *d_workspace,
                                      int64_t workspace_bytes, void *stream) {
  const char *why = check_pages(pages);
  if (!why && (!d_kv_len || !d_n_new)) why = "null lengths";
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_reserve", why);
  return run_call("mk_pages_reserve", reserve_kernel, pages, 0, d_kv_len, d_n_new,
                  std::max(pages->n_pages, pages->n_seqs), true, d_workspace, workspace_bytes, stream);
}

extern "C" mk_status mk_pages_compact(const mk_pages *pages, void *d_workspace,
                                      int64_t workspace_bytes, void *stream) {
  const char *why = check_pages(pages);
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_compact", why);
  return run_call("mk_pages_compact", compact_kernel, pages, 0, nullptr, nullptr,
                  std::max<int64_t>(pages->n_pages, (int64_t)pages->n_seqs * pages->max_pages), true,
                  d_workspace, workspace_bytes, stream);
}

extern "C" mk_status mk_pages_copy(const mk_pages *pages, int n, const int32_t *d_src,
                                   const int32_t *d_dst, void *d_workspace, int64_t workspace_bytes,
                                   void *stream) {
  const char *why = check_pages(pages);
  if (!why) why = check_list(pages, n, d_src, d_dst);
  if (why) return ops_fail(MK_ERR_ARG, "mk_pages_copy", why);
  if (n == 0) return MK_OK;
  return run_call("mk_pages_copy", copy_list_kernel, pages, n, d_src, d_dst, n, true, d_workspace,
                  workspace_bytes, stream);
}
