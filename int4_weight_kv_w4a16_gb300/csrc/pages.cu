// Pages of a paged cache on the device: counts of the places that name each page,
// a bit per free page, and the calls that take, share, move and give back pages.
//
// Whatever threads add to or take from a count commutes, and so does turning the bits of
// pages over whose count becomes zero or leaves it; a call that takes pages hands out
// the lowest free ones by rank.  So nothing depends on the order in which threads
// arrive, and no list of free pages has to be kept in order.
//
// grow, fork and compact decide in one CTA (ranks over the free bits: a word a
// thread, 32768 pages a round).  fork and compact leave a plan, and a second kernel changes
// counts and tables and copies pages with the whole GPU.
//
// The deciding CTA is a chain of loads and sums over the CTA, 3 to 4 us: to fork one of four
// sequences takes 6.0 us in all, to give back and take a token's pages for 8 sequences 5.4,
// for 256 with a window and 32 prompts among them 7.4 (a warp a sequence, one after another,
// took 14.6).  Copies are bound by memory: 500 pages of 4 layers (262 MB) moved in 86 us, 0.91
// of the copy rate; 64 half pages of 8 layers (67 MB) in 26.4 us with the decision.
#include "pages.cuh"

namespace futr {

namespace {

constexpr int kPgThreads = 256;
constexpr int kPgPlan = 1024, kPgWarps = kPgPlan / 32;   // threads of a deciding CTA
constexpr int kPgLook = 1024, kPgMaxLook = 256;          // table entries of a CTA that looks at them, most such CTAs
constexpr int kPgTile = 16384;                           // table entries of a CTA in fork

__device__ __forceinline__ int* plan_from(const PoolView& p) { return p.plan + kPlanHeader; }
__device__ __forceinline__ int* plan_to(const PoolView& p) { return plan_from(p) + p.n_pages; }
__device__ __forceinline__ int* plan_slots(const PoolView& p) { return plan_to(p) + p.n_pages; }
__device__ __forceinline__ int4* plan_seqs(const PoolView& p) {
  return reinterpret_cast<int4*>(p.plan + kPlanHeader + ((3 * (size_t)p.n_pages + 3) & ~size_t(3)));
}

// `n` more places name page id (n < 0: fewer); returns how many did before.  A page that no
// place names is free: whoever takes its count across that border turns its bit over and
// counts it among the free pages, or no longer.  Such crossings alternate, and turning over and
// adding commute, so the bits and their number follow the counts in whatever order threads
// arrive, whatever a table names.
__device__ __forceinline__ int add_places(const PoolView& p, int id, int n) {
  const int old = atomicAdd(&p.refs[id], n);
  if ((old > 0) != (old + n > 0)) {
    atomicXor(&p.free[id >> 5], 1u << (id & 31));
    atomicAdd(&p.err[2], old > 0 ? 1 : -1);
    if (old > 0 && (id >> 5) < *static_cast<volatile int*>(&p.err[3])) atomicMin(&p.err[3], id >> 5);
  }
  return old;
}

// One place fewer names page id.
__device__ __forceinline__ void release(const PoolView& p, int id) {
  if (add_places(p, id, -1) > 0) return;
  add_places(p, id, 1);   // not held: as it was
  set_err(p.err, FUTR_ERR_NOT_HELD);
}

// `n` places more name page id, which some place does already.
__device__ __forceinline__ void hold(const PoolView& p, int id, int n) {
  if (add_places(p, id, n) < 1) set_err(p.err, FUTR_ERR_NOT_HELD);
}

// An entry of a table as a page id, -1 if there is none (an id out of range counts as none).
__device__ __forceinline__ int page_of(const PoolView& p, int id) {
  if (id < 0) return -1;
  if (id < p.n_pages) return id;
  set_err(p.err, FUTR_ERR_OUT_OF_RANGE);
  return -1;
}

// The bits of word i that are pages.
__device__ __forceinline__ unsigned valid_bits(const PoolView& p, int i) {
  return p.n_pages - 32 * i >= 32 ? ~0u : (1u << (p.n_pages - 32 * i)) - 1;
}

__global__ void pages_init_kernel(const PoolView p) {
  const int i = blockIdx.x * kPgThreads + threadIdx.x;
  if (i < p.n_pages) p.refs[i] = 0;
  if (i < p.words) p.free[i] = valid_bits(p, i);
  if (i == 0) p.err[2] = p.n_pages, p.err[3] = 0, p.plan[kPlanMet] = p.plan[kPlanBad] = 0;
}

__global__ void __launch_bounds__(kPgThreads) pages_hold_kernel(const PagesArgs a) {
  pdl_trigger();
  pdl_wait();
  const long long n = (long long)a.batch * a.table_ld, step = (long long)gridDim.x * kPgThreads;
  for (long long i = (long long)blockIdx.x * kPgThreads + threadIdx.x; i < n; i += step) {
    const int id = page_of(a.p, a.table[i]);
    if (id >= 0) add_places(a.p, id, 1);
  }
}

__global__ void __launch_bounds__(kPgThreads) pages_free_kernel(const PagesArgs a) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, plog = a.c.page_log2;
  const int pos = max(0, a.pos[b]);
  const int end = (int)(((long long)pos + a.c.page - 1) >> plog);   // pages below it hold positions below pos
  // pages that only a window can hide: behind the sinks, before the first visible position
  const int s1 = a.window > 0 ? (int)(((long long)a.sinks + a.c.page - 1) >> plog) : 0;
  const int w0 = a.window > 0 ? max(0, pos - a.window + 1) >> plog : 0;
  int* row = a.table + (size_t)b * a.table_ld;
  for (int i = blockIdx.x * kPgThreads + threadIdx.x; i < a.table_ld; i += gridDim.x * kPgThreads) {
    const int e = row[i];
    if (e < 0 || (i < end && (i >= w0 || i < s1))) continue;
    row[i] = -1;
    const int id = page_of(a.p, e);
    if (id >= 0) release(a.p, id);
  }
}

// ------------------------------------------------------- the deciding CTA --

// Exclusive sum over the CTA's threads, and the total (shared: kPgWarps words).
__device__ __forceinline__ int scan(int v, int* words, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();   // the words of the call before have been read
  if (lane == 31) words[warp] = incl;
  __syncthreads();
  const int w = words[lane];
  int ws = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += t;
  }
  total = __shfl_sync(0xffffffffu, ws, 31);
  return incl - v + __shfl_sync(0xffffffffu, ws - w, warp);
}

// Whether the pages that the call's table names are held: a page that is named and free would
// be taken for a copy and written over.  All CTAs of a deciding kernel but the first look, while
// that one decides; whatever the call changes the second kernel changes, which knows what they
// found.  (In front of the decision the look cost 1 to 3 us: 128 sequences of 75 pages, forked in
// 29.9 us, took 31.2.)
__device__ __forceinline__ void look(const PagesArgs& a) {
  const long long n = (long long)a.batch * a.table_ld, step = (long long)(gridDim.x - 1) * kPgPlan;
  bool bad = false;
#pragma unroll 4
  for (long long i = (long long)(blockIdx.x - 1) * kPgPlan + threadIdx.x; i < n; i += step) {
    const int id = a.table[i];
    if ((unsigned)id < (unsigned)a.p.n_pages) bad |= a.p.refs[id] < 1;
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) a.p.plan[kPlanBad] = 1;
}

// In the second kernel: whether the call goes ahead.  (Of the CTAs that have read that it does
// not for the look's sake, the last takes that back.)
__device__ __forceinline__ bool goes_ahead(const PagesArgs& a) {
  const int ok = a.p.plan[1], bad = a.p.plan[kPlanBad];
  if (!bad) return ok;
  __syncthreads();
  if (threadIdx.x == 0) {
    set_err(a.p.err, FUTR_ERR_NOT_HELD);
    unsigned* met = reinterpret_cast<unsigned*>(a.p.plan + kPlanMet);
    if (atom_add_acq_rel_gpu(met, 1u) == gridDim.x - 1) a.p.plan[kPlanBad] = 0, *met = 0;
  }
  return false;
}

// The first `want` set bits of words [first, n) as numbers into list, in order.  Returns how
// many there were (at most want).
template <class F>
__device__ __forceinline__ int list_bits(const F& word, int first, int n, int want, int* list, int* words) {
  int done = 0;
  for (long long base = first; base < n && done < want; base += kPgPlan) {
    const int i = (int)min(base + threadIdx.x, (long long)n);
    unsigned w = i < n ? word(i) : 0u;
    int total;
    int r = done + scan(__popc(w), words, total);
    for (; w && r < want; ++r, w &= w - 1) list[r] = i * 32 + __ffs(w) - 1;
    done += total;
  }
  return min(done, want);
}

// The first `want` > 0 free pages into list; there are that many, none before word `first`.
__device__ __forceinline__ void list_free(const PoolView& p, int first, int want, int* list, int* words) {
  list_bits([&](int i) { return p.free[i]; }, first, p.words, want, list, words);
}

// A free page is named by one place.
__device__ __forceinline__ void take(const PoolView& p, int id) {
  p.refs[id] = 1;
  atomicAnd(&p.free[id >> 5], ~(1u << (id & 31)));
}

// Rows of sequence b in `grow`: its pages [i0, i1) (none: i0 == i1).
__device__ __forceinline__ void grow_pages(const PagesArgs& a, int b, int& i0, int& i1, bool report) {
  const long long n = a.start ? (long long)a.start[b + 1] - a.start[b] : 1, p0 = a.pos[b], end = p0 + n;
  i0 = i1 = 0;
  if (n == 0) return;
  if (n < 0 || p0 < 0 || end > a.c.max_pos || end > ((long long)a.table_ld << a.c.page_log2)) {
    if (report) set_err(a.p.err, FUTR_ERR_OUT_OF_RANGE);
    return;
  }
  i0 = (int)(p0 >> a.c.page_log2);
  i1 = (int)((end - 1) >> a.c.page_log2) + 1;
}

// The places that a call's rows meet, of all sequences one after another: place f is entry
// [b][i] of the table.
__global__ void __launch_bounds__(kPgPlan) pages_grow_kernel(const PagesArgs a) {
  __shared__ int words[kPgWarps];
  __shared__ int first[kPagesMaxSeqs], place[kPagesMaxSeqs];   // a sequence's first page, and its place
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int n_free = a.p.err[2], word = a.p.err[3];
  int i0 = 0, i1 = 0, places;
  if (tid < a.batch) grow_pages(a, tid, i0, i1, true);
  const int before = scan(i1 - i0, words, places);
  first[tid] = i0;
  place[tid] = before;
  __syncthreads();
  // the last sequence that begins at or before place f (of those that begin together the last
  // is the one with pages)
  auto entry = [&](int f) {
    int lo = 0;
    for (int step = kPagesMaxSeqs / 2; step > 0; step >>= 1)
      if (lo + step < a.batch && place[lo + step] <= f) lo += step;
    return a.table + (size_t)lo * a.table_ld + first[lo] + (f - place[lo]);
  };
  // those without a page: the round's, kept, and of all rounds before it
  int* list = plan_to(a.p);
  int need = 0, mine = 0, at = 0, bad = FUTR_OK;
  int* e = nullptr;
  for (int f0 = 0; f0 < places; f0 += kPgPlan) {
    e = f0 + tid < places ? entry(f0 + tid) : nullptr;
    const int id = e ? page_of(a.p, *e) : -1;
    mine = e && id < 0;
    const int held = id >= 0 ? a.p.refs[id] : 1;   // rows go to a page of their own
    if (held != 1) bad = held > 1 ? FUTR_ERR_SHARED : FUTR_ERR_NOT_HELD;
    int total;
    at = need + scan(mine, words, total);
    need += total;
  }
  if (__syncthreads_or(bad)) {
    if (bad) set_err(a.p.err, bad);
    return;
  }
  if (need == 0) return;
  if (need > n_free) {
    if (tid == 0) set_err(a.p.err, FUTR_ERR_NO_PAGES);
    return;
  }
  list_free(a.p, word, need, list, words);
  __syncthreads();
  for (int k = tid; k < need; k += kPgPlan) take(a.p, list[k]);
  if (tid == 0) {
    a.p.err[2] -= need;
    a.p.err[3] = list[need - 1] >> 5;   // the lowest are gone
  }
  if (places <= kPgPlan) {
    if (mine) *e = list[at];
    return;
  }
  need = 0;
  for (int f0 = 0; f0 < places; f0 += kPgPlan) {
    e = f0 + tid < places ? entry(f0 + tid) : nullptr;
    mine = e && (unsigned)*e >= (unsigned)a.p.n_pages;
    int total;
    at = need + scan(mine, words, total);
    need += total;
    if (mine) *e = list[at];
  }
}

__global__ void __launch_bounds__(kPgPlan) fork_plan_kernel(const PagesArgs a) {
  __shared__ int words[kPgWarps];
  __shared__ int first[kPagesMaxSeqs];   // a row's first child
  __shared__ int oldpos[kPagesMaxSeqs];
  __shared__ int s_bad;
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x > 0) return look(a);
  const int i = threadIdx.x, n_free = a.p.err[2], word = a.p.err[3];
  const int most = (int)min((long long)a.c.max_pos, (long long)a.table_ld << a.c.page_log2);
  if (i == 0) s_bad = 0;
  int parent = -1;
  if (i < a.batch) {
    parent = a.parent[i];
    first[i] = a.batch;
    oldpos[i] = a.pos[i];
  }
  __syncthreads();
  int from = -1, at = 0;
  bool others = false;   // name the written page
  if (parent >= 0 && parent < a.batch) {
    atomicMin(&first[parent], i);
    const int p = oldpos[parent];
    if (p < 0 || p > most)
      s_bad = 1;
    else {
      at = p >> a.c.page_log2;   // places below it are shared
      if (p & (a.c.page - 1)) from = page_of(a.p, a.table[(size_t)parent * a.table_ld + at]);
      if (from >= 0) others = a.p.refs[from] > 1;
    }
  } else if (i < a.batch && parent != -1) {
    s_bad = 1;
  }
  __syncthreads();
  const bool one = parent >= 0 && !s_bad && first[parent] == i;
  const bool copy = parent >= 0 && !s_bad && (!one || others) && from >= 0;
  int total;
  const int k = scan(copy, words, total);
  const bool ok = !s_bad && total <= n_free;
  if (i == 0) {
    a.p.plan[0] = ok ? total : 0;
    a.p.plan[1] = ok;
    if (!ok) set_err(a.p.err, s_bad ? FUTR_ERR_OUT_OF_RANGE : FUTR_ERR_NO_PAGES);
  }
  if (!ok) return;
  int* list = plan_to(a.p);
  if (total > 0) list_free(a.p, word, total, list, words);
  __syncthreads();
  if (i == 0 && total > 0) a.p.err[3] = list[0] >> 5;
  if (i < a.batch) {
    if (copy) {
      plan_from(a.p)[k] = from;
      plan_slots(a.p)[k] = oldpos[parent] & (a.c.page - 1);
    }
    plan_seqs(a.p)[i] = make_int4(parent, parent >= 0 ? oldpos[parent] : 0, copy ? list[k] : -1, one);
  }
}

// ------------------------------------------------------------------ copies --

// Up to kPgPiece bytes (a multiple of 16), a warp: all loads are under way before the first
// store.
constexpr int kPgPiece = 4096;
__device__ __forceinline__ void copy_piece(const uint8_t* src, uint8_t* dst, int bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* t = reinterpret_cast<uint4*>(dst);
  const int n = bytes >> 4, lane = threadIdx.x & 31;
  uint4 v[kPgPiece / 512];
#pragma unroll
  for (int j = 0; j < kPgPiece / 512; ++j)
    if (lane + 32 * j < n) v[j] = s[lane + 32 * j];
#pragma unroll
  for (int j = 0; j < kPgPiece / 512; ++j)
    if (lane + 32 * j < n) t[lane + 32 * j] = v[j];
}

// The plan's copies, a piece of up to kPgPiece bytes of a (copy, layer, head, keys or
// values) a warp at a time (warps `w` of `warps`): small pieces, so that the warps end
// together.  262 MB moved twice, with 2, 4, 6 and 8 CTAs an SM: 195, 180, 172 and 171 us.
constexpr int kPgCopyCtas = 8;
__device__ __forceinline__ void do_copies(const PagesArgs& a, int w, int warps, bool whole) {
  const int block = a.c.page * a.d, pieces = (block + kPgPiece - 1) / kPgPiece;
  const int blocks = 2 * a.c.n_kv, per = blocks * a.n_layers * pieces;   // of a page in a layer; pieces of a copy
  const int n = a.p.plan[0];
  const int *from = plan_from(a.p), *to = plan_to(a.p), *slots = plan_slots(a.p);
  const int dk = warps / per, dr = warps - dk * per;
  int k = w / per, r = w - k * per;
  while (k < n) {
    const int piece = r % pieces, q = r / pieces, layer = q / blocks, h = q - layer * blocks;
    const size_t src = (size_t)from[k] * blocks + h, dst = (size_t)to[k] * blocks + h;
    uint8_t* codes = a.c.codes + (size_t)layer * a.layer_codes;
    float* scales = a.c.scales + (size_t)layer * a.layer_scales;
    const int at = piece * kPgPiece, bytes = min(whole ? block : slots[k] * a.d, at + kPgPiece) - at;
    if (bytes > 0) copy_piece(codes + src * block + at, codes + dst * block + at, bytes);
    if (piece == 0 && (threadIdx.x & 31) == 0) scales[dst] = scales[src];
    k += dk;
    r += dr;
    if (r >= per) {
      r -= per;
      ++k;
    }
  }
}

// The first blocks change the table, columns [cols * blockIdx.x, ..) of all rows each; the
// next takes the copies' pages and moves the positions, the others copy.
__global__ void __launch_bounds__(kPgThreads) fork_apply_kernel(const PagesArgs a, int cols, int table_ctas) {
  extern __shared__ int old[];   // [batch][cols]
  pdl_trigger();
  pdl_wait();
  if (!goes_ahead(a)) return;
  const int tid = threadIdx.x, plog = a.c.page_log2;
  const int4* seqs = plan_seqs(a.p);
  if ((int)blockIdx.x == table_ctas) {
    const int copies = a.p.plan[0];
    for (int k = tid; k < copies; k += kPgThreads) take(a.p, plan_to(a.p)[k]);
    for (int i = tid; i < a.batch; i += kPgThreads) a.pos[i] = seqs[i].y;
    if (tid == 0 && copies > 0) atomicSub(&a.p.err[2], copies);
    return;
  }
  if ((int)blockIdx.x > table_ctas) {
    const int w = ((int)blockIdx.x - table_ctas - 1) * (kPgThreads / 32) + (tid >> 5);
    do_copies(a, w, ((int)gridDim.x - table_ctas - 1) * (kPgThreads / 32), false);
    return;
  }
  // a row's children; its first place that is not shared; whether its first child has a copy
  // of that place's page
  __shared__ int kids[kPagesMaxSeqs], shared[kPagesMaxSeqs];
  __shared__ uint8_t copied[kPagesMaxSeqs];
  const int c0 = blockIdx.x * cols, n = min(cols, a.table_ld - c0);
  for (int i = tid; i < a.batch; i += kPgThreads) kids[i] = 0, shared[i] = 0, copied[i] = 0;
  for (int e = tid; e < a.batch * cols; e += kPgThreads) {
    const int i = e / cols, j = e - i * cols;
    if (j < n) old[e] = a.table[(size_t)i * a.table_ld + c0 + j];
  }
  __syncthreads();
  for (int i = tid; i < a.batch; i += kPgThreads) {
    const int4 s = seqs[i];
    if (s.x >= 0) {
      atomicAdd(&kids[s.x], 1);
      shared[s.x] = s.y >> plog;   // the same for all children
      if (s.w) copied[s.x] = s.z >= 0;
    }
  }
  __syncthreads();
  for (int e = tid; e < a.batch * cols; e += kPgThreads) {
    const int i = e / cols, j = e - i * cols, c = c0 + j;
    if (j >= n) continue;
    // row i's new entry
    const int4 s = seqs[i];
    int now = -1;
    const int at = s.y >> plog;
    if (s.x >= 0) now = c == at && s.z >= 0 ? s.z : c < at || s.w ? old[s.x * cols + j] : -1;
    if (now != old[e]) a.table[(size_t)i * a.table_ld + c] = now;
    // and what becomes of its old page
    const int more = (c < shared[i] ? kids[i] : kids[i] > 0 && !(copied[i] && c == shared[i])) - 1;
    if (old[e] >= 0 && more != 0) {
      const int id = page_of(a.p, old[e]);
      if (id >= 0) {
        if (more < 0)
          release(a.p, id);
        else
          hold(a.p, id, more);
      }
    }
  }
}

__global__ void __launch_bounds__(kPgPlan) compact_plan_kernel(const PagesArgs a) {
  __shared__ int words[kPgWarps];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x > 0) return look(a);
  const PoolView& p = a.p;
  const int word = p.err[3];
  // pages of word i inside [lo, hi)
  auto inside = [&](int i) {
    const int lo = a.lo - i * 32, hi = a.hi - i * 32;
    unsigned m = hi > 0 && lo < 32 ? ~0u : 0u;
    if (lo > 0 && lo < 32) m &= ~0u << lo;
    if (hi > 0 && hi < 32) m &= ~(~0u << hi);
    return m;
  };
  int *from = plan_from(p), *to = plan_to(p), *where = plan_slots(p);
  const int moves = list_bits([&](int i) { return ~p.free[i] & inside(i) & valid_bits(p, i); }, a.lo >> 5,
                              (int)((a.hi + 31ll) >> 5), p.n_pages, from, words);
  const int room = list_bits([&](int i) { return p.free[i] & ~inside(i); }, word, p.words, moves, to, words);
  const bool ok = room == moves;
  if (threadIdx.x == 0) {
    p.plan[0] = ok ? moves : 0;
    p.plan[1] = ok;
    if (!ok) set_err(p.err, FUTR_ERR_NO_PAGES);
  }
  if (!ok) return;
  for (int i = a.lo + threadIdx.x; i < a.hi; i += kPgPlan) where[i] = i;
  __syncthreads();
  for (int k = threadIdx.x; k < moves; k += kPgPlan) where[from[k]] = to[k];
}

__global__ void __launch_bounds__(kPgThreads) compact_apply_kernel(const PagesArgs a, int table_ctas) {
  pdl_trigger();
  pdl_wait();
  if (!goes_ahead(a)) return;
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= table_ctas) {
    const int w = ((int)blockIdx.x - table_ctas) * (kPgThreads / 32) + (tid >> 5);
    do_copies(a, w, ((int)gridDim.x - table_ctas) * (kPgThreads / 32), true);
    return;
  }
  const PoolView& p = a.p;
  const int *where = plan_slots(p), *from = plan_from(p), *to = plan_to(p), moves = p.plan[0];
  const int first = blockIdx.x * kPgThreads + tid, step = table_ctas * kPgThreads;
  if (first == 0 && moves > 0) atomicMin(&p.err[3], from[0] >> 5);
  for (int k = first; k < moves; k += step) {
    const int s = from[k], t = to[k];
    p.refs[t] = p.refs[s];
    p.refs[s] = 0;
    atomicOr(&p.free[s >> 5], 1u << (s & 31));
    atomicAnd(&p.free[t >> 5], ~(1u << (t & 31)));
  }
  const long long n = (long long)a.batch * a.table_ld;
  for (long long i = first; i < n; i += step) {
    const int id = page_of(a.p, a.table[i]);
    if (id >= a.lo && id < a.hi && where[id] != id) a.table[i] = where[id];
  }
}

template <class F, class... Args>
cudaError_t pg_launch(F* f, dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}

unsigned blocks_for(long long n, long long most) {
  const long long b = (n + kPgThreads - 1) / kPgThreads;
  return (unsigned)(b < most ? b : most);
}

}  // namespace

cudaError_t launch_pages_init(const PoolView& p, cudaStream_t st) {
  pages_init_kernel<<<(unsigned)((p.n_pages + kPgThreads - 1) / kPgThreads), kPgThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_hold(const PagesArgs& a, cudaStream_t st) {
  return pg_launch(pages_hold_kernel, dim3(blocks_for((long long)a.batch * a.table_ld, 1024)), kPgThreads, 0, st, a);
}

// CTAs of a deciding kernel: one, and those that look at the table.
unsigned looking(const PagesArgs& a) {
  const long long n = ((long long)a.batch * a.table_ld + kPgLook - 1) / kPgLook;
  return 1 + (unsigned)(n < kPgMaxLook ? n : kPgMaxLook);
}

cudaError_t launch_pages_grow(const PagesArgs& a, cudaStream_t st) {
  return pg_launch(pages_grow_kernel, dim3(1), kPgPlan, 0, st, a);
}

cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t st) {
  return pg_launch(pages_free_kernel, dim3(blocks_for(a.table_ld, 64), (unsigned)a.batch), kPgThreads, 0, st, a);
}

cudaError_t launch_pages_fork(const PagesArgs& a, int sms, cudaStream_t st) {
  cudaError_t e = pg_launch(fork_plan_kernel, dim3(looking(a)), kPgPlan, 0, st, a);
  if (e != cudaSuccess) return e;
  const int most = kPgTile / a.batch, cols = a.table_ld < most ? a.table_ld : most;
  const int table_ctas = (a.table_ld + cols - 1) / cols;
  static DeviceOnce configured;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.done(dev)) {
    e = cudaFuncSetAttribute(fork_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgTile * 4);
    if (e != cudaSuccess) return e;
    configured.mark(dev);
  }
  return pg_launch(fork_apply_kernel, dim3((unsigned)(table_ctas + kPgCopyCtas * sms + 1)), kPgThreads, (size_t)a.batch * cols * 4, st,
                   a, cols, table_ctas);
}

cudaError_t launch_pages_compact(const PagesArgs& a, int sms, cudaStream_t st) {
  const cudaError_t e = pg_launch(compact_plan_kernel, dim3(looking(a)), kPgPlan, 0, st, a);
  if (e != cudaSuccess) return e;
  const int table_ctas = (int)blocks_for((long long)a.batch * a.table_ld, 64);
  return pg_launch(compact_apply_kernel, dim3((unsigned)(table_ctas + kPgCopyCtas * sms)), kPgThreads, 0, st, a, table_ctas);
}

}  // namespace futr
