// Entry points of generation with several continuations (declared in include/futr.h):
// choice of beams, order of cache slots, pages of the paged cache.  Argument checks,
// memory layouts, launches.
#include <climits>

#include "beam.cuh"
#include "pages.cuh"

namespace futr {
namespace host {
uint64_t region_after(uint64_t off, uint64_t size);
cudaError_t fill_guards_before(void* base, const uint64_t* starts, int n, cudaStream_t st);
cudaError_t check_guards_before(void* base, const uint64_t* starts, int n, int* err, cudaStream_t st);
int sm_count();
}  // namespace host
}  // namespace futr

using namespace futr;

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

template <class T>
T* at(void* base, uint64_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(base) + off);
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Nothing is thrown across the C boundary.
template <class F>
futr_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return FUTR_ERR_CUDA;
  }
}

futr_status status_of(cudaError_t e) { return e == cudaSuccess ? FUTR_OK : FUTR_ERR_CUDA; }

// Compare the guards that end at `starts`, wait, and return and clear error word 0 (words
// 0 .. n-1 of the region come back in `words`).
futr_status read_errors(void* base, const uint64_t* starts, int guards, int* err, int* words, int n, cudaStream_t s) {
  if (host::check_guards_before(base, starts, guards, err, s) != cudaSuccess) return FUTR_ERR_CUDA;
  if (cudaMemcpyAsync(words, err, n * sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FUTR_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
  if (words[0] == 0) return FUTR_OK;
  if (cudaMemsetAsync(err, 0, sizeof(int), s) != cudaSuccess) return FUTR_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
  return words[0];
}

// ------------------------------------------------------------------- beams --

struct BeamLayout {
  uint64_t err, cnt, rows, recs, total;
};

BeamLayout beam_layout(int rows, int keep, int ctas) {
  BeamLayout L{};
  const uint64_t parts = rows > ctas ? rows : ctas;
  L.err = 0;
  L.cnt = host::region_after(0, 16);
  L.rows = host::region_after(L.cnt, 2 * (uint64_t)rows * 4);
  L.recs = host::region_after(L.rows, (uint64_t)rows * beam_record(keep));
  L.total = host::region_after(L.recs, parts * beam_record(keep));
  return L;
}

bool beam_ok(const futr_beam_ws* w) { return w && w->magic == kBeamWsMagic && w->base; }

void beam_guards(const futr_beam_ws& w, uint64_t* g) {
  g[0] = w.cnt_offset;
  g[1] = w.row_offset;
  g[2] = w.rec_offset;
  g[3] = w.bytes;
}

// ------------------------------------------------------------------- pages --

struct PagesLayout {
  uint64_t refs, free, plan, err, total;
};

int pool_words(int n_pages) { return (int)(((int64_t)n_pages + 31) / 32); }

PagesLayout pages_layout(int n_pages, int max_seqs) {
  PagesLayout L{};
  L.refs = 0;
  L.free = host::region_after(0, (uint64_t)n_pages * 4);
  L.plan = host::region_after(L.free, (uint64_t)pool_words(n_pages) * 4);
  L.err = host::region_after(L.plan, (uint64_t)plan_ints(n_pages, max_seqs) * 4);
  L.total = host::region_after(L.err, 16);
  return L;
}

bool pool_ok(const futr_pages* p) { return p && p->magic == kPagesMagic && p->base; }

void pool_guards(const futr_pages& p, uint64_t* g) {
  g[0] = p.free_offset;
  g[1] = p.plan_offset;
  g[2] = p.err_offset;
  g[3] = p.bytes;
}

PoolView pool_view(const futr_pages& p) {
  PoolView v{};
  v.refs = at<int>(p.base, p.refs_offset);
  v.free = at<unsigned>(p.base, p.free_offset);
  v.plan = at<int>(p.base, p.plan_offset);
  v.err = at<int>(p.base, p.err_offset);
  v.n_pages = p.n_pages;
  v.words = pool_words(p.n_pages);
  return v;
}

// The arguments that every call on a table shares.
futr_status pages_args(const futr_paged* c, const futr_pages* pool, int batch, const int32_t* table, int table_ld,
                       PagesArgs* a) {
  if (!c || c->magic != kPagedMagic || !c->base || !pool_ok(pool) || !table) return FUTR_ERR_INVALID_ARG;
  if (c->n_pages != pool->n_pages || batch < 1 || table_ld < 1) return FUTR_ERR_INVALID_ARG;
  if (batch > pool->max_seqs) return FUTR_ERR_INVALID_ARG;
  *a = PagesArgs{};
  a->p = pool_view(*pool);
  const uint64_t blocks = (uint64_t)c->n_pages * c->shape.n_kv_heads * 2;
  a->c.codes = at<uint8_t>(c->base, 0);
  a->c.scales = at<float>(c->base, c->scale_offset);
  a->c.n_pages = c->n_pages;
  a->c.page = c->page;
  a->c.page_log2 = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  a->c.n_kv = c->shape.n_kv_heads;
  a->c.max_pos = c->max_pos;
  a->n_layers = c->n_layers;
  a->d = c->shape.head_dim;
  a->layer_codes = blocks * c->page * c->shape.head_dim;
  a->layer_scales = blocks;
  a->batch = batch;
  a->table = const_cast<int*>(table);
  a->table_ld = table_ld;
  return FUTR_OK;
}

}  // namespace

extern "C" {

futr_status futr_beam_workspace_size(int32_t rows, int32_t keep, size_t* bytes) {
  return guarded([&]() -> futr_status {
    if (!bytes) return FUTR_ERR_INVALID_ARG;
    if (rows < 1 || rows > kBeamMaxRows || keep < 1 || keep > kBeamMaxKeep) return FUTR_ERR_UNSUPPORTED;
    const int sms = host::sm_count();
    if (sms <= 0) return FUTR_ERR_CUDA;
    *bytes = (size_t)beam_layout(rows, keep, beam_part_ctas(sms)).total;
    return FUTR_OK;
  });
}

futr_status futr_beam_workspace_init(int32_t rows, int32_t keep, void* mem, size_t mem_bytes, futr_beam_ws* ws,
                                     void* stream) {
  return guarded([&]() -> futr_status {
    if (!ws || !mem) return FUTR_ERR_INVALID_ARG;
    size_t need = 0;
    const futr_status st = futr_beam_workspace_size(rows, keep, &need);
    if (st != FUTR_OK) return st;
    if (!aligned(mem, 256) || mem_bytes < need) return FUTR_ERR_INVALID_ARG;
    futr_beam_ws w{};
    w.rows = rows;
    w.keep = keep;
    w.ctas = beam_part_ctas(host::sm_count());
    const BeamLayout L = beam_layout(rows, keep, w.ctas);
    w.base = mem;
    w.bytes = L.total;
    w.err_offset = L.err;
    w.cnt_offset = L.cnt;
    w.row_offset = L.rows;
    w.rec_offset = L.recs;
    w.magic = kBeamWsMagic;
    const cudaStream_t s = as_stream(stream);
    // error word and counters start at zero
    if (cudaMemsetAsync(mem, 0, L.rows, s) != cudaSuccess) return FUTR_ERR_CUDA;
    uint64_t g[4];
    beam_guards(w, g);
    if (host::fill_guards_before(mem, g, 4, s) != cudaSuccess) return FUTR_ERR_CUDA;
    *ws = w;
    return FUTR_OK;
  });
}

futr_status futr_beam_select(const void* logits, int64_t ld, int32_t dtype, int32_t batch, int32_t beams,
                             int32_t vocab, const float* scores, const int32_t* done, int32_t end, int32_t keep,
                             int32_t stay, float* score_out, int32_t* parent, int32_t* token, int32_t* done_out,
                             const futr_beam_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!logits || !scores || !score_out || !parent || !token || !beam_ok(ws)) return FUTR_ERR_INVALID_ARG;
    if (dtype != FUTR_DTYPE_F32 && dtype != FUTR_DTYPE_BF16 && dtype != FUTR_DTYPE_F16) return FUTR_ERR_UNSUPPORTED;
    if (beams < 1 || beams > kBeamMaxBeams || keep < 1 || keep > kBeamMaxKeep) return FUTR_ERR_UNSUPPORTED;
    if (batch < 1 || vocab < 1 || ld < vocab) return FUTR_ERR_INVALID_ARG;
    if ((int64_t)batch * beams > ws->rows || keep > ws->keep) return FUTR_ERR_INVALID_ARG;
    if (end < -1 || end >= vocab || (done && end < 0) || (stay && keep != beams)) return FUTR_ERR_INVALID_ARG;
    if (score_out == scores && keep != beams) return FUTR_ERR_INVALID_ARG;
    if (done_out && done_out == done && keep != beams) return FUTR_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == FUTR_DTYPE_F32 ? 4 : 2)) return FUTR_ERR_INVALID_ARG;
    const int sms = host::sm_count();
    if (sms <= 0) return FUTR_ERR_CUDA;
    // the workspace has to fit the grid on the current device
    if (beam_part_ctas(sms) > ws->ctas) return FUTR_ERR_INVALID_ARG;
    BeamArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.scores = scores;
    a.done = done;
    a.batch = batch;
    a.beams = beams;
    a.vocab = vocab;
    a.end = end;
    a.keep = keep;
    a.stay = stay != 0;
    a.score_out = score_out;
    a.parent = parent;
    a.token = token;
    a.done_out = done_out;
    a.err = at<int>(ws->base, ws->err_offset);
    a.cnt = at<unsigned>(ws->base, ws->cnt_offset);
    a.rows = at<uint8_t>(ws->base, ws->row_offset);
    a.parts = at<uint8_t>(ws->base, ws->rec_offset);
    return status_of(launch_beam_select(a, dtype, sms, as_stream(stream)));
  });
}

futr_status futr_beam_check(const futr_beam_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!beam_ok(ws)) return FUTR_ERR_INVALID_ARG;
    uint64_t g[4];
    beam_guards(*ws, g);
    int word = 0;
    return read_errors(ws->base, g, 4, at<int>(ws->base, ws->err_offset), &word, 1, as_stream(stream));
  });
}

futr_status futr_kv_reorder(const futr_kv* kv, int32_t batch, const int32_t* parent, int32_t* pos, void* stream) {
  return guarded([&]() -> futr_status {
    if (!kv || kv->magic != kKvMagic || !kv->base || !parent || !pos || parent == pos) return FUTR_ERR_INVALID_ARG;
    if (batch < 1 || batch > kv->max_batch) return FUTR_ERR_INVALID_ARG;
    if (batch > kMaxBatch) return FUTR_ERR_UNSUPPORTED;
    const int sms = host::sm_count();
    if (sms <= 0) return FUTR_ERR_CUDA;
    return status_of(
        launch_kv_reorder(*kv, batch, parent, pos, at<int>(kv->base, kv->err_offset), sms, as_stream(stream)));
  });
}

futr_status futr_pages_size(int32_t n_pages, int32_t max_seqs, size_t* bytes) {
  if (!bytes || n_pages < 1 || max_seqs < 1) return FUTR_ERR_INVALID_ARG;
  if (max_seqs > kPagesMaxSeqs) return FUTR_ERR_UNSUPPORTED;
  *bytes = (size_t)pages_layout(n_pages, max_seqs).total;
  return FUTR_OK;
}

futr_status futr_pages_init(int32_t n_pages, int32_t max_seqs, void* mem, size_t mem_bytes, futr_pages* pool,
                            void* stream) {
  return guarded([&]() -> futr_status {
    if (!pool || !mem) return FUTR_ERR_INVALID_ARG;
    size_t need = 0;
    const futr_status st = futr_pages_size(n_pages, max_seqs, &need);
    if (st != FUTR_OK) return st;
    if (!aligned(mem, 256) || mem_bytes < need) return FUTR_ERR_INVALID_ARG;
    const PagesLayout L = pages_layout(n_pages, max_seqs);
    futr_pages p{};
    p.n_pages = n_pages;
    p.max_seqs = max_seqs;
    p.base = mem;
    p.bytes = L.total;
    p.refs_offset = L.refs;
    p.free_offset = L.free;
    p.plan_offset = L.plan;
    p.err_offset = L.err;
    p.magic = kPagesMagic;
    const cudaStream_t s = as_stream(stream);
    if (cudaMemsetAsync(at<uint8_t>(mem, L.err), 0, 16, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (launch_pages_init(pool_view(p), s) != cudaSuccess) return FUTR_ERR_CUDA;
    uint64_t g[4];
    pool_guards(p, g);
    if (host::fill_guards_before(mem, g, 4, s) != cudaSuccess) return FUTR_ERR_CUDA;
    *pool = p;
    return FUTR_OK;
  });
}

futr_status futr_pages_hold(const futr_paged* cache, const futr_pages* pool, int32_t batch, const int32_t* table,
                            int32_t table_ld, void* stream) {
  return guarded([&]() -> futr_status {
    PagesArgs a;
    const futr_status st = pages_args(cache, pool, batch, table, table_ld, &a);
    if (st != FUTR_OK) return st;
    return status_of(launch_pages_hold(a, as_stream(stream)));
  });
}

futr_status futr_pages_grow(const futr_paged* cache, const futr_pages* pool, int32_t batch, const int32_t* pos,
                            const int32_t* start, int32_t* table, int32_t table_ld, void* stream) {
  return guarded([&]() -> futr_status {
    PagesArgs a;
    const futr_status st = pages_args(cache, pool, batch, table, table_ld, &a);
    if (st != FUTR_OK) return st;
    if (!pos) return FUTR_ERR_INVALID_ARG;
    a.pos = const_cast<int*>(pos);
    a.start = start;
    return status_of(launch_pages_grow(a, as_stream(stream)));
  });
}

futr_status futr_pages_free(const futr_paged* cache, const futr_pages* pool, int32_t batch, const int32_t* pos,
                            int32_t* table, int32_t table_ld, int32_t window, int32_t sinks, void* stream) {
  return guarded([&]() -> futr_status {
    PagesArgs a;
    const futr_status st = pages_args(cache, pool, batch, table, table_ld, &a);
    if (st != FUTR_OK) return st;
    if (!pos || window < 0 || sinks < 0) return FUTR_ERR_INVALID_ARG;
    a.pos = const_cast<int*>(pos);
    a.window = window;
    a.sinks = sinks;
    return status_of(launch_pages_free(a, as_stream(stream)));
  });
}

futr_status futr_pages_fork(const futr_paged* cache, const futr_pages* pool, int32_t batch, const int32_t* parent,
                            int32_t* pos, int32_t* table, int32_t table_ld, void* stream) {
  return guarded([&]() -> futr_status {
    PagesArgs a;
    const futr_status st = pages_args(cache, pool, batch, table, table_ld, &a);
    if (st != FUTR_OK) return st;
    if (!parent || !pos || parent == pos) return FUTR_ERR_INVALID_ARG;
    const int sms = host::sm_count();
    if (sms <= 0) return FUTR_ERR_CUDA;
    a.parent = parent;
    a.pos = pos;
    return status_of(launch_pages_fork(a, sms, as_stream(stream)));
  });
}

futr_status futr_pages_compact(const futr_paged* cache, const futr_pages* pool, int32_t batch, int32_t* table,
                               int32_t table_ld, int32_t lo, int32_t hi, void* stream) {
  return guarded([&]() -> futr_status {
    PagesArgs a;
    const futr_status st = pages_args(cache, pool, batch, table, table_ld, &a);
    if (st != FUTR_OK) return st;
    if (lo < 0 || hi < lo || hi > pool->n_pages) return FUTR_ERR_INVALID_ARG;
    const int sms = host::sm_count();
    if (sms <= 0) return FUTR_ERR_CUDA;
    a.lo = lo;
    a.hi = hi;
    return status_of(launch_pages_compact(a, sms, as_stream(stream)));
  });
}

futr_status futr_pages_check(const futr_pages* pool, int32_t* n_free, void* stream) {
  return guarded([&]() -> futr_status {
    if (!pool_ok(pool)) return FUTR_ERR_INVALID_ARG;
    uint64_t g[4];
    pool_guards(*pool, g);
    int words[3] = {0, 0, 0};
    const futr_status st =
        read_errors(pool->base, g, 4, at<int>(pool->base, pool->err_offset), words, 3, as_stream(stream));
    if (n_free && st != FUTR_ERR_CUDA) *n_free = words[2];
    return st;
  });
}

}  // extern "C"
