// Entry points of the paged 8-bit cache (declared in include/futr.h): argument
// checks, memory layouts, launches.
#include <cmath>
#include <cstring>

#include "paged.cuh"

namespace futr {
namespace host {
bool shape_valid(const futr_shape* s);
bool withhold_copy();
uint64_t region_after(uint64_t off, uint64_t size);
cudaError_t fill_guards_before(void* base, const uint64_t* starts, int n, cudaStream_t st);
cudaError_t check_guards_before(void* base, const uint64_t* starts, int n, int* err, cudaStream_t st);
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

struct CacheLayout {
  uint64_t blocks, scales, rope, err, total;
};

futr_status cache_layout(const futr_shape* s, int n_layers, int n_pages, int page, int max_pos, CacheLayout* L) {
  if (!host::shape_valid(s)) return FUTR_ERR_UNSUPPORTED;
  if (n_layers < 1 || n_pages < 1 || max_pos < 1) return FUTR_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FUTR_ERR_UNSUPPORTED;
  if (max_pos > kPagedMaxPos) return FUTR_ERR_UNSUPPORTED;
  // a (page, kv-head) block is one step of the copies' outermost coordinate
  const uint64_t lp = (uint64_t)n_layers * (uint64_t)n_pages;
  if (lp * (uint64_t)s->n_kv_heads >= (1ull << 31)) return FUTR_ERR_UNSUPPORTED;
  L->blocks = lp * s->n_kv_heads;
  uint64_t off = host::region_after(0, L->blocks * 2 * page * s->head_dim);
  L->scales = off;
  off = host::region_after(off, L->blocks * 8);
  L->rope = off;
  off = host::region_after(off, (uint64_t)max_pos * (s->head_dim / 2) * 8);
  L->err = off;
  L->total = host::region_after(off, 16);
  return FUTR_OK;
}

void cache_guards(const futr_paged& c, uint64_t* g) {
  g[0] = c.scale_offset;
  g[1] = c.rope_offset;
  g[2] = c.err_offset;
  g[3] = c.bytes;
}

bool cache_ok(const futr_paged* c) { return c && c->magic == kPagedMagic && c->base; }
bool ws_ok(const futr_paged_ws* w) { return w && w->magic == kPagedWsMagic && w->base; }

struct WsLayout {
  uint64_t err, rec, total;   // counters at 0
};

WsLayout ws_layout(int head_dim, int sms) {
  WsLayout L;
  L.err = host::region_after(0, (uint64_t)paged_attn_ctas(sms) * 4);
  L.rec = host::region_after(L.err, 16);
  L.total = host::region_after(L.rec, (uint64_t)paged_rec_floats(head_dim, sms) * 4);
  return L;
}

PagedView view(const futr_paged& c, int layer) {
  PagedView v{};
  const uint64_t per_layer = (uint64_t)c.n_pages * c.shape.n_kv_heads;
  v.codes = at<uint8_t>(c.base, (uint64_t)layer * per_layer * 2 * c.page * c.shape.head_dim);
  v.scales = at<float>(c.base, c.scale_offset + (uint64_t)layer * per_layer * 8);
  v.rope = c.rope ? at<const float2>(c.base, c.rope_offset) : nullptr;
  v.n_pages = c.n_pages;
  v.page = c.page;
  v.page_log2 = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
  v.n_kv = c.shape.n_kv_heads;
  v.max_pos = c.max_pos;
  return v;
}

// The arguments that append and attention share.
futr_status check_rows(const futr_paged* c, int layer, int batch, const int32_t* pos, const int32_t* start, int n_rows,
                       const int32_t* table, int table_ld, int dtype) {
  if (!cache_ok(c) || !pos || !table) return FUTR_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->n_layers || batch < 1 || n_rows < 0 || table_ld < 1) return FUTR_ERR_INVALID_ARG;
  if (!start && n_rows != batch) return FUTR_ERR_INVALID_ARG;
  if (dtype != FUTR_DTYPE_BF16 && dtype != FUTR_DTYPE_F16) return FUTR_ERR_UNSUPPORTED;
  return FUTR_OK;
}

// Row strides of 16-bit rows of `width` elements that are read 8 at a time.
bool rows_ok(const void* p, int64_t ld, int width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0; }

}  // namespace

extern "C" {

futr_status futr_paged_size(const futr_shape* shape, int32_t n_layers, int32_t n_pages, int32_t page,
                            int32_t max_pos, size_t* bytes) {
  if (!bytes) return FUTR_ERR_INVALID_ARG;
  CacheLayout L;
  const futr_status st = cache_layout(shape, n_layers, n_pages, page, max_pos, &L);
  if (st == FUTR_OK) *bytes = (size_t)L.total;
  return st;
}

futr_status futr_paged_init(const futr_shape* shape, int32_t n_layers, int32_t n_pages, int32_t page, int32_t max_pos,
                            int32_t rope, void* mem, size_t mem_bytes, futr_paged* cache, void* stream) {
  return guarded([&]() -> futr_status {
    if (!cache || !mem) return FUTR_ERR_INVALID_ARG;
    CacheLayout L;
    const futr_status st = cache_layout(shape, n_layers, n_pages, page, max_pos, &L);
    if (st != FUTR_OK) return st;
    if (!aligned(mem, 256) || mem_bytes < L.total) return FUTR_ERR_INVALID_ARG;
    const cudaStream_t s = as_stream(stream);
    if (cudaMemsetAsync(mem, 0, L.total, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (launch_rope_table(at<float2>(mem, L.rope), max_pos, shape->head_dim, shape->rope_theta, s) != cudaSuccess)
      return FUTR_ERR_CUDA;
    futr_paged d{};
    d.shape = *shape;
    d.n_layers = n_layers;
    d.n_pages = n_pages;
    d.page = page;
    d.max_pos = max_pos;
    d.rope = rope != 0;
    d.base = mem;
    d.bytes = L.total;
    d.scale_offset = L.scales;
    d.rope_offset = L.rope;
    d.err_offset = L.err;
    d.magic = kPagedMagic;
    CUtensorMap map;
    static_assert(sizeof(map) == sizeof(d.copy_map), "a tensor map fills the descriptor's field");
    if (!make_paged_map(&map, mem, shape->head_dim, page, L.blocks)) return FUTR_ERR_CUDA;
    std::memcpy(d.copy_map, &map, sizeof(map));
    uint64_t g[4];
    cache_guards(d, g);
    if (host::fill_guards_before(mem, g, 4, s) != cudaSuccess) return FUTR_ERR_CUDA;
    *cache = d;
    return FUTR_OK;
  });
}

futr_status futr_paged_append(const futr_paged* cache, int32_t layer, int32_t batch, const int32_t* pos,
                              const int32_t* start, int32_t n_rows, const int32_t* table, int32_t table_ld,
                              const void* k, int64_t ld_k, const void* v, int64_t ld_v, int32_t dtype, void* stream) {
  return guarded([&]() -> futr_status {
    const futr_status st = check_rows(cache, layer, batch, pos, start, n_rows, table, table_ld, dtype);
    if (st != FUTR_OK) return st;
    if (n_rows == 0) return FUTR_OK;
    const int width = cache->shape.n_kv_heads * cache->shape.head_dim;
    if (!rows_ok(k, ld_k, width) || !rows_ok(v, ld_v, width)) return FUTR_ERR_INVALID_ARG;
    const PagedRows r{pos, start, table, batch, n_rows, table_ld};
    const cudaError_t e =
        launch_paged_append(view(*cache, layer), r, cache->shape.head_dim, dtype, k, ld_k, v, ld_v,
                            at<int>(cache->base, cache->err_offset), as_stream(stream));
    return e == cudaSuccess ? FUTR_OK : FUTR_ERR_CUDA;
  });
}

futr_status futr_paged_workspace_size(const futr_shape* shape, size_t* bytes) {
  return guarded([&]() -> futr_status {
    if (!bytes) return FUTR_ERR_INVALID_ARG;
    if (!host::shape_valid(shape)) return FUTR_ERR_UNSUPPORTED;
    const int sms = paged_attn_sms();
    if (sms <= 0) return FUTR_ERR_CUDA;
    *bytes = (size_t)ws_layout(shape->head_dim, sms).total;
    return FUTR_OK;
  });
}

futr_status futr_paged_workspace_init(const futr_shape* shape, void* mem, size_t mem_bytes, futr_paged_ws* ws,
                                      void* stream) {
  return guarded([&]() -> futr_status {
    if (!ws || !mem) return FUTR_ERR_INVALID_ARG;
    size_t need = 0;
    const futr_status st = futr_paged_workspace_size(shape, &need);
    if (st != FUTR_OK) return st;
    if (!aligned(mem, 256) || mem_bytes < need) return FUTR_ERR_INVALID_ARG;
    futr_paged_ws w{};
    w.head_dim = shape->head_dim;
    const int sms = paged_attn_sms();
    const WsLayout L = ws_layout(shape->head_dim, sms);
    w.ctas = paged_attn_ctas(sms);
    w.base = mem;
    w.bytes = need;
    w.err_offset = L.err;
    w.rec_offset = L.rec;
    w.magic = kPagedWsMagic;
    const cudaStream_t s = as_stream(stream);
    // counters and error words start at zero
    if (cudaMemsetAsync(mem, 0, w.rec_offset, s) != cudaSuccess) return FUTR_ERR_CUDA;
    const uint64_t g[3] = {w.err_offset, w.rec_offset, w.bytes};
    if (host::fill_guards_before(mem, g, 3, s) != cudaSuccess) return FUTR_ERR_CUDA;
    *ws = w;
    return FUTR_OK;
  });
}

futr_status futr_paged_attention(const futr_paged* cache, int32_t layer, int32_t batch, const int32_t* pos,
                                 const int32_t* start, int32_t n_rows, const int32_t* table, int32_t table_ld,
                                 const void* q, int64_t ld_q, void* out, int64_t ld_out, int32_t dtype, float scale,
                                 int32_t window, const futr_paged_ws* ws, void* stream) {
  return futr_paged_attention_sinks(cache, layer, batch, pos, start, n_rows, table, table_ld, q, ld_q, out, ld_out, dtype,
                                    scale, window, 0, ws, stream);
}

futr_status futr_paged_attention_sinks(const futr_paged* cache, int32_t layer, int32_t batch, const int32_t* pos,
                                       const int32_t* start, int32_t n_rows, const int32_t* table, int32_t table_ld,
                                       const void* q, int64_t ld_q, void* out, int64_t ld_out, int32_t dtype,
                                       float scale, int32_t window, int32_t sinks, const futr_paged_ws* ws,
                                       void* stream) {
  return guarded([&]() -> futr_status {
    const futr_status st = check_rows(cache, layer, batch, pos, start, n_rows, table, table_ld, dtype);
    if (st != FUTR_OK) return st;
    if (!ws_ok(ws) || ws->head_dim != cache->shape.head_dim || window < 0 || sinks < 0) return FUTR_ERR_INVALID_ARG;
    if (!(scale >= 0.f && std::isfinite(scale * 1.5f))) return FUTR_ERR_INVALID_ARG;   // times log2(e) below
    if (n_rows == 0) return FUTR_OK;
    const futr_shape& s = cache->shape;
    const int width = s.n_q_heads * s.head_dim;
    if (!rows_ok(q, ld_q, width) || !rows_ok(out, ld_out, width) || q == out) return FUTR_ERR_INVALID_ARG;
    // the workspace has to fit the grid on the current device
    if (paged_attn_ctas(paged_attn_sms()) > ws->ctas) return FUTR_ERR_INVALID_ARG;
    PagedAttnArgs a{};
    a.c = view(*cache, layer);
    a.r = PagedRows{pos, start, table, batch, n_rows, table_ld};
    a.q = q;
    a.out = out;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.Hkv = s.n_kv_heads;
    a.G = s.n_q_heads / s.n_kv_heads;
    a.window = window < cache->max_pos ? window : 0;   // a window of every position is none
    if (a.window > 0) {
      a.sinks = sinks < cache->max_pos ? sinks : cache->max_pos;
      a.sink_tiles = (a.sinks + 127) / 128;
      a.sink_pages = (a.sinks + cache->page - 1) / cache->page;
    }
    a.block0 = (long long)layer * cache->n_pages * s.n_kv_heads;
    const double sc = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)s.head_dim);
    a.scale_log2 = (float)(sc * 1.4426950408889634);
    a.rec = at<float>(ws->base, ws->rec_offset);
    a.cnt = at<unsigned>(ws->base, 0);
    a.err = at<int>(cache->base, cache->err_offset);
    a.stop = at<int>(ws->base, ws->err_offset);
    a.withhold = host::withhold_copy();
    CUtensorMap map;
    std::memcpy(&map, cache->copy_map, sizeof(map));
    return launch_paged_attention(a, map, s.head_dim, dtype, as_stream(stream)) == cudaSuccess ? FUTR_OK
                                                                                               : FUTR_ERR_CUDA;
  });
}

futr_status futr_paged_check(const futr_paged* cache, const futr_paged_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!cache_ok(cache) || (ws && !ws_ok(ws))) return FUTR_ERR_INVALID_ARG;
    const cudaStream_t s = as_stream(stream);
    int* err = at<int>(cache->base, cache->err_offset);
    uint64_t g[4];
    cache_guards(*cache, g);
    if (host::check_guards_before(cache->base, g, 4, err, s) != cudaSuccess) return FUTR_ERR_CUDA;
    int* stop = ws ? at<int>(ws->base, ws->err_offset) : nullptr;
    if (ws) {
      const uint64_t gw[3] = {ws->err_offset, ws->rec_offset, ws->bytes};
      if (host::check_guards_before(ws->base, gw, 3, stop, s) != cudaSuccess) return FUTR_ERR_CUDA;
    }
    int v = 0, w[2] = {0, 0};
    if (cudaMemcpyAsync(&v, err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (ws && cudaMemcpyAsync(w, stop, sizeof(w), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (v == 0 && w[0] == 0 && w[1] == 0) return FUTR_OK;
    if (v != 0 && cudaMemsetAsync(err, 0, 16, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if ((w[0] != 0 || w[1] != 0) && cudaMemsetAsync(stop, 0, 16, s) != cudaSuccess) return FUTR_ERR_CUDA;
    // a launch that gave up left its arrival counters mid-count
    if (w[1] != 0 && cudaMemsetAsync(ws->base, 0, (size_t)ws->ctas * 4, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
    return v != 0 ? v : w[0] != 0 ? w[0] : FUTR_ERR_TIMEOUT;
  });
}

}  // extern "C"
