// Entry points of the INT4 mixture-of-experts layer (declared in
// include/futr.h): argument checks, memory layouts, launches.
#include <cmath>
#include <cstring>

#include "moe.cuh"

namespace futr {
namespace host {
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

bool moe_shape_ok(const futr_moe_shape* s) {
  if (!s) return false;
  if (s->hidden <= 0 || s->hidden % 128 || s->inter <= 0 || s->inter % 128) return false;
  if (s->hidden > (1 << 20) || s->inter > (1 << 20)) return false;
  if (s->n_experts < 1 || s->n_experts > kMoeMaxExperts) return false;
  if (s->top_k < 1 || s->top_k > kMoeMaxTopK || s->top_k > s->n_experts) return false;
  if (s->group != kGroup) return false;
  return std::isfinite(s->rms_eps) && s->rms_eps >= 0.f;
}

uint64_t expert_bytes(const futr_moe_shape& s) { return moe_gu_bytes(s) + moe_down_bytes(s); }

bool ws_ok(const futr_moe_ws* w) { return w && w->magic == kMoeWsMagic && w->base; }

void ws_layout(const futr_moe_shape& s, int max_batch, int ctas, futr_moe_ws* w) {
  *w = futr_moe_ws{};
  w->shape = s;
  w->max_batch = max_batch;
  w->ctas = ctas;
  uint64_t off = host::region_after(0, 16);   // error words
  w->off_cnt = off;
  off = host::region_after(off, (uint64_t)(ctas + kRouterTiles) * 4);
  w->off_rms = off;
  off = host::region_after(off, (uint64_t)max_batch * (1 + 2 * s.top_k) * 4 + 4);   // factors, weights, choices, a count
  w->off_logits = off;
  off = host::region_after(off, (uint64_t)max_batch * s.n_experts * 4);
  w->off_x = off;
  off = host::region_after(off, (uint64_t)max_batch * (s.hidden / kGroup) * kRecBytes);
  w->off_act = off;
  off = host::region_after(off, (uint64_t)max_batch * s.top_k * (s.inter / kGroup) * kRecBytes);
  w->off_rec = off;
  w->bytes = host::region_after(off, (uint64_t)ctas * 2 * kMoeRecFloats * 4);
  w->blob_bytes = kHeaderBytes + expert_bytes(s) * s.n_experts;
  w->magic = kMoeWsMagic;
}

int ws_guards(const futr_moe_ws& w, uint64_t* g) {
  const uint64_t starts[] = {w.off_cnt, w.off_rms, w.off_logits, w.off_x, w.off_act, w.off_rec, w.bytes};
  std::memcpy(g, starts, sizeof(starts));
  return 7;
}

__global__ void moe_header_kernel(MoeHeader* dst, const MoeHeader h) { *dst = h; }

}  // namespace

extern "C" {

futr_status futr_moe_weights_size(const futr_moe_shape* shape, size_t* bytes) {
  if (!bytes) return FUTR_ERR_INVALID_ARG;
  if (!moe_shape_ok(shape)) return FUTR_ERR_UNSUPPORTED;
  *bytes = (size_t)(kHeaderBytes + expert_bytes(*shape) * shape->n_experts);
  return FUTR_OK;
}

futr_status futr_moe_pack(const futr_moe_shape* shape, int32_t expert, const float* wgate, const float* wup,
                          const float* wdown, const float* gain, void* blob, size_t blob_bytes, void* stream) {
  return guarded([&]() -> futr_status {
    size_t need = 0;
    const futr_status st = futr_moe_weights_size(shape, &need);
    if (st != FUTR_OK) return st;
    if (!wgate || !wup || !wdown || !blob || expert < 0 || expert >= shape->n_experts) return FUTR_ERR_INVALID_ARG;
    if (blob_bytes < need || !aligned(blob, 256)) return FUTR_ERR_INVALID_ARG;
    const cudaStream_t s = as_stream(stream);
    uint8_t* gu = at<uint8_t>(blob, kHeaderBytes + expert_bytes(*shape) * expert);
    if (launch_pack_expert(shape->hidden, shape->inter, wgate, wup, wdown, gain, gu, gu + moe_gu_bytes(*shape), s) !=
            cudaSuccess ||
        launch_moe_place(gu, expert_bytes(*shape) / kUnitBytes, s) != cudaSuccess)
      return FUTR_ERR_CUDA;
    const MoeHeader h{kMoeMagic, 1, shape->hidden, shape->inter, shape->n_experts};
    moe_header_kernel<<<1, 1, 0, s>>>(at<MoeHeader>(blob, 0), h);
    return cudaGetLastError() == cudaSuccess ? FUTR_OK : FUTR_ERR_CUDA;
  });
}

futr_status futr_moe_unpack(const futr_moe_shape* shape, const void* blob, int32_t expert, int32_t which,
                            int8_t* codes, uint16_t* scales, void* stream) {
  return guarded([&]() -> futr_status {
    if (!moe_shape_ok(shape)) return FUTR_ERR_UNSUPPORTED;
    if (!blob || !codes || !scales || expert < 0 || expert >= shape->n_experts) return FUTR_ERR_INVALID_ARG;
    if (which != FUTR_PROJ_GATE && which != FUTR_PROJ_UP && which != FUTR_PROJ_DOWN) return FUTR_ERR_INVALID_ARG;
    const uint8_t* gu = reinterpret_cast<const uint8_t*>(blob) + kHeaderBytes + expert_bytes(*shape) * expert;
    return launch_moe_unpack(shape->hidden, shape->inter, gu, gu + moe_gu_bytes(*shape), which, codes, scales,
                                as_stream(stream)) == cudaSuccess
               ? FUTR_OK
               : FUTR_ERR_CUDA;
  });
}

futr_status futr_moe_workspace_size(const futr_moe_shape* shape, int32_t max_batch, size_t* bytes) {
  return guarded([&]() -> futr_status {
    if (!bytes) return FUTR_ERR_INVALID_ARG;
    if (!moe_shape_ok(shape)) return FUTR_ERR_UNSUPPORTED;
    if (max_batch < 1 || max_batch > kMaxBatch) return FUTR_ERR_INVALID_ARG;
    const int ctas = moe_ctas();
    if (ctas <= 0) return FUTR_ERR_CUDA;
    futr_moe_ws w;
    ws_layout(*shape, max_batch, ctas, &w);
    *bytes = (size_t)w.bytes;
    return FUTR_OK;
  });
}

futr_status futr_moe_workspace_init(const futr_moe_shape* shape, int32_t max_batch, void* mem, size_t mem_bytes,
                                    futr_moe_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!ws || !mem) return FUTR_ERR_INVALID_ARG;
    size_t need = 0;
    const futr_status st = futr_moe_workspace_size(shape, max_batch, &need);
    if (st != FUTR_OK) return st;
    if (!aligned(mem, 256) || mem_bytes < need) return FUTR_ERR_INVALID_ARG;
    futr_moe_ws w;
    ws_layout(*shape, max_batch, moe_ctas(), &w);
    w.base = mem;
    const cudaStream_t s = as_stream(stream);
    // error words and counters start at zero
    if (cudaMemsetAsync(mem, 0, w.off_rms, s) != cudaSuccess) return FUTR_ERR_CUDA;
    uint64_t g[7];
    const int n = ws_guards(w, g);
    if (host::fill_guards_before(mem, g, n, s) != cudaSuccess) return FUTR_ERR_CUDA;
    *ws = w;
    return FUTR_OK;
  });
}

futr_status futr_moe_layer(const uint16_t* x, const float* gain, const uint16_t* router, const void* blob,
                           int32_t batch, const uint16_t* resid, uint16_t* y, int32_t* ids, float* weights,
                           const futr_moe_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!x || !router || !blob || !y || !ws_ok(ws)) return FUTR_ERR_INVALID_ARG;
    if (batch < 1 || batch > kMaxBatch) return FUTR_ERR_UNSUPPORTED;
    if (batch > ws->max_batch) return FUTR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(blob, 16) || !aligned(y, 16) || !aligned(resid, 16) ||
        !aligned(gain, 16) || !aligned(ids, 4) || !aligned(weights, 4))
      return FUTR_ERR_INVALID_ARG;
    if (moe_ctas() > ws->ctas) return FUTR_ERR_INVALID_ARG;   // a workspace of a smaller device
    const futr_moe_shape& s = ws->shape;
    MoeArgs a{};
    a.H = s.hidden;
    a.I = s.inter;
    a.E = s.n_experts;
    a.K = s.top_k;
    a.T = batch;
    a.renorm = s.renorm != 0;
    a.eps = s.rms_eps;
    a.x = reinterpret_cast<const __nv_bfloat16*>(x);
    a.gain = gain;
    a.router = reinterpret_cast<const __nv_bfloat16*>(router);
    a.blob = reinterpret_cast<const uint8_t*>(blob);
    a.gu_bytes = moe_gu_bytes(s);
    a.expert_bytes = expert_bytes(s);
    a.resid = reinterpret_cast<const __nv_bfloat16*>(resid);
    a.y = reinterpret_cast<__nv_bfloat16*>(y);
    a.ids = ids;
    a.weights = weights;
    a.err = at<int>(ws->base, 0);
    a.withhold = host::withhold_copy();
    a.cnt = at<unsigned>(ws->base, ws->off_cnt);
    a.rms = at<float>(ws->base, ws->off_rms);
    a.share = a.rms + ws->max_batch;
    a.choice = reinterpret_cast<int*>(a.share + (size_t)ws->max_batch * s.top_k);
    a.active = a.choice + (size_t)ws->max_batch * s.top_k;
    a.logits = at<float>(ws->base, ws->off_logits);
    a.xh = at<__half>(ws->base, ws->off_x);
    a.act = at<__half>(ws->base, ws->off_act);
    a.rec = at<float>(ws->base, ws->off_rec);
    return launch_moe(a, as_stream(stream)) == cudaSuccess ? FUTR_OK : FUTR_ERR_CUDA;
  });
}

futr_status futr_moe_check(const futr_moe_ws* ws, void* stream) {
  return guarded([&]() -> futr_status {
    if (!ws_ok(ws)) return FUTR_ERR_INVALID_ARG;
    const cudaStream_t s = as_stream(stream);
    int* err = at<int>(ws->base, 0);
    uint64_t g[7];
    const int n = ws_guards(*ws, g);
    if (host::check_guards_before(ws->base, g, n, err, s) != cudaSuccess) return FUTR_ERR_CUDA;
    int v[2] = {0, 0};
    if (cudaMemcpyAsync(v, err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
    if (v[0] == 0 && v[1] == 0) return FUTR_OK;
    if (cudaMemsetAsync(err, 0, 16, s) != cudaSuccess) return FUTR_ERR_CUDA;
    // a launch that gave up left its arrival counters mid-count
    if (v[1] != 0 && cudaMemsetAsync(at<uint8_t>(ws->base, ws->off_cnt), 0, (size_t)(ws->ctas + kRouterTiles) * 4, s) != cudaSuccess)
      return FUTR_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return FUTR_ERR_CUDA;
    return v[0] != 0 ? v[0] : FUTR_ERR_TIMEOUT;
  });
}

}  // extern "C"
