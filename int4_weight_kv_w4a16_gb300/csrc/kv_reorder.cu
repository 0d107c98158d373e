// The slots of the INT4 cache follow the chosen beams, in place: slot i takes what slot
// parent[i] held, in every layer and head.
//
// A thread takes 16 bytes at the same place of every slot's stream: it reads all of them
// before it writes any, so slots may trade places and one slot may go to several.
#include "pages.cuh"

namespace futr {

namespace {

constexpr int kKrThreads = 256;

struct ReorderArgs {
  uint8_t* base;
  uint64_t stream_bytes;
  int cap, d, n_kv, max_batch, batch;
  const int* parent;
  int* pos;
  int* err;
};

// Parent and tiles of 16 positions to move of slot `lane` (a full warp): tiles 0 where
// nothing moves.  False: some slot is out of range.
__device__ __forceinline__ bool read_slots(const ReorderArgs& a, int& parent, int& tiles, int& pos) {
  const int lane = threadIdx.x & 31;
  parent = lane < a.batch ? a.parent[lane] : -1;
  const int own = lane < a.batch ? a.pos[lane] : 0;
  bool bad = parent < -1 || parent >= a.batch || own < 0 || own > a.cap;
  pos = __shfl_sync(0xffffffffu, own, parent < 0 ? 0 : parent & 31);
  if (parent < 0) pos = 0;
  tiles = parent >= 0 && parent != lane ? (pos + 15) >> 4 : 0;
  return !__any_sync(0xffffffffu, bad);
}

__global__ void __launch_bounds__(kKrThreads) kv_reorder_kernel(const ReorderArgs a) {
  extern __shared__ uint4 hold[];   // [slots that move][kKrThreads]
  __shared__ int s_parent[32], s_tiles[32], s_ok;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  if (tid < 32) {
    int parent, tiles, pos;
    const bool ok = read_slots(a, parent, tiles, pos);
    s_parent[tid] = parent;
    s_tiles[tid] = ok ? tiles : 0;
    if (tid == 0) {
      s_ok = ok;
      if (!ok) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
    }
  }
  __syncthreads();
  if (!s_ok) return;
  const int h = blockIdx.y % a.n_kv, layer = blockIdx.y / a.n_kv;
  const uint64_t off = ((uint64_t)blockIdx.x * kKrThreads + tid) * 16;
  if (off >= a.stream_bytes) return;
  const uint64_t codes = (uint64_t)a.cap * a.d;
  const int tile = off < codes ? (int)(off % (codes / 2) / (8 * a.d)) : (int)((off - codes) % (2ull * a.cap) / 32);
  uint8_t* at = a.base + (((uint64_t)layer * a.max_batch) * a.n_kv + h) * a.stream_bytes + off;
  const uint64_t slot = (uint64_t)a.n_kv * a.stream_bytes;
  for (int b = 0; b < a.batch; ++b)
    if (tile < s_tiles[b]) hold[b * kKrThreads + tid] = *reinterpret_cast<const uint4*>(at + s_parent[b] * slot);
  for (int b = 0; b < a.batch; ++b)
    if (tile < s_tiles[b]) *reinterpret_cast<uint4*>(at + b * slot) = hold[b * kKrThreads + tid];
}

// The positions follow, once no CTA above reads them.
__global__ void kv_reorder_pos_kernel(const ReorderArgs a) {
  pdl_trigger();
  pdl_wait();
  int parent, tiles, pos;
  const bool ok = read_slots(a, parent, tiles, pos);
  if (ok && (int)threadIdx.x < a.batch) a.pos[threadIdx.x] = pos;
}

template <class F>
cudaError_t kr_launch(F* f, dim3 grid, int threads, size_t smem, const ReorderArgs& a, cudaStream_t st) {
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
  return cudaLaunchKernelEx(&cfg, f, a);
}

}  // namespace

cudaError_t launch_kv_reorder(const futr_kv& kv, int batch, const int* parent, int* pos, int* err, cudaStream_t st) {
  ReorderArgs a{};
  a.base = static_cast<uint8_t*>(kv.base);
  a.stream_bytes = kv.stream_bytes;
  a.cap = kv.capacity;
  a.d = kv.shape.head_dim;
  a.n_kv = kv.shape.n_kv_heads;
  a.max_batch = kv.max_batch;
  a.batch = batch;
  a.parent = parent;
  a.pos = pos;
  a.err = err;
  static DeviceOnce configured;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.done(dev)) {
    e = cudaFuncSetAttribute(kv_reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * kKrThreads * 16);
    if (e != cudaSuccess) return e;
    configured.mark(dev);
  }
  const dim3 grid((unsigned)((kv.stream_bytes / 16 + kKrThreads - 1) / kKrThreads),
                  (unsigned)(kv.n_layers * kv.shape.n_kv_heads));
  e = kr_launch(kv_reorder_kernel, grid, kKrThreads, (size_t)batch * kKrThreads * 16, a, st);
  if (e != cudaSuccess) return e;
  return kr_launch(kv_reorder_pos_kernel, dim3(1), 32, 0, a, st);
}

}  // namespace futr
