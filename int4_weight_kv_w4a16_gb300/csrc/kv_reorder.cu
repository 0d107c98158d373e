// The slots of the INT4 cache follow the chosen beams, in place: slot i takes what slot
// parent[i] held, in every layer and head.
//
// A thread takes 16 bytes at the same place of every slot's stream: it reads all that move
// before it writes any, so slots may trade places and one slot may go to several.  All of
// them are in registers at once, for as many moves as the call's batch can have: so many
// loads are in flight together (one after another through shared memory took 559 us for 32
// slots of 16 layers, 1.0 GB read and written, that take 160 here).  A stream has four runs
// (codes of keys and of values, their scales) of which the first tiles move; threads count
// through those alone.  Bound by memory: 6.3 TB/s for those, 0.93 of the copy rate.
#include "pages.cuh"

namespace futr {

namespace {

constexpr int kKrThreads = 128;

struct ReorderArgs {
  uint8_t* base;
  uint64_t stream_bytes;
  int cap, d, n_kv, n_layers, max_batch, batch;
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
  const bool bad = parent < -1 || parent >= a.batch || own < 0 || own > a.cap;
  pos = __shfl_sync(0xffffffffu, own, parent < 0 ? 0 : parent & 31);
  if (parent < 0) pos = 0;
  tiles = parent >= 0 && parent != lane ? (pos + 15) >> 4 : 0;
  return !__any_sync(0xffffffffu, bad);
}

struct Moves {
  uint64_t from[32], to[32];   // slots as offsets
  int tiles[32];               // that move
  int n, most;                 // moves, tiles of the longest
};

// The columns of all streams, C at a time in a thread, with n <= M moves.
template <int M, int C>
__device__ __forceinline__ void move_columns(const ReorderArgs& a, const Moves& mv) {
  const int tid = threadIdx.x, n = mv.n, most = mv.most;
  // columns of a stream: codes of keys, of values (d / 2 a tile each), then scales (2 each)
  const int half = a.d / 2, codes = most * half, cols = 2 * (codes + 2 * most);
  const int per = (cols + kKrThreads * C - 1) / (kKrThreads * C);
  const uint64_t code_bytes = (uint64_t)a.cap * a.d;
  const long long items = (long long)a.n_layers * a.n_kv * per;
#pragma unroll 1
  for (long long e = blockIdx.x; e < items; e += gridDim.x) {
    const int stream = (int)(e / per), first = (int)(e - (long long)stream * per) * (kKrThreads * C) + tid;
    const int layer = stream / a.n_kv, head = stream - layer * a.n_kv;
    uint8_t* at = a.base + ((uint64_t)layer * a.max_batch * a.n_kv + head) * a.stream_bytes;
    int tile[C];
    uint64_t off[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      int col = first + c * kKrThreads;
      tile[c] = 0x7fffffff;
      off[c] = 0;
      if (col < 2 * codes) {
        const bool v = col >= codes;
        if (v) col -= codes;
        tile[c] = a.d == 128 ? col >> 6 : col >> 5;
        off[c] = (v ? code_bytes / 2 : 0) + (uint64_t)col * 16;
      } else if (col < cols) {
        col -= 2 * codes;
        const bool v = col >= 2 * most;
        if (v) col -= 2 * most;
        tile[c] = col >> 1;
        off[c] = code_bytes + (v ? 2ull * a.cap : 0) + (uint64_t)col * 16;
      }
    }
    uint4 x[M][C];
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (i < n && tile[c] < mv.tiles[i]) x[i][c] = *reinterpret_cast<const uint4*>(at + mv.from[i] + off[c]);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (i < n && tile[c] < mv.tiles[i]) *reinterpret_cast<uint4*>(at + mv.to[i] + off[c]) = x[i][c];
  }
}

// M: most moves of the batch.  Few moves of up to 8 slots take more columns at once, 8 loads a
// thread at least: one slot of 32 layers at 900 positions, from memory, 13.1 us (two loads: 15.3);
// of 9 to 32 slots up to 8 moves take a column a thread (1, 2, 4 and 8 of 32, 16 layers of 1500
// positions: 21.5, 31.2, 42.8, 64.8 us; one of 4 slots 7.9).  Three CTAs an
// SM (168 registers) for 32 moves: 170 us, two (189) 187; for 16 (147 us) four would not hold
// the data (223).
template <int M>
__global__ void __launch_bounds__(kKrThreads, M > 16 ? 3 : 2) kv_reorder_kernel(const ReorderArgs a) {
  __shared__ Moves mv;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  if (tid < 32) {
    int parent, tiles, pos;
    const bool ok = read_slots(a, parent, tiles, pos);
    if (!ok) tiles = 0;
    const unsigned votes = __ballot_sync(0xffffffffu, tiles > 0);
    const uint64_t slot = (uint64_t)a.n_kv * a.stream_bytes;
    if (tiles > 0) {
      const int i = __popc(votes & ((1u << tid) - 1));
      mv.from[i] = parent * slot;
      mv.to[i] = tid * slot;
      mv.tiles[i] = tiles;
    }
    const int most = __reduce_max_sync(0xffffffffu, tiles);
    if (tid == 0) {
      mv.n = __popc(votes);
      mv.most = most;
      if (!ok) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
    }
  }
  __syncthreads();
  const int n = mv.n;
  if (n == 0) return;
  if constexpr (M > 8) {
    if (n > 8) {
      move_columns<M, 1>(a, mv);
      return;
    }
  } else {
    if (n == 1) {
      move_columns<1, 8>(a, mv);
      return;
    }
    if (n == 2) {
      move_columns<2, 4>(a, mv);
      return;
    }
    if (n <= 4) {
      move_columns<4, 2>(a, mv);
      return;
    }
  }
  if constexpr (M > 4) move_columns<8, 1>(a, mv);
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
cudaError_t kr_launch(F* f, int grid, int threads, const ReorderArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

// CTAs: those that run at once, several times, so that late ones find what is left.  Times 1,
// 2, 4 and 6: one slot 13.8, 13.1, 13.6, 14.1 us; 16 147.7, 147.2, 145.0, 148.6; 32 174, 172,
// 165, 159.
template <int M>
constexpr int kKrWaves = M > 16 ? 6 : M > 8 ? 4 : 2;

template <int M>
int kr_ctas(int dev, int sms) {
  return kKrWaves<M> * sms * remembered(occ_key(dev, M, 0, 0), [&]() {
           int n = 0;
           if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv_reorder_kernel<M>, kKrThreads, 0) != cudaSuccess ||
               n < 1) {
             cudaGetLastError();
             return 1;
           }
           return n;
         });
}

template <int M>
cudaError_t kr_run(const ReorderArgs& a, int dev, int sms, cudaStream_t st) {
  const long long most = (long long)a.n_layers * a.n_kv * (long long)((a.stream_bytes / 16 + kKrThreads - 1) / kKrThreads);
  const int ctas = kr_ctas<M>(dev, sms);
  return kr_launch(kv_reorder_kernel<M>, most < ctas ? (int)most : ctas, kKrThreads, a, st);
}

}  // namespace

cudaError_t launch_kv_reorder(const futr_kv& kv, int batch, const int* parent, int* pos, int* err, int sms,
                              cudaStream_t st) {
  ReorderArgs a{};
  a.base = static_cast<uint8_t*>(kv.base);
  a.stream_bytes = kv.stream_bytes;
  a.cap = kv.capacity;
  a.d = kv.shape.head_dim;
  a.n_kv = kv.shape.n_kv_heads;
  a.n_layers = kv.n_layers;
  a.max_batch = kv.max_batch;
  a.batch = batch;
  a.parent = parent;
  a.pos = pos;
  a.err = err;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = batch <= 4    ? kr_run<4>(a, dev, sms, st)
      : batch <= 8  ? kr_run<8>(a, dev, sms, st)
      : batch <= 16 ? kr_run<16>(a, dev, sms, st)
                    : kr_run<32>(a, dev, sms, st);
  if (e != cudaSuccess) return e;
  return kr_launch(kv_reorder_pos_kernel, 1, 32, a, st);
}

}  // namespace futr
