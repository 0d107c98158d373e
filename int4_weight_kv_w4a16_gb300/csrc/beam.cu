// The best continuations of each prompt's beams:
//   value(w, v) = score_w + x_wv - L_w,   L_w = log sum_u exp(x_wu)
// the `keep` largest of a prompt's beams * vocab values, equal ones by (w, v).
//
// L_w is the same for a whole row, so a row's candidates are its `keep` largest
// logits (equal ones by the lowest token), compared as they are; only those meet the
// other beams' in fp64.  One pass over the logits:
//   parts  a CTA takes a part of a row in tiles of 4096, a thread 16 logits of a tile in
//          registers: running maximum and sum of exponentials per thread, and every logit
//          that reaches a threshold goes to a list in shared memory.  The threshold starts
//          at (about) the keep-th largest of the 256 threads' maxima of the first tile: so
//          many logits reach it at least, and few more.  A list that fills up is cut down
//          to its keep largest, and the threshold follows.
//   rows   the parts' sums and lists of a row become one.
//   beams  the rows' candidates of a prompt, by value.
// A list's entries are keys (logit in an order-preserving 32-bit form, then the inverted
// token), all different, so the order in which threads add to it has no effect.
//
// Selecting the k largest of a list: bisection of the key's value, one count over the
// CTA a step, until k keys are at or above it.
#include <cfloat>
#include <climits>
#include <cstring>

#include "beam.cuh"

namespace futr {

namespace {

constexpr int kBmThreads = 256, kBmWarps = kBmThreads / 32;
constexpr int kBmPer = 16;                        // logits of a thread in a tile
constexpr int kBmTile = kBmThreads * kBmPer;
constexpr int kBmList = 1024;                     // entries of a part's list
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bm_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving unsigned form of a float (no NaN; -0 counts as +0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ (~(uint32_t)((int32_t)o >> 31) | 0x80000000u));
}
constexpr uint32_t kLowest = 0x00800000u;   // ordered(-FLT_MAX)

__device__ __forceinline__ unsigned long long ordered64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return u ^ ((unsigned long long)((long long)u >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ unsigned long long make_key(float x, int v) {
  return ((unsigned long long)ordered(x) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}
__device__ __forceinline__ float key_logit(unsigned long long k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_token(unsigned long long k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

// Sum over the CTA; `turn` alternates between calls (two sets of words).
__device__ __forceinline__ int cta_sum(int v, int* words, int turn) {
  const int s = __reduce_add_sync(0xffffffffu, v);
  int* w = words + (turn & 1) * kBmWarps;
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = s;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kBmWarps; ++i) t += w[i];
  return t;
}

// The value T that exactly k of the CTA's keys reach (at most N a thread, 0 = none), all
// different; at most k keys: 1 (every key reaches it).  `turn` counts the sums made.
template <int N>
__device__ __forceinline__ unsigned long long select_key(const unsigned long long (&key)[N], int k, int* words,
                                                         int& turn) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) n += key[i] != 0;
  if (cta_sum(n, words, turn++) <= k) return 1;
  // invariant: more than k keys reach lo, fewer than k reach hi
  unsigned long long lo = 1, hi = ~0ull;
  while (hi - lo > 1) {
    const unsigned long long mid = lo + ((hi - lo) >> 1);
    n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += key[i] >= mid;
    n = cta_sum(n, words, turn++);
    if (n == k) return mid;
    if (n > k)
      lo = mid;
    else
      hi = mid;
  }
  return hi;   // not reached: keys differ, so some value has exactly k above it
}

template <int kType>
struct Vec;
template <>
struct Vec<FUTR_DTYPE_F32> {
  using T = float;
};
template <>
struct Vec<FUTR_DTYPE_BF16> {
  using T = uint16_t;
};
template <>
struct Vec<FUTR_DTYPE_F16> {
  using T = uint16_t;
};

template <int kType>
__device__ __forceinline__ float logit_of(typename Vec<kType>::T u) {
  if constexpr (kType == FUTR_DTYPE_F32)
    return u;
  else if constexpr (kType == FUTR_DTYPE_BF16)
    return __uint_as_float((uint32_t)u << 16);
  else
    return __half2float(__ushort_as_half(u));
}

// The W logits from token W * vec on (vec < v1; -inf behind the row's end): one 16-byte load,
// or two that a row off such a boundary lies across; single ones at its ends.
template <int kType>
__device__ __forceinline__ void load_vec(const typename Vec<kType>::T* x, int vec, int v1, int vocab, float* v) {
  using T = typename Vec<kType>::T;
  constexpr int W = 16 / sizeof(T);
  const long long e = (long long)vec * W;
  const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15), off = shift / (int)sizeof(T);
  uint32_t u[9] = {};
  if (vec < v1 && shift == 0 && e + W <= vocab) {
    const uint4 p = __ldcs(reinterpret_cast<const uint4*>(x + e));
    u[0] = p.x, u[1] = p.y, u[2] = p.z, u[3] = p.w;
  } else if (vec < v1 && shift != 0 && e >= off && e - off + 2 * W <= vocab) {
    const uint4* a = reinterpret_cast<const uint4*>(x + e - off);
    const uint4 p = a[0], q = a[1];
    u[0] = p.x, u[1] = p.y, u[2] = p.z, u[3] = p.w, u[4] = q.x, u[5] = q.y, u[6] = q.z, u[7] = q.w;
    if (shift & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
    }
    if (shift & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(u[i], u[i + 1], (shift & 3) * 8);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = vec < v1 && e + i < vocab ? logit_of<kType>(x[e + i]) : -INFINITY;
    return;
  }
  T t[W];
  memcpy(t, u, 16);
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = logit_of<kType>(t[i]);
}

// Rows that are not read: without a finite score, or ended.
__device__ __forceinline__ bool row_read(const BeamArgs& a, int row) {
  const float s = a.scores[row];
  return s >= -FLT_MAX && s <= FLT_MAX && !(a.done && a.done[row] != 0);
}

template <int kType>
__global__ void __launch_bounds__(kBmThreads) beam_parts_kernel(const BeamArgs a) {
  using T = typename Vec<kType>::T;
  constexpr int W = 16 / sizeof(T);       // logits of a 16-byte vector
  constexpr int NV = kBmPer / W;          // vectors of a thread in a tile
  __shared__ unsigned long long list[kBmList];
  __shared__ int words[2 * kBmWarps];
  __shared__ int s_n[3];                  // entries that a tile adds, three tiles in turn
  __shared__ float s_m[kBmWarps];
  __shared__ double s_s[kBmWarps];
  __shared__ int s_out;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.splits, part = blockIdx.x % a.splits, K = a.keep;
  pdl_trigger();
  pdl_wait();
  if (!row_read(a, row)) return;
  uint8_t* rec = a.parts + ((size_t)row * a.splits + part) * beam_record(K);
  // the row in vectors of W logits from its first on, wherever it lies: equal rows have
  // equal sums
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.ld;
  const int nv = (a.vocab - 1) / W + 1;
  const int v0 = (int)((long long)nv * part / a.splits), v1 = (int)((long long)nv * (part + 1) / a.splits);
  if (tid < 3) s_n[tid] = 0;
  if (tid == 0) s_out = 0;
  __syncthreads();
  int turn = 0, n = 0, tile = 0;          // sums made, entries of the list, tiles
  float m = -INFINITY, s = 0.f;
  unsigned long long thr = 1;
  float thr_x = -FLT_MAX;                 // a logit below it does not reach thr
  for (int at = v0; at < v1; at += kBmThreads * NV, ++tile) {
    float v[kBmPer];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_vec<kType>(x, at + tid + kBmThreads * j, v1, a.vocab, v + j * W);
    float top = v[0];
#pragma unroll
    for (int i = 1; i < kBmPer; ++i) top = fmaxf(top, v[i]);
    if (top > m) {
      s *= bm_ex2((m - top) * kLog2e);    // (the first time 2^-inf = 0)
      m = top;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kBmPer; i += 2) {
      s0 += bm_ex2((v[i] - ref) * kLog2e);
      s1 += bm_ex2((v[i + 1] - ref) * kLog2e);
    }
    s += s0 + s1;                         // a NaN or +inf in the row makes it a NaN
    if (tile == 0) {
      // the threshold: K or a few more of the threads' maxima reach it
      const uint32_t o = ordered(top);
      uint32_t lo = kLowest, hi = 0xFF7FFFFFu;   // ordered(FLT_MAX)
      if (cta_sum(o >= lo, words, turn++) > K) {
        while (lo < hi) {
          const uint32_t mid = lo + ((hi - lo + 1) >> 1);
          const int c = cta_sum(o >= mid, words, turn++);
          if (c >= K) lo = mid; else hi = mid - 1;
          if (c >= K && c <= K + K / 4) break;
        }
        thr = (unsigned long long)lo << 32;
        thr_x = unordered(lo);
      }
    }
    auto token = [&](int i) { return (at + tid + kBmThreads * (i / W)) * W + i % W; };
    unsigned reach = 0;
    if (top >= thr_x) {
#pragma unroll
      for (int i = 0; i < kBmPer; ++i) {
        if (v[i] >= thr_x && make_key(v[i], token(i)) >= thr) reach |= 1u << i;
      }
    }
    const int c = __popc(reach);
    int* counter = &s_n[tile % 3];
    int to = 0;
    if (c) to = atomicAdd(counter, c);
    __syncthreads();
    const int more = *counter;
    if (tid == 0) s_n[(tile + 2) % 3] = 0;   // last read before this tile's barrier, next used two tiles on
    if (n + more <= kBmList) {
      to += n;
#pragma unroll
      for (int i = 0; i < kBmPer; ++i)
        if (reach >> i & 1)
          list[to++] = make_key(v[i], token(i));
      n += more;
    } else {
      // too many at once: one logit a thread at a time, the list cut down between
#pragma unroll 1
      for (int i = -1; i < kBmPer; ++i) {
        if (i >= 0) {
          float xi = v[0];
#pragma unroll
          for (int q = 1; q < kBmPer; ++q) xi = q == i ? v[q] : xi;
          const unsigned long long key = (reach >> i & 1) ? make_key(xi, token(i)) : 0;
          const bool in = key >= thr && key != 0;
          const unsigned votes = __ballot_sync(0xffffffffu, in);
          int* w = words + (turn++ & 1) * kBmWarps;
          if (lane == 0) w[warp] = __popc(votes);
          __syncthreads();
          int before = 0, all = 0;
#pragma unroll
          for (int q = 0; q < kBmWarps; ++q) {
            before += q < warp ? w[q] : 0;
            all += w[q];
          }
          if (in) list[n + before + __popc(votes & ((1u << lane) - 1))] = key;
          n += all;
        }
        if (n > kBmList - kBmThreads) {
          __syncthreads();
          unsigned long long key[kBmList / kBmThreads];
#pragma unroll
          for (int q = 0; q < kBmList / kBmThreads; ++q) {
            const int p = tid + q * kBmThreads;
            key[q] = p < n ? list[p] : 0;
          }
          thr = select_key(key, K, words, turn);
          thr_x = unordered((uint32_t)(thr >> 32) < kLowest ? kLowest : (uint32_t)(thr >> 32));
          __syncthreads();   // every key has been read
          if (tid == 0) s_out = 0;
          __syncthreads();
#pragma unroll
          for (int q = 0; q < kBmList / kBmThreads; ++q)
            if (key[q] >= thr) list[atomicAdd(&s_out, 1)] = key[q];
          __syncthreads();
          n = s_out;
        }
      }
    }
  }
  // the part's K largest
  __syncthreads();
  {
    unsigned long long key[kBmList / kBmThreads];
#pragma unroll
    for (int q = 0; q < kBmList / kBmThreads; ++q) {
      const int p = tid + q * kBmThreads;
      key[q] = p < n ? list[p] : 0;
    }
    thr = select_key(key, K, words, turn);
    if (tid == 0) s_out = 0;
    __syncthreads();
    unsigned long long* out = reinterpret_cast<unsigned long long*>(rec + 16);
#pragma unroll
    for (int q = 0; q < kBmList / kBmThreads; ++q)
      if (key[q] >= thr) out[atomicAdd(&s_out, 1)] = key[q];
    __syncthreads();
    for (int i = s_out + tid; i < K; i += kBmThreads) out[i] = 0;
  }
  // its maximum and sum
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBmWarps; ++i) M = fmaxf(M, s_m[i]);
  // (a thread without a logit has the sum 0, or a NaN)
  double S = m == -INFINITY ? (double)s : (double)s * (double)bm_ex2((m - M) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
  if (lane == 0) s_s[warp] = S;
  __syncthreads();
  if (tid == 0) {
    double sum = 0.0;
    for (int i = 0; i < kBmWarps; ++i) sum += s_s[i];
    *reinterpret_cast<float*>(rec) = M;
    reinterpret_cast<double*>(rec)[1] = sum;
  }
}

// A row's parts become one: log-sum, and the K largest keys.  A row with an infinity or
// NaN has no keys.
constexpr int kBmMaxKeys = 16;   // keys of a thread: up to 64 parts of 64 keys

__global__ void __launch_bounds__(kBmThreads) beam_rows_kernel(const BeamArgs a) {
  __shared__ int words[2 * kBmWarps];
  __shared__ int s_out;
  __shared__ double s_lse;
  const int tid = threadIdx.x, row = blockIdx.x, K = a.keep;
  pdl_trigger();
  pdl_wait();
  uint8_t* rec = a.rows + (size_t)row * beam_record(K);
  unsigned long long* out = reinterpret_cast<unsigned long long*>(rec + 16);
  if (!row_read(a, row)) {
    const float sc = a.scores[row];
    const bool bad = !(sc <= FLT_MAX);   // NaN or +inf
    const bool ended = !bad && sc >= -FLT_MAX;   // (a finite score that is not read: done)
    for (int i = tid; i < K; i += kBmThreads) out[i] = i == 0 && ended ? make_key(0.f, a.end) : 0;
    if (tid == 0) {
      reinterpret_cast<double*>(rec)[1] = 0.0;
      if (bad) set_err(a.err, FUTR_ERR_NOT_FINITE);
    }
    return;
  }
  const uint8_t* parts = a.parts + (size_t)row * a.splits * beam_record(K);
  if (tid == 0) s_out = 0;
  if (tid < 32) {
    float M = -INFINITY;
    for (int p = tid; p < a.splits; p += 32) M = fmaxf(M, *reinterpret_cast<const float*>(parts + p * beam_record(K)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    double S = 0.0;
    for (int p = tid; p < a.splits; p += 32) {
      const float m = *reinterpret_cast<const float*>(parts + p * beam_record(K));
      const double s = reinterpret_cast<const double*>(parts + p * beam_record(K))[1];
      S += m == -INFINITY ? s : s * exp((double)m - (double)M);   // (no logit: 0, or a NaN)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    if (tid == 0) {
      const bool bad = !(S <= DBL_MAX) || M == INFINITY;
      if (bad) set_err(a.err, FUTR_ERR_NOT_FINITE);
      s_lse = bad || M == -INFINITY ? (double)INFINITY : (double)M + log(S);
    }
  }
  __syncthreads();
  const double lse = s_lse;
  int turn = 0;
  unsigned long long key[kBmMaxKeys];
#pragma unroll
  for (int q = 0; q < kBmMaxKeys; ++q) {
    const int i = tid + q * kBmThreads;
    key[q] = 0;
    if (i < a.splits * K && lse < (double)INFINITY)
      key[q] = reinterpret_cast<const unsigned long long*>(parts + (size_t)(i / K) * beam_record(K) + 16)[i % K];
  }
  const unsigned long long thr = select_key(key, K, words, turn);
#pragma unroll
  for (int q = 0; q < kBmMaxKeys; ++q)
    if (key[q] >= thr) out[atomicAdd(&s_out, 1)] = key[q];
  __syncthreads();
  for (int i = s_out + tid; i < K; i += kBmThreads) out[i] = 0;
  if (tid == 0) reinterpret_cast<double*>(rec)[1] = lse;
}

// A prompt's beams: the K best of their candidates, by value, equal ones by (w, v).
constexpr int kBmCands = kBeamMaxBeams * kBeamMaxKeep / kBmThreads;   // of a thread

__global__ void __launch_bounds__(kBmThreads) beam_pick_kernel(const BeamArgs a) {
  __shared__ int words[2 * kBmWarps];
  __shared__ int s_out;
  __shared__ unsigned long long s_val[kBeamMaxKeep];      // the chosen: ordered value, place (w, v), value
  __shared__ long long s_at[kBeamMaxKeep];
  __shared__ float s_f[kBeamMaxKeep];
  __shared__ int s_rank[kBeamMaxKeep];
  const int tid = threadIdx.x, b = blockIdx.x, W = a.beams, K = a.keep;
  pdl_trigger();
  pdl_wait();
  if (tid == 0) s_out = 0;
  unsigned long long val[kBmCands];
  long long at[kBmCands];
  float f[kBmCands];
#pragma unroll
  for (int q = 0; q < kBmCands; ++q) {
    const int i = tid + q * kBmThreads, w = i / K;
    val[q] = 0;
    if (i < W * K) {
      const uint8_t* rec = a.rows + ((size_t)b * W + w) * beam_record(K);
      const unsigned long long key = reinterpret_cast<const unsigned long long*>(rec + 16)[i % K];
      if (key != 0) {
        const double v = (double)a.scores[b * W + w] + ((double)key_logit(key) - reinterpret_cast<const double*>(rec)[1]);
        val[q] = ordered64(v);
        at[q] = ((long long)w << 32) | (uint32_t)key_token(key);
        f[q] = (float)v;
      }
    }
  }
  // the largest value that at least K candidates reach
  int turn = 0, n = 0;
#pragma unroll
  for (int q = 0; q < kBmCands; ++q) n += val[q] != 0;
  unsigned long long lo = 1;
  int left = 0;                 // of those at lo itself, how many are chosen
  bool all = true;              // every candidate that reaches lo is chosen
  if (cta_sum(n, words, turn++) > K) {
    unsigned long long hi = ~0ull;   // fewer than K reach hi
    int above = 0;                   // that reach hi
    all = false;
    while (hi - lo > 1) {
      const unsigned long long mid = lo + ((hi - lo) >> 1);
      n = 0;
#pragma unroll
      for (int q = 0; q < kBmCands; ++q) n += val[q] >= mid;
      n = cta_sum(n, words, turn++);
      if (n >= K) lo = mid; else hi = mid, above = n;
      if (n == K) {
        all = true;
        break;
      }
    }
    left = K - above;
  }
  __syncthreads();
  // equal values at the border: the lowest places
  if (!all) {
    for (int k = 0; k < left; ++k) {
      long long best = LLONG_MAX;
#pragma unroll
      for (int q = 0; q < kBmCands; ++q)
        if (val[q] == lo && at[q] < best) best = at[q];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const long long other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other < best ? other : best;
      }
      __shared__ long long s_best[kBmWarps];
      if ((tid & 31) == 0) s_best[tid >> 5] = best;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kBmWarps; ++i) best = s_best[i] < best ? s_best[i] : best;
#pragma unroll
      for (int q = 0; q < kBmCands; ++q)
        if (val[q] == lo && at[q] == best) {
          const int to = atomicAdd(&s_out, 1);
          s_val[to] = lo, s_at[to] = best, s_f[to] = f[q];
          val[q] = 0;
        }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kBmCands; ++q)
      if (val[q] == lo) val[q] = 0;
  }
#pragma unroll
  for (int q = 0; q < kBmCands; ++q)
    if (val[q] >= lo) {
      const int to = atomicAdd(&s_out, 1);
      s_val[to] = val[q], s_at[to] = at[q], s_f[to] = f[q];
    }
  __syncthreads();
  const int got = s_out;
  // their order
  if (tid < got) {
    int r = 0;
    for (int i = 0; i < got; ++i)
      r += s_val[i] > s_val[tid] || (s_val[i] == s_val[tid] && s_at[i] < s_at[tid]);
    s_rank[r] = tid;
  }
  __syncthreads();
  // a beam's best child in its place, the others in the places left
  __shared__ int s_slot[kBeamMaxKeep];
  if (a.stay && tid == 0) {
    unsigned taken = 0;
    for (int i = 0; i < got; ++i) {
      const unsigned w = 1u << (int)(s_at[s_rank[i]] >> 32);
      s_slot[i] = taken & w ? -1 : (int)(s_at[s_rank[i]] >> 32);
      taken |= w;
    }
    int next = 0;
    for (int i = 0; i < K; ++i) {
      if (i < got && s_slot[i] >= 0) continue;
      while (taken >> next & 1) ++next;
      s_slot[i] = next;
      taken |= 1u << next;
    }
  }
  __syncthreads();
  if (tid < K) {
    const size_t o = (size_t)b * K + (a.stay ? s_slot[tid] : tid);
    if (tid < got) {
      const int c = s_rank[tid], token = (int)(uint32_t)s_at[c];
      a.score_out[o] = s_f[c];
      a.parent[o] = b * W + (int)(s_at[c] >> 32);
      a.token[o] = token;
      if (a.done_out) a.done_out[o] = token == a.end;
    } else {
      a.score_out[o] = -INFINITY;
      a.parent[o] = -1;
      a.token[o] = a.end < 0 ? 0 : a.end;
      if (a.done_out) a.done_out[o] = 0;
    }
  }
}

template <class F>
cudaError_t bm_launch(F* f, unsigned grid, const BeamArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kBmThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

}  // namespace

int beam_part_ctas(int sms) { return 4 * sms; }

cudaError_t launch_beam_select(const BeamArgs& args, int dtype, int sms, cudaStream_t st) {
  BeamArgs a = args;
  const int rows = a.batch * a.beams;
  // parts: as many CTAs as run at once, no part below a tile, 64 at most (the rows kernel's keys)
  int splits = beam_part_ctas(sms) / rows;
  const int tiles = (a.vocab + kBmTile - 1) / kBmTile;
  splits = splits < tiles ? splits : tiles;
  a.splits = splits < 1 ? 1 : splits > 64 ? 64 : splits;
  const unsigned grid = (unsigned)(rows * a.splits);
  cudaError_t e = dtype == FUTR_DTYPE_F32    ? bm_launch(beam_parts_kernel<FUTR_DTYPE_F32>, grid, a, st)
                  : dtype == FUTR_DTYPE_BF16 ? bm_launch(beam_parts_kernel<FUTR_DTYPE_BF16>, grid, a, st)
                                             : bm_launch(beam_parts_kernel<FUTR_DTYPE_F16>, grid, a, st);
  if (e != cudaSuccess) return e;
  e = bm_launch(beam_rows_kernel, (unsigned)rows, a, st);
  if (e != cudaSuccess) return e;
  return bm_launch(beam_pick_kernel, (unsigned)a.batch, a, st);
}

}  // namespace futr
