// The best continuations of each prompt's beams:
//   value(w, v) = score_w + x_wv - L_w,   L_w = log sum_u exp(x_wu)
// the `keep` largest of a prompt's beams * vocab values, equal ones by (w, v).
//
// L_w is the same for a whole row, so a row's candidates are its `keep` largest
// logits (equal ones by the lowest token), compared as they are; only those meet the
// other beams', as sums in fp64.  One pass over the logits, one kernel:
//   part   a CTA takes a part of a row in tiles, a thread 32 logits of a tile in registers:
//          running maximum and sum of exponentials per thread, and every logit that reaches
//          a threshold goes to a list in shared memory.
//          The threshold starts at (about) the keep-th largest of the threads' maxima of the
//          first tile: so many logits reach it at least, and few more.  A list that grows is cut
//          down to its keep largest, and the threshold follows.
//   row    the CTA that ends a row's last part makes one list and sum of all (where a
//          prompt's parts are too many for the next step by themselves).
//   pick   the CTA that ends a prompt's last row: log-sums, then the candidates by value.
// A list's entries are keys (logit in an order-preserving 32-bit form, then the inverted
// token), all different, so the order in which threads add to it has no effect; sums are
// added in the order of threads and parts.
//
// Short lists are put in order by counting, for each entry, those before it; of long ones
// the k largest are found by bisection, a count over the CTA a step.
//
// 256 rows of 128256 fp32 logits (131 MB) take 31.5 us, of which the tiles some 16 (at the
// rate of memory), the way to the first threshold 4 and the steps behind the last tile 6; 4
// rows 9.0 us, the same steps; 256 rows of bf16 27.5 us.  Waits for instructions are among the
// largest of a few rows, so the rare steps are out of line (34.1 and 9.1 us with them in line,
// where the rest took 31.2 and 8.7).  Not faster: a ring of bulk copies in place of the loads
// (39 us), and a persistent kernel whose ring runs on through its parts (42).
#include <cfloat>
#include <climits>
#include <type_traits>

#include "beam.cuh"

namespace futr {

namespace {

constexpr int kBmThreads = 256, kBmWarps = kBmThreads / 32;
constexpr int kBmLogits = 32;                     // logits of a thread in a tile
constexpr int kBmList = 1024;                     // entries of a part's list
constexpr int kBmCut = 64;                        // entries of a list that is cut, at least
constexpr int kBmShort = kBmThreads;              // entries that are put in order by counting
constexpr int kBmOne = 2048;                      // most candidates of a prompt that are picked from at once
constexpr int kBmMaxParts = 64;                   // parts of a row
constexpr int kBmPerSm = 4;                       // CTAs an SM
constexpr int kBmMaxWaves = 4;                    // parts of all rows, in CTAs that run at once
constexpr double kBmStart = 4.0;                  // what a part costs beside its logits, in halves of tiles
constexpr double kBmByRow = 6.0;                  // and the row's step
constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 numbers side by side, as one instruction takes them.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  return (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float pair_lo(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float pair_hi(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

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

// A sum in two fp32 parts, hi the sum rounded: some 2^-46 of its size (fp64 adds take 16
// times an fp32 one's time here, and exp and log some 30 of them: 5 of 20 us for one prompt).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two x, float y) {
  const float s = x.hi + y, t = s - x.hi;
  const float e = (x.hi - (s - t)) + (y - t) + x.lo;   // (the first two terms: what s lost, exactly)
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
__device__ __forceinline__ Two add(Two x, Two y) { return add(add(x, y.hi), y.lo); }

// A candidate's place in the order of a prompt, in two words: larger values first (an
// order-preserving form of the fp64, its last five bits cut off), then lower beams; the second
// word, the key turned over, larger logits and then lower tokens.  A beam's values grow with
// its logits or stay equal (each step of x - M + C rounds to the nearest), so its candidates are in
// the order of their logits.
constexpr unsigned long long kBeamBits = 31;
__device__ __forceinline__ unsigned long long place_of(double v, int beam) {
  const long long u = __double_as_longlong(v + 0.0);   // (-0 counts as +0)
  return ((unsigned long long)(u ^ (u >> 63 | (long long)(1ull << 63))) & ~kBeamBits) | (kBeamBits - beam);
}
__device__ __forceinline__ double value_at(unsigned long long place) {
  const long long u = (long long)(place & ~kBeamBits);
  return __longlong_as_double(u ^ (~(u >> 63) | (long long)(1ull << 63)));
}

// log x of x.hi >= 2^-100: x.hi = 2^e f with f near 1, whose logarithm is small enough for
// fp32 (an error of 2^-26 at most, where log x itself, rounded, has 2^-21).
__device__ __forceinline__ Two log_of(Two x) {
  constexpr double ln2 = 0.69314718055994530942;
  constexpr float ln2_hi = (float)ln2, ln2_lo = (float)(ln2 - (double)(float)ln2);
  const int u = __float_as_int(x.hi), e = (u - __float_as_int(0.75f)) >> 23;
  const float f = __int_as_float(u - e * (1 << 23)), p = (float)e * ln2_hi;
  const float rest = fmaf((float)e, ln2_hi, -p) + (float)e * ln2_lo;
  return add(add(add(Two{p, 0.f}, logf(f)), rest), __fdiv_rn(x.lo, x.hi));
}

__device__ __forceinline__ unsigned long long make_key(float x, int v) {
  return ((unsigned long long)ordered(x) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}
__device__ __forceinline__ float key_logit(unsigned long long k) { return unordered((uint32_t)(k >> 32)); }

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

// The largest and the smallest nonzero of the CTA's values (0 and ~0: there are none).
template <int N>
__device__ __forceinline__ void cta_range(const unsigned long long (&v)[N], unsigned long long* words,
                                          unsigned long long& lo, unsigned long long& hi) {
  lo = ~0ull, hi = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    hi = v[i] > hi ? v[i] : hi;
    lo = v[i] != 0 && v[i] < lo ? v[i] : lo;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
    hi = h > hi ? h : hi;
    lo = l < lo ? l : lo;
  }
  __syncthreads();   // the words of the call before have been read
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = hi, words[kBmWarps + (threadIdx.x >> 5)] = lo;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBmWarps; ++i) {
    hi = words[i] > hi ? words[i] : hi;
    lo = words[kBmWarps + i] < lo ? words[kBmWarps + i] : lo;
  }
}

// How many of the CTA's values reach t.
template <int N>
__device__ __forceinline__ int cta_reach(const unsigned long long (&v)[N], unsigned long long t, int* words, int& turn) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) n += v[i] >= t;
  return cta_sum(n, words, turn++);
}

// The value that exactly k of the CTA's keys reach, all different (0: none); 1, which all
// reach, where there are at most k.  `range`: words for cta_range; `turn` counts the sums.
template <int N>
__device__ __forceinline__ unsigned long long select_key(const unsigned long long (&v)[N], int k, int* words,
                                                         unsigned long long* range, int& turn) {
  unsigned long long lo, hi;
  cta_range(v, range, lo, hi);
  if (hi == 0 || cta_reach(v, lo, words, turn) <= k) return 1;
  ++hi;   // invariant: more than k reach lo, fewer than k reach hi
  while (hi - lo > 1) {
    const unsigned long long mid = lo + ((hi - lo) >> 1);
    const int n = cta_reach(v, mid, words, turn);
    if (n == k) return mid;
    if (n > k)
      lo = mid;
    else
      hi = mid;
  }
  return hi;
}

// A value that at least k of the CTA's threads' values reach, and few more (0 where fewer
// than k are not 0): the k-th largest of the ceil(k / 4) largest of each of the 8 warps.
// Each warp counts for its own of these those above, a half of the lanes over a half of them.
// (Counting for each of the 256 values took 2.4 us, 3.5 with four CTAs an SM; every warp for
// all of k = 64's 128 values 6 and 13.)
__device__ __forceinline__ uint32_t reached(uint32_t v, int k, uint32_t* all, int* words) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, each = (k + 3) >> 2;   // 1 .. 16
  uint32_t mine = 0;
  for (int i = 0; i < each; ++i) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, v);
    if ((lane & 15) == i) mine = top;
    if (lane == __ffs(__ballot_sync(0xffffffffu, v == top)) - 1) v = 0;   // of equal values one goes
  }
  const int n = each * kBmWarps;
  if (lane < each) all[warp * each + lane] = mine;
  __syncthreads();
  int above = 0;
#pragma unroll 4
  for (int i = lane & 16 ? n / 2 : 0; i < (lane & 16 ? n : n / 2); i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(all + i);
    above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
  }
  above += __shfl_xor_sync(0xffffffffu, above, 16);
  // the least of those that fewer than k exceed
  uint32_t low = __reduce_min_sync(0xffffffffu, (lane & 15) < each && above < k ? mine : ~0u);
  if (lane == 0) words[warp] = (int)low;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBmWarps; ++i) low = min(low, (uint32_t)words[i]);
  return low;
}

template <int kType>
using Logit = std::conditional_t<kType == FUTR_DTYPE_F32, float, uint16_t>;

// Logit i of 16 bytes.
template <int kType>
__device__ __forceinline__ float logit_of(const uint32_t (&u)[4], int i) {
  if constexpr (kType == FUTR_DTYPE_F32)
    return __uint_as_float(u[i]);
  else if constexpr (kType == FUTR_DTYPE_BF16)
    return __uint_as_float(i & 1 ? u[i >> 1] & 0xffff0000u : u[i >> 1] << 16);
  else
    return __half2float(__ushort_as_half((uint16_t)(i & 1 ? u[i >> 1] >> 16 : u[i >> 1] & 0xffffu)));
}

// The 16 bytes from byte `shift` of two blocks on.
__device__ __forceinline__ void shifted(const uint4& p, const uint4& q, int shift, uint32_t (&u)[4]) {
  uint32_t w[9] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w, 0};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = __funnelshift_r(w[i], w[i + 1], (shift & 3) * 8);
}

// The logits from token W * vec on (vec < v1; -inf behind the row's end) as they are: one
// 16-byte load, or two that a row off such a boundary lies across; single ones at its ends.
// Wherever a row lies, a thread gets the same tokens: equal rows have equal sums.
template <int kType>
__device__ __forceinline__ void load_vec(const Logit<kType>* x, int vec, int v1, int vocab, uint32_t (&u)[4]) {
  using T = Logit<kType>;
  constexpr int W = 16 / sizeof(T);
  constexpr uint32_t none = kType == FUTR_DTYPE_F32 ? 0xff800000u : kType == FUTR_DTYPE_BF16 ? 0xff80u : 0xfc00u;
  const long long e = (long long)vec * W;
  const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15), off = shift / (int)sizeof(T);
  if (vec < v1 && shift == 0 && e + W <= vocab) {
    const uint4 p = __ldcs(reinterpret_cast<const uint4*>(x + e));
    u[0] = p.x, u[1] = p.y, u[2] = p.z, u[3] = p.w;
  } else if (vec < v1 && shift != 0 && e >= off && e - off + 2 * W <= vocab) {
    const uint4* a = reinterpret_cast<const uint4*>(x + e - off);
    shifted(a[0], a[1], shift, u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint32_t t = none;
      if (vec < v1 && e + i < vocab) {
        if constexpr (sizeof(T) == 4)
          t = __float_as_uint(x[e + i]);
        else
          t = x[e + i];
      }
      u[i * (int)sizeof(T) / 4] |= t << (8 * (i * (int)sizeof(T) % 4));
    }
  }
}

// Rows that are not read: without a finite score, or ended.
__device__ __forceinline__ bool row_read(const BeamArgs& a, int row) {
  const float s = a.scores[row];
  return s >= -FLT_MAX && s <= FLT_MAX && !(a.done && a.done[row] != 0);
}

// Shared memory of a CTA.
struct BmShared {
  union {
    unsigned long long list[kBmList + 2];   // a part's list
    ulonglong2 cand[kBmOne];                // pick: candidates, as place_of has it
  };
  uint4 all[kBeamMaxKeep / 2];   // the warps' largest values: 2 keep, rounded up
  unsigned long long range[2 * kBmWarps];
  int words[2 * kBmWarps], warps[kBmWarps];
  int n[3];                   // entries that a tile adds, three tiles in turn
  int out;
  unsigned last;
  Two sum[kBmWarps];
  float top[kBmWarps];
  // a beam's value: logit - most + base; base -inf: it offers nothing, most inf: it has ended
  float most[kBeamMaxBeams];
  Two base[kBeamMaxBeams];
  // the chosen, best first: value, row, token; their places
  float f[kBeamMaxKeep];
  int beam[kBeamMaxKeep], token[kBeamMaxKeep], slot[kBeamMaxKeep];
};

__device__ __forceinline__ unsigned long long* keys_of(uint8_t* rec) {
  return reinterpret_cast<unsigned long long*>(rec + 16);
}

__device__ __forceinline__ void put_stats(uint8_t* rec, float M, Two S) {
  *reinterpret_cast<float4*>(rec) = make_float4(M, S.hi, S.lo, 0.f);
}

__device__ __forceinline__ Two warp_sum(Two s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = add(s, Two{__shfl_down_sync(0xffffffffu, s.hi, o), __shfl_down_sync(0xffffffffu, s.lo, o)});
  return Two{__shfl_sync(0xffffffffu, s.hi, 0), __shfl_sync(0xffffffffu, s.lo, 0)};
}

// The entries of the list that reach thr, to the front of it or to a record.
template <int N>
__device__ __forceinline__ void put_keys(BmShared& sh, const unsigned long long (&key)[N], unsigned long long thr,
                                         unsigned long long* to) {
  __syncthreads();   // the list has been read
  if (threadIdx.x == 0) sh.out = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (key[q] >= thr) to[atomicAdd(&sh.out, 1)] = key[q];
  __syncthreads();
}

__device__ __forceinline__ void read_list(const BmShared& sh, int n, unsigned long long (&key)[kBmList / kBmThreads]) {
#pragma unroll
  for (int q = 0; q < kBmList / kBmThreads; ++q) {
    const int p = threadIdx.x + q * kBmThreads;
    key[q] = p < n ? sh.list[p] : 0;
  }
}

// The list's n <= kBmShort entries in order, the K largest of them at `to` (n > K, or all).
__device__ __forceinline__ void sort_list(BmShared& sh, int n, int K, unsigned long long* to) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.list[n] = 0;   // (the count goes by twos)
  __syncthreads();
  const unsigned long long key = tid < n ? sh.list[tid] : 0;
  int rank = 0;
  if ((tid & ~31) < n) {
    for (int i = 0; i < n; i += 2) {
      const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&sh.list[i]);
      rank += (k2.x > key) + (k2.y > key);
    }
  }
  __syncthreads();   // the list has been read
  if (tid < n && rank < K) to[rank] = key;
  __syncthreads();
}

// The list's K largest of n > K to the front of it or to a record; the least of them, or a
// value between it and the next.  (Out of line, as what follows: rare, and the way past it is
// fetched in each call.)
__device__ __noinline__ unsigned long long cut_list(BmShared& sh, int n, int K, unsigned long long* to) {
  unsigned long long key[kBmList / kBmThreads];
  int turn = 0;
  __syncthreads();
  read_list(sh, n, key);
  const unsigned long long thr = select_key(key, K, sh.words, sh.range, turn);
  put_keys(sh, key, thr, to);
  return thr;
}

// A tile's logits x (kBmLogits a thread, W in a row, from vector `at` on) that reach thr to the
// list of n entries, one a thread at a time, the list cut down between; its entries.
template <int W>
__device__ __noinline__ int crowded_tile(BmShared& sh, const float* x, int at, int K, int n, unsigned long long& thr) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
  for (int i = 0; i < kBmLogits; ++i) {
    if (n > kBmList - kBmThreads) {
      thr = cut_list(sh, n, K, sh.list);
      n = K;
    }
    const int token = (at + tid + kBmThreads * (i / W)) * W + i % W;
    const unsigned long long key = x[i] >= -FLT_MAX ? make_key(x[i], token) : 0;
    const bool in = key != 0 && key >= thr;
    const unsigned votes = __ballot_sync(0xffffffffu, in);
    __syncthreads();   // the words have been read
    if (lane == 0) sh.words[warp] = __popc(votes);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < kBmWarps; ++q) {
      before += q < warp ? sh.words[q] : 0;
      all += sh.words[q];
    }
    if (in) sh.list[n + before + __popc(votes & ((1u << lane) - 1))] = key;
    n += all;
  }
  return n;
}

// A part of a row: its record.
template <int kType>
__device__ __forceinline__ void do_part(const BeamArgs& a, BmShared& sh, int row, int part, uint8_t* rec) {
  using T = Logit<kType>;
  constexpr int W = 16 / sizeof(T);            // logits of a vector
  constexpr int P = kBmLogits, V = P / W;      // logits and vectors of a thread in a tile
  constexpr int kStep = kBmThreads * V;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.keep;
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.ld;
  const int nv = (a.vocab - 1) / W + 1;
  const int v0 = (int)((long long)nv * part / a.splits), v1 = (int)((long long)nv * (part + 1) / a.splits);
  const int shift = (int)(reinterpret_cast<uintptr_t>(x) & 15);
  int n = 0, tile = 0;                         // entries of the list, tiles
  const int kCut = max(2 * K, kBmCut);         // entries above which the list is cut
  float m = -INFINITY, s = 0.f;                // maximum, sum of 2^((x - m) log2 e)
  unsigned long long thr = 1;
  float thr_x = -FLT_MAX;                      // a logit below it does not reach thr
  if (tid < 3) sh.n[tid] = 0;
  __syncthreads();
  for (int at = v0; at < v1; at += kStep, ++tile) {
    uint32_t u[V][4];
    // a tile that lies in the part and the row as a whole, on 16-byte boundaries or off them,
    // without checks (256 rows of 50257 logits, most of them off: 26.7 us with checks for every
    // vector, 24.0 without)
    const bool whole = at + kStep <= v1 && (long long)(at + kStep + (shift != 0)) * W <= a.vocab;
    if (whole && shift == 0) {
      const uint4* p = reinterpret_cast<const uint4*>(x) + at + tid;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint4 q = __ldcs(p + kBmThreads * j);
        u[j][0] = q.x, u[j][1] = q.y, u[j][2] = q.z, u[j][3] = q.w;
      }
    } else if (whole && at > 0) {
      const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(x) - shift) + at + tid;
#pragma unroll
      for (int j = 0; j < V; ++j) shifted(p[kBmThreads * j], p[kBmThreads * j + 1], shift, u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) load_vec<kType>(x, at + tid + kBmThreads * j, v1, a.vocab, u[j]);
    }
    auto logit = [&](int i) { return logit_of<kType>(u[i / W], i % W); };
    auto token = [&](int i) { return (at + tid + kBmThreads * (i / W)) * W + i % W; };
    // maxima of 8 logits, and of all
    float tops[P / 8], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < P / 8; ++j) {
      tops[j] = logit(8 * j);
#pragma unroll
      for (int i = 1; i < 8; ++i) tops[j] = fmaxf(tops[j], logit(8 * j + i));
      top = fmaxf(top, tops[j]);
    }
    if (top > m) {
      s *= bm_ex2((m - top) * kLog2e);         // (the first time 2^-inf = 0)
      m = top;
    }
    const float at_m = m == -INFINITY ? 0.f : m;
    if (fabsf(at_m) <= 0x1p20f) {
      // 2^(x log2 e - ref), two logits an instruction where there is one; ref is m log2 e
      // rounded, what that lost is put back
      const float ref = __fmul_rn(at_m, kLog2e), lost = fmaf(at_m, kLog2e, -ref);
      const uint64_t c2 = pair_of(kLog2e, kLog2e), r2 = pair_of(-ref, -ref);
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const uint64_t e = pair_fma(pair_of(logit(i), logit(i + 1)), c2, r2);
        sum = pair_add(sum, pair_of(bm_ex2(pair_lo(e)), bm_ex2(pair_hi(e))));
      }
      s = fmaf(pair_lo(sum) + pair_hi(sum), bm_ex2(-lost), s);   // a NaN or +inf in the row makes it one
    } else {   // a row that masks have left nothing but their own large values, or so
#pragma unroll 1
      for (int j = 0; j < V; ++j) {
        uint32_t t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = u[0][i];
#pragma unroll
        for (int q = 1; q < V; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = q == j ? u[q][i] : t[i];
#pragma unroll
        for (int i = 0; i < W; ++i) s += bm_ex2((logit_of<kType>(t, i) - at_m) * kLog2e);
      }
    }
    if (tile == 0) {
      const uint32_t lo = reached(top > -INFINITY ? ordered(top) : 0u, K, reinterpret_cast<uint32_t*>(sh.all), sh.warps);
      if (lo >= kLowest) {
        thr = (unsigned long long)lo << 32;
        thr_x = unordered(lo);
      }
    }
    int* counter = &sh.n[tile % 3];
    if (top >= thr_x) {
#pragma unroll
      for (int j = 0; j < P / 8; ++j)
        if (tops[j] >= thr_x) {
#pragma unroll
          for (int i = 8 * j; i < 8 * j + 8; ++i)
            if (logit(i) >= thr_x) {
              const unsigned long long key = make_key(logit(i), token(i));
              if (key >= thr) {
                const int to = n + atomicAdd(counter, 1);
                if (to < kBmList) sh.list[to] = key;
              }
            }
        }
    }
    __syncthreads();
    const int more = *counter;
    if (tid == 0) sh.n[(tile + 2) % 3] = 0;    // last read before this tile's barrier, next used two tiles on
    if (n + more <= kBmList) {
      n += more;
      if (more > 0 && n > kCut && at + kStep < v1) {
        if (n <= kBmShort) {
          sort_list(sh, n, K, sh.list);
          thr = sh.list[K - 1];
        } else {
          thr = cut_list(sh, n, K, sh.list);
        }
        thr_x = unordered((uint32_t)(thr >> 32));
        n = K;
      }
      continue;
    }
    // too many at once: what the tile added is dropped, and added a logit a thread at a time,
    // the list cut down between
    float all[P];
#pragma unroll
    for (int i = 0; i < P; ++i) all[i] = logit(i);
    n = crowded_tile<W>(sh, all, at, K, n, thr);
    thr_x = unordered(max((uint32_t)(thr >> 32), kLowest));
  }
  // the part's K largest
  __syncthreads();
  if (n <= K) {
    for (int i = tid; i < K; i += kBmThreads) keys_of(rec)[i] = i < n ? sh.list[i] : 0;
  } else if (n <= kBmShort) {
    sort_list(sh, n, K, keys_of(rec));
  } else {
    cut_list(sh, n, K, keys_of(rec));
  }
  // its maximum and sum
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) sh.top[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kBmWarps; ++i) M = fmaxf(M, sh.top[i]);
  // (a thread without a logit has the sum 0, or a NaN)
  Two S{m == -INFINITY ? s : s * bm_ex2((m - M) * kLog2e), 0.f};
  S = warp_sum(S);
  if (lane == 0) sh.sum[warp] = S;
  __syncthreads();
  if (tid < 32) {
    S = tid < kBmWarps ? sh.sum[tid] : Two{0.f, 0.f};
#pragma unroll
    for (int o = kBmWarps / 2; o > 0; o >>= 1)
      S = add(S, Two{__shfl_down_sync(0xffffffffu, S.hi, o), __shfl_down_sync(0xffffffffu, S.lo, o)});
    if (tid == 0) put_stats(rec, M, S);
  }
}

// The maximum and the sum of `n` records (a warp; n up to kBmMaxParts): in all lanes.
__device__ __forceinline__ void join_sums(const uint8_t* recs, int n, size_t step, float& M, Two& S) {
  const int lane = threadIdx.x & 31;
  float m[kBmMaxParts / 32];
  Two s[kBmMaxParts / 32];
  M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBmMaxParts / 32; ++i) {
    const int p = lane + 32 * i;
    m[i] = -INFINITY;
    s[i] = Two{0.f, 0.f};
    if (p < n) {
      const float4 r = __ldcg(reinterpret_cast<const float4*>(recs + p * step));
      m[i] = r.x;
      s[i] = Two{r.y, r.z};
    }
    M = fmaxf(M, m[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  S = Two{0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kBmMaxParts / 32; ++i) {
    // (no logit: 0, or a NaN)
    const float w = m[i] == -INFINITY ? 1.f : bm_ex2((m[i] - M) * kLog2e);
    S = add(S, Two{s[i].hi * w, fmaf(s[i].hi, w, -(s[i].hi * w)) + s[i].lo * w});
  }
  S = warp_sum(S);
}

// i / d for i d < 2^32, by ceil(2^32 / d) (0: d is 1).
__device__ __forceinline__ int quotient(int i, uint32_t by) { return by ? (int)__umulhi((uint32_t)i, by) : i; }
uint32_t quotient_by(int d) { return d == 1 ? 0 : (uint32_t)(((1ull << 32) + d - 1) / d); }

// Which entry of record r index i takes: the records' entries one after another, each turned
// by 5 against the one before, so that a thread (every 256th index) does not get the best of
// all of them.
__device__ __forceinline__ int entry_of(const BeamArgs& a, int i, int r) {
  const int t = i - r * a.keep + 5 * r;
  return t - quotient(t, a.by_keep) * a.keep;
}

// A row's parts become one record.
__device__ __noinline__ void do_row(const BeamArgs& a, BmShared& sh, int row) {
  const int tid = threadIdx.x, K = a.keep;
  const size_t step = beam_record(K);
  const uint8_t* parts = a.parts + (size_t)row * a.splits * step;
  uint8_t* rec = a.rows + (size_t)row * step;
  if (tid < 32) {
    float M;
    Two S;
    join_sums(parts, a.splits, step, M, S);
    if (tid == 0) put_stats(rec, M, S);
  }
  if (tid == 0) sh.out = 0;
  constexpr int N = kBmMaxParts * kBeamMaxKeep / kBmThreads;
  unsigned long long key[N];
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int i = tid + q * kBmThreads, r = quotient(i, a.by_keep);
    key[q] = 0;
    if (i < a.splits * K)
      key[q] = __ldcg(reinterpret_cast<const unsigned long long*>(parts + (size_t)r * step + 16) + entry_of(a, i, r));
    top = max(top, (uint32_t)(key[q] >> 32));
  }
  const uint32_t low = reached(top, K, reinterpret_cast<uint32_t*>(sh.all), sh.warps);
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (key[q] != 0 && (uint32_t)(key[q] >> 32) >= low) {
      const int to = atomicAdd(&sh.out, 1);
      if (to < kBmShort) sh.list[to] = key[q];
    }
  __syncthreads();
  const int n = sh.out;
  if (n <= K) {
    for (int i = tid; i < K; i += kBmThreads) keys_of(rec)[i] = i < n ? sh.list[i] : 0;
  } else if (n <= kBmShort) {
    sort_list(sh, n, K, keys_of(rec));
  } else {
    int turn = 0;
    put_keys(sh, key, select_key(key, K, sh.words, sh.range, turn), keys_of(rec));
  }
}

// A prompt's beams: the K best of their candidates, `lists` records a beam.
__device__ __forceinline__ void do_pick(const BeamArgs& a, BmShared& sh, int b, const uint8_t* recs, int lists) {
  const int tid = threadIdx.x, warp = tid >> 5, W = a.beams, K = a.keep;
  const size_t step = beam_record(K);
  recs += (size_t)b * W * lists * step;
  // the candidates' keys, on their way before the sums are looked at (those of beams that
  // offer nothing, or have ended, are not used)
  constexpr int N = kBmOne / kBmThreads;
  unsigned long long key[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int i = tid + q * kBmThreads, r = quotient(i, a.by_keep);
    key[q] = 0;
    if (i < W * lists * K)
      key[q] = __ldcg(reinterpret_cast<const unsigned long long*>(recs + (size_t)r * step + 16) + entry_of(a, i, r));
  }
  for (int w = warp; w < W; w += kBmWarps) {
    const int row = b * W + w;
    const float score = a.scores[row];
    float most = 0.f;
    Two base{-INFINITY, 0.f};
    if (!(score <= FLT_MAX)) {   // NaN or +inf
      if ((tid & 31) == 0) set_err(a.err, FUTR_ERR_NOT_FINITE);
    } else if (row_read(a, row)) {
      float M;
      Two S;
      join_sums(recs + (size_t)w * lists * step, lists, step, M, S);
      const bool bad = !(S.hi <= FLT_MAX) || M == INFINITY;
      if (bad && (tid & 31) == 0) set_err(a.err, FUTR_ERR_NOT_FINITE);
      if (!bad && M > -INFINITY) {
        const Two l = log_of(S);
        most = M;
        base = Two{score, 0.f};
        if (l.hi > 0.f) base = add(add(base, -l.hi), -l.lo);   // S holds e^0: less than 1 it is by roundings alone
      }
    } else if (score >= -FLT_MAX) {
      most = INFINITY;
      base = Two{score, 0.f};
    }
    if ((tid & 31) == 0) sh.most[w] = most, sh.base[w] = base;
  }
  if (tid == 0) sh.out = 0;
  __syncthreads();
  // the candidates' values in fp32 decide that most are not chosen: they are off by 4 u A at
  // most, u = 2^-24 and A the largest of the best beam's base (no value of its beam is above it)
  // and of the bound by which `keep` of them lie, so those within 2^-20 A of it (16 u) may be
  uint32_t near[N], top = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int i = tid + q * kBmThreads;
    near[q] = 0;
    if (i < W * lists * K) {
      const int w = quotient(i, lists > 1 ? a.by_beam : a.by_keep);
      const float most = sh.most[w], base = sh.base[w].hi;
      float v = -INFINITY;
      if (most == INFINITY) {
        if (i == w * lists * K) v = base;
        key[q] = ~(unsigned long long)(uint32_t)a.end;
      } else if (key[q] != 0) {
        v = (key_logit(key[q]) - most) + base;
      }
      if (v >= -FLT_MAX) near[q] = ordered(v);   // (below it: as little as a logit of -inf)
      top = max(top, near[q]);
    }
  }
  const float best = unordered(__reduce_max_sync(0xffffffffu, ordered((tid & 31) < W ? sh.base[tid & 31].hi : -INFINITY)));
  uint32_t low = reached(top, K, reinterpret_cast<uint32_t*>(sh.all), sh.warps);
  if (low != 0) {
    const float bound = unordered(low);
    low = max(1u, ordered(fmaf(fmaxf(fabsf(bound), fabsf(best)), -0x1p-20f, bound)));
  }
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (near[q] != 0 && near[q] >= low) {
      const int i = tid + q * kBmThreads, w = quotient(i, lists > 1 ? a.by_beam : a.by_keep);
      sh.cand[atomicAdd(&sh.out, 1)] = make_ulonglong2((unsigned)w, ~key[q]);
    }
  __syncthreads();
  const int n = sh.out, got = min(n, K);
  // their places, by fp64 (0.3 us; of all candidates 0.5 to 3)
#pragma unroll 1
  for (int c = tid; c < n; c += kBmThreads) {
    const int w = (int)sh.cand[c].x;
    const float most = sh.most[w];
    const double base = (double)sh.base[w].hi + sh.base[w].lo;
    sh.cand[c].x = place_of(most == INFINITY ? base : ((double)key_logit(~sh.cand[c].y) - most) + base, w);
  }
  __syncthreads();
  // their order
#pragma unroll 1
  for (int c = tid; c < n; c += kBmThreads) {
    const ulonglong2 my = sh.cand[c];
    int r = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const ulonglong2 t = sh.cand[i];
      r += (t.x > my.x) | ((t.x == my.x) & (t.y < my.y));
    }
    if (r < K) {
      sh.f[r] = fmaxf((float)value_at(my.x), -FLT_MAX);
      sh.beam[r] = (int)(kBeamBits - (my.x & kBeamBits));
      sh.token[r] = (int)(uint32_t)my.y;
    }
  }
  __syncthreads();
  // a beam's best child in its place, the others in the places left
  if (a.stay) {
    if (tid == 0) {
      unsigned taken = 0;
      for (int i = 0; i < got; ++i) {
        const int w = sh.beam[i];
        sh.slot[i] = taken >> w & 1 ? -1 : w;
        taken |= 1u << w;
      }
      int next = 0;
      for (int i = 0; i < K; ++i) {
        if (i < got && sh.slot[i] >= 0) continue;
        while (taken >> next & 1) ++next;
        sh.slot[i] = next;
        taken |= 1u << next;
      }
    }
    __syncthreads();
  }
  if (tid < K) {
    const size_t o = (size_t)b * K + (a.stay ? sh.slot[tid] : tid);
    if (tid < got) {
      a.score_out[o] = sh.f[tid];
      a.parent[o] = b * W + sh.beam[tid];
      a.token[o] = sh.token[tid];
      if (a.done_out) a.done_out[o] = sh.token[tid] == a.end;
    } else {
      a.score_out[o] = -INFINITY;
      a.parent[o] = -1;
      a.token[o] = a.end < 0 ? 0 : a.end;
      if (a.done_out) a.done_out[o] = 0;
    }
  }
}

// True in the CTA that arrives last of `n` at a counter, which starts over; what the
// others wrote before is there.
__device__ __forceinline__ bool arrive_last(BmShared& sh, unsigned* counter, unsigned n) {
  __syncthreads();
  if (threadIdx.x == 0) {
    sh.last = atom_add_acq_rel_gpu(counter, 1u) == n - 1;
    if (sh.last) *counter = 0u;
  }
  __syncthreads();
  return sh.last != 0;
}

template <int kType>
__global__ void __launch_bounds__(kBmThreads, kBmPerSm) beam_kernel(const BeamArgs a) {
  __shared__ BmShared sh;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x / a.splits, part = blockIdx.x % a.splits, b = row / a.beams;
  if (row_read(a, row)) do_part<kType>(a, sh, row, part, a.parts + (size_t)blockIdx.x * beam_record(a.keep));
  if (a.by_row) {
    if (!arrive_last(sh, a.cnt + a.batch + row, (unsigned)a.splits)) return;
    if (row_read(a, row)) do_row(a, sh, row);
    if (!arrive_last(sh, a.cnt + b, (unsigned)a.beams)) return;
    do_pick(a, sh, b, a.rows, 1);
  } else {
    if (!arrive_last(sh, a.cnt + b, (unsigned)(a.beams * a.splits))) return;
    do_pick(a, sh, b, a.parts, a.splits);
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

int beam_part_ctas(int sms) { return kBmPerSm * kBmMaxWaves * sms; }

cudaError_t launch_beam_select(const BeamArgs& args, int dtype, int sms, cudaStream_t st) {
  BeamArgs a = args;
  const long long rows = (long long)a.batch * a.beams, slots = (long long)kBmPerSm * sms;
  // parts of a row: those that end soonest, by waves of CTAs, in halves of tiles (4096
  // logits); a part costs about kBmStart more.  256 rows of 128256 logits in 1, 2, 3, 4 and 7
  // parts: 47, 33.5, 43, 39 and 44 us; 4 rows in 8, 16, 32 and 64: 9.7, 9.0, 9.0 and 11.
  const int tiles = (a.vocab - 1) / (kBmThreads * kBmLogits / 2) + 1;
  double best = 1e30;
  a.splits = 1;
  for (int s = 1; s <= kBmMaxParts && s <= tiles && (s == 1 || rows * s <= beam_part_ctas(sms)); ++s) {
    const double cost = (double)((rows * s + slots - 1) / slots) * ((double)tiles / s + kBmStart) +
                        (a.beams * s * a.keep > kBmOne ? kBmByRow : 0.0);
    if (cost < best * 0.98) {
      best = cost;
      a.splits = s;
    }
  }
  a.by_row = a.beams * a.splits * a.keep > kBmOne;
  a.by_keep = quotient_by(a.keep);
  a.by_beam = quotient_by(a.keep * a.splits);
  const unsigned grid = (unsigned)(rows * a.splits);
  return dtype == FUTR_DTYPE_F32    ? bm_launch(beam_kernel<FUTR_DTYPE_F32>, grid, a, st)
         : dtype == FUTR_DTYPE_BF16 ? bm_launch(beam_kernel<FUTR_DTYPE_BF16>, grid, a, st)
                                    : bm_launch(beam_kernel<FUTR_DTYPE_F16>, grid, a, st);
}

}  // namespace futr
