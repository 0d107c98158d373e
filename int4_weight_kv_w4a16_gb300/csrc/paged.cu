// Append to the paged 8-bit cache: RoPE, page scale, e4m3 codes, in one pass
// over the new rows.
//
//   k'_i = k_i cos a - k_{i+d/2} sin a,  k'_{i+d/2} = k_{i+d/2} cos a + k_i sin a,
//   a = p theta^(-2i/d)   (fp32 products, each rounded, from the fp32 table)
//   s = max(s_old, 2^e),  2^e the smallest power of two with amax <= 448 2^e
//   code = e4m3(x / s);   where s > s_old, an old code c becomes e4m3(c s_old / s)
//
// One CTA per (touched page, kv-head, K or V): it alone writes that page's
// codes and scale, so there are no atomics and the result does not depend on
// any order.  A group of d/8 lanes takes one row, a lane the elements 4 i .. 4 i + 3
// and their rotation partners d/2 further on, so that a table entry is read once and
// nothing is exchanged.  A thread holds up to four rows from the maximum to the
// codes: page / 4 rows at a time, whatever the page.
//
// Bound by memory for prompts (2 bytes read and 1 written per element): 64 MB take
// 16.4 us (3.9 TB/s; 9.5 us at the copy rate; the rest is the start of a CTA, four
// waves of them).  Two rows a thread took 21 us where four and eight took 18.4, and
// reading the rows a second time instead of keeping them 36.  Bound by latency for
// single tokens, whose chain is: row bounds -> table entry -> old scale, and beside
// it row -> rotation -> maximum: 2.3 us for one, 3.2 us for 32 sequences.
#include <cuda_fp8.h>

#include "paged.cuh"

namespace futr {

namespace {

constexpr int kAppRounds = 4;                                 // rows a thread holds
constexpr int kAppMaxThreads = 128 * (128 / 8) / kAppRounds;   // page 128, head dim 128

// e4m3 of x in [-448, 448] (saturating), as bits; and back.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Exponent of the page scale for a largest magnitude amax: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int x = (int)(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kPagedMinExp ? kPagedMinExp : e;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <bool kHalf>
__device__ __forceinline__ void widen8(const uint2& lo, const uint2& hi, float (&x)[8]) {
  const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kHalf) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

struct AppendArgs {
  PagedView c;
  PagedRows r;
  const uint16_t* src[2];   // K, V rows
  long long ld[2];
  int* err;
};

template <int D, bool kHalf>
__global__ void __launch_bounds__(kAppMaxThreads) paged_append_kernel(const AppendArgs a) {
  constexpr int L = D / 8;                            // lanes of a row
  __shared__ float s_max[kAppMaxThreads / 32];
  __shared__ int s_found[5];
  const int threads = blockDim.x, rows = threads / L;   // rows at a time
  const int tid = threadIdx.x, lane = tid & 31, lg = tid % L, rg = tid / L;
  const int kvh = blockIdx.y, which = blockIdx.z;
  pdl_trigger();
  pdl_wait();
  // one warp of the grid looks every sequence over (the search below stops early)
  if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0 && tid >= threads - 32)
    for (int s = lane; s < a.r.batch; s += 32) {
      int r0, nn, pp;
      if (!paged_seq(a.r, a.c, s, r0, nn, pp)) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
    }
  // the touched page of this CTA: sequences in order, each with the pages that
  // its new rows meet; one warp looks for all (every warp by itself: 18.4 us for the
  // prompts that take 16.4)
  int item = blockIdx.x, row0 = 0, n = 0, p0 = 0, b = -1;
  for (int b0 = 0; b0 < a.r.batch && tid < 32; b0 += 32) {
    int rr = 0, nn = 0, pp = 0, pages = 0;
    if (b0 + lane < a.r.batch) {
      paged_seq(a.r, a.c, b0 + lane, rr, nn, pp);
      if (nn > 0) pages = ((pp + nn - 1) >> a.c.page_log2) - (pp >> a.c.page_log2) + 1;
    }
    int incl = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > item);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      row0 = __shfl_sync(0xffffffffu, rr, src);
      n = __shfl_sync(0xffffffffu, nn, src);
      p0 = __shfl_sync(0xffffffffu, pp, src);
      item -= __shfl_sync(0xffffffffu, incl - pages, src);
      break;
    }
    item -= __shfl_sync(0xffffffffu, incl, 31);
  }
  if (tid == 0) {
    s_found[0] = b;
    s_found[1] = item;
    s_found[2] = row0;
    s_found[3] = n;
    s_found[4] = p0;
  }
  __syncthreads();
  b = s_found[0], item = s_found[1], row0 = s_found[2], n = s_found[3], p0 = s_found[4];
  if (b < 0) return;   // the grid is an upper bound
  const int page = a.c.page, pi = (p0 >> a.c.page_log2) + item;
  const int id = a.r.table[(size_t)b * a.r.table_ld + pi];
  const int base = pi << a.c.page_log2;
  const int lo = max(base, p0) - base, hi = min(base + page, p0 + n) - base;   // slots [lo, hi) are new
  const uint16_t* src = (which ? a.src[1] : a.src[0]) + (size_t)kvh * D + 4 * lg;
  const long long ld = which ? a.ld[1] : a.ld[0];
  const bool rotate = which == 0 && a.c.rope != nullptr;

  // The rows, all of them on their way before the page number is looked at.
  float x[kAppRounds][8];
  {
    uint2 raw[kAppRounds][2];
    float4 cs[kAppRounds][2];
#pragma unroll
    for (int i = 0; i < kAppRounds; ++i) {
      const int slot = lo + i * rows + rg;
      raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
      if (slot < hi) {
        const uint16_t* row = src + (size_t)(row0 + base + slot - p0) * ld;
        raw[i][0] = *reinterpret_cast<const uint2*>(row);
        raw[i][1] = *reinterpret_cast<const uint2*>(row + D / 2);
        if (rotate) {
          const float4* t = reinterpret_cast<const float4*>(a.c.rope + (size_t)(base + slot) * (D / 2) + 4 * lg);
          cs[i][0] = t[0];
          cs[i][1] = t[1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAppRounds; ++i) {
      widen8<kHalf>(raw[i][0], raw[i][1], x[i]);
      if (rotate && lo + i * rows + rg < hi) {
        const float c[4] = {cs[i][0].x, cs[i][0].z, cs[i][1].x, cs[i][1].z};
        const float n[4] = {cs[i][0].y, cs[i][0].w, cs[i][1].y, cs[i][1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float l = x[i][j], u = x[i][4 + j];
          x[i][j] = __fsub_rn(__fmul_rn(l, c[j]), __fmul_rn(u, n[j]));
          x[i][4 + j] = __fadd_rn(__fmul_rn(u, c[j]), __fmul_rn(l, n[j]));
        }
      }
    }
  }
  if (id < 0 || id >= a.c.n_pages) {
    if (tid == 0) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
    return;
  }
  const size_t blk = ((size_t)id * a.c.n_kv + kvh) * 2 + which;
  uint8_t* codes = a.c.codes + blk * page * D;
  float* scale = a.c.scales + blk;
  // a page whose slot 0 is written starts over
  const float s_old = lo == 0 ? 0.f : *scale;

  // largest magnitude; what is not finite is stored as 0 and reported
  float m = 0.f, none = 0.f;   // none: 0 times every element, 0 unless one is not finite
#pragma unroll
  for (int i = 0; i < kAppRounds; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m = fmaxf(m, fabsf(x[i][j]));
      none = fmaf(x[i][j], 0.f, none);
    }
  if (none != 0.f) {
    set_err(a.err, FUTR_ERR_NOT_FINITE);
    m = 0.f;
#pragma unroll
    for (int i = 0; i < kAppRounds; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(fabsf(x[i][j]) <= 3.4028234e38f)) x[i][j] = 0.f;
        m = fmaxf(m, fabsf(x[i][j]));
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_max[tid >> 5] = m;
  __syncthreads();   // every thread has read the old scale by now, too
  for (int w = 0; w < threads / 32; ++w) m = fmaxf(m, s_max[w]);
  const float s_new = fmaxf(s_old, pow2(scale_exp(m)));
  const float inv = __uint_as_float((254u << 23) - __float_as_uint(s_new));   // of a power of two: exact
  if (tid == 0 && s_new != s_old) *scale = s_new;
  if ((__float_as_uint(s_new) & 0x7FFFFFu) != 0u || s_new > 0x1p120f) {
    // an old scale that is no power of two as they are made here, but a program's own:
    // the rows are divided by it, x[0] a turn
#pragma unroll 1
    for (int slot = lo + rg; slot < hi; slot += rows) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __fdiv_rn(x[0][4 * h + j], s_new);
        *(reinterpret_cast<uint32_t*>(codes + (size_t)slot * D + h * (D / 2)) + lg) =
            e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
      }
#pragma unroll
      for (int i = 0; i + 1 < kAppRounds; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = x[i + 1][j];
    }
    return;
  }
  if (s_old > 0.f && s_new > s_old) {
    // the page's other slots at the new scale, 8 codes a thread
    const float ratio = s_old * inv;
    for (int i = tid; i < page * L; i += threads) {
      const int slot = i / L;
      if (slot >= lo && slot < hi) continue;
      uint2* at = reinterpret_cast<uint2*>(codes) + i;
      uint2 u = *at;
      uint32_t w[2] = {u.x, u.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 f0 = e4m3x2_to_f32(w[j] & 0xFFFFu), f1 = e4m3x2_to_f32(w[j] >> 16);
        w[j] = e4m3x2(f0.x * ratio, f0.y * ratio) | (e4m3x2(f1.x * ratio, f1.y * ratio) << 16);
      }
      *at = make_uint2(w[0], w[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kAppRounds; ++i) {
    const int slot = lo + i * rows + rg;
    if (slot < hi) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *(reinterpret_cast<uint32_t*>(codes + (size_t)slot * D + h * (D / 2)) + lg) =
            e4m3x2(x[i][4 * h] * inv, x[i][4 * h + 1] * inv) |
            (e4m3x2(x[i][4 * h + 2] * inv, x[i][4 * h + 3] * inv) << 16);
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& c, const PagedRows& r, int d, int dtype, const void* k, long long ld_k,
                                const void* v, long long ld_v, int* err, cudaStream_t st) {
  AppendArgs a{c, r, {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v)}, {ld_k, ld_v}, err};
  // touched pages: a sequence of n rows meets at most (n - 1) / page + 2, one row exactly 1
  const long long rows = r.n_rows, per = r.start ? 2 : 1;
  const long long bound = r.start ? rows / c.page + per * (rows < r.batch ? rows : r.batch) : r.batch;
  const long long items = bound < rows ? bound : rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)items, (unsigned)c.n_kv, 2);
  // a page's rows in four rounds; a single row's CTA has a row's lanes and some more,
  // for the page's other codes when the scale grows
  cfg.blockDim = dim3(r.start ? (unsigned)(c.page * (d / 8) / kAppRounds) : 64u);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool half = dtype == FUTR_DTYPE_F16;
  if (d == 128)
    return half ? cudaLaunchKernelEx(&cfg, paged_append_kernel<128, true>, a)
                : cudaLaunchKernelEx(&cfg, paged_append_kernel<128, false>, a);
  return half ? cudaLaunchKernelEx(&cfg, paged_append_kernel<64, true>, a)
              : cudaLaunchKernelEx(&cfg, paged_append_kernel<64, false>, a);
}

}  // namespace futr
