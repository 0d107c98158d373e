// Causal grouped-query attention over the paged 8-bit cache, for any number of
// new rows per sequence.
//
//   x_j = scale * q'.k_j  (k_j = code * key scale),  visible max(0, p - window + 1) <= j <= p
//   and, with sinks, j < sinks (j <= p); the tiles in between are not in a row tile's run
//   o   = sum_j 2^(x_j log2 e) v_j / sum_j 2^(x_j log2 e)
//
// A row tile is up to 8 rows of one sequence that share a kv-head (row = new token
// x query head of the group).  Its work is a run of 128-position
// tiles; all runs of the call, one after the other, are cut into equal
// contiguous shares, one per CTA of a grid that fills the GPU once.  The cut is
// made on the device from the sequences' lengths, so ragged batches balance
// and a captured launch follows lengths that change.  A run that spans several
// CTAs leaves one record (m, l, O) per CTA; the CTA that arrives last adds them
// in CTA order: no result depends on timing.
//
// In a CTA warp 4 streams tiles (tensor copies, one per page, swizzled so that
// the fragment reads below meet no bank conflicts) through a ring, warps 0..3
// take 32 positions of each tile:
//   S^T = K q'^T: mma.m16n8k16 f16, A = 16 positions of key codes converted in
//     registers (exact: e4m3 is a subset of f16), B = the rows as columns;
//   w = 2^(x + log2(value scale) - M + 14), M the running maximum of that exponent:
//     the value scale rides in the exponent, so w <= 2^14 is a safe f16 whatever
//     the scales are, and the normalizer adds w / value scale in fp32 (2^14 is in
//     both and cancels; with w <= 1 a weight below 2^-24 of the largest became 0 or
//     2^-24 in the products but not in the normalizer);
//   O^T += V^T w: A = value codes, converted the same way; the score fragment
//     becomes the B operand by an 8x8 register transpose.
// The query enters as f16, each row divided by a power of two near its largest
// element (put back in the score's factor): 11 significant bits, below what bf16
// rows resolve; f16 rows, which resolve more, in two parts (22 bits; an output's
// error is then its own rounding, 2.0e-4, instead of 4.3e-4).  The second MMAs cost
// drafted tokens nothing (10.3 us), 32 ragged sequences of D = 128 34.6 us instead of
// 33.3.  The weights enter as f16: 11 bits down to 2^-28 of the largest, next to the 4 of
// the values they multiply.
// All sums are fp32.
//
// Bound by memory while a sequence has one row tile (the codes are read once, 2 d
// bytes a position and kv-head); further tiles of a sequence read them from L2.  32
// ragged sequences of 512 to 4096 positions (148 MB): 33.3 us, 4.4 TB/s; four of 20K
// to 50K (269 MB): 51.3 us, 5.2 TB/s; the copies alone, in equal shares of tiles, 30
// and 48.5 us.  One sequence of 1024 positions: 8.0 us, the latency of share -> page
// id -> tile -> join.  16 sequences with a window of 4096 and 4 sinks (135 MB): 30.8 us, and
// 29.8 without the sinks.
#include <climits>

#include "paged_dev.cuh"

namespace futr {

namespace {

constexpr int kPaCW = 4;                        // consumer warps
constexpr int kPaThreads = (kPaCW + 1) * 32;
// Blocks of 8 rows (MMA columns) in a row tile.  Two cost registers that one CTA in
// two then lacks: 8 sequences of 16 rows over 4000 positions take 50 us with two and
// 25 us with one (D = 128), 20 and 18 us (D = 64).
constexpr int NT = 1;
constexpr float kTopWeight = 14.f;   // log2 of the largest weight
constexpr int kPaRows = 8 * NT;
// An item's start and join count as three tiles in the cut.  With 0, 2, 3, 4 and 6: 32
// ragged sequences 36.8, 33.3, 33.3, 33.8, 35.3 us; four long ones 53.8, 52.0, 51.2, 51.2,
// 51.5; drafted tokens (D = 64) 13.2, 11.5, 10.4, 10.5, 11.0.
template <bool kSinks>
constexpr Rows kPaWork{kPaRows, 3, kSinks};

template <int D>
struct PaLayout {
  static constexpr int R = kPaRows;
  static constexpr int kRing = D == 128 ? 2 : 4;                // 64 KB of tiles: two CTAs share an SM's memory
  static constexpr int kStage = 2 * kPaTile * D;                // K and V codes
  static constexpr int kScale = kRing * kStage;                 // [ring][sub-tiles] float4 (ks, lv, 1/vs, -)
  static constexpr int kQ = kScale + kRing * kPaSub * 16;       // query fragments [D/16][NT][32][parts] uint2
  static constexpr int kQs = kQ + (D / 16) * NT * 32 * 16;      // [R] score factors
  static constexpr int kOLd = D + 4;
  static constexpr int kO = kQs + R * 4;                        // [4 warps][R][kOLd] fp32
  static constexpr int kM = kO + kPaCW * R * kOLd * 4;          // [4 warps][R]
  static constexpr int kL = kM + kPaCW * R * 4;                 // [4 warps][R]
  static constexpr int kBar = kL + kPaCW * R * 4;
  static constexpr int kBytes = kBar + 2 * kRing * 8 + 32;
};

__device__ __forceinline__ void pa_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kPaCW * 32) : "memory"); }

// ---------------------------------------------------------------- consumer --

// f16 parts of a query element, by the rows' type
template <bool kHalf>
constexpr int kQueryParts = kHalf ? 2 : 1;

// The consumers' current item, in shared memory: its bounds are read where they
// are needed instead of being held in registers through the tile loop.
struct PaItem {
  Walk w;
  Cut cut;
  int active;                    // this CTA has a share
  int first, count, valid;       // tiles of this CTA's part (from number `first` on), rows of the tile
  int written;                   // positions below it exist
  int hi_min, lo_max;            // positions [lo_max, hi_min] are visible to every row
  int hi_max, lo_min;            // positions that some row sees
  int back;                      // a row at p sees positions >= p - back
  int hi[kPaRows];                  // each row's position
};

template <int D, int kParts>
struct PaWarp {
  float m[NT][2], l[NT][2], o[D / 16][NT][4];
  float qs[NT][2];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
  }

  // 32 positions from pos0, in two halves of 16: key codes at ks[h], value codes
  // at vs[h] (16 rows of D bytes each, swizzled by the copy), sc[h] = (key scale,
  // log2 and inverse of the value scale); qf: the query fragments; positions
  // below it.written exist.  Two halves at a time: their products are
  // independent chains, and they share one maximum.
  template <bool kSinks>
  __device__ __forceinline__ void tile32(const uint8_t* const (&ks)[2], const uint8_t* const (&vs)[2],
                                         const float4 (&sc)[2], const __half* qf, const PaItem& it, int pos0, int sinks) {
    constexpr int CH = D / 64;   // 16-byte chunks of a lane's key dims
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int swz = D == 128 ? g : (g >> 1) & 3;   // rows g and g + 8 share it
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][nt][e] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int ch = (CH * t + j) ^ swz;
      uint32_t w[2][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 k = *reinterpret_cast<const uint4*>(ks[h] + (g + 8 * r) * D + ch * 16);
          w[h][r][0] = k.x; w[h][r][1] = k.y; w[h][r][2] = k.z; w[h][r][3] = k.w;
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t af[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cvt4(w[h][0][i], af[h][0], af[h][2]);
          cvt4(w[h][1][i], af[h][1], af[h][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2* q = reinterpret_cast<const uint2*>(qf + (((4 * j + i) * NT + nt) * 32 + lane) * 4 * kParts);
          const uint2 q0 = q[0];
#pragma unroll
          for (int h = 0; h < 2; ++h) mma_f16_16816(s[h][nt], af[h], q0.x, q0.y);
          if (kParts == 2) {
            const uint2 q1 = q[1];
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_f16_16816(s[h][nt], af[h], q1.x, q1.y);
          }
        }
      }
    }
    // positions below end[h] of a half exist (a missing page: none of them)
    int end[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) end[h] = sc[h].y == -INFINITY ? 0 : it.written;
    const bool all = (pos0 >= it.lo_max || (kSinks && pos0 + 31 < sinks)) && pos0 + 31 <= it.hi_min && end[0] > 0 && end[1] > 0;
    uint32_t bt[2][NT], bb[2][NT];
    bool moved = false;
    float corr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = sc[h].x * qs[nt][e];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = fmaf(s[h][nt][2 * r + e], f, sc[h].y);
            if (!all) {
              const int p = pos0 + 16 * h + 8 * r + g, top = it.hi[8 * nt + 2 * t + e];
              if (p > top || (p < top - it.back && !(kSinks && p < sinks)) || p >= end[h]) x = -INFINITY;
            }
            s[h][nt][2 * r + e] = x;
            mx = fmaxf(mx, x);
          }
        }
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        const float mn = fmaxf(m[nt][e], mx);
        // (nothing visible yet: 2^(-inf - 0) = 0)
        corr[nt][e] = pa_ex2(m[nt][e] - (mn == -INFINITY ? 0.f : mn));
        const float ref = mn == -INFINITY ? 0.f : mn - kTopWeight;
        moved |= m[nt][e] != mn;
        m[nt][e] = mn;
        float sum = l[nt][e] * corr[nt][e];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float wa = pa_ex2(s[h][nt][e] - ref), wb = pa_ex2(s[h][nt][2 + e] - ref);
          s[h][nt][e] = wa;
          s[h][nt][2 + e] = wb;
          sum = fmaf(wa + wb, sc[h].z, sum);
        }
        l[nt][e] = sum;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bt[h][nt] = movmatrix_trans(pack_half2(s[h][nt][0], s[h][nt][1]));
        bb[h][nt] = movmatrix_trans(pack_half2(s[h][nt][2], s[h][nt][3]));
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[j][nt][0] *= corr[nt][0];
          o[j][nt][1] *= corr[nt][1];
          o[j][nt][2] *= corr[nt][0];
          o[j][nt][3] *= corr[nt][1];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // slots that no row has been written to may hold anything, NaN codes
      // included: their codes are cleared (a weight of 0 alone would not do)
      const int p1 = pos0 + 16 * h;
      uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
      if (p1 + 16 > end[h]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) keep[i] = p1 + 2 * t + (i & 1) + 8 * (i >> 1) < end[h] ? ~0u : 0u;
      }
#pragma unroll
      for (int jj = 0; jj < D / 64; ++jj) {
        // dims 64 jj + 8 g .. + 7 of positions 2t, 2t + 1, 2t + 8, 2t + 9
        uint2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * t + (i & 1) + 8 * (i >> 1);
          const int ch = (4 * jj + (g >> 1)) ^ (D == 128 ? row & 7 : (row >> 1) & 3);
          v[i] = *reinterpret_cast<const uint2*>(vs[h] + row * D + ch * 16 + (g & 1) * 8);
          v[i].x &= keep[i];
          v[i].y &= keep[i];
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t v0 = q ? v[0].y : v[0].x, v1 = q ? v[1].y : v[1].x, v2 = q ? v[2].y : v[2].x,
                         v3 = q ? v[3].y : v[3].x;
          uint32_t a0[4], a1[4];   // rows g, g + 8: dims 4q, 4q + 1 (a0) and 4q + 2, 4q + 3 (a1)
          cvt4(__byte_perm(v0, v1, 0x5140), a0[0], a0[1]);
          cvt4(__byte_perm(v2, v3, 0x5140), a0[2], a0[3]);
          cvt4(__byte_perm(v0, v1, 0x7362), a1[0], a1[1]);
          cvt4(__byte_perm(v2, v3, 0x7362), a1[2], a1[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(o[4 * jj + 2 * q][nt], a0, bt[h][nt], bb[h][nt]);
            mma_f16_16816(o[4 * jj + 2 * q + 1][nt], a1, bt[h][nt], bb[h][nt]);
          }
        }
      }
    }
  }
};

// Rows warp, warp + 4, ... of the tile: rotated, divided by a power of two and
// stored as f16 into their places in the B fragments; their score factors to
// qs.  The loads of all of a warp's rows are in flight together.
template <int D, bool kHalf>
__device__ __forceinline__ void load_queries(const PagedAttnArgs& a, const Walk& w, int valid, __half* qf, float* qs) {
  constexpr int J = D / 32, CH = D / 64, RW = 8 * NT / kPaCW;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t u[RW][J];
  float2 cs[RW][J / 2];
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const int r = warp + kPaCW * k;
    if (r < valid) {
      const int row = w.rt * 8 * NT + r, i = row / a.G, head = w.kvh * a.G + row - i * a.G;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)(w.row0 + i) * a.ld_q + (size_t)head * D;
#pragma unroll
      for (int j = 0; j < J; ++j) u[k][j] = q[lane + 32 * j];
      if (a.c.rope) {
#pragma unroll
        for (int j = 0; j < J / 2; ++j) cs[k][j] = a.c.rope[(size_t)(w.p0 + i) * (D / 2) + lane + 32 * j];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const int r = warp + kPaCW * k;
    float x[J], factor = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = 0.f;
    if (r < valid) {
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] = widen<kHalf>(u[k][j]);
      if (a.c.rope) {
#pragma unroll
        for (int j = 0; j < J / 2; ++j) {
          const float x1 = x[j], x2 = x[j + J / 2];
          x[j] = x1 * cs[k][j].x - x2 * cs[k][j].y;
          x[j + J / 2] = x2 * cs[k][j].x + x1 * cs[k][j].y;
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) mx = fmaxf(mx, fabsf(x[j]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // exponent of the largest element, kept where 2^e and 2^-e are normal
      const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126);
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] *= inv;
      factor = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = lane + 32 * j, t = i / (16 * CH), rem = i % (16 * CH), ks = (rem / 16) * 4 + (rem % 16) / 4;
      const __half hi = __float2half_rn(x[j]);
      __half* at = qf + ((ks * NT + (r >> 3)) * 32 + (r & 7) * 4 + t) * 4 * kQueryParts<kHalf> + (i & 3);
      at[0] = hi;
      if (kHalf) at[4] = __float2half_rn(x[j] - __half2float(hi));
    }
    if (lane == 0) qs[r] = factor;
  }
}

// The records r0 and rn[0 .. nc - 1] (m [R], l [R], O [R][D] each) added into
// s_o and s_l in this order, in one pass with a running maximum: a thread takes
// 4 dims of a row, eight records in flight.
template <int D, int R>
__device__ __forceinline__ void sum_records(const float* r0, const float* rn, int nc, int valid, float* s_o, int ld,
                                         float* s_l) {
  constexpr size_t step = (size_t)2 * R * (D + 2);
  for (int e = threadIdx.x; e < valid * (D / 4); e += kPaCW * 32) {
    const int r = e / (D / 4), q = e - r * (D / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
    constexpr int kU = 8;
#pragma unroll 1
    for (int k = -1; k < nc; k += kU) {
      float4 v[kU];
      float mm[kU], ll[kU], mx = M;
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        mm[i] = -INFINITY;
        if (k + i < nc) {
          const float* src = k + i < 0 ? r0 : rn + (size_t)(k + i) * step;
          mm[i] = __ldcg(src + r);
          ll[i] = __ldcg(src + R + r);
          v[i] = __ldcg(reinterpret_cast<const float4*>(src + 2 * R) + e);
        }
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) mx = fmaxf(mx, mm[i]);
      const float ref = mx == -INFINITY ? 0.f : mx, f = pa_ex2(M - ref);
      acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
      L *= f;
      M = mx;
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (k + i < nc) {
          const float wt = pa_ex2(mm[i] - ref);
          acc.x = fmaf(v[i].x, wt, acc.x);
          acc.y = fmaf(v[i].y, wt, acc.y);
          acc.z = fmaf(v[i].z, wt, acc.z);
          acc.w = fmaf(v[i].w, wt, acc.w);
          L = fmaf(ll[i], wt, L);
        }
    }
    *reinterpret_cast<float4*>(s_o + r * ld + 4 * q) = acc;
    if (q == 0) s_l[r] = L;
  }
}

template <int D, bool kHalf, bool kSinks>
__global__ void __launch_bounds__(kPaThreads, 2)
    paged_attn_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap map) {
  using Lay = PaLayout<D>;
  constexpr int R = Lay::R, kPaRing = Lay::kRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* s_scale = reinterpret_cast<float4*>(smem + Lay::kScale);
  __half* qf = reinterpret_cast<__half*>(smem + Lay::kQ);
  float* s_qs = reinterpret_cast<float*>(smem + Lay::kQs);
  float* s_o = reinterpret_cast<float*>(smem + Lay::kO);
  float* s_m = reinterpret_cast<float*>(smem + Lay::kM);
  float* s_l = reinterpret_cast<float*>(smem + Lay::kL);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* empty = full + kPaRing;
  volatile int* s_dead = reinterpret_cast<volatile int*>(empty + kPaRing);   // a wait ran out
  volatile int* s_issued = s_dead + 1;
  volatile int* s_last = s_dead + 2;
  volatile int* s_snap = s_dead + 3;                                          // s_dead as the consumers saw it together
  __shared__ PaItem s_item;
  __shared__ float s_tot[2 * R];   // a part's (or the whole item's) maxima and normalizers
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kPaRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kPaCW);
    }
    fence_mbar_init();
    *s_dead = 0;
    *s_issued = 0;
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const int cta = blockIdx.x;
  const int page = a.c.page, plog = a.c.page_log2;

  if (warp == kPaCW) {
    // ---------------------------------------------------------- producer --
    Walk w;
    Cut cut;
    if (!find_share(a, kPaWork<kSinks>, cta, gridDim.x, w, cut, false)) return;
    int issued = 0;
    const bool ok = produce_tiles<D>(a, &map, kPaWork<kSinks>, w, smem, s_scale, full, empty, kPaRing, cut.total, issued);
    if (!ok) {
      pa_timeout(a);
      *s_dead = 1;
    }
    if (lane == 0) *s_issued = issued;
  } else {
    // ---------------------------------------------------------- consumers --
    const int g = lane >> 2, t = lane & 3;
    // where a sub-tile's codes lie in a stage
    int koff[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = 32 * warp + 16 * h;   // first position in the tile
      koff[h] = (p >> plog) * (2 * page * D) + (p & (page - 1)) * D;
    }
    const int voff = page * D;
    PaWarp<D, kQueryParts<kHalf>> aw;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    PaItem& it = s_item;
    if (warp == 0) {
      Walk w;
      Cut cut;
      const bool active = find_share(a, kPaWork<kSinks>, cta, gridDim.x, w, cut, cta == 0);
      if (lane == 0) {
        it.w = w;
        it.cut = cut;
        it.active = active;
      }
    }
    pa_sync();
    if (!it.active) return;
    for (bool more = true; more;) {
      if (tid == 0) {
        const Walk& c = it.w;
        it.first = first_number(kPaWork<kSinks>, c.t) + (int)(c.u - c.item0);
        it.count = (int)(min(c.u1, c.item0 + (c.t.t1 - c.t.t0)) - c.u);
        it.valid = min(R, c.n * a.G - c.rt * R);
        it.written = c.p0 + c.n;
        it.hi_min = c.p0 + (c.rt * R) / a.G;
        it.hi_max = c.p0 + (c.rt * R + it.valid - 1) / a.G;
        it.back = a.window > 0 ? a.window - 1 : 0x3fffffff;
        it.lo_min = it.hi_min - it.back;
        it.lo_max = it.hi_max - it.back;
      }
      pa_sync();
      const int valid = it.valid, count = it.count;
      if (tid < R) it.hi[tid] = it.w.p0 + (it.w.rt * R + min(tid, valid - 1)) / a.G;
      load_queries<D, kHalf>(a, it.w, valid, qf, s_qs);
      pa_sync();
      aw.init();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) aw.qs[nt][e] = s_qs[8 * nt + 2 * t + e];
      int pos0 = it.first * kPaTile + 32 * warp;
      for (int i = 0; i < count; ++i, pos0 += kPaTile) {
        if (ok && !pa_wait(&full[slot], phase, a)) {
          ok = false;
          pa_timeout(a);
          *s_dead = 1;
        }
        if (kSinks) pos0 = tile_of(a, kPaWork<kSinks>, it.w.t, it.first + i) * kPaTile + 32 * warp;
        if (ok && pos0 <= it.hi_max && (pos0 + 31 >= it.lo_min || (kSinks && pos0 < a.sinks))) {
          const uint8_t* st = smem + slot * Lay::kStage;
          const uint8_t* ks[2] = {st + koff[0], st + koff[1]};
          const uint8_t* vs[2] = {ks[0] + voff, ks[1] + voff};
          const float4 sc[2] = {s_scale[slot * kPaSub + 2 * warp], s_scale[slot * kPaSub + 2 * warp + 1]};
          aw.template tile32<kSinks>(ks, vs, sc, qf, it, pos0, a.sinks);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == kPaRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // ---- the four warps' (m, l, O) to shared memory, each at its own maximum
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = aw.l[nt][e];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
          const int r = 8 * nt + 2 * t + e;
          if (g == 0) {
            s_m[warp * R + r] = aw.m[nt][e];
            s_l[warp * R + r] = v;
          }
          if (r < valid) {
            float2* p = reinterpret_cast<float2*>(s_o + (warp * R + r) * Lay::kOLd + 8 * g);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
              p[32 * (j >> 2) + (j & 3)] = make_float2(aw.o[j][nt][e], aw.o[j][nt][2 + e]);
          }
        }
      if (tid == 0) *s_snap = *s_dead;   // one value for every branch below
      pa_sync();
      // the sums over the four warps, in warp order: a thread takes 4 dims of a
      // row; they stay where warp 0's were
      for (int e = tid; e < valid * (D / 4); e += kPaCW * 32) {
        const int r = e / (D / 4), q = e - r * (D / 4);
        const float M = fmaxf(fmaxf(s_m[r], s_m[R + r]), fmaxf(s_m[2 * R + r], s_m[3 * R + r]));
        const float ref = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int k = 0; k < kPaCW; ++k) {
          const float f = pa_ex2(s_m[k * R + r] - ref);
          const float4 v = *reinterpret_cast<const float4*>(s_o + (k * R + r) * Lay::kOLd + 4 * q);
          L = fmaf(s_l[k * R + r], f, L);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
        *reinterpret_cast<float4*>(s_o + r * Lay::kOLd + 4 * q) = acc;
        if (q == 0) {
          s_tot[r] = M;
          s_tot[R + r] = L;
        }
      }
      pa_sync();
      // ---- a whole item: the rows; a part of one: a record, and the CTA that
      // arrives last adds the records in CTA order
      const Walk& c = it.w;
      const long long item1 = c.item0 + (c.t.t1 - c.t.t0);
      const bool whole = c.u == c.item0 && c.u + count == item1;
      const int dead = *s_snap;
      bool write = whole && !dead;
      if (!whole && !dead) {
        float* rec = a.rec + ((size_t)cta * 2 + (c.item0 < c.u ? 0 : 1)) * (R * (D + 2));
        for (int r = tid; r < 2 * R; r += kPaCW * 32) rec[r] = s_tot[r];
        for (int e = tid; e < valid * (D / 4); e += kPaCW * 32) {
          const int r = e / (D / 4), q = e - r * (D / 4);
          reinterpret_cast<float4*>(rec + 2 * R)[e] = *reinterpret_cast<const float4*>(s_o + r * Lay::kOLd + 4 * q);
        }
        pa_sync();
        // the CTAs of this item: those whose shares hold its first and last unit
        const int c0 = it.cut.owner(c.item0), c1 = it.cut.owner(item1 - 1);
        if (tid == 0) {
          const unsigned arrived = atom_add_acq_rel_gpu(&a.cnt[c0], 1u);
          *s_last = arrived == (unsigned)(c1 - c0) ? 1 : 0;
          if (*s_last) a.cnt[c0] = 0u;
        }
        pa_sync();
        if (*s_last) {
          write = true;
          // CTA c0's second slot, then the others' first
          sum_records<D, R>(a.rec + ((size_t)c0 * 2 + 1) * (R * (D + 2)), a.rec + (size_t)(c0 + 1) * 2 * (R * (D + 2)),
                            c1 - c0, valid, s_o, Lay::kOLd, s_tot + R);
          pa_sync();
        }
      }
      if (write) {
        for (int e = tid; e < valid * (D / 8); e += kPaCW * 32) {
          const int r = e / (D / 8), q = e - r * (D / 8);
          const int row = c.rt * R + r, i = row / a.G, head = c.kvh * a.G + row - i * a.G;
          const float L = s_tot[R + r], inv = L != 0.f ? __fdiv_rn(1.0f, L) : 0.f;   // a row that sees nothing: zeros
          const float4* p = reinterpret_cast<const float4*>(s_o + r * Lay::kOLd + 8 * q);
          const float4 v0 = p[0], v1 = p[1];
          uint4 u;
          u.x = narrow2<kHalf>(v0.x * inv, v0.y * inv);
          u.y = narrow2<kHalf>(v0.z * inv, v0.w * inv);
          u.z = narrow2<kHalf>(v1.x * inv, v1.y * inv);
          u.w = narrow2<kHalf>(v1.z * inv, v1.w * inv);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(c.row0 + i) * a.ld_out + (size_t)head * D +
                                    8 * q) = u;
        }
      }
      more = c.u + count + kPaWork<kSinks>.pad < c.u1;
      if (more) {
        pa_sync();   // the sums, the query fragments and the item are free again
        if (tid == 0) {
          it.w.u += count;
          it.w.next_item(a, kPaWork<kSinks>);
        }
      }
    }
  }
  __syncthreads();
  if (*s_dead && tid == 0) drain_ring(full, kPaRing, *s_issued);
}

template <int D>
size_t pa_smem() {
  return (size_t)PaLayout<D>::kBytes + 1024;
}

template <int D, bool kHalf, bool kSinks>
cudaError_t pa_configure(int dev) {
  static DeviceOnce configured;
  if (configured.done(dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, kHalf, kSinks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)pa_smem<D>());
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(paged_attn_kernel<D, kHalf, kSinks>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  configured.mark(dev);
  return cudaSuccess;
}

constexpr int kPaMaxPerSm = 2;   // CTAs an SM that any variant is launched with at most

template <int D, bool kHalf, bool kSinks>
int pa_per_sm(int dev) {
  return remembered(occ_key(dev, D, kHalf + 2 * kSinks, 0), [&]() {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_attn_kernel<D, kHalf, kSinks>, kPaThreads,
                                                      pa_smem<D>()) != cudaSuccess ||
        n < 1) {
      cudaGetLastError();
      return 1;
    }
    return n < kPaMaxPerSm ? n : kPaMaxPerSm;
  });
}

int sm_count(int dev) {
  return remembered(occ_key(dev, 0, 0, 0), [&]() {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
  });
}

template <int D, bool kHalf, bool kSinks>
cudaError_t pa_launch(const PagedAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = pa_configure<D, kHalf, kSinks>(dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count(dev) * pa_per_sm<D, kHalf, kSinks>(dev)));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = pa_smem<D>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel<D, kHalf, kSinks>, a, map);
}

template <bool kSinks>
cudaError_t pa_launch_any(const PagedAttnArgs& a, const CUtensorMap& map, int d, bool half, cudaStream_t st) {
  if (d == 128) return half ? pa_launch<128, true, kSinks>(a, map, st) : pa_launch<128, false, kSinks>(a, map, st);
  return half ? pa_launch<64, true, kSinks>(a, map, st) : pa_launch<64, false, kSinks>(a, map, st);
}

// Rows (tokens x query heads of a kv-head) a sequence, on average, from which on the
// many-row kernel is faster.  It costs the same for any number up to 128, these tiles
// of 8 rows their number; but it has an SM for a CTA, which few (sequence, kv-head)
// pairs do not fill.  In us, these / that, after 4000 positions: 64 pairs, D = 128, 32
// rows 44 / 43, 48 rows 62 / 43, 64 rows 80 / 44; D = 64, 40 rows 38 / 38, 64 rows
// 56 / 38; 32 pairs, D = 128, 48 rows 36 / 29; D = 64, 48 rows 27 / 26; 16 pairs, D = 128,
// 48 rows 23 / 24; D = 64, 64 rows 22 / 22; 8 pairs after 8000, D = 128, 64 rows
// 27 / 30, 96 rows 35 / 31.  Where contexts are short or kv-heads few the two meet later:
// 64 pairs after 500, D = 64, 64 rows 20 / 20; 32 sequences of 2 kv-heads after 1000,
// D = 64, 64 rows 25 / 25.
constexpr int kTcPairs = 32;
int tc_min_rows(const PagedAttnArgs& a, int d) {
  return (long long)a.r.batch * a.Hkv < kTcPairs ? 80 : d == 128 ? 48 : 64;
}
// Where sequences may differ much (their rows are on the device), both kernels, each
// for its sequences: from 1024 rows on in all, where a chunk among single tokens costs
// the tiles of 8 rows more than two launches, and below 256 a sequence on average,
// where the single tokens are worth one.  31 single tokens and a chunk of 512 tokens
// after 2000 positions (G = 4): 85 us, by the tiles of 8 rows alone 253; with a chunk
// of 256 73 and 136; 64 sequences of 5 drafted tokens, where the many-row kernel finds
// nothing, 145 and 139.  Single tokens alone have no chunk (64 of G = 16 after 1000
// positions 36 with both, 32 with one): the rows beyond one token a sequence have to be
// worth one.
constexpr int kBothMinRows = 1024, kBothMaxRows = 256, kBothMinChunk = 512;

}  // namespace

// Floats of all CTAs' records on a device with `sms` SMs: two CTAs an SM of these
// kernels, or one of the many-row kernel.
size_t paged_rec_floats(int d, int sms) {
  const size_t few = (size_t)sms * kPaMaxPerSm * 2 * kPaRows * (d + 2), many = (size_t)sms * paged_tc_rec_floats(d);
  return few > many ? few : many;
}

int paged_attn_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return sm_count(dev);
}

int paged_attn_ctas(int sms) { return sms * kPaMaxPerSm; }

cudaError_t launch_paged_attention(const PagedAttnArgs& args, const CUtensorMap& map, int d, int dtype, cudaStream_t st) {
  PagedAttnArgs a = args;
  a.rows_lo = 0;
  a.rows_hi = INT_MAX;
  const long long rows = (long long)a.r.n_rows * a.G, batch = a.r.batch;
  const int least = tc_min_rows(a, d);
  const bool many = rows >= least * batch;
  const bool both = a.r.start && batch > 1 && rows >= kBothMinRows && rows < kBothMaxRows * batch &&
                    rows - batch * a.G >= kBothMinChunk;
  if (many || both) {
    if (both) a.rows_lo = least;
    const cudaError_t e = launch_paged_attention_tc(a, map, d, dtype, paged_attn_sms(), st);
    if (e != cudaSuccess || !both) return e;
    a.rows_lo = 0;
    a.rows_hi = least;
  }
  const bool half = dtype == FUTR_DTYPE_F16;
  return a.sinks > 0 ? pa_launch_any<true>(a, map, d, half, st) : pa_launch_any<false>(a, map, d, half, st);
}

// Codes as [blocks][2 page][d] bytes, a block per (page, kv-head), copied whole;
// rows of 128 (64) bytes with the 128-byte (64-byte) swizzle.
bool make_paged_map(CUtensorMap* m, const void* codes, int d, int page, uint64_t blocks) {
  static std::atomic<void*> entry{nullptr};
  void* p = entry.load(std::memory_order_acquire);
  if (!p) {
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    entry.store(p, std::memory_order_release);
  }
  using Fn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                          const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                          CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)(2 * page), blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)(2 * page) * d};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)(2 * page), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return reinterpret_cast<Fn>(p)(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box,
                                 elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace futr
