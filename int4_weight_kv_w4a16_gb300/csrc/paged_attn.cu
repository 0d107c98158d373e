// Causal grouped-query attention over the paged 8-bit cache, for any number of
// new rows per sequence.
//
//   x_j = scale * q'.k_j  (k_j = code * key scale),  visible max(0, p - window + 1) <= j <= p
//   o   = sum_j 2^(x_j log2 e) v_j / sum_j 2^(x_j log2 e)
//
// A row tile is up to R = 8 NT rows of one sequence that share a kv-head (row =
// new token x query head of the group).  Its work is a run of 64-position
// tiles; all runs of the call, one after the other, are cut into equal
// contiguous shares, one per CTA of a grid that fills the GPU once.  The cut is
// made on the device from the sequences' lengths, so ragged batches balance
// and a captured launch follows lengths that change.  A run that spans several
// CTAs leaves one record (m, l, O) per CTA; the CTA that arrives last adds them
// in CTA order: no result depends on timing.
//
// In a CTA warp 4 streams tiles (2- or 3-D tensor copies, one per page up to 64
// positions, swizzled so that the fragment reads below meet no bank conflicts)
// through a ring, warps 0..3 take 16 positions of each tile:
//   S^T = K q'^T: mma.m16n8k16 f16, A = 16 positions of key codes converted in
//     registers (exact: e4m3 is a subset of f16), B = the rows as columns;
//   w = 2^(x + log2(value scale) - M), M the running maximum of that exponent:
//     the value scale rides in the exponent, so w <= 1 is a safe f16 whatever
//     the scales are, and the normalizer adds w / value scale in fp32;
//   O^T += V^T w: A = value codes, converted the same way; the score fragment
//     becomes the B operand by an 8x8 register transpose.
// The query enters as f16, each row divided by a power of two near its largest
// element (put back in the score's factor): 11 significant bits, an order
// below the cache's own 4; so do the weights.  All sums are fp32.
//
// Bound by memory while R <= 16 (the codes are read once, 2 d bytes a position
// and kv-head), by the tensor pipe for long row runs.
#include "paged.cuh"

namespace futr {

namespace {

constexpr int kPaCW = 4;                        // consumer warps
constexpr int kPaThreads = (kPaCW + 1) * 32;
constexpr int kPaTile = 64;                     // positions of a tile
constexpr int kPaRing = 4;
constexpr unsigned long long kPaWaitNs = 1000000000ull;

template <int D, int NT>
struct PaLayout {
  static constexpr int R = 8 * NT;
  static constexpr int kStage = 2 * kPaTile * D;                // K and V codes
  static constexpr int kScale = kPaRing * kStage;               // [ring][4 sub-tiles] float4 (ks, lv, 1/vs, -)
  static constexpr int kQ = kScale + kPaRing * 4 * 16;          // query fragments [D/16][NT][32] uint2
  static constexpr int kQs = kQ + (D / 16) * NT * 32 * 8;       // [R] score factors
  static constexpr int kOLd = D + 4;
  static constexpr int kO = kQs + R * 4;                        // [R][kOLd] fp32
  static constexpr int kM = kO + R * kOLd * 4;                  // [4 warps][R]
  static constexpr int kL = kM + kPaCW * R * 4;                 // [4 warps][R]
  static constexpr int kBar = kL + kPaCW * R * 4;
  static constexpr int kBytes = kBar + 2 * kPaRing * 8 + 32;
};

__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, const int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long dl = global_ns() + kPaWaitNs;
  return mbar_wait_until(bar, parity, dl, err);
}

__device__ __forceinline__ void pa_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kPaCW * 32) : "memory"); }

__device__ __forceinline__ float pa_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cvt4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ shares --

// Row tile rt of a sequence (n rows from position p0, G query heads a kv-head,
// R rows a tile): its 64-position tiles [t0, t1).
struct TileRange {
  int t0, t1;
};
__device__ __forceinline__ TileRange row_tile(int n, int p0, int G, int R, int window, int rt) {
  const int rows = n * G, r0 = rt * R, r1 = min(rows, r0 + R) - 1;
  const int first = p0 + r0 / G, last = p0 + r1 / G;
  const int lo = window > 0 ? max(0, first - window + 1) : 0;
  return {lo / kPaTile, last / kPaTile + 1};
}

__device__ __forceinline__ long long seq_tiles(int n, int p0, int G, int R, int window) {
  long long w = 0;
  const int nrt = (n * G + R - 1) / R;
  for (int rt = 0; rt < nrt; ++rt) {
    const TileRange t = row_tile(n, p0, G, R, window, rt);
    w += t.t1 - t.t0;
  }
  return w;
}

// The position of a CTA in the call's work: sequence b, kv-head, row tile and
// the next 64-position tile.  Every warp keeps its own copy and steps it the
// same way.
struct Walk {
  int b, kvh, rt, row0, n, p0;
  long long per_head;      // tiles of one kv-head of sequence b
  long long u, u1;         // this CTA's share [u, u1), u advancing
  long long item0;         // unit index of the current item's first tile
  TileRange t;

  // Enter sequence b (rows known); the item that holds unit `at` of its units.
  __device__ __forceinline__ void enter(const PagedAttnArgs& a, int R, long long at, long long base) {
    kvh = (int)(at / per_head);
    long long rem = at - (long long)kvh * per_head;
    rt = 0;
    t = row_tile(n, p0, a.G, R, a.window, 0);
    while (rem >= t.t1 - t.t0) {
      rem -= t.t1 - t.t0;
      ++rt;
      t = row_tile(n, p0, a.G, R, a.window, rt);
    }
    item0 = base + at - rem;
  }

  // Step to the item after the current one (its units start at item0 + tiles).
  __device__ __forceinline__ void next_item(const PagedAttnArgs& a, int R) {
    item0 += t.t1 - t.t0;
    ++rt;
    if (rt * R >= n * a.G) {
      rt = 0;
      if (++kvh == a.Hkv) {
        kvh = 0;
        do {
          ++b;
          paged_seq(a.r, a.c, b, row0, n, p0);
        } while (n == 0);   // u < u1: a later sequence has rows
        per_head = seq_tiles(n, p0, a.G, R, a.window);
      }
    }
    t = row_tile(n, p0, a.G, R, a.window, rt);
  }
};

// Units of the whole call and the share of CTA `cta` of `ctas` (a full warp).
// Returns the number of CTAs that get a share.
__device__ __forceinline__ int find_share(const PagedAttnArgs& a, int R, int cta, int ctas, Walk& w, long long& total,
                                          bool report) {
  const int lane = threadIdx.x & 31;
  total = 0;
  for (int b0 = 0; b0 < a.r.batch; b0 += 32) {
    long long units = 0;
    if (b0 + lane < a.r.batch) {
      int row0, n, p0;
      if (!paged_seq(a.r, a.c, b0 + lane, row0, n, p0) && report) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
      units = seq_tiles(n, p0, a.G, R, a.window) * a.Hkv;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    total += units;
  }
  const int use = (int)(total < ctas ? total : ctas);
  if (cta >= use) return use;
  w.u = total * cta / use;
  w.u1 = total * (cta + 1) / use;
  long long before = 0;
  for (int b0 = 0; b0 < a.r.batch; b0 += 32) {
    int row0 = 0, n = 0, p0 = 0;
    long long per = 0;
    if (b0 + lane < a.r.batch) {
      paged_seq(a.r, a.c, b0 + lane, row0, n, p0);
      per = seq_tiles(n, p0, a.G, R, a.window);
    }
    long long incl = per * a.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > w.u);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.b = b0 + src;
      w.row0 = __shfl_sync(0xffffffffu, row0, src);
      w.n = __shfl_sync(0xffffffffu, n, src);
      w.p0 = __shfl_sync(0xffffffffu, p0, src);
      w.per_head = __shfl_sync(0xffffffffu, per, src);
      const long long base = before + __shfl_sync(0xffffffffu, incl - per * a.Hkv, src);
      w.enter(a, R, w.u - base, base);
      return use;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return 0;   // not reached: u < total
}

// ---------------------------------------------------------------- consumer --

template <int D, int NT>
struct PaWarp {
  float m[NT][2], l[NT][2], o[D / 16][NT][4];
  float qs[NT][2];
  int hi[NT][2], lo[NT][2];   // visible positions of this lane's columns
  int hi_min, lo_max;         // positions [lo_max, hi_min] are visible to every row

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

  // 16 positions from pos0: key codes at ks_, value codes at vs_ (16 rows of D
  // bytes each, swizzled by the copy), sc = (key scale, log2 and inverse of the
  // value scale); qf: the query fragments.  `written`: positions below it exist.
  __device__ __forceinline__ void sub_tile(const uint8_t* ks_, const uint8_t* vs_, float4 sc, const uint2* qf, int pos0,
                                           int written) {
    constexpr int CH = D / 64;   // 16-byte chunks of a lane's key dims
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int swz = D == 128 ? g : (g >> 1) & 3;   // rows g and g + 8 share it
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int ch = (CH * t + j) ^ swz;
      const uint4 k0 = *reinterpret_cast<const uint4*>(ks_ + g * D + ch * 16);
      const uint4 k1 = *reinterpret_cast<const uint4*>(ks_ + (g + 8) * D + ch * 16);
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t af[4];
        cvt4(w0[i], af[0], af[2]);
        cvt4(w1[i], af[1], af[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = qf[((4 * j + i) * NT + nt) * 32 + lane];
          mma_f16_16816(s[nt], af, q.x, q.y);
        }
      }
    }
    const int pa = pos0 + g, pb = pa + 8;
    const bool all = pos0 >= lo_max && pos0 + 15 <= hi_min;
    uint32_t bt[NT], bb[NT];
    bool moved = false;
    float corr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = sc.x * qs[nt][e];
        float xa = fmaf(s[nt][e], f, sc.y), xb = fmaf(s[nt][2 + e], f, sc.y);
        if (!all) {
          if (pa > hi[nt][e] || pa < lo[nt][e]) xa = -INFINITY;
          if (pb > hi[nt][e] || pb < lo[nt][e]) xb = -INFINITY;
        }
        float mx = fmaxf(xa, xb);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        const float mn = fmaxf(m[nt][e], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;   // nothing visible yet: 2^(-inf - 0) = 0
        corr[nt][e] = pa_ex2(m[nt][e] - ref);
        moved |= m[nt][e] != mn;
        m[nt][e] = mn;
        s[nt][e] = pa_ex2(xa - ref);
        s[nt][2 + e] = pa_ex2(xb - ref);
        l[nt][e] = fmaf(s[nt][e] + s[nt][2 + e], sc.z, l[nt][e] * corr[nt][e]);
      }
      bt[nt] = movmatrix_trans(pack_half2(s[nt][0], s[nt][1]));
      bb[nt] = movmatrix_trans(pack_half2(s[nt][2], s[nt][3]));
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
    // slots that no row has been written to may hold anything, NaN codes
    // included: their codes are cleared (a weight of 0 alone would not do)
    uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};
    if (pos0 + 16 > written) {
#pragma unroll
      for (int i = 0; i < 4; ++i) keep[i] = pos0 + 2 * t + (i & 1) + 8 * (i >> 1) < written ? ~0u : 0u;
    }
#pragma unroll
    for (int jj = 0; jj < D / 32; ++jj) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * t + (i & 1) + 8 * (i >> 1);
        const int ch = (2 * jj + (g >> 2)) ^ (D == 128 ? row & 7 : (row >> 1) & 3);
        v[i] = *reinterpret_cast<const uint32_t*>(vs_ + row * D + ch * 16 + (g & 3) * 4) & keep[i];
      }
      uint32_t p0a, p0b, p1a, p1b, p2a, p2b, p3a, p3b;   // dims 0..3 of this lane, position pairs a, b
      cvt4(__byte_perm(v[0], v[1], 0x5140), p0a, p1a);
      cvt4(__byte_perm(v[0], v[1], 0x7362), p2a, p3a);
      cvt4(__byte_perm(v[2], v[3], 0x5140), p0b, p1b);
      cvt4(__byte_perm(v[2], v[3], 0x7362), p2b, p3b);
      const uint32_t a0[4] = {p0a, p1a, p0b, p1b}, a1[4] = {p2a, p3a, p2b, p3b};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16_16816(o[2 * jj][nt], a0, bt[nt], bb[nt]);
        mma_f16_16816(o[2 * jj + 1][nt], a1, bt[nt], bb[nt]);
      }
    }
  }
};

template <bool kHalf>
__device__ __forceinline__ float widen(uint16_t u) {
  return kHalf ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}

template <bool kHalf>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if (kHalf) return pack_half2(a, b);
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Row r of the tile (one warp): rotated, divided by a power of two and stored
// as f16 into its place in the B fragments; its score factor to qs[r].
template <int D, int NT, bool kHalf>
__device__ __forceinline__ void load_query(const PagedAttnArgs& a, const Walk& w, int r, int valid, __half* qf,
                                           float* qs) {
  constexpr int J = D / 32, CH = D / 64;
  const int lane = threadIdx.x & 31;
  float x[J];
#pragma unroll
  for (int j = 0; j < J; ++j) x[j] = 0.f;
  float factor = 0.f;
  if (r < valid) {
    const int row = w.rt * 8 * NT + r, i = row / a.G, head = w.kvh * a.G + row - i * a.G;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)(w.row0 + i) * a.ld_q + (size_t)head * D;
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] = widen<kHalf>(q[lane + 32 * j]);
    if (a.c.rope) {
      const float2* cs = a.c.rope + (size_t)(w.p0 + i) * (D / 2);
#pragma unroll
      for (int j = 0; j < J / 2; ++j) {
        const float2 f = cs[lane + 32 * j];
        const float x1 = x[j], x2 = x[j + J / 2];
        x[j] = x1 * f.x - x2 * f.y;
        x[j + J / 2] = x2 * f.x + x1 * f.y;
      }
    }
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) mx = fmaxf(mx, fabsf(x[j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // exponent of the largest element, kept where 2^e and 2^-e are normal
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < J; ++j) x[j] *= inv;
    factor = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int i = lane + 32 * j, t = i / (16 * CH), rem = i % (16 * CH), ks = (rem / 16) * 4 + (rem % 16) / 4;
    qf[((ks * NT + (r >> 3)) * 32 + (r & 7) * 4 + t) * 4 + (i & 3)] = __float2half_rn(x[j]);
  }
  if (lane == 0) qs[r] = factor;
}

template <int D, int NT, bool kHalf>
__global__ void __launch_bounds__(kPaThreads, NT <= 2 ? 3 : 2)
    paged_attn_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap map) {
  using Lay = PaLayout<D, NT>;
  constexpr int R = Lay::R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* s_scale = reinterpret_cast<float4*>(smem + Lay::kScale);
  uint2* qf = reinterpret_cast<uint2*>(smem + Lay::kQ);
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
  Walk w;
  long long total;
  const int cta = blockIdx.x;
  const int ctas = find_share(a, R, cta, gridDim.x, w, total, cta == 0 && warp == 0);
  if (cta >= ctas) return;
  const int page = a.c.page, plog = a.c.page_log2;

  if (warp == kPaCW) {
    // ---------------------------------------------------------- producer --
    // copies of a tile: whole (page, kv-head) blocks, keys then values, for
    // pages up to 64 positions; else 64 rows of keys and 64 of values
    const int ppt = page >= kPaTile ? 1 : kPaTile / page;   // pages of a tile
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (w.u < w.u1 && ok) {
      const int first = w.t.t0 + (int)(w.u - w.item0);
      const int count = (int)(min(w.u1, w.item0 + (w.t.t1 - w.t.t0)) - w.u);
      const int end = min(w.p0 + w.n, (first + count) * kPaTile);   // positions needed
      // page ids and scales, 32 pages a round (one per lane), one round ahead
      const int pg0 = (first * kPaTile) >> plog, pg1 = (end - 1) >> plog;
      const int* tab = a.r.table + (size_t)w.b * a.r.table_ld;
      auto fetch = [&](int pg, int& id, float2& s) {
        id = pg <= pg1 ? tab[pg] : 0;
        if (id < 0 || id >= a.c.n_pages) {
          set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
          id = -1;
        }
        s = make_float2(0.f, 0.f);
        if (id >= 0) s = reinterpret_cast<const float2*>(a.c.scales)[(size_t)id * a.Hkv + w.kvh];
      };
      int id, id_next = 0, base = pg0;
      float2 sc, sc_next = make_float2(0.f, 0.f);
      fetch(base + lane, id, sc);
      if (base + 32 <= pg1) fetch(base + 32 + lane, id_next, sc_next);
      for (int i = 0; i < count && ok; ++i) {
        const int pos = (first + i) * kPaTile, pg = pos >> plog;
        if (pg >= base + 32) {   // 32 is a multiple of the pages of a tile and base of their number: no tile straddles
          base += 32;
          id = id_next;
          sc = sc_next;
          if (base + 32 <= pg1) fetch(base + 32 + lane, id_next, sc_next);
        }
        if (issued >= kPaRing && !pa_wait(&empty[slot], phase ^ 1u, a.err)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + slot * Lay::kStage;
        // the 4 sub-tiles' scales
        const int mine = lane < 4 ? ((pos + 16 * lane) >> plog) - base : 0;
        const float kscale = __shfl_sync(0xffffffffu, sc.x, mine & 31), vscale = __shfl_sync(0xffffffffu, sc.y, mine & 31);
        const int myid = __shfl_sync(0xffffffffu, id, mine & 31);
        if (lane < 4) {
          // log2 of the value scale, its power of two apart (a scale of 0, a
          // page never written, counts as the smallest; a missing page as
          // not visible)
          float lv = (float)kPagedMinExp, inv = __uint_as_float((uint32_t)(127 - kPagedMinExp) << 23);
          if (vscale > 0.f) {
            const uint32_t u = __float_as_uint(vscale);
            lv = (float)((int)(u >> 23) - 127) + log2f(__uint_as_float((u & 0x7FFFFFu) | 0x3F800000u));
            inv = __fdiv_rn(1.0f, vscale);
          }
          if (myid < 0) lv = -INFINITY;
          s_scale[slot * 4 + lane] = make_float4(kscale, lv, inv, 0.f);
        }
        __syncwarp();
        if (page <= kPaTile) {
          const int last = min(ppt, ((end - 1 - pos) >> plog) + 1);   // pages of this tile
          const uint32_t bytes = (uint32_t)(2 * page * D);
          const int zid = __shfl_sync(0xffffffffu, id, (pg - base + lane) & 31);
          const bool have = lane < last && zid >= 0;
          const unsigned mask = __ballot_sync(0xffffffffu, have);
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes * __popc(mask));
          __syncwarp();
          if (have)
            tma_3d(smem_u32(st + lane * bytes), &map, 0, (int)(a.block0 + (long long)zid * a.Hkv + w.kvh), &full[slot]);
        } else {
          const int zid = __shfl_sync(0xffffffffu, id, (pg - base) & 31);
          if (lane == 0) {
            const int z = (int)(a.block0 + (long long)zid * a.Hkv + w.kvh), y = pos & (page - 1);
            mbar_arrive_expect_tx(&full[slot], zid >= 0 ? Lay::kStage : 0u);
            if (zid >= 0) {
              tma_3d(smem_u32(st), &map, y, z, &full[slot]);
              tma_3d(smem_u32(st + kPaTile * D), &map, page + y, z, &full[slot]);
            }
          }
        }
        ++issued;
        if (++slot == kPaRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
      w.u += count;
      if (w.u < w.u1) w.next_item(a, R);
    }
    if (!ok) {
      record_timeout(a.err);
      *s_dead = 1;
    }
    if (lane == 0) *s_issued = issued;
  } else {
    // ---------------------------------------------------------- consumers --
    const int g = lane >> 2, t = lane & 3;
    // where a sub-tile's codes lie in a stage
    const int pin = 16 * warp;                               // first position in the tile
    const int koff = page <= kPaTile ? (pin >> plog) * (2 * page * D) + (pin & (page - 1)) * D : pin * D;
    const int voff = koff + (page <= kPaTile ? page * D : kPaTile * D);
    PaWarp<D, NT> aw;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (w.u < w.u1) {
      const int first = w.t.t0 + (int)(w.u - w.item0);
      const int count = (int)(min(w.u1, w.item0 + (w.t.t1 - w.t.t0)) - w.u);
      const int valid = min(R, w.n * a.G - w.rt * R);
      for (int r = warp; r < R; r += kPaCW) load_query<D, NT, kHalf>(a, w, r, valid, reinterpret_cast<__half*>(qf), s_qs);
      pa_sync();
      aw.init();
      aw.hi_min = 0x7fffffff;
      aw.lo_max = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          aw.qs[nt][e] = s_qs[r];
          const int p = w.p0 + (w.rt * R + min(r, valid - 1)) / a.G;
          aw.hi[nt][e] = p;
          aw.lo[nt][e] = a.window > 0 ? p - a.window + 1 : 0;
        }
      aw.hi_min = w.p0 + (w.rt * R) / a.G;
      aw.lo_max = a.window > 0 ? w.p0 + (w.rt * R + valid - 1) / a.G - a.window + 1 : 0;
      const int written = w.p0 + w.n;
      for (int i = 0; i < count; ++i) {
        if (ok && !pa_wait(&full[slot], phase, a.err)) {
          ok = false;
          record_timeout(a.err);
          *s_dead = 1;
        }
        const int pos0 = (first + i) * kPaTile + pin;
        if (ok && pos0 < written && s_scale[slot * 4 + warp].y != -INFINITY)
          aw.sub_tile(smem + slot * Lay::kStage + koff, smem + slot * Lay::kStage + voff, s_scale[slot * 4 + warp], qf,
                      pos0, written);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        if (++slot == kPaRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // ---- the four warps' (m, l, O): common maximum, then O added in shared
      // memory, each warp on its own quarter of the dims per round
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = aw.l[nt][e];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
          if (g == 0) {
            s_m[warp * R + 8 * nt + 2 * t + e] = aw.m[nt][e];
            s_l[warp * R + 8 * nt + 2 * t + e] = v;
          }
        }
      if (tid == 0) *s_snap = *s_dead;   // one value for every branch below
      pa_sync();
      float f[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          const float M = fmaxf(fmaxf(s_m[r], s_m[R + r]), fmaxf(s_m[2 * R + r], s_m[3 * R + r]));
          f[nt][e] = M == -INFINITY ? 0.f : pa_ex2(aw.m[nt][e] - M);
        }
#pragma unroll
      for (int k = 0; k < kPaCW; ++k) {
        // round k: quarter (warp + k) mod 4 of the D / 16 row tiles
#pragma unroll
        for (int qd = 0; qd < kPaCW; ++qd)
          if (qd == ((warp + k) & 3)) {
#pragma unroll
            for (int jq = 0; jq < D / 64; ++jq) {
              const int j = qd * (D / 64) + jq;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float2* p = reinterpret_cast<float2*>(s_o + (8 * nt + 2 * t + e) * Lay::kOLd + 32 * (j >> 1) + 4 * g +
                                                        2 * (j & 1));
                  float2 v = make_float2(aw.o[j][nt][e] * f[nt][e], aw.o[j][nt][2 + e] * f[nt][e]);
                  if (k > 0) {
                    const float2 c = *p;
                    v.x += c.x;
                    v.y += c.y;
                  }
                  *p = v;
                }
            }
          }
        pa_sync();
      }
      // ---- a whole item: the rows; a part of one: a record, and the CTA that
      // arrives last adds the records in CTA order
      const long long item1 = w.item0 + (w.t.t1 - w.t.t0);
      const bool whole = w.u == w.item0 && w.u + count == item1;
      const int dead = *s_snap;
      bool write = whole && !dead;
      if (!whole && !dead) {
        float* rec = a.rec + ((size_t)cta * 2 + (w.item0 < w.u ? 0 : 1)) * (R * (D + 2));
        for (int r = tid; r < valid; r += kPaCW * 32) {
          const float M = fmaxf(fmaxf(s_m[r], s_m[R + r]), fmaxf(s_m[2 * R + r], s_m[3 * R + r]));
          float L = 0.f;
#pragma unroll
          for (int k = 0; k < kPaCW; ++k)
            L += s_m[k * R + r] == -INFINITY ? 0.f : s_l[k * R + r] * pa_ex2(s_m[k * R + r] - M);
          rec[r] = M;
          rec[R + r] = L;
        }
        for (int e = tid; e < valid * (D / 4); e += kPaCW * 32) {
          const int r = e / (D / 4), c = e - r * (D / 4);
          reinterpret_cast<float4*>(rec + 2 * R)[e] = *reinterpret_cast<const float4*>(s_o + r * Lay::kOLd + 4 * c);
        }
        pa_sync();
        // the CTAs of this item: those whose shares hold its first and last unit
        const int c0 = (int)(((w.item0 + 1) * ctas - 1) / total), c1 = (int)((item1 * ctas - 1) / total);
        if (tid == 0) {
          const unsigned arrived = atom_add_acq_rel_gpu(&a.cnt[c0], 1u);
          *s_last = arrived == (unsigned)(c1 - c0) ? 1 : 0;
          if (*s_last) a.cnt[c0] = 0u;
        }
        pa_sync();
        if (*s_last) {
          write = true;
          // maximum and normalizer of each row into s_m, s_l of warp 0
          const size_t step = (size_t)2 * R * (D + 2);
          const float* r0 = a.rec + ((size_t)c0 * 2 + 1) * (R * (D + 2));   // CTA c0's second slot
          const float* rn = a.rec + (size_t)(c0 + 1) * step;                 // the others' first
          const int nc = c1 - c0;                                            // others
          for (int r = warp; r < valid; r += kPaCW) {
            float M = lane == 0 ? __ldcg(r0 + r) : -INFINITY;
            for (int k = lane; k < nc; k += 32) M = fmaxf(M, __ldcg(rn + k * step + r));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            float L = 0.f;
            if (M != -INFINITY) {
              if (lane == 0) L = __ldcg(r0 + R + r) * pa_ex2(__ldcg(r0 + r) - M);
              for (int k = lane; k < nc; k += 32) L += __ldcg(rn + k * step + R + r) * pa_ex2(__ldcg(rn + k * step + r) - M);
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            }
            if (lane == 0) {
              s_m[r] = M;
              s_l[r] = L;
            }
          }
          pa_sync();
          for (int e = tid; e < valid * (D / 4); e += kPaCW * 32) {
            const int r = e / (D / 4), c = e - r * (D / 4);
            const float M = s_m[r] == -INFINITY ? 0.f : s_m[r];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kU = 8;   // records in flight
            for (int k = -1; k < nc; k += kU) {
              float4 v[kU];
              float mm[kU];
#pragma unroll
              for (int i = 0; i < kU; ++i)
                if (k + i < nc) {
                  const float* src = k + i < 0 ? r0 : rn + (size_t)(k + i) * step;
                  mm[i] = __ldcg(src + r);
                  v[i] = __ldcg(reinterpret_cast<const float4*>(src + 2 * R) + e);
                }
#pragma unroll
              for (int i = 0; i < kU; ++i)
                if (k + i < nc) {
                  const float wt = pa_ex2(mm[i] - M);
                  acc.x = fmaf(v[i].x, wt, acc.x);
                  acc.y = fmaf(v[i].y, wt, acc.y);
                  acc.z = fmaf(v[i].z, wt, acc.z);
                  acc.w = fmaf(v[i].w, wt, acc.w);
                }
            }
            *reinterpret_cast<float4*>(s_o + r * Lay::kOLd + 4 * c) = acc;
          }
          pa_sync();
        }
      } else if (write) {
        for (int r = tid; r < valid; r += kPaCW * 32) {
          const float M = fmaxf(fmaxf(s_m[r], s_m[R + r]), fmaxf(s_m[2 * R + r], s_m[3 * R + r]));
          float L = 0.f;
#pragma unroll
          for (int k = 0; k < kPaCW; ++k)
            L += s_m[k * R + r] == -INFINITY ? 0.f : s_l[k * R + r] * pa_ex2(s_m[k * R + r] - M);
          s_l[r] = L;   // this thread alone reads and writes row r of warp 0's sums
        }
        pa_sync();
      }
      if (write) {
        for (int e = tid; e < valid * (D / 8); e += kPaCW * 32) {
          const int r = e / (D / 8), c = e - r * (D / 8);
          const int row = w.rt * R + r, i = row / a.G, head = w.kvh * a.G + row - i * a.G;
          const float L = s_l[r], inv = L != 0.f ? __fdiv_rn(1.0f, L) : 0.f;   // a row that sees nothing: zeros
          const float4* p = reinterpret_cast<const float4*>(s_o + r * Lay::kOLd + 8 * c);
          const float4 v0 = p[0], v1 = p[1];
          uint4 u;
          u.x = narrow2<kHalf>(v0.x * inv, v0.y * inv);
          u.y = narrow2<kHalf>(v0.z * inv, v0.w * inv);
          u.z = narrow2<kHalf>(v1.x * inv, v1.y * inv);
          u.w = narrow2<kHalf>(v1.z * inv, v1.w * inv);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(w.row0 + i) * a.ld_out + (size_t)head * D +
                                    8 * c) = u;
        }
      }
      w.u += count;
      if (w.u < w.u1) {
        w.next_item(a, R);
        pa_sync();   // s_o, s_m, s_l and the query fragments are free again
      }
    }
  }
  __syncthreads();
  if (*s_dead && tid == 0) drain_ring(full, kPaRing, *s_issued);
}

template <int D, int NT, bool kHalf>
size_t pa_smem() {
  return (size_t)PaLayout<D, NT>::kBytes + 1024;
}

template <int D, int NT, bool kHalf>
cudaError_t pa_configure(int dev) {
  static DeviceOnce configured;
  if (configured.done(dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, NT, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)pa_smem<D, NT, kHalf>());
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(paged_attn_kernel<D, NT, kHalf>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  configured.mark(dev);
  return cudaSuccess;
}

constexpr int kPaMaxPerSm = 3;   // CTAs an SM that any variant is launched with at most

template <int D, int NT, bool kHalf>
int pa_per_sm(int dev) {
  return remembered(occ_key(dev, D, NT * 2 + kHalf, 0), [&]() {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_attn_kernel<D, NT, kHalf>, kPaThreads,
                                                      pa_smem<D, NT, kHalf>()) != cudaSuccess ||
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

template <int D, int NT, bool kHalf>
cudaError_t pa_launch(const PagedAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = pa_configure<D, NT, kHalf>(dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count(dev) * pa_per_sm<D, NT, kHalf>(dev)));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = pa_smem<D, NT, kHalf>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel<D, NT, kHalf>, a, map);
}

template <int D, bool kHalf>
cudaError_t pa_launch_nt(const PagedAttnArgs& a, const CUtensorMap& map, cudaStream_t st) {
  // rows of a tile: one new token's group where every sequence has one row,
  // else 32 rows (several tokens of a group, or a chunk's tiles)
  const int rows = a.r.start == nullptr || a.r.n_rows <= a.r.batch ? a.G : 32;
  if (rows <= 8) return pa_launch<D, 1, kHalf>(a, map, st);
  if (rows <= 16) return pa_launch<D, 2, kHalf>(a, map, st);
  return pa_launch<D, 4, kHalf>(a, map, st);
}

}  // namespace

constexpr int kPaMaxRows = 32;

size_t paged_rec_floats(int d) { return (size_t)2 * kPaMaxRows * (d + 2); }

int paged_attn_ctas(int d) {
  (void)d;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return sm_count(dev) * kPaMaxPerSm;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, const CUtensorMap& map, int d, int dtype, cudaStream_t st) {
  const bool half = dtype == FUTR_DTYPE_F16;
  if (d == 128) return half ? pa_launch_nt<128, true>(a, map, st) : pa_launch_nt<128, false>(a, map, st);
  return half ? pa_launch_nt<64, true>(a, map, st) : pa_launch_nt<64, false>(a, map, st);
}

// Codes as [blocks][2 page][d] bytes, a block per (page, kv-head); boxes of
// a whole block up to pages of 64, else of 64 rows; rows of 128 (64) bytes
// with the 128-byte (64-byte) swizzle.
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
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)(page <= kPaTile ? 2 * page : kPaTile), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  return reinterpret_cast<Fn>(p)(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box,
                                 elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                 d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace futr
