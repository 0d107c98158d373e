// Attention over the paged 8-bit cache for many rows a sequence (chunks of a
// prompt), on the 5th-generation tensor cores.  The mathematics, the roundings
// and the cut of the work are those of paged_attn.cu; a row tile has 256 rows,
// two halves of 128 = the lanes of tensor memory.
//
// One CTA an SM, 14 warps:
//   warp 12      streams tiles of 128 positions (8-bit codes) into a ring;
//   warps 8-11   widen a tile's codes to f16 (exact) into operand buffers, keys (one)
//                and values (two, so that the next tile's are ready when this one's
//                products end): rows of 128 bytes (64 dims) with the 128-byte
//                swizzle, which is a K-major operand for Q K^T and an MN-major one
//                for P V; once for all 256 rows;
//   warp 13      issues the MMAs (kind::f16, M 128, fp32 accumulators):
//                S_h = Q_h K^T (operands in shared memory) and O_h += P_h V (P in
//                tensor memory), ordered P_0 V, S_0 of the next tile, P_1 V, S_1 of
//                the next tile, so that the softmax of one half runs under the
//                products of the other;
//   warps 0-7    the softmax: a thread per row reads its 128 scores from tensor
//                memory twice (maximum, then weights), and writes the weights as f16
//                over the scores it has read, where they are P V's A operand.
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (D columns each).
//
// The query of f16 rows has two f16 parts, as in paged_attn.cu.  At D = 128 the second
// takes the shared memory of a value buffer and of a stage of the ring, so that the
// next tile's copy and values wait for this one's products.
//
// The running reference M of a row follows its maximum only when that has grown
// by more than 2^4: weights, 2^11 at the reference, stay below f16's 2^16, the
// normalizer is fp32, and O, in tensor memory, is rescaled a few times an item instead
// of every tile.  A weight has 11 bits down to 2^-25 of the largest, and is nothing
// below 2^-36 of it.
//
// Bound by the tensor cores in principle (4 x 256 x 128 x D flops a tile take 2048
// cycles at D = 128).  Measured on four prompts' chunks of 512 rows after contexts to
// 8K, 32 heads over 8, D = 128: 82 us, 0.59 PFLOP/s of the seen positions (a reference that
// lags by 2^8: 1.5 us less).  A CTA's
// 20 tiles take some 5200 cycles each (a half's softmax, 3300 while it shares the
// schedulers with the other half's and the widening, and its products, 1024, follow
// one another); the start, the queries of two parts and the records of split items
// take a third of the time.  Steps of 64 positions, whose products could run under
// the softmax, took 104 us where this took 98: twice the reads of the queries from
// shared memory.
#include "paged_dev.cuh"

namespace futr {

namespace {

constexpr int kTcRows = 256, kTcHalf = 128;
// An item's start (queries) and end (records) count as four tiles in the cut: CTAs with
// three items ended last.  With 0, 3, 4, 5, 6 and 8 the chunks above take 98.1, 87.6,
// 86.0, 86.6, 88.0 and 90.8 us.
template <bool kSinks>
constexpr Rows kTcWork{kTcRows, 4, kSinks};
constexpr int kTcThreads = 14 * 32;
constexpr int kTcSoft = 8 * 32;                 // softmax threads
constexpr float kTiny = 1.17549435e-38f;
constexpr float kRefWeight = 11.f, kRefLag = 4.f;   // log2 of the weight at a row's reference, and of what the maximum may exceed it by

// f16 parts of a query element: two for f16 rows, as few rows have them, so that a
// row's error does not depend on the kernel its batch takes.  The chunks of the head
// comment with f16 rows: an error of 2.1e-4 in 104 us, with one part 4.3e-4 in 84 (the
// products of the scores lie between a half's softmaxes); four chunks of up to 256 rows
// after 4000 positions, D = 64: 40.5 and 37.8.
template <bool kHalf>
constexpr int kTcParts = kHalf ? 2 : 1;

template <int D, bool kHalf>
struct TcLayout {
  static constexpr int kParts = kTcParts<kHalf>;
  static constexpr bool kTight = D == 128 && kParts == 2;        // 227 KB hold one of each
  static constexpr int kValues = kTight ? 1 : 2;                 // value buffers
  static constexpr int kRing = kTight ? 1 : 2;                   // stages of 8-bit tiles
  static constexpr int kOp = kTcHalf * D * 2;                    // one f16 operand of 128 rows
  static constexpr int kQ = 0;                                   // [half][part]
  static constexpr int kK = kQ + 2 * kParts * kOp;
  static constexpr int kV = kK + kOp;
  static constexpr int kStage = kV + kValues * kOp;              // ring of 8-bit tiles
  static constexpr int kRaw = kStage + kRing * 2 * kPaTile * D;  // [ring][sub-tiles] float4
  static constexpr int kScale = kRaw + kRing * kPaSub * 16;      // [2][sub-tiles] float4, by tile parity
  static constexpr int kQs = kScale + 2 * kPaSub * 16;           // [256] score factors
  static constexpr int kBar = kQs + kTcRows * 4;
  static constexpr int kBytes = kBar + 24 * 8 + 64;
};

struct TcItem {
  Walk w;
  Cut cut;
  int active;
  int first, count, valid;       // tiles of this CTA's part (from number `first` on), rows of the tile
};

__device__ __forceinline__ void tc_soft_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kTcSoft) : "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane; the values are there after tc_wait_ld.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}

// The wait for loads, tied to the values it makes valid.
__device__ __forceinline__ void tc_wait_ld32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Shared-memory operand descriptor with the 128-byte swizzle: rows of 128 bytes in
// 8-row atoms of 1 KB (stride 1024); `lead`: bytes between 64-element blocks of an
// MN-major operand (a K-major operand's block is one row wide: unused).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t tc_desc_lo(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

// Instruction descriptors: D fp32, A and B f16, M = 128; N = 128 (scores), N = D
// with B MN-major (bit 16: values as [position][dim]).
constexpr uint32_t kIdescS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
template <int D>
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (((uint32_t)D >> 3) << 17) | ((128u >> 4) << 24);

// The issuer's instructions: the whole warp comes here and one elected lane issues, so
// that the operands stay in uniform registers.  Descriptors as their low words (the
// high word is the same for all).
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tc_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Byte offset of dim i of row r in an f16 operand (blocks of 64 dims, swizzled rows).
__device__ __forceinline__ int tc_at(int r, int i) {
  return (i >> 6) * (kTcHalf * 128) + r * 128 + ((((i & 63) >> 3) ^ (r & 7)) << 4) + (i & 7) * 2;
}

// The rows of one half that belong to this softmax warp (32 of them), rotated,
// divided by a power of two and stored as f16 (rows past `valid` as zeros); their
// score factors to qs.  16 lanes take a row, a lane D / 32 rotation pairs of it; the
// loads of eight rows are in flight together.  (A warp a row: 84.2 us for the chunks of the
// head comment, 6.5 of them an item's first queries, that take 5.5 here.  Their way to L2
// while the item before is still at work changed nothing.)
template <int D, bool kHalf>
__device__ __forceinline__ void tc_load_queries(const PagedAttnArgs& a, const Walk& w, int valid, int half, uint8_t* q16,
                                                float* qs) {
  constexpr int P = D / 32, RW = 4;   // pairs of a lane, steps of two rows at a time
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, sub = lane >> 4, at = P * (lane & 15);
  uint32_t lo[RW][P / 2], hi[RW][P / 2];
  float2 cs[RW][P];
  auto load = [&](int r0) {
    const int row = w.rt * kTcRows + kTcHalf * half + r0 + sub;
    int i = row / a.G, g = row - i * a.G;
#pragma unroll
    for (int k = 0; k < RW; ++k) {
#pragma unroll
      for (int j = 0; j < P / 2; ++j) lo[k][j] = hi[k][j] = 0u;
#pragma unroll
      for (int j = 0; j < P; ++j) cs[k][j] = make_float2(1.f, 0.f);
      if (kTcHalf * half + r0 + 2 * k + sub < valid) {
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)(w.row0 + i) * a.ld_q +
                            (size_t)(w.kvh * a.G + g) * D + at;
        if (P == 4) {
          const uint2 l = *reinterpret_cast<const uint2*>(q), h = *reinterpret_cast<const uint2*>(q + D / 2);
          lo[k][0] = l.x, lo[k][P / 2 - 1] = l.y;
          hi[k][0] = h.x, hi[k][P / 2 - 1] = h.y;
        } else {
          lo[k][0] = *reinterpret_cast<const uint32_t*>(q);
          hi[k][0] = *reinterpret_cast<const uint32_t*>(q + D / 2);
        }
        if (a.c.rope) {
          const float4* c = reinterpret_cast<const float4*>(a.c.rope + (size_t)(w.p0 + i) * (D / 2) + at);
#pragma unroll
          for (int j = 0; j < P / 2; ++j) {
            const float4 c2 = c[j];
            cs[k][2 * j] = make_float2(c2.x, c2.y);
            cs[k][2 * j + 1] = make_float2(c2.z, c2.w);
          }
        }
      }
      g += 2;   // two rows on
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (g >= a.G) {
          g -= a.G;
          ++i;
        }
    }
  };
#pragma unroll 1
  for (int r0 = 32 * warp; r0 < 32 * warp + 32; r0 += 2 * RW) {
    load(r0);
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const int r = r0 + 2 * k + sub;
      float x[2][P], mx = 0.f;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float x1 = widen<kHalf>((uint16_t)(lo[k][j / 2] >> (16 * (j & 1)))),
                    x2 = widen<kHalf>((uint16_t)(hi[k][j / 2] >> (16 * (j & 1))));
        x[0][j] = x1 * cs[k][j].x - x2 * cs[k][j].y;
        x[1][j] = x2 * cs[k][j].x + x1 * cs[k][j].y;
        mx = fmaxf(mx, fmaxf(fabsf(x[0][j]), fabsf(x[1][j])));
      }
      // the largest magnitudes of both rows: magnitudes order like their bits
      const uint32_t m0 = __reduce_max_sync(0xffffffffu, sub ? 0u : __float_as_uint(mx));
      const uint32_t m1 = __reduce_max_sync(0xffffffffu, sub ? __float_as_uint(mx) : 0u);
      const int e = min(max((int)((sub ? m1 : m0) >> 23) - 127, -126), 126);   // (2^-e is normal, too)
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* dst = q16 + tc_at(r, at + h * (D / 2));
        float v[P];
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = x[h][j] * inv;
#pragma unroll
        for (int part = 0; part < kTcParts<kHalf>; ++part) {
          if (P == 4)
            *reinterpret_cast<uint2*>(dst + part * (kTcHalf * D * 2)) =
                make_uint2(pack_half2(v[0], v[1]), pack_half2(v[P - 2], v[P - 1]));
          else
            *reinterpret_cast<uint32_t*>(dst + part * (kTcHalf * D * 2)) = pack_half2(v[0], v[1]);
#pragma unroll
          for (int j = 0; j < P; ++j) v[j] -= __half2float(__float2half_rn(v[j]));
        }
      }
      if ((lane & 15) == 0)
        qs[kTcHalf * half + r] =
            kTcHalf * half + r < valid ? __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2 : 0.f;
    }
  }
}

// The 16-column factors and terms of 32 columns: x = s f + b.
struct TcScale {
  float f0, f1, b0, b1;
};

// The columns of a tile that a row sees: low .. top, and those below `sink`.
struct TcSight {
  int low, top, sink;
};

// What it does not see of the chunk of 32 at column c to -inf.
template <bool kSinks>
__device__ __forceinline__ void tc_mask(float (&x)[32], int c, const TcSight& v) {
  const uint32_t hole = (uint32_t)max(0, v.low - v.sink);   // columns from `sink` on, before `low`
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (c + j > v.top || (kSinks ? (uint32_t)(c + j - v.sink) < hole : c + j < v.low)) x[j] = -INFINITY;
}

// The largest s f + b of 32 columns (f > 0; -inf where nothing is seen).
__device__ __forceinline__ float tc_max(const float (&s)[32], const TcScale& t) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    m0 = fmaxf(m0, s[j]);
    m1 = fmaxf(m1, s[16 + j]);
  }
  return fmaxf(fmaf(m0, t.f0, t.b0), fmaf(m1, t.f1, t.b1));
}

// Their weights 2^(s f + b - ref) as f16, and the sums of each 16.  (A masked score
// of -inf has weight 0: f > 0 wherever a position is seen; a row whose factor is 0
// has weights that nothing reads.)
__device__ __forceinline__ void tc_weights(const float (&s)[32], const TcScale& t, float ref, uint32_t (&h)[16],
                                           float& sum0, float& sum1) {
  const float b0 = t.b0 - ref, b1 = t.b1 - ref;
  float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    float w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = pa_ex2(fmaf(s[j + i], j < 16 ? t.f0 : t.f1, j < 16 ? b0 : b1));
      q[(j >> 4) * 2 + i] += w[i];
    }
    h[j >> 1] = pack_half2(w[0], w[1]);
  }
  sum0 = q[0] + q[1];
  sum1 = q[2] + q[3];
}

__device__ __forceinline__ TcScale tc_scale_of(const float4* sc, int c, float qf) {
  const float4 s0 = sc[2 * c], s1 = sc[2 * c + 1];
  // (a factor of 0 must not meet a masked score of -inf)
  return TcScale{fmaxf(s0.x * qf, kTiny), fmaxf(s1.x * qf, kTiny), s0.y, s1.y};
}

// What a warp's rows see of the chunk of 32 columns at column c: nothing, all of it, or some
// see some.  A warp's 32 rows are few tokens, so the borders of a tile that is cut (by a
// row's own position, its window, the sinks) lie in one or two of its chunks.
// (Comparisons for all four: 74 us for the fp16 chunks of a window of 1000 with 100 sinks
// that took 69.5 so, 85.8 for the chunks of the head comment that took 84.2.)
enum TcChunk { kNone, kSome, kAll };
template <bool kSinks>
__device__ __forceinline__ TcChunk tc_chunk(int c, const TcSight& v) {
  const bool all = c + 31 <= v.top && (c >= v.low || (kSinks && c + 31 < v.sink));
  if (__all_sync(0xffffffffu, all)) return kAll;
  const bool none = c > v.top || (c + 31 < v.low && !(kSinks && c < v.sink));
  return __all_sync(0xffffffffu, none) ? kNone : kSome;
}

// A row's maximum over the tile, chunks of 32 columns.  With and without a mask
// apart: the comparisons would cost every tile half as much again.  Rolled loops over
// 32 columns: with 64 a turn those chunks took 101 us where this took 93, unrolled 132 (the roles' code
// no longer fits the instruction cache); a row's 128 scores held in registers, by a
// split of the CTA's registers between the roles, 104 where this took 100.
template <bool kCut, bool kSinks>
__device__ __forceinline__ float tc_row_max(uint32_t ts, const float4* sc, float qf, const TcSight& v) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const TcChunk seen = kCut ? tc_chunk<kSinks>(32 * c, v) : kAll;
    if (seen == kNone) continue;
    float x[32];
    tc_ld32(ts + 32 * c, x);
    const TcScale t = tc_scale_of(sc, c, qf);
    tc_wait_ld32(x);
    if (seen == kSome) tc_mask<kSinks>(x, 32 * c, v);
    mx = fmaxf(mx, tc_max(x, t));
  }
  return mx;
}

// Its weights, over scores that have been read (chunk c's to columns 16 c .. 16 c +
// 15); returns their sum with each 16 columns times their inverse value scale.
template <bool kCut, bool kSinks>
__device__ __forceinline__ float tc_row_weights(uint32_t ts, const float4* sc, float qf, float ref,
                                                const TcSight& v) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t h[16];
    const TcChunk seen = kCut ? tc_chunk<kSinks>(32 * c, v) : kAll;
    if (seen == kNone) {
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = 0u;
      tc_st16(ts + 16 * c, h);
      continue;
    }
    float x[32];
    tc_ld32(ts + 32 * c, x);
    const TcScale t = tc_scale_of(sc, c, qf);
    tc_wait_ld32(x);
    if (seen == kSome) tc_mask<kSinks>(x, 32 * c, v);
    float sum0, sum1;
    tc_weights(x, t, ref, h, sum0, sum1);
    sum = fmaf(sum0, sc[2 * c].z, fmaf(sum1, sc[2 * c + 1].z, sum));
    tc_st16(ts + 16 * c, h);
  }
  return sum;
}

// An item that spans CTAs: how many follow its first CTA (0: nothing to join), and
// its rows.
struct TcJoin {
  int others, row0, kvh, rt, valid;
};

// The bounds of the current part from its walk (one thread).
__device__ __forceinline__ void tc_set(const PagedAttnArgs& a, Rows s, TcItem& it) {
  const Walk& c = it.w;
  it.first = first_number(s, c.t) + (int)(c.u - c.item0);
  it.count = (int)(min(c.u1, c.item0 + (c.t.t1 - c.t.t0)) - c.u);
  it.valid = min(kTcRows, c.n * a.G - c.rt * kTcRows);
}

template <int D, bool kHalf, bool kSinks>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_attn_tc_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap map) {
  using Lay = TcLayout<D, kHalf>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* s_raw = reinterpret_cast<float4*>(smem + Lay::kRaw);
  float4* s_scale = reinterpret_cast<float4*>(smem + Lay::kScale);
  float* s_qs = reinterpret_cast<float*>(smem + Lay::kQs);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);   // [ring] a tile's codes have landed
  uint64_t* empty = full + 2;            // [ring] they are widened
  uint64_t* qready = empty + 2;          // [2] the queries of a half are in place
  uint64_t* kready = qready + 2;         // keys widened
  uint64_t* kfree = kready + 1;          // both halves' scores are done
  uint64_t* vready = kfree + 1;          // [2] values widened, by the tile's parity
  uint64_t* vfree = vready + 2;          // [2] both halves' P V are done
  uint64_t* sfull = vfree + 2;           // [2] scores of a half in tensor memory, scales in shared memory
  uint64_t* pready = sfull + 2;          // [2] weights of a half in tensor memory
  uint64_t* odone = pready + 2;          // [2] P V of a half is done
  volatile int* s_dead = reinterpret_cast<volatile int*>(odone + 2);   // a wait ran out
  volatile int* s_issued = s_dead + 1;
  volatile int* s_snap = s_dead + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(odone + 2) + 4;
  __shared__ TcItem s_item;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Lay::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&vready[h], 4);
      mbar_init(&vfree[h], 1);
      mbar_init(&qready[h], 4);
      mbar_init(&sfull[h], 5);   // the MMAs and the four widening warps
      mbar_init(&pready[h], 4);
      mbar_init(&odone[h], 1);
    }
    mbar_init(kready, 4);
    mbar_init(kfree, 1);
    fence_mbar_init();
    *s_dead = 0;
    *s_issued = 0;
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *s_tmem, 0);
  pdl_trigger();
  pdl_wait();
  const int cta = blockIdx.x, page = a.c.page, plog = a.c.page_log2;
  TcItem& it = s_item;
  if (warp == 0) {
    Walk w;
    Cut cut;
    const bool active = find_share(a, kTcWork<kSinks>, cta, gridDim.x, w, cut, cta == 0);
    if (lane == 0) {
      it.w = w;
      it.cut = cut;
      it.active = active;
    }
  }
  __syncthreads();
  // each role steps its own copy
  const bool active = it.active;
  Walk w = it.w;
  __syncthreads();
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {   // in dead mode: nothing to wait for
    if (ok && !pa_wait(bar, parity, a)) {
      ok = false;
      pa_timeout(a);
      *s_dead = 1;
    }
    return ok;
  };

  auto vbuf = [](uint32_t t) { return Lay::kValues == 2 ? t & 1u : 0u; };   // tile t's value buffer

  if (warp == 12) {
    // ---------------------------------------------------------- producer --
    if (active) {
      int issued = 0;
      if (!produce_tiles<D>(a, &map, kTcWork<kSinks>, w, smem + Lay::kStage, s_raw, full, empty, Lay::kRing,
                            it.cut.total, issued)) {
        pa_timeout(a);
        *s_dead = 1;
      }
      if (lane == 0) *s_issued = issued;
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------ issuer --
    if (active) {
      uint32_t t = 0, done[2] = {0, 0};   // tiles begun; P V issued by half
      uint32_t part = 0, part1 = 0;       // parts, and parts with a second half
      const uint32_t q16 = tc_desc_lo(smem_u32(smem + Lay::kQ), 16), k16 = tc_desc_lo(smem_u32(smem + Lay::kK), 16);
      const uint32_t v16 = tc_desc_lo(smem_u32(smem + Lay::kV), kTcHalf * 128);
      auto scores = [&](int h) {
#pragma unroll
        for (int part = 0; part < Lay::kParts; ++part)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * (kTcHalf * 128) + (ks & 3) * 32) >> 4;
            tc_mma_ss(tm + 128 * h, q16 + (h * Lay::kParts + part) * (Lay::kOp >> 4) + off, k16 + off, kIdescS,
                      part + ks > 0);
          }
        tc_commit(&sfull[h]);
      };
      auto values = [&](int h, bool first) {
#pragma unroll
        for (int ks = 0; ks < kPaTile / 16; ++ks)
          tc_mma_ts(tm + 256 + D * h, tm + 128 * h + 8 * ks, v16 + vbuf(t) * (Lay::kOp >> 4) + ks * (2048 >> 4),
                    kIdescO<D>, !first || ks > 0);
        tc_commit(&odone[h]);
        ++done[h];
      };
      while (w.u < w.u1 && ok) {
        const int count = (int)(min(w.u1, w.item0 + (w.t.t1 - w.t.t0)) - w.u);
        const int nh = min(kTcRows, w.n * a.G - w.rt * kTcRows) > kTcHalf ? 2 : 1;
        // the first tile's scores
        if (!wait(kready, t & 1u)) break;
        for (int h = 0; h < nh; ++h) {
          if (!wait(&qready[h], (h == 0 ? part : part1) & 1u)) break;
          tc_fence_after();
          scores(h);
        }
        if (!ok) break;
        tc_commit(kfree);
        for (int i = 0; i < count && ok; ++i, ++t) {
          const bool more = i + 1 < count;
          if (!wait(&vready[t & 1], (t >> 1) & 1u)) break;
          for (int h = 0; h < nh && ok; ++h) {
            if (!wait(&pready[h], done[h] & 1u)) break;
            tc_fence_after();
            values(h, i == 0);
            if (h + 1 == nh) tc_commit(&vfree[t & 1]);
            if (more) {
              if (h == 0 && !wait(kready, (t + 1) & 1u)) break;
              tc_fence_after();
              scores(h);
              if (h + 1 == nh) tc_commit(kfree);
            }
          }
        }
        w.u += count;
        ++part;
        part1 += nh - 1;
        if (w.u < w.u1) w.next_item(a, kTcWork<kSinks>);
      }
      // the buffers' last releases, which no other tile waits for, have to arrive while
      // this CTA's shared memory is its own
      if (t > 0) wait(kfree, (t - 1) & 1u);
      for (uint32_t i = t > 2 ? t - 2 : 0; i < t; ++i) wait(&vfree[i & 1], (i >> 1) & 1u);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- widening --
    // A quarter-warp takes 4 chunks (of 16 codes) of rows r and r ^ 5: neither its
    // reads of the 8-bit rows nor its writes of the f16 rows meet a bank twice.
    if (active) {
      constexpr int kQr = D / 64;                       // column quarters of 64 codes
      const int wg = warp - 8, l = lane & 7, qd = lane >> 3;
      const int rl = (l >> 2) ? (qd ^ 5) : qd;          // row within 8
      // offsets of this lane's chunk: in the f16 operand, and of its four rows in a tile
      const int r0 = 32 * wg + rl;
      const int d0 = r0 * 128 + (((2 * (l & 3)) ^ rl) << 4), d1 = r0 * 128 + (((2 * (l & 3) + 1) ^ rl) << 4);
      const int sr = D == 128 ? rl : (rl >> 1) & 3;
      int src[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r = r0 + 8 * g;
        src[g] = (r >> plog) * (2 * page * D) + (r & (page - 1)) * D;
      }
      uint32_t t = 0, told[2] = {0, 0};   // tiles; arrivals at sfull by half
      while (w.u < w.u1) {
        const int first = first_number(kTcWork<kSinks>, w.t) + (int)(w.u - w.item0);
        const int count = (int)(min(w.u1, w.item0 + (w.t.t1 - w.t.t0)) - w.u);
        const int nh = min(kTcRows, w.n * a.G - w.rt * kTcRows) > kTcHalf ? 2 : 1;
        for (int i = 0; i < count; ++i, ++t) {
          const int slot = t % Lay::kRing;
          wait(&full[slot], (t / Lay::kRing) & 1u);
          const uint8_t* st = smem + Lay::kStage + slot * (2 * kPaTile * D);
          const float4 raw = s_raw[slot * kPaSub + (lane & (kPaSub - 1))];
          // what was never written, or lies on a missing page, becomes zeros
          const int left = w.p0 + w.n - tile_of(a, kTcWork<kSinks>, w.t, first + i) * kPaTile;   // written positions from the tile's first
          const unsigned gone = __ballot_sync(0xffffffffu, lane < kPaSub && raw.y == -INFINITY);
          const bool plain = left >= kPaTile && gone == 0u;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            // the operand buffer is free once the MMAs of the tile before (values in two
            // buffers: of the one before that) have read it
            const uint32_t prev = t - (kv ? Lay::kValues : 1);
            if (t >= (kv ? Lay::kValues : 1)) wait(kv ? &vfree[prev & 1] : kfree, kv ? (prev >> 1) & 1u : prev & 1u);
            uint8_t* dst = smem + (kv ? Lay::kV + vbuf(t) * Lay::kOp : Lay::kK);
            const uint8_t* from = st + kv * page * D;
            if (ok) {
#pragma unroll 2
              for (int g = 0; g < 4; ++g) {
#pragma unroll
                for (int h = 0; h < kQr; ++h) {
                  uint4 v = *reinterpret_cast<const uint4*>(from + src[g] + (((4 * h + (l & 3)) ^ sr) << 4));
                  if (!plain) {
                    const int r = r0 + 8 * g;
                    if (r >= left || ((gone >> (r >> 4)) & 1u)) v = make_uint4(0u, 0u, 0u, 0u);
                  }
                  uint4 o0, o1;
                  cvt4(v.x, o0.x, o0.y);
                  cvt4(v.y, o0.z, o0.w);
                  cvt4(v.z, o1.x, o1.y);
                  cvt4(v.w, o1.z, o1.w);
                  *reinterpret_cast<uint4*>(dst + d0 + g * 1024 + h * (kTcHalf * 128)) = o0;
                  *reinterpret_cast<uint4*>(dst + d1 + g * 1024 + h * (kTcHalf * 128)) = o1;
                }
              }
            }
            if (kv == 0 && wg == 0 && lane < kPaSub) s_scale[(t & 1) * kPaSub + lane] = raw;
            tc_proxy_fence();
            // (an arrival counts for this tile once the tile before is complete)
            if (kv == 0)
              for (int h = 0; h < nh; ++h)
                if (told[h]++ > 0) wait(&sfull[h], told[h] & 1u);
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(kv ? &vready[t & 1] : kready);
              if (kv == 0)
                for (int h = 0; h < nh; ++h) mbar_arrive(&sfull[h]);
              else
                mbar_arrive(&empty[slot]);
            }
          }
        }
        w.u += count;
        if (w.u < w.u1) w.next_item(a, kTcWork<kSinks>);
      }
    }
  } else {
    // ----------------------------------------------------------- softmax --
    TcJoin join{};
    const int half = warp >> 2, row = tid & (kTcHalf - 1);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tm + lanes + 128 * half, to = tm + lanes + 256 + D * half;
    if (active) {
      uint32_t t = 0, mine = 0;   // tiles of the CTA; tiles of this half
      for (bool more = true; more;) {
        if (tid == 0) tc_set(a, kTcWork<kSinks>, it);
        tc_soft_sync();
        const int count = it.count, valid = it.valid;
        const bool here = kTcHalf * half < valid;
        const int r = kTcHalf * half + row, myrow = it.w.rt * kTcRows + min(r, valid - 1);
        if (r < valid) {   // all rows on their way at once: the loads below take eight at a time
          const int i = myrow / a.G;
          const uint16_t* q = static_cast<const uint16_t*>(a.q) + (size_t)(it.w.row0 + i) * a.ld_q +
                              (size_t)(it.w.kvh * a.G + myrow - i * a.G) * D;
          for (int l = 0; l < D / 64; ++l) tc_prefetch(q + 64 * l);
          if (a.c.rope)
            for (int l = myrow - i * a.G; l < D / 32; l += a.G)
              tc_prefetch(a.c.rope + (size_t)(it.w.p0 + i) * (D / 2) + 16 * l);
        }
        float M = -INFINITY, L = 0.f;
        if (here) {
          tc_load_queries<D, kHalf>(a, it.w, valid, half, smem + Lay::kQ + half * Lay::kParts * Lay::kOp, s_qs);
          tc_proxy_fence();
          tc_fence_before();   // (the item's products follow the reads of the last one's sums)
          __syncwarp();
          if (lane == 0) mbar_arrive(&qready[half]);
          const float qf = s_qs[r];   // this warp wrote it
          const int p = it.w.p0 + myrow / a.G, back = a.window > 0 ? a.window - 1 : 0x3fffffff;
          for (int i = 0; i < count; ++i, ++mine) {
            const int pos0 = tile_of(a, kTcWork<kSinks>, it.w.t, it.first + i) * kPaTile;
            wait(&sfull[half], mine & 1u);
            tc_fence_after();
            const float4* sc = s_scale + ((t + i) & 1) * kPaSub;
            const int top = p - pos0, low = top - back;   // columns low .. top are visible
            const TcSight v{low, top, kSinks ? max(0, a.sinks - pos0) : 0};
            const bool cut = __any_sync(0xffffffffu, top < kPaTile - 1 || low > 0);
            const float mx = cut ? tc_row_max<true, kSinks>(ts, sc, qf, v)
                                 : tc_row_max<false, kSinks>(ts, sc, qf, v);
            // the reference moves when the maximum has outgrown it (or it has none yet)
            const bool grow = mx > M + kRefLag || (M == -INFINITY && mx > M);
            if (__any_sync(0xffffffffu, grow)) {
              const float now = grow ? mx : M;
              const float corr = M == now ? 1.f : pa_ex2(M - now);
              M = now;
              L *= corr;
              if (i > 0) {
                wait(&odone[half], (mine - 1) & 1u);   // the sums so far are complete
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  float o[32];
                  tc_ld32(to + 32 * c, o);
                  tc_wait_ld32(o);
#pragma unroll
                  for (int j = 0; j < 32; ++j) o[j] *= corr;
                  tc_st32(to + 32 * c, o);
                }
              }
            }
            const float ref = M == -INFINITY ? 0.f : M - kRefWeight;
            L += cut ? tc_row_weights<true, kSinks>(ts, sc, qf, ref, v)
                     : tc_row_weights<false, kSinks>(ts, sc, qf, ref, v);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[half]);
          }
          wait(&odone[half], (mine - 1) & 1u);
          tc_fence_after();
        }
        t += count;
        // ---- a whole item: its rows; a part of one: a record, which the joining kernel
        // adds to the others
        const Walk& c = it.w;
        const long long item1 = c.item0 + (c.t.t1 - c.t.t0);
        const bool whole = c.u == c.item0 && c.u + count == item1;
        if (tid == 0) *s_snap = *s_dead;
        tc_soft_sync();
        const bool live = *s_snap == 0;
        constexpr size_t kRecRow = kTcRows, kRec = (size_t)kTcRows * (D + 2);
        float* rec = a.rec + ((size_t)cta * 2 + (c.item0 < c.u ? 0 : 1)) * kRec;
        const bool row_ok = r < valid;
        const int i = myrow / a.G, head = c.kvh * a.G + myrow - i * a.G;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (size_t)(c.row0 + i) * a.ld_out + (size_t)head * D;
        if (live && here) {
          const float inv = L != 0.f ? __fdiv_rn(1.0f, L) : 0.f;   // a row that sees nothing: zeros
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            float o[32];
            tc_ld32(to + 32 * k, o);
            tc_wait_ld32(o);
            if (row_ok && whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint4 u;
                u.x = narrow2<kHalf>(o[8 * j] * inv, o[8 * j + 1] * inv);
                u.y = narrow2<kHalf>(o[8 * j + 2] * inv, o[8 * j + 3] * inv);
                u.z = narrow2<kHalf>(o[8 * j + 4] * inv, o[8 * j + 5] * inv);
                u.w = narrow2<kHalf>(o[8 * j + 6] * inv, o[8 * j + 7] * inv);
                *reinterpret_cast<uint4*>(out + 32 * k + 8 * j) = u;
              }
            } else if (row_ok) {
              // [dim quad][row] float4: neighbouring rows side by side
#pragma unroll
              for (int j = 0; j < 8; ++j)
                reinterpret_cast<float4*>(rec + 2 * kRecRow)[(8 * k + j) * kTcRows + r] =
                    make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
          if (row_ok && !whole) {
            rec[r] = M;
            rec[kRecRow + r] = L;
          }
        }
        // the CTA with an item's beginning describes the join
        if (!whole && live && c.item0 == c.u && tid == 0)
          join = TcJoin{it.cut.owner(item1 - 1) - cta, c.row0, c.kvh, c.rt, valid};
        more = c.u + count + kTcWork<kSinks>.pad < c.u1;
        if (more) {
          tc_soft_sync();   // the item's bounds are read no more
          if (tid == 0) {
            it.w.u += count;
            it.w.next_item(a, kTcWork<kSinks>);
          }
        }
      }
    }
    if (tid == 0) reinterpret_cast<TcJoin*>(a.rec + (size_t)gridDim.x * 2 * kTcRows * (D + 2))[cta] = join;
  }
  // every MMA has been waited for (odone, vfree), or, after a time-out, gets its time here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*s_dead && tid == 0) drain_ring(full, Lay::kRing, *s_issued);
  if (*s_dead && tid == 32) {
    const unsigned long long dl = global_ns() + 1000000ull;   // 1 ms: far longer than what is in flight takes
    while (global_ns() < dl) {
    }
  }
  __syncthreads();
  __syncwarp();
  if (warp == 13)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
}

// Joins the records of split items, in CTA order: block (c, y) rows 32 y .. 32 y + 31
// of the item that begins in CTA c, a lane per row, a warp per eighth of its dims.
// A kernel of its own, so that every SM takes part: the CTA that arrived last would
// read 133 KB a part by itself, 19 of them for one sequence of 256 rows over 8000
// positions: a call of 73 us became one of 46 (36.5 by now).  Where items have few parts
// it costs a launch: 96 us for the chunks above, 93 without it (both in equal shares of
// tiles).
constexpr int kTcJoinRows = 32;

template <int D, bool kHalf>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedAttnArgs a, int ctas) {
  constexpr size_t kRecRow = kTcRows, kRec = (size_t)kTcRows * (D + 2);
  constexpr int Q = D / 32;   // dim quads of a thread
  const int cta = blockIdx.x, r = kTcJoinRows * blockIdx.y + (threadIdx.x & 31), q0 = Q * (threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  const TcJoin join = reinterpret_cast<const TcJoin*>(a.rec + (size_t)ctas * 2 * kRec)[cta];
  if (join.others == 0 || r >= join.valid || a.stop[1] != 0) return;   // (after a time-out parts may be missing)
  const float* r0 = a.rec + ((size_t)cta * 2 + 1) * kRec + r;         // its CTA's second slot
  const float* rn = a.rec + (size_t)(cta + 1) * 2 * kRec + r;         // the others' first
  const int nc = join.others;
  float top = *r0;
#pragma unroll 4
  for (int k = 0; k < nc; ++k) top = fmaxf(top, rn[(size_t)k * 2 * kRec]);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int j = 0; j < Q; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = -1; k < nc; ++k) {
    const float* src = k < 0 ? r0 : rn + (size_t)k * 2 * kRec;
    const float wt = pa_ex2(src[0] - ref);
    sum = fmaf(src[kRecRow], wt, sum);
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const float4 v = reinterpret_cast<const float4*>(src - r + 2 * kRecRow)[(q0 + j) * kTcRows + r];
      acc[j].x = fmaf(v.x, wt, acc[j].x);
      acc[j].y = fmaf(v.y, wt, acc[j].y);
      acc[j].z = fmaf(v.z, wt, acc[j].z);
      acc[j].w = fmaf(v.w, wt, acc[j].w);
    }
  }
  const float inv = sum != 0.f ? __fdiv_rn(1.0f, sum) : 0.f;
  const int row = join.rt * kTcRows + r, i = row / a.G, head = join.kvh * a.G + row - i * a.G;
  uint16_t* out = static_cast<uint16_t*>(a.out) + (size_t)(join.row0 + i) * a.ld_out + (size_t)head * D + 4 * q0;
#pragma unroll
  for (int j = 0; j < Q; j += 2) {
    uint4 u;
    u.x = narrow2<kHalf>(acc[j].x * inv, acc[j].y * inv);
    u.y = narrow2<kHalf>(acc[j].z * inv, acc[j].w * inv);
    u.z = narrow2<kHalf>(acc[j + 1].x * inv, acc[j + 1].y * inv);
    u.w = narrow2<kHalf>(acc[j + 1].z * inv, acc[j + 1].w * inv);
    *reinterpret_cast<uint4*>(out + 4 * j) = u;
  }
}

template <int D, bool kHalf>
size_t tc_smem() {
  return (size_t)TcLayout<D, kHalf>::kBytes + 1024;
}

template <int D, bool kHalf, bool kSinks>
cudaError_t tc_launch(const PagedAttnArgs& a, const CUtensorMap& map, int ctas, cudaStream_t st) {
  static DeviceOnce configured;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.done(dev)) {
    e = cudaFuncSetAttribute(paged_attn_tc_kernel<D, kHalf, kSinks>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)tc_smem<D, kHalf>());
    if (e != cudaSuccess) return e;
    configured.mark(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = tc_smem<D, kHalf>();
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<D, kHalf, kSinks>, a, map);
  if (e != cudaSuccess) return e;
  // rows of a tile: no sequence has more than all of them
  const long long rows = (long long)a.r.n_rows * a.G;
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)((rows < kTcRows ? rows : kTcRows) + kTcJoinRows - 1) / kTcJoinRows);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kHalf>, a, ctas);
}

template <bool kSinks>
cudaError_t tc_launch_any(const PagedAttnArgs& a, const CUtensorMap& map, int d, bool half, int ctas, cudaStream_t st) {
  if (d == 128)
    return half ? tc_launch<128, true, kSinks>(a, map, ctas, st) : tc_launch<128, false, kSinks>(a, map, ctas, st);
  return half ? tc_launch<64, true, kSinks>(a, map, ctas, st) : tc_launch<64, false, kSinks>(a, map, ctas, st);
}

}  // namespace

size_t paged_tc_rec_floats(int d) { return (size_t)2 * kTcRows * (d + 2) + sizeof(TcJoin) / 4; }

cudaError_t launch_paged_attention_tc(const PagedAttnArgs& a, const CUtensorMap& map, int d, int dtype, int ctas,
                                      cudaStream_t st) {
  const bool half = dtype == FUTR_DTYPE_F16;
  return a.sinks > 0 ? tc_launch_any<true>(a, map, d, half, ctas, st) : tc_launch_any<false>(a, map, d, half, ctas, st);
}

}  // namespace futr
