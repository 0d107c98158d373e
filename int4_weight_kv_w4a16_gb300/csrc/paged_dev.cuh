// Device code of the paged attention kernels (paged_attn.cu: few rows a sequence,
// paged_attn_tc.cu: many): waits and copies, and the cut of a call's work into
// equal shares.
#pragma once

#include "paged.cuh"

namespace futr {
namespace {

constexpr int kPaTile = 128;                    // positions of a tile: 32 a warp
constexpr int kPaSub = kPaTile / 16;            // 16-position sub-tiles: what one page is a multiple of
constexpr unsigned long long kPaWaitNs = 1000000000ull;

__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, const PagedAttnArgs& a) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long dl = global_ns() + kPaWaitNs;
  return mbar_wait_until(bar, parity, dl, a.stop);
}

// A wait ran out: the workspace is out of use until a check with it; the cache
// reports it, too, for a check without.
__device__ __forceinline__ void pa_timeout(const PagedAttnArgs& a) {
  record_timeout(a.stop);
  set_err(a.err, FUTR_ERR_TIMEOUT);
}

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

// ------------------------------------------------------------------ shares --

// a / b for a >= 0, b > 0, on the path to the first copy: unit counts are small
// numbers in all but the longest calls, and there one fp32 division, off by one
// at most, with its remainder checked costs a fraction of an integer division.
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 21) != 0) return a / b;
  int q = (int)__fdividef((float)(int)a, (float)(int)b);
  const int r = (int)a - q * (int)b;
  if (r < 0) --q;
  if (r >= (int)b) ++q;
  return q;
}

// Sequence b of the call: no rows where they are another launch's.
__device__ __forceinline__ bool my_seq(const PagedAttnArgs& a, int b, int& row0, int& n, int& p0) {
  const bool ok = paged_seq(a.r, a.c, b, row0, n, p0);
  if (n * a.G < a.rows_lo || n * a.G >= a.rows_hi) n = 0;
  return ok;
}

// What a kernel makes of rows: R rows a row tile, whose start (queries, the join of
// its parts) counts as much as `pad` tiles of positions.  The units of an item are
// `pad` that hold nothing, then its tiles.  sinks: the call has some (a constant: the
// kernels without them would be 1 to 3 % slower, 10.8 us for the drafted tokens that take
// 10.4).
struct Rows {
  int R, pad;
  bool sinks;
};

// Row tile rt of a sequence (n rows from position p0, R rows a tile): its tiles, those
// of the sinks first, then those from the first that its window meets.  They have
// consecutive numbers: without sinks the tiles' own, t0 .. t1 - 1; with sinks 0 .. t1 - t0
// - 1, the sinks' tiles their own, the others' t0 less.
struct TileRange {
  int t0, t1;
};
__device__ __forceinline__ int first_number(Rows s, const TileRange& t) { return s.sinks ? 0 : t.t0; }
__device__ __forceinline__ int tile_of(const PagedAttnArgs& a, Rows s, const TileRange& t, int number) {
  return s.sinks && number >= a.sink_tiles ? t.t0 + number : number;
}
__device__ __forceinline__ TileRange row_tile(const PagedAttnArgs& a, Rows s, int n, int p0, int rt) {
  int first = p0, last = p0;
  if (n > 1) {
    const int r0 = rt * s.R, r1 = min(n * a.G, r0 + s.R) - 1;
    first = p0 + r0 / a.G;
    last = p0 + r1 / a.G;
  }
  // (sinks that reach the window's tiles: one run from tile 0)
  const int lo = a.window > 0 ? max(0, first - a.window + 1) / kPaTile : 0;
  return {s.sinks ? lo - min(lo, a.sink_tiles) : lo, last / kPaTile + 1};
}

// The units of a sequence and kv-head.
__device__ __forceinline__ long long seq_units(const PagedAttnArgs& a, int n, int p0, Rows s) {
  long long w = 0;
  const int nrt = (n * a.G + s.R - 1) / s.R;
#pragma unroll 1
  for (int rt = 0; rt < nrt; ++rt) {
    const TileRange t = row_tile(a, s, n, p0, rt);
    w += s.pad + t.t1 - t.t0;
  }
  return w;
}

// `total` units cut into `use` shares: the first `rem` of per + 1, the others of per.
struct Cut {
  long long total, per;
  int use, rem;
  __device__ __forceinline__ void set(long long units, int ctas) {
    total = units;
    use = (int)(units < ctas ? units : ctas);
    per = units <= ctas ? 1 : quot(units, ctas);
    rem = (int)(units - per * use);
  }
  __device__ __forceinline__ long long begin(int cta) const { return per * cta + min(cta, rem); }
  __device__ __forceinline__ int owner(long long u) const {
    const long long big = (per + 1) * rem;
    return (int)(u < big ? quot(u, per + 1) : rem + (per == 1 ? u - big : quot(u - big, per)));
  }
};

// The position of a CTA in the call's work: sequence b, kv-head, row tile and
// the next tile.  The producer warp keeps one copy, the consumers another.
struct Walk {
  int b, kvh, rt, row0, n, p0;
  long long per_head;      // units of one kv-head of sequence b
  long long u, u1;         // this CTA's share [u, u1), u advancing
  long long item0;         // unit index of the current item's first tile
  TileRange t;

  // Enter sequence b (rows known); the item that holds unit `at` of its units.
  __device__ __forceinline__ void enter(const PagedAttnArgs& a, Rows s, long long at, long long base) {
    kvh = (int)quot(at, per_head);
    long long rem = at - (long long)kvh * per_head;
    rt = 0;
    t = row_tile(a, s, n, p0, 0);
#pragma unroll 1
    while (rem >= s.pad + t.t1 - t.t0) {
      rem -= s.pad + t.t1 - t.t0;
      ++rt;
      t = row_tile(a, s, n, p0, rt);
    }
    item0 = base + at - rem + s.pad;
    u = max(u, item0);
  }

  // Step to the first tile of the item after the current one, which is done (it may
  // lie behind this share).
  __device__ __forceinline__ void next_item(const PagedAttnArgs& a, Rows s) {
    item0 += t.t1 - t.t0 + s.pad;
    u = item0;
    ++rt;
    if (rt * s.R >= n * a.G) {
      rt = 0;
      if (++kvh == a.Hkv) {
        kvh = 0;
        do {
          ++b;
          my_seq(a, b, row0, n, p0);
        } while (n == 0);   // u < u1: a later sequence has rows
        per_head = seq_units(a, n, p0, s);
      }
    }
    t = row_tile(a, s, n, p0, rt);
  }
};

// The call's units, their cut, and the share of CTA `cta` (a full warp).  False:
// it has no tile.
__device__ __forceinline__ bool find_share(const PagedAttnArgs& a, Rows s, int cta, int ctas, Walk& w, Cut& cut,
                                           bool report) {
  const int lane = threadIdx.x & 31;
  int row0 = 0, n = 0, p0 = 0;   // of sequence b0 + lane
  long long per = 0, incl = 0;   // its units per kv-head; all units of this round's sequences up to it
  auto look = [&](int b0) {
    n = 0;
    per = 0;
    if (b0 + lane < a.r.batch) {
      if (!my_seq(a, b0 + lane, row0, n, p0) && report) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
      per = seq_units(a, n, p0, s);
    }
    incl = per * a.Hkv;
#pragma unroll 1
    for (int o = 1; o < 32 && o < a.r.batch; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
  };
  const int top = min(31, a.r.batch - 1);   // a lane whose prefix sum is complete
  long long total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.r.batch; b0 += 32) {
    look(b0);
    total += __shfl_sync(0xffffffffu, incl, top);
  }
  cut.set(total, ctas);
  if (cta >= cut.use) return false;
  w.u = cut.begin(cta);
  w.u1 = cut.begin(cta + 1);
  long long before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.r.batch; b0 += 32) {
    if (a.r.batch > 32) look(b0);   // up to 32 sequences: still at hand
    const unsigned hit = __ballot_sync(0xffffffffu, lane <= top && before + incl > w.u);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.b = b0 + src;
      w.row0 = __shfl_sync(0xffffffffu, row0, src);
      w.n = __shfl_sync(0xffffffffu, n, src);
      w.p0 = __shfl_sync(0xffffffffu, p0, src);
      w.per_head = __shfl_sync(0xffffffffu, per, src);
      const long long base = before + __shfl_sync(0xffffffffu, incl - per * a.Hkv, src);
      w.enter(a, s, w.u - base, base);
      return w.u < w.u1;
    }
    before += __shfl_sync(0xffffffffu, incl, top);
  }
  return false;   // not reached: u < total
}

// ---------------------------------------------------------------- producer --

// The tiles of a CTA's share into a ring of stages (a full warp): a tile's pages as
// whole (page, kv-head) blocks, keys then values, and the scales of its 16-position
// sub-tiles, (key scale, log2 and inverse of the value scale, 0).  False: a wait
// ran out (`issued` stages are under way or done).  total: the call's units.
template <int D>
__device__ __forceinline__ bool produce_tiles(const PagedAttnArgs& a, const CUtensorMap* map, Rows s, Walk& w,
                                              uint8_t* stages, float4* s_scale, uint64_t* full, uint64_t* empty,
                                              int ring, long long total, int& issued) {
  const int lane = threadIdx.x & 31, page = a.c.page, plog = a.c.page_log2;
  const int ppt = kPaTile >> plog;   // pages of a tile
  const uint32_t bytes = (uint32_t)(2 * page * D);
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  if (a.withhold && w.u1 == total) return ok;
  while (w.u < w.u1 && ok) {
    const int first = first_number(s, w.t) + (int)(w.u - w.item0);
    const int count = (int)(min(w.u1, w.item0 + (w.t.t1 - w.t.t0)) - w.u);
    const int last = tile_of(a, s, w.t, first + count - 1) * kPaTile;
    const int end = min(w.p0 + w.n, last + kPaTile);   // positions needed
    // page ids and scales, 32 pages a round (one per lane), one round ahead; pages are
    // numbered as their tiles are
    const int tlog = 7 - plog;
    const int pg0 = first << tlog;
    const int pg1 = s.sinks ? ((first + count - 1) << tlog) + ((end - 1 - last) >> plog) : (end - 1) >> plog;
    // (pages before the first row's window, behind the sinks, are not looked at: a program
    // may have given them back)
    const int seen = a.window > 0 ? max(0, w.p0 + w.rt * s.R / a.G - a.window + 1) >> plog : 0;
    const int* tab = a.r.table + (size_t)w.b * a.r.table_ld;
    auto fetch = [&](int pg, int& id, float2& sc) {
      // its place in the table
      const int at = s.sinks ? (tile_of(a, s, w.t, pg >> tlog) << tlog) + (pg & (ppt - 1)) : pg;
      const bool look = pg <= pg1 && (at >= seen || (s.sinks && at < a.sink_pages));
      id = look ? tab[at] : -1;
      if (id < 0 || id >= a.c.n_pages) {
        if (look) set_err(a.err, FUTR_ERR_OUT_OF_RANGE);
        id = -1;
      }
      sc = make_float2(0.f, 0.f);
      if (id >= 0) sc = reinterpret_cast<const float2*>(a.c.scales)[(size_t)id * a.Hkv + w.kvh];
    };
    int id, id_next = 0, base = pg0;
    float2 sc, sc_next = make_float2(0.f, 0.f);
    fetch(base + lane, id, sc);
    if (base + 32 <= pg1) fetch(base + 32 + lane, id_next, sc_next);
    for (int i = 0; i < count && ok; ++i) {
      const int pos = (first + i) * kPaTile, pg = pos >> plog;
      if (pg >= base + 32) {   // 32 and pg0 are multiples of the pages of a tile: no tile straddles
        base += 32;
        id = id_next;
        sc = sc_next;
        if (base + 32 <= pg1) fetch(base + 32 + lane, id_next, sc_next);
      }
      if (issued >= ring && !pa_wait(&empty[slot], phase ^ 1u, a)) {
        ok = false;
        break;
      }
      uint8_t* st = stages + slot * (2 * kPaTile * D);
      // the copies need the page ids only: they are under way while the
      // scales, loaded with the ids, arrive
      const int zid = __shfl_sync(0xffffffffu, id, (pg - base + lane) & 31);
      const bool have = lane < ppt && zid >= 0;
      const unsigned mask = __ballot_sync(0xffffffffu, have);
      if (have)
        tma_3d(smem_u32(st + lane * bytes), map, 0, (int)(a.block0 + (long long)zid * a.Hkv + w.kvh), &full[slot]);
      const int from = (((pos + 16 * (lane & (kPaSub - 1))) >> plog) - base) & 31;   // the page of sub-tile `lane`
      const float kscale = __shfl_sync(0xffffffffu, sc.x, from), vscale = __shfl_sync(0xffffffffu, sc.y, from);
      const int myid = __shfl_sync(0xffffffffu, id, from);
      if (lane < kPaSub) {
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
        s_scale[slot * kPaSub + lane] = make_float4(kscale, lv, inv, 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes * __popc(mask));
      ++issued;
      if (++slot == ring) {
        slot = 0;
        phase ^= 1u;
      }
    }
    w.u += count;
    if (w.u < w.u1) w.next_item(a, s);
  }
  return ok;
}

}  // namespace
}  // namespace futr
