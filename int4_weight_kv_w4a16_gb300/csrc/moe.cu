// Mixture-of-experts layer for 1..32 tokens with INT4 experts.
//
//   r_t = 1 / sqrt(mean x_t^2 + eps);  l_te = r_t sum_k (x_tk g_k) Wr_ek
//   the K largest l_te (equal ones: lowest expert first), p = softmax(l_t),
//   w = p of the chosen (divided by their sum if asked)
//   y_t = resid_t + sum_j w_tj Wd_e (silu(r_t W'g_e x_t) * (r_t W'u_e x_t)),  e = e_tj
//
// Three kernels with programmatic dependent launch:
//   router   the logits, a CTA per two experts and eight tokens, which also leaves
//            its part of the tokens as f16; the CTA that arrives last for its eight
//            tokens picks their experts, a warp per token;
//   gate/up  streams the chosen experts' gate/up units once;
//   down     streams their down units once, beginning before gate/up has ended.
// Every CTA of the expert kernels sorts the (token, expert) pairs by expert itself,
// on every SM at once: less time than one CTA takes to do it for the others and
// hand it over.
// Above 8 tokens a fourth adds down's parts.
//
// The expert kernels are bound by the weight stream: 17 tokens through 8 of 128
// experts (4096 x 1536, 830 MB) take 172 us, 4.8 TB/s; 32 through 2 of 8 (4096 x
// 14336, 726 MB) 193 us, 3.8 TB/s, where the unpacking and the products of up to 16
// columns take as long as the stream; one token through 2 of 8 (181 MB) 49 us, some
// 15 of them the router, the starts and the ends of three kernels.  All units of the
// chosen experts form one run, cut into equal contiguous shares, one per CTA of a
// grid that fills the GPU; the cut is made on the device from the routing.  A
// unit (128 rows x 128 inputs) comes by one bulk copy, the record of each of the
// expert's tokens (128 inputs) by one more; four warps unpack the
// nibbles straight into f16 A fragments and the tokens are the N side, so an
// expert costs its own tokens' columns only.  A row block that spans CTAs leaves
// one record per CTA, added in CTA order by the one that arrives last.  Down
// runs over (row block, expert, group) with the expert inside: the experts of a
// row block meet in one fp32 tile per token in shared memory, so y needs no
// second pass.
//
// The products.  A nibble u = code + 8 is masked into the f16 1 + u/16 (rows g of an
// MMA tile) or 1 + u/256 (rows g + 8); one addition makes it code/16 or code/256, both
// exact, and 16 (256) is multiplied in once at the end.  With the nibbles as masked, and
// accumulators that start at -1.5 (-1.03125) times the inputs' sum, the additions are
// saved (listed calls 2 to 8 % faster), but what the accumulators hold is then up to 264
// times what the codes leave: inputs of one sign, 16384 of them, cost an output 3.1e-4.
//
// Rounding: inputs are f16 (x divided by a power of two near its RMS, so bf16
// values keep all their bits down to 2^-14 of it; w * silu * up, the routing
// weight inside, by one at the largest of each 64: 11 bits).  Everything else is
// fp32 until y.
#include "moe.cuh"

namespace futr {

namespace {

constexpr int kMoeCW = 4;
constexpr int kMoeThreads = (kMoeCW + 1) * 32;
constexpr int kMoeMaxPerSm = 3;
constexpr int kRouterThreads = 512;
constexpr int kRouterE = 2;        // experts of a router CTA
constexpr int kRouterSlices = kRouterThreads / 32 / kRouterE;   // parts of the inputs: a warp's share
constexpr unsigned long long kMoeWaitNs = 1000000000ull;

__device__ __forceinline__ bool moe_wait(uint64_t* bar, uint32_t parity, const int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long dl = global_ns() + kMoeWaitNs;
  return mbar_wait_until(bar, parity, dl, err);
}

__device__ __forceinline__ void moe_sync() { asm volatile("bar.sync 1, %0;" ::"r"(kMoeCW * 32) : "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 2^e at the leading bit of v >= 0 (1 for 0, and bounded so that 2^-e is normal).
__device__ __forceinline__ float pow2_at(float v) {
  const int e = min(max((int)(__float_as_uint(v) >> 23) - 127, -120), 120);
  return v > 0.f ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.f;
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// Whether the blob holds this layer's experts.  Where it does not, nothing behind its
// header is read: its units may end before the layer's would.
__device__ __forceinline__ bool own_blob(const MoeArgs& a) {
  const MoeHeader* h = reinterpret_cast<const MoeHeader*>(a.blob);
  return (h->magic == kMoeMagic) & (h->hidden == a.H) & (h->inter == a.I) & (h->n_experts == a.E);   // loads side by side
}

// ------------------------------------------------------------------ router --

// Floats in ascending order as unsigned integers in ascending order above 0 (NaN: below -inf).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t u = __float_as_uint(v + 0.f);   // -0 counts as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The experts of token t (a warp): the K largest logits, equal ones by the lowest
// index, and their weights.  Expert lane + 32 i in v[i].
__device__ __forceinline__ void pick_experts(const MoeArgs& a, int t) {
  constexpr int kV = kMoeMaxExperts / 32;
  const int lane = threadIdx.x & 31;
  float v[kV];
  uint32_t key[kV];   // the order of v; 0: taken, absent
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kV; ++i) v[i] = lane + 32 * i < a.E ? __ldcg(a.logits + (size_t)t * a.E + lane + 32 * i) : 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    key[i] = lane + 32 * i < a.E ? order_key(v[i]) : 0u;
    nan |= v[i] != v[i];
  }
  nan = __any_sync(0xffffffffu, nan);
  float mine = 0.f, top = 0.f;   // lane j: the j-th choice
  int mine_id = 0;
#pragma unroll 1
  for (int j = 0; j < a.K; ++j) {
    uint32_t bk = key[0];
    float bv = v[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < kV; ++i)
      if (32 * i < a.E && key[i] > bk) {
        bk = key[i];
        bv = v[i];
        bi = i;
      }
    const uint32_t best = __reduce_max_sync(0xffffffffu, bk);
    const int id = __reduce_min_sync(0xffffffffu, bk == best ? lane + 32 * bi : 0x7fffffff);
    const float val = __shfl_sync(0xffffffffu, bv, id & 31);
    if ((id & 31) == lane) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (i == id >> 5) key[i] = 0u;
    }
    if (j == 0) top = val;
    if (lane == j) {
      mine = val;
      mine_id = id;
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (32 * i < a.E) sum += lane + 32 * i < a.E ? expf(v[i] - top) : 0.f;
  sum = warp_sum(sum);
  float w = lane < a.K ? __fdiv_rn(expf(mine - top), sum) : 0.f;
  if (a.renorm) w = __fdiv_rn(w, warp_sum(w));
  if (nan) w = __int_as_float(0x7fc00000);
  if (lane < a.K) {
    const int p = t * a.K + lane;
    a.choice[p] = mine_id;
    a.share[p] = w;
    if (a.ids) a.ids[p] = mine_id;
    if (a.weights) a.weights[p] = w;
  }
}

__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a) {
  __shared__ float s_dot[kRouterE][kRouterSlices][kRouterT], s_sq[kRouterSlices][kRouterT];
  __shared__ float s_factor[kRouterT];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int et = blockIdx.x, t0 = blockIdx.y * kRouterT, nt = min(kRouterT, a.T - t0);
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0 && !own_blob(a)) set_err(a.err, FUTR_ERR_BAD_BLOB);
  // warp = (expert, slice): every kRouterSlices-th chunk of 256 inputs
  {
    const int el = warp / kRouterSlices, sl = warp % kRouterSlices, e = et * kRouterE + el;
    float acc[kRouterT], ss[kRouterT];
#pragma unroll
    for (int t = 0; t < kRouterT; ++t) acc[t] = ss[t] = 0.f;
    if (e < a.E || el == 0) {
      const __nv_bfloat16* wr = a.router + (size_t)min(e, a.E - 1) * a.H;
      for (int j = 256 * sl + 8 * lane; j < a.H; j += 256 * kRouterSlices) {
        float w[8];
        const uint4 wv = *reinterpret_cast<const uint4*>(wr + j);
        uint4 xv[kRouterT];
#pragma unroll
        for (int t = 0; t < kRouterT; ++t)
          if (t < nt) xv[t] = *reinterpret_cast<const uint4*>(a.x + (size_t)(t0 + t) * a.H + j);
        float g[8];
        if (a.gain) {
          const float4 g0 = *reinterpret_cast<const float4*>(a.gain + j), g1 = *reinterpret_cast<const float4*>(a.gain + j + 4);
          g[0] = g0.x; g[1] = g0.y; g[2] = g0.z; g[3] = g0.w;
          g[4] = g1.x; g[5] = g1.y; g[6] = g1.z; g[7] = g1.w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = 1.f;
        }
        const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[2 * i] = __uint_as_float(wu[i] << 16);
          w[2 * i + 1] = __uint_as_float(wu[i] & 0xffff0000u);
        }
#pragma unroll
        for (int t = 0; t < kRouterT; ++t)
          if (t < nt) {
            const uint32_t xu[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
            float s = 0.f, q = 0.f;   // sums of 8 first: a short chain of additions
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float lo = __uint_as_float(xu[i] << 16), hi = __uint_as_float(xu[i] & 0xffff0000u);
              s = fmaf(__fmul_rn(lo, g[2 * i]), w[2 * i], s);
              s = fmaf(__fmul_rn(hi, g[2 * i + 1]), w[2 * i + 1], s);
              q = fmaf(lo, lo, fmaf(hi, hi, q));
            }
            acc[t] += s;
            ss[t] += q;
          }
      }
    }
#pragma unroll
    for (int t = 0; t < kRouterT; ++t)
      if (t < nt) {
        const float s = warp_sum(acc[t]);
        if (lane == 0) s_dot[el][sl][t] = s;
        if (el == 0) {
          const float q = warp_sum(ss[t]);
          if (lane == 0) s_sq[sl][t] = q;
        }
      }
  }
  __syncthreads();
  if (tid < kRouterE * kRouterT) {
    const int el = tid / kRouterT, t = tid % kRouterT, e = et * kRouterE + el;
    if (t < nt) {
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int i = 0; i < kRouterSlices; ++i) {
        s += s_dot[el][i][t];
        q += s_sq[i][t];
      }
      const float mean = __fdiv_rn(q, (float)a.H);
      const float r = a.eps > 0.f ? __fdiv_rn(1.0f, sqrtf(mean + a.eps)) : 1.f;
      if (e < a.E) a.logits[(size_t)(t0 + t) * a.E + e] = r * s;
      if (el == 0) {
        const float f = pow2_at(sqrtf(mean));
        s_factor[t] = pow2_inverse(f);
        if (et == 0) a.rms[t0 + t] = r * f;
      }
    }
  }
  __syncthreads();
  // this CTA's part of its tokens as f16 records: a warp per record of 128 inputs
  const int ng = a.H / kGroup;
  for (int i = warp; ; i += kRouterThreads / 32) {
    const int t = i % kRouterT, g = et + i / kRouterT * (int)gridDim.x;
    if (g >= ng) break;
    if (t >= nt) continue;
    const uint2 v = *reinterpret_cast<const uint2*>(a.x + (size_t)(t0 + t) * a.H + g * kGroup + 4 * lane);
    const float f = s_factor[t];
    const __half2 h0 = __floats2half2_rn(__uint_as_float(v.x << 16) * f, __uint_as_float(v.x & 0xffff0000u) * f);
    const __half2 h1 = __floats2half2_rn(__uint_as_float(v.y << 16) * f, __uint_as_float(v.y & 0xffff0000u) * f);
    __half* rec = a.xh + ((size_t)(t0 + t) * ng + g) * kRecHalves;
    reinterpret_cast<uint2*>(rec)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  }
  // the last CTA of these tokens picks their experts
  __syncthreads();
  if (tid == 0) {
    s_last = atom_add_acq_rel_gpu(a.cnt + blockIdx.y, 1u) == gridDim.x - 1 ? 1 : 0;
    if (s_last) a.cnt[blockIdx.y] = 0u;
  }
  __syncthreads();
  if (s_last && warp < nt) pick_experts(a, t0 + warp);
}

// The routing, in shared memory.  A pair is one (token, chosen expert); pairs
// are ordered by expert, then token.
struct MoeRoute {
  unsigned mask[kMoeMaxExperts];             // tokens of each expert
  // the runs of at most C pairs of one expert: an expert of more pairs has several
  int n_active;
  uint16_t off[kMoeMaxPairs + 1];            // first pair of each
  uint16_t first[kMoeMaxExperts];            // first pair of each expert
  uint16_t pick[kMoeMaxPairs];               // of each pair: its place in the choices
  uint8_t expert[kMoeMaxPairs];              // its expert, ascending
  uint8_t token[kMoeMaxPairs];               // of each pair
};

// From the choices, by all threads of the CTA.  C: columns that one pass over an
// expert's units takes.
template <int C>
__device__ __forceinline__ void make_route(const MoeArgs& a, MoeRoute& rt) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pairs = a.T * a.K;
  constexpr int kP = (kMoeMaxPairs + kMoeThreads - 1) / kMoeThreads, kV = kMoeMaxExperts / 32;
  int id[kP], t[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int p = tid + i * kMoeThreads;
    id[i] = p < pairs ? __ldcg(a.choice + p) : 0;
    t[i] = p / a.K;
  }
  for (int i = tid; i < kMoeMaxExperts; i += kMoeThreads) rt.mask[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kP; ++i)
    if (tid + i * kMoeThreads < pairs) atomicOr(&rt.mask[id[i]], 1u << t[i]);
  __syncthreads();
  // experts in use and the first pair of each: prefix sums, eight experts a lane
  if (warp == 0) {
    unsigned m[kV];
    int n = 0, used = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      m[i] = rt.mask[kV * lane + i];
      n += __popc(m[i]);
      used += (__popc(m[i]) + C - 1) / C;
    }
    int both = n | (used << 16);   // at most 512 each
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, both, o);
      if (lane >= o) both += x;
    }
    if (lane == 31) {
      rt.n_active = both >> 16;
      rt.off[both >> 16] = (uint16_t)(both & 0xffff);
    }
    int pn = (both & 0xffff) - n, pu = (both >> 16) - used;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      rt.first[kV * lane + i] = (uint16_t)pn;
      const int cnt = __popc(m[i]);
      for (int c = 0; c < cnt; c += C) {
        rt.expert[pu] = (uint8_t)(kV * lane + i);
        rt.off[pu] = (uint16_t)(pn + c);
        ++pu;
      }
      pn += cnt;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kP; ++i)
    if (tid + i * kMoeThreads < pairs) {
      const int at = rt.first[id[i]] + __popc(rt.mask[id[i]] & ((1u << t[i]) - 1u));
      rt.token[at] = (uint8_t)t[i];
      rt.pick[at] = (uint16_t)(tid + i * kMoeThreads);
    }
  __syncthreads();
}

// ---------------------------------------------------------- expert kernels --

template <int NT>
struct MoeLayout {
  // three CTAs an SM; with 32 columns two
  static constexpr int kRing = NT == 1 ? 6 : NT == 2 ? 4 : 5;
  static constexpr int kStage = kUnitBytes + 8 * NT * kRecBytes;  // unit, then [8 NT] records
  static constexpr int kRed = kRing * kStage;                    // [columns, down: tokens][kRedLd] fp32
  static constexpr int kBar = kRed + (NT == 1 ? 8 : kMaxBatch) * kRedLd * 4;
  static constexpr int kBytes = kBar + 2 * kRing * 8 + 16;
};

// The four f16x2 registers of a word (see moe.cuh): the placed nibbles read 1 + u/16
// (rows g) and 1 + u/256 (rows g + 8); less 1.5 and 1.03125 they are code/16 and
// code/256, exact.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b32 s, a, b, c, d;\n\t"
      "prmt.b32 s, %4, %4, 0x2301;\n\t"
      "lop3.b32 a, %4, 0x03C003C0, %5, 0xEA;\n\t"
      "lop3.b32 b, %4, 0x003C003C, %5, 0xEA;\n\t"
      "lop3.b32 c, s, 0x03C003C0, %5, 0xEA;\n\t"
      "lop3.b32 d, s, 0x003C003C, %5, 0xEA;\n\t"
      "add.rn.f16x2 %0, a, %6;\n\t"
      "add.rn.f16x2 %1, b, %7;\n\t"
      "add.rn.f16x2 %2, c, %6;\n\t"
      "add.rn.f16x2 %3, d, %7;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w), "r"(0x3C003C00u), "r"(0xBE00BE00u), "r"(0xBC20BC20u));
}
constexpr float kUnitA = 16.f, kUnitB = 256.f;

// One unit times NT tiles of 8 columns for this warp's 32 rows, the group's
// product times the rows' scales into acc.  Down: the two halves of the inputs
// have factors of their own.
template <int NT, bool kDown>
__device__ __forceinline__ void moe_unit(const uint8_t* st, const int (&xrow)[NT], const int (&col)[NT],
                                         float (&acc)[2][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2;
  const __half* tile = reinterpret_cast<const __half*>(st + kUnitBytes);
  const uint4* wt = reinterpret_cast<const uint4*>(st + 2 * warp * 1024);
  const __half* sc = reinterpret_cast<const __half*>(st + kUnitCodeBytes);
  uint32_t words[2][8];
  float s_lo[2], s_hi[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint4 w0 = wt[64 * m + lane], w1 = wt[64 * m + 32 + lane];
    words[m][0] = w0.x; words[m][1] = w0.y; words[m][2] = w0.z; words[m][3] = w0.w;
    words[m][4] = w1.x; words[m][5] = w1.y; words[m][6] = w1.z; words[m][7] = w1.w;
    const int r0 = (2 * warp + m) * 16 + gr;
    s_lo[m] = __half2float(sc[r0]);
    s_hi[m] = __half2float(sc[r0 + 8]);
  }
  // factors of this lane's two columns of each tile
  float2 tail[NT][2];
  if (kDown) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        tail[nt][i] = *reinterpret_cast<const float2*>(tile + (col[nt] + i) * kRecHalves + kGroup);
  }
  float d[2][NT][4], part[2][NT][4];
#pragma unroll
  for (int kp = 0; kp < 4; ++kp) {
    if (kp == 0 || (kDown && kp == 2)) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (kp == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) part[m][nt][i] = d[m][nt][i] * tail[nt][i & 1].x;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) d[m][nt][i] = 0.f;
        }
    }
    uint32_t b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) ldmatrix_x4(b[nt], tile + xrow[nt] + 32 * kp);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t af[4];
        codes4(words[m][2 * kp + h], af);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(d[m][nt], af, b[nt][2 * h], b[nt][2 * h + 1]);
      }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = kDown ? fmaf(d[m][nt][i], tail[nt][i & 1].y, part[m][nt][i]) : d[m][nt][i];
        acc[m][nt][i] = fmaf(i < 2 ? s_lo[m] : s_hi[m], v, acc[m][nt][i]);
      }
}

// The run of units of a kernel.  Gate/up: item = (expert, row block), its
// units the input groups.  Down: item = row block, its units (expert, group).
template <bool kDown>
struct MoeRun {
  int ng, n_rb, active;   // groups of a unit row, row blocks, experts in use
  int item_len;           // units of an item
  __device__ __forceinline__ MoeRun(const MoeArgs& a, int n) : active(n) {
    ng = (kDown ? a.I : a.H) / kGroup;
    n_rb = kDown ? a.H / kRowsPerBlock : 2 * a.I / kRowsPerBlock;
    item_len = kDown ? ng * n : ng;
  }
  // The least units of a share.  Down: a row block's parts are added one after the
  // other, a part in about a third of a unit's time: with few units, parts and units a
  // part balance near the root of the item.  Without / with it, 8 tokens through 4 of
  // 128 experts of 640 x 512 35 / 24 us, 1 through 2 of 8 of 1024 x 3584 20 / 18, 20
  // through the same 32.9 / 34.5; larger layers the same within 2 %.
  __device__ __forceinline__ int least() const { return kDown ? max(1, (int)sqrtf((float)item_len * (1.f / 3.f))) : 1; }
  __device__ __forceinline__ int total() const { return kDown ? n_rb * item_len : n_rb * item_len * active; }
  // row block and active-expert index of unit u; the units of that (row
  // block, expert) end before `end`
  __device__ __forceinline__ void at(int u, int& rb, int& ai, int& g, int& end) const {
    if (kDown) {
      rb = u / item_len;
      const int rem = u - rb * item_len;
      ai = rem / ng;
      g = rem - ai * ng;
    } else {
      const int item = u / ng;
      ai = item / n_rb;
      rb = item - ai * n_rb;
      g = u - item * ng;
    }
    end = u - g + ng;
  }
};

// The run cut into shares, one per CTA: the first `rem` of per + 1 units, the
// others of per.  Whole items where that costs at most a few units more than equal
// shares: an item that two CTAs share costs both a record and an arrival, about
// the time of eight units (8.4 KB each at a CTA's part of the memory bandwidth).
struct MoeCut {
  int use, per, rem, len;   // len: units that a share is a multiple of
  __device__ __forceinline__ MoeCut(int total, int item_len, int ctas, int least) {
    const int items = total / item_len, most = (items + ctas - 1) / ctas;
    len = (long long)most * item_len * ctas <= total + 8LL * ctas ? item_len : 1;
    const int n = total / len;
    use = min(len == 1 ? n / least : n, ctas);
    per = n / use;
    rem = n - per * use;
  }
  __device__ __forceinline__ int begin(int cta) const { return (per * cta + min(cta, rem)) * len; }
  __device__ __forceinline__ int owner(int u) const {
    const int n = u / len, big = (per + 1) * rem;
    return n < big ? n / (per + 1) : rem + (n - big) / per;
  }
};

// More than 8 tokens: the records of a down row block (14 of 16 KB at 32 tokens on
// 152 SMs) are added by a kernel of their own, by 8 tokens; the one CTA that arrives
// last would read them alone, for longer than a launch takes (32 tokens through 2 of
// 8 experts 199 us so, 193 with the kernel; through 8 of 128 of 2048 x 768 96 and 79).  With up to 8 tokens the launch costs
// what it saves (1 to 8 tokens through five layers: within 1 us either way).
__host__ __device__ inline bool sums_apart(int T) { return T > 8; }

// A CTA's place in its ring of stages.
struct MoeRing {
  int slot;
  uint32_t phase;
  bool ok;
};

// The units u .. end - 1 of one (row block, expert) with n <= 8 NT columns, and
// their sums into this warp's 32 rows of the tile red[column][row].  Down:
// column = token, added expert by expert (a token has one column per expert, and
// only this warp touches these rows).
template <int NT, int NTL, bool kDown>
__device__ __forceinline__ void run_units(const MoeArgs& a, uint8_t* smem, float* red, uint64_t* full, uint64_t* empty,
                                          volatile int* s_dead, const uint8_t* token, int n, int units, MoeRing& ring) {
  using Lay = MoeLayout<NTL>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
  // columns past n read column 0: they only feed MMA columns that are not stored
  int xrow[NT], col[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = 8 * nt + (lane & 7);
    xrow[nt] = (c < n ? c : 0) * kRecHalves + 8 * (lane >> 3);
    col[nt] = 8 * nt + 2 * t4 + 1 < 8 * NTL ? 8 * nt + 2 * t4 : 0;
  }
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;
#pragma unroll 1
  for (int u = 0; u < units; ++u) {
    if (ring.ok && !moe_wait(&full[ring.slot], ring.phase, a.err)) {
      ring.ok = false;
      record_timeout(a.err);
      *s_dead = 1;
    }
    if (ring.ok) moe_unit<NT, kDown>(smem + ring.slot * Lay::kStage, xrow, col, acc);
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[ring.slot]);
    if (++ring.slot == Lay::kRing) {
      ring.slot = 0;
      ring.phase ^= 1u;
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = 8 * nt + 2 * t4 + i;
      if (c < n) {
        float* p = red + (kDown ? token[c] : c) * kRedLd + 32 * warp + gr;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float lo = kUnitA * acc[m][nt][i], hi = kUnitB * acc[m][nt][2 + i];
          p[16 * m] = kDown ? p[16 * m] + lo : lo;
          p[16 * m + 8] = kDown ? p[16 * m + 8] + hi : hi;
        }
      }
    }
  __syncwarp();
}

__device__ __forceinline__ uint2 out4(const MoeArgs& a, size_t o, float4 v) {
  if (a.resid) {
    const uint2 ru = *reinterpret_cast<const uint2*>(a.resid + o);
    v.x += __uint_as_float(ru.x << 16);
    v.y += __uint_as_float(ru.x & 0xffff0000u);
    v.z += __uint_as_float(ru.y << 16);
    v.w += __uint_as_float(ru.y & 0xffff0000u);
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Records r0 and rn[0 .. nc - 1], float4 i of each, added in this order.
__device__ __forceinline__ float4 sum_parts(const float4* r0, const float4* rn, int nc, int i) {
  constexpr size_t step = (size_t)2 * kMoeRecFloats / 4;
  constexpr int kU = 8;   // records in flight
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k = -1; k < nc; k += kU) {
    float4 v[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (k + j < nc) v[j] = __ldcg(k + j < 0 ? r0 + i : rn + (size_t)(k + j) * step + i);
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (k + j < nc) {
        s.x += v[j].x; s.y += v[j].y; s.z += v[j].z; s.w += v[j].w;
      }
  }
  return s;
}

template <int NT, bool kDown>
__global__ void __launch_bounds__(kMoeThreads, NT == 4 ? 2 : 3) moe_expert_kernel(const MoeArgs a) {
  using Lay = MoeLayout<NT>;
  constexpr int kMoeRing = Lay::kRing;
  extern __shared__ __align__(128) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + Lay::kRed);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* empty = full + kMoeRing;
  volatile int* s_dead = reinterpret_cast<volatile int*>(empty + kMoeRing);   // a wait ran out
  volatile int* s_snap = s_dead + 1;     // as the consumers saw it together
  volatile int* s_last = s_dead + 2;
  volatile int* s_issued = s_dead + 3;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMoeRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kMoeCW);
    }
    fence_mbar_init();
    *s_dead = 0;
    *s_issued = 0;
  }
  __syncthreads();
  // Gate/up waits for the router, then lets down start.  Down starts once
  // every gate/up CTA has passed its wait, so the choices are complete; its
  // weights do not depend on gate/up, only the activations do.
  if (!kDown) {
    pdl_wait();
    pdl_trigger();
  } else {
    pdl_trigger();
  }
  const bool own = own_blob(a);   // the same for all CTAs; looked at below, when the choices are there, too
  __shared__ MoeRoute s_route;
  make_route<8 * NT>(a, s_route);
  const MoeRoute* rt = &s_route;
  const MoeRun<kDown> run(a, rt->n_active);
  const int total = run.total();
  const MoeCut cut(total, run.item_len, (int)gridDim.x, run.least());
  const int cta = blockIdx.x;
  if (cta >= cut.use) return;
  if (!own) {
    if (kDown) pdl_wait();   // down's end is the call's
    return;
  }
  const int u0 = cut.begin(cta), u1 = cut.begin(cta + 1);

  if (warp == kMoeCW) {
    // ---------------------------------------------------------- producer --
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    bool waited = !kDown;
    int rows_due = 0;   // down: stages whose activations wait for gate/up
    const __half* due[kMoeRing];
    int due_bytes[kMoeRing];
    for (int u = !kDown && a.withhold && cta == 0 ? u1 : u0; u < u1 && ok;) {
      int rb, ai, g, end;
      run.at(u, rb, ai, g, end);
      end = min(end, u1);
      const int e = rt->expert[ai], off = rt->off[ai], n = rt->off[ai + 1] - off;
      const uint8_t* w = a.blob + kHeaderBytes + (size_t)e * a.expert_bytes + (kDown ? a.gu_bytes : 0) +
                         ((size_t)rb * run.ng + g) * kUnitBytes;
      // Gate/up: this lane's token's records (lanes n..31 have none).  Down: the
      // expert's records of a group lie side by side, one copy (with a copy each the
      // 32 tokens took 189 us, with one 184).
      const int lanes = kDown ? 1 : n, rec_bytes = kDown ? n * kRecBytes : kRecBytes;
      const size_t step = kDown ? (size_t)a.T * a.K * kRecHalves : kRecHalves;
      const __half* row = kDown ? a.act + g * step + (size_t)off * kRecHalves : a.xh + g * step;
      if (!kDown && lane < n) row += (size_t)rt->token[off + lane] * run.ng * kRecHalves;
      for (; u < end; ++u) {
        if (issued >= kMoeRing) {
          if (!moe_wait(&empty[slot], phase ^ 1u, a.err)) {
            ok = false;
            break;
          }
        }
        uint8_t* st = smem + slot * Lay::kStage;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[slot], kUnitBytes + n * kRecBytes);
          bulk_g2s(st, w, kUnitBytes, &full[slot]);
        }
        if (waited) {
          if (lane < lanes) bulk_g2s(st + kUnitBytes + lane * kRecBytes, row, rec_bytes, &full[slot]);
        } else {
          // the ring's first stages: weights now, activations after the wait
#pragma unroll
          for (int i = 0; i < kMoeRing; ++i)
            if (i == rows_due) {
              due[i] = row;
              due_bytes[i] = rec_bytes;
            }
          ++rows_due;
          if (rows_due == kMoeRing || u + 1 == u1) {
            pdl_wait();
            waited = true;
#pragma unroll
            for (int i = 0; i < kMoeRing; ++i)
              if (i < rows_due && lane == 0)   // (down only)
                bulk_g2s(smem + i * Lay::kStage + kUnitBytes, due[i], due_bytes[i], &full[i]);
          }
        }
        w += kUnitBytes;
        row += step;
        ++issued;
        if (++slot == kMoeRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      record_timeout(a.err);
      *s_dead = 1;
    }
    if (lane == 0) *s_issued = issued;
  } else {
    // ---------------------------------------------------------- consumers --
    if (kDown) pdl_wait();   // records and counters are gate/up's until it has ended
    if (kDown && cta == 0 && tid == 0) *a.active = rt->n_active;
    MoeRing ring{0, 0u, true};
    for (int u = u0; u < u1;) {
      // one item's part in this share
      const int item = u / run.item_len, i0 = item * run.item_len, i1 = i0 + run.item_len;
      const int seg0 = u, seg1 = min(i1, u1);
      int rb = 0, ai = 0, g, end, off = 0, n = 0;
      if (kDown) {
        for (int c = 0; c < a.T; ++c) red[c * kRedLd + 32 * warp + lane] = 0.f;
        __syncwarp();
      }
      while (u < seg1) {
        run.at(u, rb, ai, g, end);
        end = min(end, seg1);
        off = rt->off[ai];
        n = rt->off[ai + 1] - off;
        const uint8_t* token = rt->token + off;
        if (NT == 1 || n <= 8)
          run_units<1, NT, kDown>(a, smem, red, full, empty, s_dead, token, n, end - u, ring);
        else if (NT == 2 || n <= 16)
          run_units<2, NT, kDown>(a, smem, red, full, empty, s_dead, token, n, end - u, ring);
        else
          run_units<4, NT, kDown>(a, smem, red, full, empty, s_dead, token, n, end - u, ring);
        u = end;
      }
      const int cols = kDown ? a.T : n;
      if (tid == 0) *s_snap = *s_dead;
      moe_sync();
      bool write = !*s_snap;
      const bool apart = kDown && sums_apart(a.T);
      if (write && (seg0 != i0 || seg1 != i1)) {
        // a part: this CTA's record, then the last arrival adds them in CTA order
        float* rec = a.rec + ((size_t)cta * 2 + (i0 < seg0 ? 0 : 1)) * kMoeRecFloats;
        for (int i = tid; i < cols * 32; i += kMoeCW * 32) {
          const int c = i >> 5, q = i & 31;
          reinterpret_cast<float4*>(rec)[i] = *reinterpret_cast<const float4*>(red + c * kRedLd + 4 * q);
        }
        moe_sync();
        const int c0 = cut.owner(i0), c1 = cut.owner(i1 - 1);
        if (!apart && tid == 0) {
          *s_last = atom_add_acq_rel_gpu(&a.cnt[kRouterTiles + c0], 1u) == (unsigned)(c1 - c0) ? 1 : 0;
          if (*s_last) a.cnt[kRouterTiles + c0] = 0u;
        }
        moe_sync();
        write = !apart && *s_last != 0;
        if (write) {
          const float4* r0 = reinterpret_cast<const float4*>(a.rec + ((size_t)c0 * 2 + 1) * kMoeRecFloats);
          const float4* rn = reinterpret_cast<const float4*>(a.rec + (size_t)(c0 + 1) * 2 * kMoeRecFloats);
          for (int i = tid; i < cols * 32; i += kMoeCW * 32)
            *reinterpret_cast<float4*>(red + (i >> 5) * kRedLd + 4 * (i & 31)) = sum_parts(r0, rn, c1 - c0, i);
          moe_sync();
        }
      }
      if (write) {
        if (kDown) {
          for (int i = tid; i < cols * 32; i += kMoeCW * 32) {
            const int c = i >> 5, q = i & 31;
            const size_t o = (size_t)c * a.H + (size_t)rb * kRowsPerBlock + 4 * q;
            *reinterpret_cast<uint2*>(a.y + o) = out4(a, o, *reinterpret_cast<const float4*>(red + c * kRedLd + 4 * q));
          }
        } else {
          // a warp per column: outputs 64 rb .. 64 rb + 63 of pair off + c, half a record
          for (int c = warp; c < cols; c += kMoeCW) {
            const float r = a.rms[rt->token[off + c]], wt = a.share[rt->pick[off + c]];
            float v[2], mx = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float gt = r * red[c * kRedLd + 2 * lane + h], up = r * red[c * kRedLd + 64 + 2 * lane + h];
              v[h] = wt * (__fdiv_rn(gt, 1.0f + expf(-gt)) * up);
              mx = fmaxf(mx, fabsf(v[h]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float f = pow2_at(mx), inv = pow2_inverse(f);
            const __half2 hv = __floats2half2_rn(v[0] * inv, v[1] * inv);
            __half* rec = a.act + ((size_t)(rb >> 1) * (a.T * a.K) + off + c) * kRecHalves;
            reinterpret_cast<__half2*>(rec + 64 * (rb & 1))[lane] = hv;
            if (lane == 0) reinterpret_cast<float*>(rec + kGroup)[rb & 1] = f;
          }
        }
      }
      moe_sync();   // the tile is free again
    }
  }
  __syncthreads();
  if (*s_dead && tid == 0) drain_ring(full, kMoeRing, *s_issued);
}

// y from the records of down: a CTA per row block and eight tokens, a thread per
// four outputs.
__global__ void __launch_bounds__(256) moe_sum_kernel(const MoeArgs a) {
  pdl_trigger();
  pdl_wait();
  if (!own_blob(a)) return;
  const MoeRun<true> run(a, *a.active);
  const MoeCut cut(run.total(), run.item_len, a.down_ctas, run.least());
  const int rb = blockIdx.x, t = 8 * blockIdx.y + (threadIdx.x >> 5), q = threadIdx.x & 31;
  if (t >= a.T) return;
  const int i0 = rb * run.item_len, c0 = cut.owner(i0), c1 = cut.owner(i0 + run.item_len - 1);
  if (c0 == c1) return;   // one CTA had the whole row block, and wrote it
  const float4* r0 = reinterpret_cast<const float4*>(a.rec + ((size_t)c0 * 2 + 1) * kMoeRecFloats);
  const float4* rn = reinterpret_cast<const float4*>(a.rec + (size_t)(c0 + 1) * 2 * kMoeRecFloats);
  const size_t o = (size_t)t * a.H + (size_t)rb * kRowsPerBlock + 4 * q;
  *reinterpret_cast<uint2*>(a.y + o) = out4(a, o, sum_parts(r0, rn, c1 - c0, 32 * t + q));
}

template <int NT, bool kDown>
cudaError_t moe_configure(int dev) {
  static DeviceOnce configured;
  if (configured.done(dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(moe_expert_kernel<NT, kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       MoeLayout<NT>::kBytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(moe_expert_kernel<NT, kDown>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  configured.mark(dev);
  return cudaSuccess;
}

template <int NT, bool kDown>
int moe_per_sm(int dev) {
  return remembered(occ_key(dev, NT, kDown, 0), [&]() {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, moe_expert_kernel<NT, kDown>, kMoeThreads,
                                                      MoeLayout<NT>::kBytes) != cudaSuccess ||
        n < 1) {
      cudaGetLastError();
      return 1;
    }
    return n < kMoeMaxPerSm ? n : kMoeMaxPerSm;
  });
}

int moe_sms(int dev) {
  return remembered(occ_key(dev, 0, 0, 0), [&]() {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
  });
}

template <class Kernel>
cudaError_t moe_go(Kernel k, dim3 grid, int threads, size_t smem, cudaStream_t st, const MoeArgs& a) {
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
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int NT>
cudaError_t launch_experts(MoeArgs a, int dev, cudaStream_t st) {
  cudaError_t e = moe_configure<NT, false>(dev);
  if (e == cudaSuccess) e = moe_configure<NT, true>(dev);
  if (e != cudaSuccess) return e;
  const int sms = moe_sms(dev);
  e = moe_go(moe_expert_kernel<NT, false>, dim3((unsigned)(sms * moe_per_sm<NT, false>(dev))), kMoeThreads,
             MoeLayout<NT>::kBytes, st, a);
  if (e != cudaSuccess) return e;
  a.down_ctas = sms * moe_per_sm<NT, true>(dev);
  e = moe_go(moe_expert_kernel<NT, true>, dim3((unsigned)a.down_ctas), kMoeThreads, MoeLayout<NT>::kBytes, st, a);
  if (e != cudaSuccess || !sums_apart(a.T)) return e;
  return moe_go(moe_sum_kernel, dim3((unsigned)(a.H / kRowsPerBlock), (unsigned)((a.T + 7) / 8)), 256, 0, st, a);
}

// ----------------------------------------------------------------- packing --

__host__ __device__ inline uint32_t place_word(uint32_t w) {
  uint32_t r = 0;
  for (int h = 0; h < 2; ++h) {
    const uint32_t u0 = (w >> (16 * h)) & 15u, u1 = (w >> (16 * h + 4)) & 15u, u2 = (w >> (16 * h + 8)) & 15u,
                   u3 = (w >> (16 * h + 12)) & 15u;
    r |= ((u0 << 6) | (u1 << 2) | (u3 << 10) | ((u2 & 3u) << 14) | (u2 >> 2)) << (16 * h);
  }
  return r;
}

__host__ __device__ inline uint32_t plain_word(uint32_t w) {
  uint32_t r = 0;
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = (w >> (16 * h)) & 0xFFFFu;
    const uint32_t u0 = (v >> 6) & 15u, u1 = (v >> 2) & 15u, u2 = ((v >> 14) & 3u) | ((v & 3u) << 2), u3 = (v >> 10) & 15u;
    r |= (u0 | (u1 << 4) | (u2 << 8) | (u3 << 12)) << (16 * h);
  }
  return r;
}

// One CTA per unit.
__global__ void __launch_bounds__(256) moe_place_kernel(uint8_t* units) {
  uint32_t* w = reinterpret_cast<uint32_t*>(units + (size_t)blockIdx.x * kUnitBytes);
  for (int i = threadIdx.x; i < kUnitCodeBytes / 4; i += 256) w[i] = place_word(w[i]);
}

struct MoeUnpackArgs {
  const uint8_t* sec;
  int rows, cols, n_groups;
  int map;  // 0 identity, 1 gate rows, 2 up rows
  int8_t* codes;
  uint16_t* scales;
};

__global__ void __launch_bounds__(256) moe_unpack_kernel(const MoeUnpackArgs a) {
  const size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= (size_t)a.rows * a.cols) return;
  const int R = (int)(e / a.cols), C = (int)(e % a.cols);
  const int SR = a.map == 0 ? R : 128 * (R / 64) + 64 * (a.map - 1) + (R % 64);
  const int rb = SR >> 7, lr = SR & 127, rt = lr >> 4, rr = lr & 15;
  const int grp = C >> 7, cc = C & 127, ks = cc >> 4, kk = cc & 15;
  const int slot = (rr >> 3) + 2 * (kk >> 3) + 4 * (kk & 1);
  const int lane = 4 * (rr & 7) + ((kk & 7) >> 1);
  const uint8_t* unit = a.sec + ((size_t)rb * a.n_groups + grp) * kUnitBytes;
  const uint32_t word = plain_word(reinterpret_cast<const uint32_t*>(unit)[rt * 256 + (ks >> 2) * 128 + lane * 4 + (ks & 3)]);
  a.codes[e] = (int8_t)((int)((word >> (4 * slot)) & 0xF) - 8);
  if (cc == 0) a.scales[(size_t)R * a.n_groups + grp] = reinterpret_cast<const uint16_t*>(unit + kUnitCodeBytes)[lr];
}

}  // namespace

int moe_ctas() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return moe_sms(dev) * kMoeMaxPerSm;
}

cudaError_t launch_moe(const MoeArgs& a, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = moe_go(moe_router_kernel, dim3((unsigned)((a.E + kRouterE - 1) / kRouterE), (unsigned)((a.T + kRouterT - 1) / kRouterT)),
             kRouterThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  // Columns of a pass: an expert has at most T tokens.  Above 16, passes of 16 (three
  // CTAs an SM) unless experts have more than 8 tokens on average, where many would
  // have to be streamed twice.  In passes of 16 / of 32, at two tokens an expert: 32
  // through 8 of 128 of 2048 x 768 79 / 88 us, through 4 of 60 of 2048 x 1408 72 / 74; at
  // six: 24 through 2 of 8 of 4096 x 14336 182 / 197; at 16: 32 through 2 of 4 of 4096 x
  // 14336 163 / 161, 4 of 8 of 4096 x 4096 112 / 110.  At eight, where the rule changes
  // sides, the layer's size decides, which it does not know: 2 of 8 of 4096 x 14336
  // 193 / 212, x 8192 139 / 137, x 4096 87 / 84, x 2048 60 / 55.
  if (a.T <= 8) return launch_experts<1>(a, dev, st);
  if (a.T <= 16 || a.T * a.K <= 8 * a.E) return launch_experts<2>(a, dev, st);
  return launch_experts<4>(a, dev, st);
}

cudaError_t launch_moe_place(uint8_t* units, size_t n_units, cudaStream_t st) {
  moe_place_kernel<<<(unsigned)n_units, 256, 0, st>>>(units);
  return cudaGetLastError();
}

cudaError_t launch_moe_unpack(int hidden, int inter, const uint8_t* gu, const uint8_t* down, int which, int8_t* codes,
                              uint16_t* scales, cudaStream_t st) {
  const bool is_down = which == FUTR_PROJ_DOWN;
  MoeUnpackArgs a{};
  a.map = which == FUTR_PROJ_GATE ? 1 : which == FUTR_PROJ_UP ? 2 : 0;
  a.rows = is_down ? hidden : inter;
  a.cols = is_down ? inter : hidden;
  a.sec = is_down ? down : gu;
  a.n_groups = a.cols / kGroup;
  a.codes = codes;
  a.scales = scales;
  const size_t n = (size_t)a.rows * a.cols;
  moe_unpack_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace futr
