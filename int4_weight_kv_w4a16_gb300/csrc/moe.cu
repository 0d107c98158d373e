// Mixture-of-experts layer for 1..32 tokens with INT4 experts.
//
//   r_t = 1 / sqrt(mean x_t^2 + eps);  l_te = r_t sum_k (x_tk g_k) Wr_ek
//   the K largest l_te (equal ones: lowest expert first), p = softmax(l_t),
//   w = p of the chosen (divided by their sum if asked)
//   y_t = resid_t + sum_j w_tj Wd_e (silu(r_t W'g_e x_t) * (r_t W'u_e x_t)),  e = e_tj
//
// Three kernels with programmatic dependent launch:
//   router   a warp per expert and four tokens; the CTA that arrives last picks
//            the experts of every token and sorts the (token, expert) pairs by expert;
//   gate/up  streams the chosen experts' gate/up units once;
//   down     streams their down units once, beginning before gate/up has ended.
// The expert kernels are bound by the weight stream.  All units of the chosen
// experts form one run, cut into equal contiguous shares, one per CTA of a
// grid that fills the GPU; the cut is made on the device from the routing.  A
// unit (128 rows x 128 inputs) comes by one bulk copy, the 128 inputs of each
// of the expert's tokens by one 256-byte copy each; four warps unpack the
// nibbles straight into bf16 A fragments (as the block's projections do) and
// the tokens are the N side, so an expert costs its own tokens' columns only.
// A row block that spans CTAs leaves one record per CTA, added in CTA order by
// the one that arrives last.  Down runs over (row block, expert, group) with
// the expert inside: the experts of a row block meet in one fp32 tile per
// token in shared memory, so y needs no second pass.
//
// Rounding: the activation w * silu * up is rounded to bf16 between the two
// expert kernels (it is the B operand of the down product), the routing weight
// inside, so the weighted sum over experts is an fp32 sum.  Everything else is
// fp32 until y.
#include "moe.cuh"

namespace futr {

namespace {

constexpr int kMoeCW = 4;
constexpr int kMoeThreads = (kMoeCW + 1) * 32;
constexpr int kMoeMaxPerSm = 3;
constexpr int kRouterThreads = 256;
constexpr int kRouterTokens = 4;   // tokens of a router warp
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

// ------------------------------------------------------------------ router --

__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const MoeArgs a) {
  __shared__ int s_last;
  __shared__ int s_id[kMoeMaxPairs];
  __shared__ float s_w[kMoeMaxPairs];
  __shared__ unsigned s_mask[kMoeMaxExperts];   // tokens of each expert
  __shared__ int s_off[kMoeMaxExperts];
  __shared__ int s_sum[2][kRouterThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int task = blockIdx.x * (kRouterThreads / 32) + warp;
  const int e = task % a.E, t0 = task / a.E * kRouterTokens;
  if (task == 0 && lane == 0) {
    const MoeHeader* h = reinterpret_cast<const MoeHeader*>(a.blob);
    if (h->magic != kMoeMagic || h->hidden != a.H || h->inter != a.I || h->n_experts != a.E)
      set_err(a.err, FUTR_ERR_BAD_BLOB);
  }
  if (t0 < a.T) {
    const int nt = min(kRouterTokens, a.T - t0);
    float acc[kRouterTokens] = {}, ss[kRouterTokens] = {};
    const __nv_bfloat16* wr = a.router + (size_t)e * a.H;
#pragma unroll 4
    for (int j = 8 * lane; j < a.H; j += 256) {
      float w[8], g[8];
      const uint4 wv = *reinterpret_cast<const uint4*>(wr + j);
      const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = __uint_as_float(wu[i] << 16);
        w[2 * i + 1] = __uint_as_float(wu[i] & 0xffff0000u);
        g[2 * i] = g[2 * i + 1] = 1.f;
      }
      if (a.gain) {
        const float4 g0 = *reinterpret_cast<const float4*>(a.gain + j), g1 = *reinterpret_cast<const float4*>(a.gain + j + 4);
        g[0] = g0.x; g[1] = g0.y; g[2] = g0.z; g[3] = g0.w;
        g[4] = g1.x; g[5] = g1.y; g[6] = g1.z; g[7] = g1.w;
      }
#pragma unroll
      for (int t = 0; t < kRouterTokens; ++t)
        if (t < nt) {
          const uint4 xv = *reinterpret_cast<const uint4*>(a.x + (size_t)(t0 + t) * a.H + j);
          const uint32_t xu[4] = {xv.x, xv.y, xv.z, xv.w};
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
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t)
      if (t < nt) {
        const float s = warp_sum(acc[t]), q = warp_sum(ss[t]);
        const float r = a.eps > 0.f ? __fdiv_rn(1.0f, sqrtf(__fdiv_rn(q, (float)a.H) + a.eps)) : 1.f;
        if (lane == 0) {
          a.logits[(size_t)(t0 + t) * a.E + e] = r * s;
          if (e == 0) a.route->rms[t0 + t] = r;
        }
      }
  }
  __syncthreads();
  if (tid == 0) {
    s_last = atom_add_acq_rel_gpu(a.cnt + a.n_cnt, 1u) == gridDim.x - 1 ? 1 : 0;
    if (s_last) a.cnt[a.n_cnt] = 0u;
  }
  __syncthreads();
  if (!s_last) return;

  // the choice of experts: a warp per token, expert lane + 32 i in v[i]
  for (int i = tid; i < kMoeMaxExperts; i += kRouterThreads) s_mask[i] = 0u;
  __syncthreads();
  constexpr int kV = kMoeMaxExperts / 32;
  for (int t = warp; t < a.T; t += kRouterThreads / 32) {
    float v[kV], mx = -INFINITY, sum = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      v[i] = lane + 32 * i < a.E ? __ldcg(a.logits + (size_t)t * a.E + lane + 32 * i) : -INFINITY;
      mx = fmaxf(mx, v[i]);
      nan |= v[i] != v[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    nan = __any_sync(0xffffffffu, nan);
#pragma unroll
    for (int i = 0; i < kV; ++i) sum += lane + 32 * i < a.E ? expf(v[i] - mx) : 0.f;
    sum = warp_sum(sum);
    unsigned taken = 0u;   // this lane's chosen experts
    float chosen = 0.f, total = 0.f;   // lane j: weight of the j-th choice
    int chosen_id = 0;
    for (int j = 0; j < a.K; ++j) {
      // largest value, then lowest index; NaN ranks with -inf
      float bv = -INFINITY;
      int bi = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int id = lane + 32 * i;
        const float c = v[i] != v[i] ? -INFINITY : v[i];
        if (id < a.E && !((taken >> i) & 1u) && (bi == 0x7fffffff || c > bv)) {
          bv = c;
          bi = id;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) {
          bv = ov;
          bi = oi;
        }
      }
      if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
      const float w = nan ? __int_as_float(0x7fc00000) : __fdiv_rn(expf(bv - mx), sum);
      total += w;
      if (lane == j) {
        chosen = w;
        chosen_id = bi;
      }
    }
    if (a.renorm) chosen = __fdiv_rn(chosen, total);
    if (lane < a.K) {
      const int p = t * a.K + lane;
      s_id[p] = chosen_id;
      s_w[p] = chosen;
      atomicOr(&s_mask[chosen_id], 1u << t);
      if (a.ids) a.ids[p] = chosen_id;
      if (a.weights) a.weights[p] = chosen;
    }
  }
  __syncthreads();
  // experts in use and the first pair of each: prefix sums over the experts
  {
    const unsigned mask = tid < a.E ? s_mask[tid] : 0u;
    const int n = __popc(mask), used = n > 0;
    int pn = n, pu = used;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, pn, o), y = __shfl_up_sync(0xffffffffu, pu, o);
      if (lane >= o) {
        pn += x;
        pu += y;
      }
    }
    if (lane == 31) {
      s_sum[0][warp] = pn;
      s_sum[1][warp] = pu;
    }
    __syncthreads();
    int bn = 0, bu = 0;
    for (int w = 0; w < warp; ++w) {
      bn += s_sum[0][w];
      bu += s_sum[1][w];
    }
    s_off[tid] = bn + pn - n;
    if (used) {
      a.route->expert[bu + pu - 1] = tid;
      a.route->off[bu + pu - 1] = bn + pn - n;
    }
    if (tid == kRouterThreads - 1) {
      a.route->n_active = bu + pu;
      a.route->off[bu + pu] = bn + pn;
    }
  }
  __syncthreads();
  for (int p = tid; p < a.T * a.K; p += kRouterThreads) {
    const int t = p / a.K, id = s_id[p];
    const int at = s_off[id] + __popc(s_mask[id] & ((1u << t) - 1u));
    a.route->token[at] = t;
    a.route->weight[at] = s_w[p];
  }
}

// ---------------------------------------------------------- expert kernels --

template <int NT>
struct MoeLayout {
  static constexpr int kRing = NT == 4 ? 5 : 6;                      // two CTAs an SM at the least
  static constexpr int kStage = kUnitBytes + 8 * NT * kTileLd * 2;   // unit, then [8 NT][136] bf16
  static constexpr int kRed = kRing * kStage;                        // [8 NT][kRedLd] fp32
  static constexpr int kBar = kRed + 8 * NT * kRedLd * 4;
  static constexpr int kBytes = kBar + 2 * kRing * 8 + 16;
};

// One unit times n_nt tiles of 8 columns for this warp's 32 rows: the group's
// product in fp32, then times the rows' scales into acc.
template <int NT>
__device__ __forceinline__ void moe_unit(const uint8_t* st, const int (&xrow)[NT], int n_nt, float (&acc)[2][NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2;
  const __nv_bfloat16* tile = reinterpret_cast<const __nv_bfloat16*>(st + kUnitBytes);
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
  float d[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[m][nt][i] = 0.f;
#pragma unroll
  for (int kp = 0; kp < 4; ++kp) {
    uint32_t b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      if (nt < n_nt) ldmatrix_x4(b[nt], tile + xrow[nt] + 32 * kp);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t af[4];
        nib4_bf16x2(words[m][2 * kp + h], af);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (nt < n_nt) mma_bf16_16816(d[m][nt], af, b[nt][2 * h], b[nt][2 * h + 1]);
      }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc[m][nt][0] = fmaf(s_lo[m], d[m][nt][0], acc[m][nt][0]);
      acc[m][nt][1] = fmaf(s_lo[m], d[m][nt][1], acc[m][nt][1]);
      acc[m][nt][2] = fmaf(s_hi[m], d[m][nt][2], acc[m][nt][2]);
      acc[m][nt][3] = fmaf(s_hi[m], d[m][nt][3], acc[m][nt][3]);
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

template <int NT, bool kDown>
__global__ void __launch_bounds__(kMoeThreads, NT == 1 ? 3 : 2) moe_expert_kernel(const MoeArgs a) {
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
  // every gate/up CTA has passed its wait, so the routing is complete; its
  // weights do not depend on gate/up, only the activations do.
  if (!kDown) {
    pdl_wait();
    pdl_trigger();
  } else {
    pdl_trigger();
  }
  const MoeRoute* rt = a.route;
  const MoeRun<kDown> run(a, rt->n_active);
  const int total = run.total();
  const int cta = blockIdx.x, ctas = min(total, (int)gridDim.x);
  if (cta >= ctas) return;
  const int u0 = (int)((long long)total * cta / ctas), u1 = (int)((long long)total * (cta + 1) / ctas);
  const int K = kDown ? a.I : a.H;   // inputs of the product

  if (warp == kMoeCW) {
    // ---------------------------------------------------------- producer --
    int slot = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    bool waited = !kDown;
    int rows_due = 0;   // down: stages whose activations wait for gate/up
    const __nv_bfloat16* due[kMoeRing];
    int due_n[kMoeRing];
    for (int u = u0; u < u1 && ok;) {
      int rb, ai, g, end;
      run.at(u, rb, ai, g, end);
      end = min(end, u1);
      const int e = rt->expert[ai], off = rt->off[ai], n = rt->off[ai + 1] - off;
      const uint8_t* w = a.blob + kHeaderBytes + (size_t)e * a.expert_bytes + (kDown ? a.gu_bytes : 0) +
                         ((size_t)rb * run.ng + g) * kUnitBytes;
      // this lane's token row (columns n..31 have none)
      const __nv_bfloat16* row = nullptr;
      if (lane < n) row = kDown ? a.act + (size_t)(off + lane) * K : a.x + (size_t)rt->token[off + lane] * K;
      row += (size_t)g * kGroup;
      for (; u < end; ++u) {
        if (issued >= kMoeRing) {
          if (!moe_wait(&empty[slot], phase ^ 1u, a.err)) {
            ok = false;
            break;
          }
        }
        uint8_t* st = smem + slot * Lay::kStage;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[slot], kUnitBytes + n * kGroup * 2);
          bulk_g2s(st, w, kUnitBytes, &full[slot]);
        }
        if (waited) {
          if (lane < n) bulk_g2s(st + kUnitBytes + lane * kTileLd * 2, row, kGroup * 2, &full[slot]);
        } else {
          // the ring's first stages: weights now, activations after the wait
#pragma unroll
          for (int i = 0; i < kMoeRing; ++i)
            if (i == rows_due) {
              due[i] = row;
              due_n[i] = n;
            }
          ++rows_due;
          if (rows_due == kMoeRing || u + 1 == u1) {
            pdl_wait();
            waited = true;
#pragma unroll
            for (int i = 0; i < kMoeRing; ++i)
              if (i < rows_due && lane < due_n[i])
                bulk_g2s(smem + i * Lay::kStage + kUnitBytes + lane * kTileLd * 2, due[i], kGroup * 2, &full[i]);
          }
        }
        w += kUnitBytes;
        row += kGroup;
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
    const int gr = lane >> 2, t4 = lane & 3;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
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
        const int n_nt = (n + 7) >> 3;
        int xrow[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int c = 8 * nt + (lane & 7);
          xrow[nt] = (c < n ? c : 0) * kTileLd + 8 * (lane >> 3);
        }
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;
        for (; u < end; ++u) {
          if (ok && !moe_wait(&full[slot], phase, a.err)) {
            ok = false;
            record_timeout(a.err);
            *s_dead = 1;
          }
          if (ok) moe_unit<NT>(smem + slot * Lay::kStage, xrow, n_nt, acc);
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[slot]);
          if (++slot == kMoeRing) {
            slot = 0;
            phase ^= 1u;
          }
        }
        // this warp's 32 rows of the tile red[column][row]; down: column = token,
        // added expert by expert (a token has one column per expert, and only
        // this warp touches these rows)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = 8 * nt + 2 * t4 + i;
            if (c < n) {
              float* p = red + (kDown ? rt->token[off + c] : c) * kRedLd + 32 * warp + gr;
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                p[16 * m] = kDown ? p[16 * m] + acc[m][nt][i] : acc[m][nt][i];
                p[16 * m + 8] = kDown ? p[16 * m + 8] + acc[m][nt][2 + i] : acc[m][nt][2 + i];
              }
            }
          }
        __syncwarp();
      }
      const int cols = kDown ? a.T : n;
      if (tid == 0) *s_snap = *s_dead;
      moe_sync();
      bool write = !*s_snap;
      if (write && (seg0 != i0 || seg1 != i1)) {
        // a part: this CTA's record, then the last arrival adds them in CTA order
        float* rec = a.rec + ((size_t)cta * 2 + (i0 < seg0 ? 0 : 1)) * kMoeRecFloats;
        for (int i = tid; i < cols * 32; i += kMoeCW * 32) {
          const int c = i >> 5, q = i & 31;
          reinterpret_cast<float4*>(rec)[i] = *reinterpret_cast<const float4*>(red + c * kRedLd + 4 * q);
        }
        moe_sync();
        const int c0 = (int)(((long long)(i0 + 1) * ctas - 1) / total), c1 = (int)(((long long)i1 * ctas - 1) / total);
        if (tid == 0) {
          *s_last = atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0) ? 1 : 0;
          if (*s_last) a.cnt[c0] = 0u;
        }
        moe_sync();
        write = *s_last != 0;
        if (write) {
          const float4* r0 = reinterpret_cast<const float4*>(a.rec + ((size_t)c0 * 2 + 1) * kMoeRecFloats);
          const float4* rn = reinterpret_cast<const float4*>(a.rec + (size_t)(c0 + 1) * 2 * kMoeRecFloats);
          constexpr size_t step = (size_t)2 * kMoeRecFloats / 4;
          const int nc = c1 - c0;
          for (int i = tid; i < cols * 32; i += kMoeCW * 32) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kU = 8;   // records in flight
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
            *reinterpret_cast<float4*>(red + (i >> 5) * kRedLd + 4 * (i & 31)) = s;
          }
          moe_sync();
        }
      }
      if (write) {
        if (kDown) {
          for (int i = tid; i < cols * 32; i += kMoeCW * 32) {
            const int c = i >> 5, q = i & 31;
            const size_t o = (size_t)c * a.H + (size_t)rb * kRowsPerBlock + 4 * q;
            float4 v = *reinterpret_cast<const float4*>(red + c * kRedLd + 4 * q);
            if (a.resid) {
              const uint2 ru = *reinterpret_cast<const uint2*>(a.resid + o);
              v.x += __uint_as_float(ru.x << 16);
              v.y += __uint_as_float(ru.x & 0xffff0000u);
              v.z += __uint_as_float(ru.y << 16);
              v.w += __uint_as_float(ru.y & 0xffff0000u);
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(a.y + o) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          }
        } else {
          for (int i = tid; i < cols * 64; i += kMoeCW * 32) {
            const int c = i >> 6, j = i & 63;
            const float r = rt->rms[rt->token[off + c]];
            const float gt = r * red[c * kRedLd + j], up = r * red[c * kRedLd + 64 + j];
            const float s = __fdiv_rn(gt, 1.0f + expf(-gt)) * up;
            a.act[(size_t)(off + c) * a.I + (size_t)rb * 64 + j] = __float2bfloat16_rn(rt->weight[off + c] * s);
          }
        }
      }
      moe_sync();   // the tile is free again
    }
  }
  __syncthreads();
  if (*s_dead && tid == 0) drain_ring(full, kMoeRing, *s_issued);
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
cudaError_t moe_go(Kernel k, int grid, int threads, size_t smem, cudaStream_t st, const MoeArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
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
cudaError_t launch_experts(const MoeArgs& a, int dev, cudaStream_t st) {
  cudaError_t e = moe_configure<NT, false>(dev);
  if (e == cudaSuccess) e = moe_configure<NT, true>(dev);
  if (e != cudaSuccess) return e;
  const int sms = moe_sms(dev);
  e = moe_go(moe_expert_kernel<NT, false>, sms * moe_per_sm<NT, false>(dev), kMoeThreads, MoeLayout<NT>::kBytes, st, a);
  if (e != cudaSuccess) return e;
  return moe_go(moe_expert_kernel<NT, true>, sms * moe_per_sm<NT, true>(dev), kMoeThreads, MoeLayout<NT>::kBytes, st, a);
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
  const int tasks = a.E * ((a.T + kRouterTokens - 1) / kRouterTokens), warps = kRouterThreads / 32;
  e = moe_go(moe_router_kernel, (tasks + warps - 1) / warps, kRouterThreads, 0, st, a);
  if (e != cudaSuccess) return e;
  // an expert has at most T tokens
  if (a.T <= 8) return launch_experts<1>(a, dev, st);
  if (a.T <= 16) return launch_experts<2>(a, dev, st);
  return launch_experts<4>(a, dev, st);
}

}  // namespace futr
