// Distillation of a student's row against a teacher's top logits: loss,
// gradient, or both (the formulas: include/specverify_rows.h).
//
// With K the listed tokens, e_v = 2^((s_v - mt) c) over the tokens outside K
// (mt their maximum, c = log2(e) / temperature) and S the row's whole sum,
//
//   gradient outside K = (w / T) A e_v,  A = 2^((mt - M) c) / S - p_t / sum e
//   gradient in K      = (w / T) (q_j - p_j)
//
// so the dense part of the gradient is one exponential and one product per
// element, and only the k listed tokens need the teacher.
//
// distill_kernel: a cluster of C CTAs owns a row, each a slice held in
// registers from one read of HBM (U vectors per thread).  While the vectors
// are on their way every CTA forms the teacher's softmax and the student's
// weights at the listed tokens (two-float: the loss is a small difference of
// logarithms).  A bitmap of the slice's listed tokens takes them out of the
// slice, so the mass outside K is a sum of its own terms.  The CTAs push
// (maximum, sum) into each other's shared memory, one cluster barrier, and
// the gradient leaves from the registers: a row is read once and written
// once.  Rows beyond the cluster's registers are taken in chunks and read
// twice.
//
// It is the form for lists of more than 256 tokens and rows beyond the
// persistent form's reach (sv_distill_pipe.cuh, which is two to three times as
// fast: the loss of 1024 rows of 152064 bf16, k = 128: 225 us here, 91 there;
// with the gradient 284 and 135), bound by the latency of a row's phases, of
// which two CTAs an SM overlap.
//
// distill_backward_kernel forms the gradient from the forward pass's row
// statistics: no reduction, one CTA per slice.  HBM: 2048 rows of 128256 bf16 in
// 150 us (a tenth of weight 0), 6.6 TB/s of logits read and gradient written.
#pragma once

#include "sv_rows.cuh"

namespace sv {
namespace rows {

constexpr int kDiThreads = 512;
constexpr int kDiWarps = kDiThreads / 32;
constexpr int kDiMaxC = 8;           // CTAs per cluster
constexpr int kDiBwThreads = 256;
constexpr int kDiBwU = 8;            // vectors per thread of the backward kernel

struct DistillParams {
  int R, V, k;
  int C, SV, NCK;                    // CTAs per row, vectors per CTA, chunks of them
  float c, c_lo;                     // log2(e) / temperature
  double inv_t;                      // 1 / temperature
  const void* student;
  const int32_t* indices;
  const float* logprobs;
  const float* tail;
  const float* weight;
  const float* grad_loss;            // backward
  int up_stride;                     // 0: grad_loss is one value
  int stop;                          // persistent form: the cluster's row at which it gives up (tests; -1: none)
  float* loss;
  float* stats;                      // [R][8]: mt, A, teacher maximum, 1 / Z, M, 1 / S, listed twice, usable
  void* grad;
};

// Beyond this a divergence is called infinite.
constexpr float kDiFar = 1.0e30f;

// w ((lp - tm) - (s - kr) / temperature): a listed token's term of the loss,
// up to the row's constants.
__device__ __forceinline__ F2 distill_term(F2 w, float lp, float tm, float s, float kr, F2 inv_t) {
  return f2_mul(w, f2_add(two_diff(lp, tm), f2_neg(f2_mul(two_diff(s, kr), inv_t))));
}

// The loss of a row of weight 1 (all lanes of a warp; the three logarithms
// side by side), in two-float throughout: sum_j p_j (ln p_j - ln q_j) + p_t
// (ln p_t - ln q_t), with the row's constants (ln Z, ln S) taken out of the
// sums.  E1: the sum of the listed tokens' terms.
__device__ __forceinline__ float distill_loss(F2 Z, F2 S, F2 st, F2 E1, F2 wt, float ltail, float tm, float mt, float km,
                                              float M, bool infinite, F2 inv_t, const float* tab) {
  const int lane = threadIdx.x & 31;
  const F2 mine = lane == 0 ? Z : lane == 1 ? S : st;
  const F2 lg = mine.hi > 0.f ? f2_log(mine, tab) : F2{-INFINITY, 0.f};
  const F2 lz{__shfl_sync(0xffffffffu, lg.hi, 0), __shfl_sync(0xffffffffu, lg.lo, 0)};
  const F2 ls{__shfl_sync(0xffffffffu, lg.hi, 1), __shfl_sync(0xffffffffu, lg.lo, 1)};
  const F2 lt{__shfl_sync(0xffffffffu, lg.hi, 2), __shfl_sync(0xffffffffu, lg.lo, 2)};
  const float kr = km == -INFINITY ? M : km;
  const bool tail = wt.hi != 0.f;
  if (!(S.hi > 0.f && S.hi < INFINITY) || Z.hi != Z.hi) return __uint_as_float(0x7fffffffu);
  // p wants what q has nothing of, or less than float32 can say
  if (infinite || (M - kr) * inv_t.hi > kDiFar || (tail && (!(st.hi > 0.f) || (mt - kr) * inv_t.hi < -kDiFar)))
    return INFINITY;
  F2 e = E1;
  if (tail) e = f2_add(e, f2_mul(wt, f2_add(two_diff(ltail, tm), f2_neg(f2_add(f2_mul(two_diff(mt, kr), inv_t), lt)))));
  const float q = e.hi * __frcp_rn(Z.hi);            // e / Z: a quotient and its remainder's
  const F2 rem = f2_add(e, f2_neg(f2_mul(Z, F2{q, 0.f})));
  F2 sum = f2_norm(q, rem.hi * __frcp_rn(Z.hi));
  sum = f2_add(sum, f2_add(ls, f2_neg(lz)));
  return f2_add(sum, f2_mul(two_diff(M, kr), inv_t)).hi;
}

// 2^(d (c + c_lo)), d <= 0: the weight of a value that lies d below its
// reference.  One exponential, corrected to first order for the product's
// rounding and for c_lo: the instruction's 2^-22 is what is left, as in every
// term outside the list (the fused call has two-float weights here because
// its loss, a small difference, needs them).
__device__ __forceinline__ float weight_fast(float d, float c, float c_lo) {
  const float p = d * c;
  if (p < -150.f) return 0.f;   // also where the product leaves float32's range
  const float y = ex2_approx(p), e = fmaf(d, c_lo, fmaf(d, c, -p));
  return fmaf(y * 6.931471825e-01f, e, y);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Store v at the address `local` has in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void push_f4(const float4* local, int rank, float4 v) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(local), d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(d), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <typename T, int U>
struct DistillSmem {
  uint32_t bits[kDiThreads * U * Tr<T>::VW / 32];   // the chunk's listed tokens
  int sid[kMaxK];                                   // listed tokens (-1: ignored)
  float sw[kMaxK];                                  // the teacher's weights, relative to its maximum
  float sq[kMaxK];                                  // the student's, relative to km
  float sx[kMaxK];                                  // the student's logits at the listed tokens
  float tab[128];
  float4 part[kDiMaxC];                             // (maximum, sum, twice) of every CTA of the cluster
  float fred[kDiWarps];
  F2 f2red[kDiWarps];
  int twice;
  int infinite;                                     // a listed token the teacher wants has no student mass
  // the row's statistics, by warp 0
  float mt, A, M, invS, Es;                         // Es = 2^((mk - M) c)
  F2 S, st;
};

template <typename T>
__device__ __forceinline__ void zero_slice_of(const Window<T>& g, int v0, int v1, int first, int step) {
  for (int v = v0 + first; v < v1; v += step) g.store(v, make_uint4(0u, 0u, 0u, 0u));
}
template <typename T>
__device__ __forceinline__ void zero_slice(const Window<T>& g, int v0, int v1) {
  zero_slice_of(g, v0, v1, (int)threadIdx.x, (int)blockDim.x);
}

template <typename T, int U, bool GRAD>
__global__ void __launch_bounds__(kDiThreads, 2) distill_kernel(const DistillParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  constexpr int CH = kDiThreads * U;                // vectors per chunk
  __shared__ __align__(16) DistillSmem<T, U> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / p.C, rank = blockIdx.x - r * p.C;
  const Window<T, const T> win(static_cast<const T*>(p.student), (size_t)r, p.V);
  const Window<T> gwin(static_cast<T*>(p.grad), (size_t)r, p.V);
  const int NV = win.vectors();
  const int v0 = min(rank * p.SV, NV), v1 = min(v0 + p.SV, NV);
  const int k = p.k;
  const F2 c{p.c, p.c_lo};
  const float wgt = p.weight ? __ldg(p.weight + r) : 1.f;
  if (wgt == 0.f) {                                 // the same for the whole cluster
    if (GRAD) zero_slice(gwin, v0, v1);
    if (rank == 0 && tid == 0) {
      p.loss[r] = 0.f;
      if (p.stats) p.stats[(size_t)r * 8 + 7] = 0.f;
    }
    return;
  }
  cluster_arrive();                                 // waited for before the first push: every CTA has started

  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = v0 + u * kDiThreads + tid;
    x[u] = v < v1 && v < v0 + CH ? win.load(v) : make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
  }

  // ---- the teacher, and the student at the listed tokens
  load_exp2_table(sm.tab);
  if (tid == 0) sm.twice = sm.infinite = 0;
  const float ltail = p.tail ? __ldg(p.tail + r) : -INFINITY;
  float tm = ltail != ltail ? INFINITY : ltail, km = -INFINITY;   // a NaN makes the maximum +inf, and the row NaN
  float lpv[2], sv_[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int j = tid + q * kDiThreads;
    lpv[q] = sv_[q] = -INFINITY;
    if (j < k) {
      int id = __ldg(p.indices + (size_t)r * k + j);
      if ((unsigned)id >= (unsigned)p.V) id = -1;
      if (id >= 0) {
        lpv[q] = __ldg(p.logprobs + (size_t)r * k + j);
        sv_[q] = Elem<T>::load(win.base + win.a0 + id);
        tm = fmaxf(tm, lpv[q] != lpv[q] ? INFINITY : lpv[q]);
        km = fmaxf(km, sv_[q]);
      }
      sm.sid[j] = id;
      sm.sx[j] = sv_[q];
    }
  }
  tm = block_max_n<kDiWarps>(tm, sm.fred);
  km = block_max_n<kDiWarps>(km, sm.fred);
  if (!(tm > -INFINITY)) {                          // nothing to learn from (the same for the whole cluster)
    cluster_wait();
    if (GRAD) zero_slice(gwin, v0, v1);
    if (rank == 0 && tid == 0) {
      p.loss[r] = 0.f;
      if (p.stats) p.stats[(size_t)r * 8 + 7] = 0.f;
    }
    return;
  }
  const F2 l2e{kLog2eHi, kLog2eLo}, inv_t = f2_from(p.inv_t);
  F2 Z{0.f, 0.f}, WK{0.f, 0.f}, E1{0.f, 0.f};
  const F2 wt = p.tail ? weight_f2(ltail, tm, l2e, sm.tab) : F2{0.f, 0.f};
  const float kr = km == -INFINITY ? 0.f : km;      // the reference of the listed tokens' logarithms
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int j = tid + q * kDiThreads;
    if (j < k) {
      F2 w{0.f, 0.f}, ws{0.f, 0.f};
      if (sm.sid[j] >= 0) {
        w = weight_f2(lpv[q], tm, l2e, sm.tab);
        ws = weight_f2(sv_[q], km, c, sm.tab);
        Z = f2_add(Z, w);
        WK = f2_add(WK, ws);
        if (w.hi != 0.f) {
          if ((sv_[q] - kr) * inv_t.hi < -kDiFar) sm.infinite = 1;
          else E1 = f2_add(E1, distill_term(w, lpv[q], tm, sv_[q], kr, inv_t));
        }
      }
      sm.sw[j] = w.hi;
      sm.sq[j] = ws.hi;
    }
  }
  Z = f2_add(block_sum_f2_n<kDiWarps>(Z, sm.f2red), wt);
  WK = block_sum_f2_n<kDiWarps>(WK, sm.f2red);
  if (rank == 0) E1 = block_sum_f2_n<kDiWarps>(E1, sm.f2red);

  // ---- the slice without the listed tokens: (maximum, sum)
  float m = -INFINITY;
  F2 s{0.f, 0.f};
  for (int ch = 0; ch < p.NCK; ++ch) {
    const int c0 = v0 + ch * CH;
    if (ch > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = c0 + u * kDiThreads + tid;
        x[u] = v < v1 ? win.load(v) : make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
      }
    }
    __syncthreads();
    for (int i = tid; i < CH * VW / 32; i += kDiThreads) sm.bits[i] = 0u;
    __syncthreads();
    const int p0 = c0 * VW - win.a0;                // row index of the chunk's first element
    const int pn = min(CH, v1 - c0) * VW;
    for (int j = tid; j < k; j += kDiThreads) {
      const int o = sm.sid[j] - p0;
      if (sm.sid[j] >= 0 && o >= 0 && o < pn) {
        const uint32_t bit = 1u << (o & 31);
        if (atomicOr(&sm.bits[o >> 5], bit) & bit) sm.twice = 1;
      }
    }
    __syncthreads();
    float tmx = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int lv = u * kDiThreads + tid;
      const uint32_t b = (sm.bits[lv * VW / 32] >> (lv * VW % 32)) & ((1u << VW) - 1u);
      if (b) {
#pragma unroll
        for (int t = 0; t < VW; ++t)
          if ((b >> t) & 1u) TR::put(x[u], t, Elem<T>::kNegInf);
      }
      tmx = fmaxf(tmx, TR::template vmax<false>(x[u]));
    }
    const float mc = block_max_n<kDiWarps>(tmx, sm.fred);
    const float ref = mc == -INFINITY ? 0.f : mc;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < VW; t += 4) {
        s0 += ex2_approx((TR::get(x[u], t) - ref) * p.c);
        s1 += ex2_approx((TR::get(x[u], t + 1) - ref) * p.c);
        s2 += ex2_approx((TR::get(x[u], t + 2) - ref) * p.c);
        s3 += ex2_approx((TR::get(x[u], t + 3) - ref) * p.c);
      }
    const F2 sc = block_sum_f2_n<kDiWarps>(f2_add(f2_add(F2{s0, 0.f}, F2{s1, 0.f}), f2_add(F2{s2, 0.f}, F2{s3, 0.f})),
                                           sm.f2red);
    if (ch == 0) {
      m = mc;
      s = sc;
    } else {
      const float mn = fmaxf(m, mc);
      const F2 a = m == mn ? s : f2_mul(s, weight_f2(m, mn, c, sm.tab));
      const F2 b = mc == mn ? sc : f2_mul(sc, weight_f2(mc, mn, c, sm.tab));
      s = f2_add(a, b);
      m = mn;
    }
  }

  // ---- the row: every CTA hands its part to all
  cluster_wait();                                   // all CTAs of the cluster run
  if (tid < p.C) push_f4(&sm.part[rank], tid, make_float4(m, s.hi, s.lo, sm.twice ? 1.f : 0.f));
  cluster_arrive();
  cluster_wait();
  const bool twice = __syncthreads_or(tid < p.C && sm.part[tid < p.C ? tid : 0].w != 0.f);
  if (twice) {                                      // a token's weight counts once, whatever the list says
    // (from shared memory: in place, other CTAs write the row's gradient from here on)
    F2 w1{0.f, 0.f};
    for (int j = tid; j < k; j += kDiThreads) {
      bool first = sm.sid[j] >= 0;
      for (int i = 0; i < j && first; ++i) first = sm.sid[i] != sm.sid[j];
      if (first) w1 = f2_add(w1, weight_f2(sm.sx[j], km, c, sm.tab));
    }
    WK = block_sum_f2_n<kDiWarps>(w1, sm.f2red);
  }
  if (warp == 0) {
    const float4 v = lane < p.C ? sm.part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    float mt = v.x;
#pragma unroll
    for (int o = kDiMaxC / 2; o >= 1; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    F2 st{v.y, v.z};
    if (v.x != mt) st = v.x == -INFINITY ? st : f2_mul(st, weight_f2(v.x, mt, c, sm.tab));
#pragma unroll
    for (int o = kDiMaxC / 2; o >= 1; o >>= 1) st = f2_add(st, f2_shfl_xor(st, o));
    if (lane == 0) {
      const float M = fmaxf(mt, km);
      const F2 Et = mt == M ? F2{1.f, 0.f} : weight_f2(mt, M, c, sm.tab);
      const F2 Ek = km == M ? F2{1.f, 0.f} : weight_f2(km, M, c, sm.tab);
      const F2 tailm = mt == M ? st : f2_mul(st, Et);
      const F2 S = f2_add(tailm, km == M ? WK : f2_mul(WK, Ek));
      const bool good = S.hi > 0.f && S.hi < INFINITY;
      const float nan = __uint_as_float(0x7fffffffu);
      const float invS = good ? f2_rcp(S) : nan;
      const float pt = wt.hi * f2_rcp(Z);
      const bool some = st.hi > 0.f;
      sm.mt = mt == -INFINITY ? 0.f : mt;
      // (without mass outside nothing is to be formed there, but a teacher's NaN shows)
      sm.A = !good || pt != pt ? nan : !some ? 0.f : Et.hi * invS - (pt == 0.f ? 0.f : pt * f2_rcp(st));
      sm.M = M;
      sm.invS = invS;
      sm.Es = Ek.hi;
      sm.S = S;
      sm.st = st;
      if (!good) sm.mt = 0.f;
      if (rank == 0 && p.stats) {
        float4* o = reinterpret_cast<float4*>(p.stats + (size_t)r * 8);
        o[0] = make_float4(sm.mt, sm.A, tm, f2_rcp(Z));
        o[1] = make_float4(M, invS, twice ? 1.f : 0.f, 1.f);
      }
    }
  }
  __syncthreads();

  if (GRAD) {
    const float sc = (float)((double)wgt * p.inv_t);
    const float mt = sm.mt, gA = sc * sm.A;
    for (int ch = 0; ch < p.NCK; ++ch) {
      const int c0 = v0 + ch * CH;
      if (p.NCK > 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = c0 + u * kDiThreads + tid;
          if (v < v1) x[u] = win.load(v);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = c0 + u * kDiThreads + tid;
        if (v < v1) {
          float g[VW];
#pragma unroll
          for (int t = 0; t < VW; ++t) g[t] = gA * ex2_approx((TR::get(x[u], t) - mt) * p.c);
          gwin.store(v, Elem<T>::pack(g));
        }
      }
    }
    __syncthreads();                                // the listed tokens of the slice go on top
    const int p0 = v0 * VW - win.a0, p1 = v1 * VW - win.a0;
    const float invZ = f2_rcp(Z), qs = sm.Es * sm.invS;
    for (int j = tid; j < k; j += kDiThreads) {
      const int id = sm.sid[j];
      if (id < 0 || id < p0 || id >= p1) continue;
      float w = sm.sw[j];
      if (twice) {
        w = 0.f;
        for (int i = 0; i < k; ++i)
          if (sm.sid[i] == id) w += sm.sw[i];
      }
      Elem<T>::store(gwin.base + gwin.a0 + id, sc * (sm.sq[j] * qs - w * invZ));
    }
  }
  if (rank == 0 && warp == 0) {
    const float l = distill_loss(Z, sm.S, sm.st, E1, wt, ltail, tm, sm.mt, km, sm.M, sm.infinite, inv_t, sm.tab);
    if (lane == 0) p.loss[r] = wgt * l;
  }
}

template <typename T>
__global__ void __launch_bounds__(kDiBwThreads, 4) distill_backward_kernel(const DistillParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  constexpr int U = kDiBwU;
  const int tid = threadIdx.x, k = p.k;
  const int r = blockIdx.x / p.C, h = blockIdx.x - r * p.C;
  const Window<T, const T> win(static_cast<const T*>(p.student), (size_t)r, p.V);
  const Window<T> gwin(static_cast<T*>(p.grad), (size_t)r, p.V);
  const int NV = win.vectors();
  const int v0 = min(h * p.SV, NV), v1 = min(v0 + p.SV, NV);
  const float wgt = p.weight ? __ldg(p.weight + r) : 1.f;
  const float up = __ldg(p.grad_loss + (size_t)r * p.up_stride);
  const float* st = p.stats + (size_t)r * 8;
  if (wgt == 0.f || up == 0.f || __ldg(st + 7) == 0.f) {
    zero_slice(gwin, v0, v1);
    return;
  }
  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = v0 + u * kDiBwThreads + tid;
    if (v < v1) x[u] = win.load(v);
  }
  // the listed tokens of the slice: their gradient, before anything is written over the student
  const float sc = (float)((double)wgt * (double)up * p.inv_t);
  const int p0 = v0 * VW - win.a0, p1 = v1 * VW - win.a0;
  const int32_t* idx = p.indices + (size_t)r * k;
  const float* lp = p.logprobs + (size_t)r * k;
  const float tm = __ldg(st + 2), invZ = __ldg(st + 3), M = __ldg(st + 4), invS = __ldg(st + 5);
  const bool twice = __ldg(st + 6) != 0.f;
  int kid[4];
  float kg[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = tid + q * kDiBwThreads;
    kid[q] = -1;
    if (j < k) {
      const int id = __ldg(idx + j);
      if (id >= 0 && id < p.V && id >= p0 && id < p1) {
        float w = 0.f;
        if (twice) {
          for (int i = 0; i < k; ++i)
            if (__ldg(idx + i) == id) w += weight_fast(__ldg(lp + i) - tm, kLog2eHi, kLog2eLo);
        } else {
          w = weight_fast(__ldg(lp + j) - tm, kLog2eHi, kLog2eLo);
        }
        const float q_j = weight_fast(Elem<T>::load(win.base + win.a0 + id) - M, p.c, p.c_lo) * invS;
        kid[q] = id;
        kg[q] = sc * (q_j - w * invZ);
      }
    }
  }
  const float mt = __ldg(st), gA = sc * __ldg(st + 1);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = v0 + u * kDiBwThreads + tid;
    if (v < v1) {
      float g[VW];
#pragma unroll
      for (int t = 0; t < VW; ++t) g[t] = gA * ex2_approx((TR::get(x[u], t) - mt) * p.c);
      gwin.store(v, Elem<T>::pack(g));
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (kid[q] >= 0) Elem<T>::store(gwin.base + gwin.a0 + kid[q], kg[q]);
}

}  // namespace rows
}  // namespace sv
