// Distillation over many rows: a persistent cluster of C CTAs takes row after
// row, so that loading, summing, exchanging and writing overlap between
// neighbouring rows instead of following one another within each.
//
// Per CTA, 16 streaming warps own the CTA's slice of every row through a ring
// of kDpStages cp.async stages private to each thread (a thread reads back
// only what it copied), and 8 list warps own what the teacher's list needs,
// one listed token per thread.  In iteration t
//
//   A  streaming warps: row t without its listed tokens -> (maximum, sum) per warp
//      list warp 0:     row t - 1's statistics from the parts of all C CTAs
//   -- block barrier
//   B  streaming warps: row t - 1's gradient, out of the ring; row t + 2 into it
//      list warps:      row t's part to all CTAs (one cluster barrier, waited
//                       for at the end of the iteration); the listed tokens of
//                       row t - 2 on top of its gradient, and its loss; the
//                       list of row t + 2, whose loads were issued an
//                       iteration earlier
//
// so every dependent chain (the gather of the listed tokens, the two-float
// sums, the exchange, the float64 logarithms of the loss) has at least half an
// iteration in which the streaming warps have work of their own.  The forward
// pass alone has no B for the streaming warps; there the cluster barrier is
// waited for at the end of the next A.
//
// Bound: HBM, with the exponentials close behind (two per element at 16 per
// clock and SM: 77 % of the time the bytes of a bf16 row take).
#pragma once

#include "sv_distill.cuh"

namespace sv {
namespace rows {

constexpr int kDpSt = 512;              // streaming threads
constexpr int kDpLi = 256;              // list threads: the largest list
constexpr int kDpThreads = kDpSt + kDpLi;
constexpr int kDpU = 8;                 // vectors per streaming thread and row
constexpr int kDpSlice = kDpSt * kDpU;  // vectors per CTA and row
constexpr int kDpStages = 3;
constexpr int kDpLists = 6;             // rows whose lists are alive

struct DpList {
  int sid[kDpLi];                       // listed tokens (-1: ignored)
  float sw[kDpLi], sq[kDpLi];           // the teacher's and the student's weights
  float tm, km, ltail, wgt;
  F2 Z, WK, E1, wt;
  int live;                             // 0: weight 0, 1: nothing to learn from, 2: a row
  int infinite, twice;
};
struct DpStat {
  float mt, A, M, invS, Es;
  F2 S, st;
  int twice;
};
template <typename T>
struct DpSmem {
  uint4 ring[kDpStages][kDpU][kDpSt];
  uint32_t bits[2][kDpSlice * Tr<T>::VW / 32];
  DpList list[kDpLists];
  DpStat stat[kDpLists];
  float4 part[3][kDiMaxC];              // a row's parts: read while the next row's may be arriving
  float4 wpart[2][kDpSt / 32];
  F2 lsum[kDpLi / 32][3];
  float2 lmax[kDpLi / 32];
  float tab[128];
};

__device__ __forceinline__ void list_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
static_assert(kDpLi == 256, "list_barrier");

// The statistics of a row from the C parts (one warp; lane 0 writes).
__device__ __forceinline__ void dp_statistics(const float4* part, int C, const DpList& L, int k, F2 c, const float* tab,
                                              DpStat& out, float* stats) {
  const int lane = threadIdx.x & 31;
  const float4 v = lane < C ? part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  const bool twice = __any_sync(0xffffffffu, v.w != 0.f);
  float mt = v.x;
#pragma unroll
  for (int o = kDiMaxC / 2; o >= 1; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
  F2 st{v.y, v.z};
  if (v.x != mt) st = v.x == -INFINITY ? st : f2_mul(st, weight_f2(v.x, mt, c, tab));
#pragma unroll
  for (int o = kDiMaxC / 2; o >= 1; o >>= 1) st = f2_add(st, f2_shfl_xor(st, o));
  F2 WK = L.WK;
  if (twice) {                          // a token's weight counts once, whatever the list says
    WK = F2{0.f, 0.f};
    for (int j = lane; j < k; j += 32) {
      bool first = L.sid[j] >= 0;
      for (int i = 0; i < j && first; ++i) first = L.sid[i] != L.sid[j];
      if (first) WK = f2_add(WK, F2{L.sq[j], 0.f});
    }
    WK = warp_sum_f2(WK);
  }
  if (lane == 0) {
    const float km = L.km;
    const float M = fmaxf(mt, km);
    const F2 Et = mt == M ? F2{1.f, 0.f} : weight_f2(mt, M, c, tab);
    const F2 Ek = km == M ? F2{1.f, 0.f} : weight_f2(km, M, c, tab);
    const F2 S = f2_add(mt == M ? st : f2_mul(st, Et), km == M ? WK : f2_mul(WK, Ek));
    const bool good = S.hi > 0.f && S.hi < INFINITY;
    const float nan = __uint_as_float(0x7fffffffu);
    const float invS = good ? f2_rcp(S) : nan;
    const float invZ = f2_rcp(L.Z);
    const float pt = L.wt.hi * invZ;
    const bool some = st.hi > 0.f;
    out.mt = mt == -INFINITY || !good ? 0.f : mt;
    out.A = !good ? nan : !some ? 0.f : Et.hi * invS - (pt == 0.f ? 0.f : pt * f2_rcp(st));
    out.M = M;
    out.invS = invS;
    out.Es = Ek.hi;
    out.S = S;
    out.st = st;
    out.twice = twice;
    if (stats) {
      float4* o = reinterpret_cast<float4*>(stats);
      o[0] = make_float4(out.mt, out.A, L.tm, invZ);
      o[1] = make_float4(M, invS, twice ? 1.f : 0.f, L.live == 2 ? 1.f : 0.f);
    }
  }
}

// The loss of a row (one warp: the three logarithms side by side).
__device__ __forceinline__ void dp_loss(const DpList& L, const DpStat& s, double inv_t, float* loss) {
  const int lane = threadIdx.x & 31;
  if (L.live != 2) {
    if (lane == 0) *loss = 0.f;
    return;
  }
  const F2 mine = lane == 0 ? L.Z : lane == 1 ? s.S : s.st;
  const double lg = log(f2_double(mine));
  const double lz = __shfl_sync(0xffffffffu, lg, 0), ls = __shfl_sync(0xffffffffu, lg, 1),
               lt = __shfl_sync(0xffffffffu, lg, 2);
  if (lane == 0) {
    const double kr = L.km == -INFINITY ? 0.0 : (double)L.km;
    double e = f2_double(L.E1);
    if (L.wt.hi != 0.f)
      e += f2_double(L.wt) * (((double)L.ltail - (double)L.tm) - (((double)s.mt - kr) * inv_t + lt));
    double l = e / f2_double(L.Z) - lz + ls + ((double)s.M - kr) * inv_t;
    if (!(s.S.hi > 0.f && s.S.hi < INFINITY)) l = __longlong_as_double(0x7fffffffffffffffll);
    else if (L.infinite && l == l) l = (double)INFINITY;
    *loss = (float)((double)L.wgt * l);
  }
}

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kDpThreads, 1) distill_pipe_kernel(const DistillParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DpSmem<T>& sm = *reinterpret_cast<DpSmem<T>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.C, rank = blockIdx.x % C;
  const int g = blockIdx.x / C, NG = gridDim.x / C;
  const int n = (p.R - g + NG - 1) / NG;            // rows of this cluster: g, g + NG, ...
  const int k = p.k;
  const F2 c{p.c, p.c_lo};
  const bool streaming = tid < kDpSt;
  const T* student = static_cast<const T*>(p.student);
  cluster_arrive();                                 // waited for before the first push: every CTA has started

  // ---- streaming warps: the ring
  auto issue = [&](int i) {                         // row i of the cluster into its stage
    if (i < n) {
      const int r = g + i * NG;
      if (!p.weight || __ldg(p.weight + r) != 0.f) {
        const Window<T, const T> win(student, (size_t)r, p.V);
        const int v0 = min(rank * p.SV, win.vectors()), v1 = min(v0 + p.SV, win.vectors());
        uint4(*st)[kDpSt] = sm.ring[i % kDpStages];
#pragma unroll
        for (int u = 0; u < kDpU; ++u) {
          const int v = v0 + u * kDpSt + tid;
          if (v < v1) {
            if (win.whole(v)) {
              const unsigned sa = (unsigned)__cvta_generic_to_shared(&st[u][tid]);
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa), "l"(win.base + (size_t)v * VW) : "memory");
            } else {
              st[u][tid] = win.load(v);
            }
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // ---- list warps: a listed token per thread, loads an iteration ahead of their use
  const int lt = tid - kDpSt, lw = lt >> 5;
  int id1 = -1, id2 = -1;                           // of the row whose student value is loaded, and of the next
  float lp1 = -INFINITY, lp2 = -INFINITY, s1 = -INFINITY;
  auto load_list = [&](int i, int& id, float& lp) {
    id = -1;
    lp = -INFINITY;
    if (i < n && lt < k) {
      const size_t r = g + (size_t)i * NG;
      const int v = __ldg(p.indices + r * k + lt);
      if ((unsigned)v < (unsigned)p.V) id = v;
      lp = __ldg(p.logprobs + r * k + lt);
    }
  };
  auto load_student = [&](int i, int id) {
    if (id < 0) return -INFINITY;
    return Elem<T>::load(student + ((size_t)g + (size_t)i * NG) * p.V + id);
  };
  // the list of row i from (id1, lp1, s1)
  auto prepare = [&](int i) {
    if (i >= n) return;                             // the same for all list threads
    const int r = g + i * NG;
    DpList& L = sm.list[i % kDpLists];
    uint32_t* bits = sm.bits[i & 1];
    for (int w = lt; w < kDpSlice * VW / 32; w += kDpLi) bits[w] = 0u;
    const float wgt = p.weight ? __ldg(p.weight + r) : 1.f;
    const float ltail = p.tail ? __ldg(p.tail + r) : -INFINITY;
    if (lt == 0) L.infinite = L.twice = 0;
    const bool on = id1 >= 0;
    const float lp = on ? lp1 : -INFINITY, s = on ? s1 : -INFINITY;
    float tm = lp != lp ? INFINITY : lp, km = s;    // a NaN makes the maximum +inf, and the row NaN
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, m));
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, m));
    }
    if (lane == 0) sm.lmax[lw] = make_float2(tm, km);
    list_barrier();
    tm = ltail != ltail ? INFINITY : ltail;
    km = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDpLi / 32; ++w) {
      tm = fmaxf(tm, sm.lmax[w].x);
      km = fmaxf(km, sm.lmax[w].y);
    }
    const F2 l2e{kLog2eHi, kLog2eLo};
    F2 w{0.f, 0.f}, ws{0.f, 0.f}, e1{0.f, 0.f};
    if (lw * 32 < k) {                              // warps with listed tokens
      const float kr = km == -INFINITY ? 0.f : km;
      if (on) {
        w = weight_f2(lp, tm, l2e, sm.tab);
        ws = weight_f2(s, km, c, sm.tab);
        if (w.hi != 0.f) {
          if (s == -INFINITY) {
            L.infinite = 1;
          } else {
            e1 = f2_mul(w, f2_from(((double)lp - (double)tm) - ((double)s - (double)kr) * p.inv_t));
          }
        }
        const Window<T, const T> win(student, (size_t)r, p.V);
        const int v0 = min(rank * p.SV, win.vectors()), v1 = min(v0 + p.SV, win.vectors());
        const int o = id1 + win.a0 - v0 * VW;
        if (o >= 0 && o < (v1 - v0) * VW) {
          const uint32_t bit = 1u << (o & 31);
          if (atomicOr(&bits[o >> 5], bit) & bit) L.twice = 1;
        }
      }
      const F2 a = warp_sum_f2(w), b = warp_sum_f2(ws), d = warp_sum_f2(e1);
      if (lane == 0) {
        sm.lsum[lw][0] = a;
        sm.lsum[lw][1] = b;
        sm.lsum[lw][2] = d;
      }
    }
    L.sid[lt] = id1;
    L.sw[lt] = w.hi;
    L.sq[lt] = ws.hi;
    list_barrier();
    if (lw == 1) {                                  // (warp 0 has the exchange to do)
      F2 a{0.f, 0.f}, b{0.f, 0.f}, d{0.f, 0.f};
      if (lane < (k + 31) / 32) {
        a = sm.lsum[lane][0];
        b = sm.lsum[lane][1];
        d = sm.lsum[lane][2];
      }
#pragma unroll
      for (int m = kDpLi / 64; m >= 1; m >>= 1) {
        a = f2_add(a, f2_shfl_xor(a, m));
        b = f2_add(b, f2_shfl_xor(b, m));
        d = f2_add(d, f2_shfl_xor(d, m));
      }
      if (lane == 0) {
        const F2 wt = p.tail ? weight_f2(ltail, tm, l2e, sm.tab) : F2{0.f, 0.f};
        L.Z = f2_add(a, wt);
        L.WK = b;
        L.E1 = d;
        L.wt = wt;
        L.tm = tm;
        L.km = km;
        L.ltail = ltail;
        L.wgt = wgt;
        L.live = wgt == 0.f ? 0 : tm > -INFINITY ? 2 : 1;
      }
    }
  };

  for (int i = tid; i < 128; i += kDpThreads) sm.tab[i] = i < 64 ? __ldg(kExp2Hi + i) : __ldg(kExp2Lo + i - 64);
  __syncthreads();
  if (streaming) {
    issue(0);
    issue(1);
    if (!GRAD) issue(2);
  } else {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      load_list(i, id1, lp1);
      s1 = load_student(i, id1);
      prepare(i);
      list_barrier();
    }
    load_list(2, id1, lp1);
    s1 = load_student(2, id1);
    load_list(3, id2, lp2);
  }
  cluster_wait();                                   // every CTA of the cluster has started
  __syncthreads();

#pragma unroll 1
  for (int t = 0; t <= n + 1; ++t) {                // (the last row's list and loss come two iterations later)
    // ---------------------------------------------------------------- A
    if (streaming) {
      if (t < n) {
        asm volatile("cp.async.wait_group %0;" ::"n"(GRAD ? 1 : 2) : "memory");
        if (sm.list[t % kDpLists].live != 0) {
          const int r = g + t * NG;
          const Window<T, const T> win(student, (size_t)r, p.V);
          const int v0 = min(rank * p.SV, win.vectors()), v1 = min(v0 + p.SV, win.vectors());
          const uint4(*st)[kDpSt] = sm.ring[t % kDpStages];
          const unsigned char* bits = reinterpret_cast<const unsigned char*>(sm.bits[t & 1]);
          uint4 x[kDpU];
          float m = -INFINITY;
#pragma unroll
          for (int u = 0; u < kDpU; ++u) {
            const int lv = u * kDpSt + tid;
            x[u] = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
            if (v0 + lv < v1) x[u] = st[u][tid];
            const uint32_t b = VW == 8 ? bits[lv] : (bits[lv >> 1] >> ((lv & 1) * 4)) & 15u;
            if (b) {
#pragma unroll
              for (int e = 0; e < VW; ++e)
                if ((b >> e) & 1u) TR::put(x[u], e, Elem<T>::kNegInf);
            }
            m = fmaxf(m, TR::template vmax<false>(x[u]));
          }
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float ref = m == -INFINITY ? 0.f : m, rho = ref * p.c;
          float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f, fix = 1.f;
          if (fabsf(rho) < kNear) {
            // one multiply-add and one exponential a term; the rounding of rho leaves at the end
            fix = ex2_approx(-fmaf(ref, p.c, -rho));
#pragma unroll
            for (int u = 0; u < kDpU; ++u)
#pragma unroll
              for (int e = 0; e < VW; e += 4) {
                a0 += ex2_approx(fmaf(TR::get(x[u], e), p.c, -rho));
                a1 += ex2_approx(fmaf(TR::get(x[u], e + 1), p.c, -rho));
                a2 += ex2_approx(fmaf(TR::get(x[u], e + 2), p.c, -rho));
                a3 += ex2_approx(fmaf(TR::get(x[u], e + 3), p.c, -rho));
              }
          } else {                                  // enormous logits or a tiny temperature: the difference first
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
#pragma unroll 1
              for (int e = 0; e < VW; ++e) a0 += ex2_approx((TR::get(x[u], e) - ref) * p.c);
            }
          }
          F2 s = f2_add(f2_add(F2{a0, 0.f}, F2{a1, 0.f}), f2_add(F2{a2, 0.f}, F2{a3, 0.f}));
          s = f2_mul(warp_sum_f2(s), F2{fix, 0.f});
          if (lane == 0) sm.wpart[t & 1][warp] = make_float4(m, s.hi, s.lo, 0.f);
        }
      }
      if (!GRAD) issue(t + 3);
    } else if (GRAD && lw == 0 && t >= 1 && t - 1 < n) {
      dp_statistics(sm.part[(t - 1) % 3], C, sm.list[(t - 1) % kDpLists], k, c, sm.tab, sm.stat[(t - 1) % kDpLists], nullptr);
    }
    if (!GRAD && t >= 1) cluster_wait();            // row t - 1's parts are in
    __syncthreads();
    // ---------------------------------------------------------------- B
    if (streaming) {
      cluster_arrive();
      if (GRAD) {
        if (t >= 1 && t - 1 < n) {
          const int i = t - 1, r = g + i * NG;
          const Window<T> gwin(static_cast<T*>(p.grad), (size_t)r, p.V);
          const int v0 = min(rank * p.SV, gwin.vectors()), v1 = min(v0 + p.SV, gwin.vectors());
          const DpList& L = sm.list[i % kDpLists];
          const uint4(*st)[kDpSt] = sm.ring[i % kDpStages];
          const bool row = L.live == 2;
          const float mt = row ? sm.stat[i % kDpLists].mt : 0.f, rho = mt * p.c;
          float gA = row ? (float)((double)L.wgt * p.inv_t) * sm.stat[i % kDpLists].A : 0.f;
          if (!row) {
            zero_slice_of(gwin, v0, v1, tid, kDpSt);
          } else if (fabsf(rho) < kNear) {
            gA *= ex2_approx(-fmaf(mt, p.c, -rho));
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
              const int v = v0 + u * kDpSt + tid;
              if (v < v1) {
                const uint4 x = st[u][tid];
                float gr[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) gr[e] = gA * ex2_approx(fmaf(TR::get(x, e), p.c, -rho));
                gwin.store(v, Elem<T>::pack(gr));
              }
            }
          } else {
#pragma unroll 1
            for (int u = 0; u < kDpU; ++u) {
              const int v = v0 + u * kDpSt + tid;
              if (v < v1) {
                const uint4 x = st[u][tid];
                float gr[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) gr[e] = gA * ex2_approx((TR::get(x, e) - mt) * p.c);
                gwin.store(v, Elem<T>::pack(gr));
              }
            }
          }
        }
        issue(t + 2);
      }
    } else {
      if (lw == 0) {
        if (t < n && sm.list[t % kDpLists].live != 0) {
          // the CTA's part of row t: 16 warps' (maximum, sum)
          const float4 v = lane < kDpSt / 32 ? sm.wpart[t & 1][lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
          float m = v.x;
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = __shfl_sync(0xffffffffu, m, 0);
          F2 s{v.y, v.z};
          if (v.x != m) s = v.x == -INFINITY ? F2{0.f, 0.f} : f2_mul(s, weight_f2(v.x, m, c, sm.tab));
          if (lane >= kDpSt / 32) s = F2{0.f, 0.f};
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) s = f2_add(s, f2_shfl_xor(s, o));
          s = F2{__shfl_sync(0xffffffffu, s.hi, 0), __shfl_sync(0xffffffffu, s.lo, 0)};
          if (lane < C)
            push_f4(&sm.part[t % 3][rank], lane, make_float4(m, s.hi, s.lo, sm.list[t % kDpLists].twice ? 1.f : 0.f));
        }
        __syncwarp();
      }
      cluster_arrive();
      if (!GRAD && lw == 0 && t >= 1 && t - 1 < n)
        dp_statistics(sm.part[(t - 1) % 3], C, sm.list[(t - 1) % kDpLists], k, c, sm.tab, sm.stat[(t - 1) % kDpLists],
                      rank == 0 && p.stats ? p.stats + (size_t)(g + (t - 1) * NG) * 8 : nullptr);
      if (t >= 2 && t - 2 < n) {
        const int i = t - 2, r = g + i * NG;
        const DpList& L = sm.list[i % kDpLists];
        const DpStat& s = sm.stat[i % kDpLists];
        if (GRAD && L.live == 2 && lt < k && L.sid[lt] >= 0) {
          const int id = L.sid[lt];
          const Window<T> gwin(static_cast<T*>(p.grad), (size_t)r, p.V);
          const int v0 = min(rank * p.SV, gwin.vectors()), v1 = min(v0 + p.SV, gwin.vectors());
          const int o = id + gwin.a0;
          if (o >= v0 * VW && o < v1 * VW) {
            float w = L.sw[lt];
            if (s.twice) {
              w = 0.f;
              for (int j = 0; j < k; ++j)
                if (L.sid[j] == id) w += L.sw[j];
            }
            Elem<T>::store(gwin.base + o,
                           (float)((double)L.wgt * p.inv_t) * (L.sq[lt] * (s.Es * s.invS) - w * f2_rcp(L.Z)));
          }
        }
        if (rank == 0 && lw == kDpLi / 32 - 1) dp_loss(L, s, p.inv_t, p.loss + r);
      }
      // the list of row t + 2, and the loads of the rows behind it
      const float s2 = load_student(t + 3, id2);
      int id3;
      float lp3;
      load_list(t + 4, id3, lp3);
      prepare(t + 2);
      id1 = id2;
      lp1 = lp2;
      s1 = s2;
      id2 = id3;
      lp2 = lp3;
    }
    if (GRAD) cluster_wait();
  }
  if (!GRAD) cluster_wait();
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace rows
}  // namespace sv
