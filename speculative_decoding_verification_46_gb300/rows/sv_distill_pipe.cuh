// Distillation over many rows: a persistent cluster of C CTAs takes row after
// row, so that loading, summing, exchanging and writing overlap between
// neighbouring rows instead of following one another within each.
//
// The warps of a CTA have four roles and wait for one another only where one
// needs what another made, through mbarriers in shared memory: a warp that
// finds its barrier complete goes on alone, so the streaming warps drift
// apart and keep the pipes busy with different phases.  (With named barriers,
// which make all waiting warps meet, half of the time went to the slowest of
// them.)
//
//   streaming (22 warps)  own the CTA's slice of every row through a ring of
//       kDpStages cp.async stages private to each thread (a thread reads back
//       only what it copied).  Per row t: sum the slice without its listed
//       tokens to (maximum, sum); then write row t - 1's gradient out of the
//       ring and start loading row t + 2 into the stage that frees.
//   list (two groups of up to 2 warps, a row each in turn)  the teacher's
//       softmax and the student's weights at the listed tokens (two-float),
//       the bitmap that takes the tokens out of the streams, and at the end
//       the tokens' own gradient on top of the dense one.  The loads of a
//       list are issued a row of the group before they are used.
//   parts (1 warp)  the CTA's part of row t to all CTAs of the cluster.
//   statistics (1 warp)  from the C parts the row's statistics, and its loss;
//       the CTAs take the losses in turn.
//
// So every dependent chain - gather, two-float sums, exchange, logarithms -
// has a whole row's streaming time to finish in.  The forward pass alone is
// the same without the gradient.
//
// Every wait is bounded.  A role that gives up notes it in every CTA of the
// cluster and leaves its loop, the others follow as their own waits run out,
// and when all have left, losses, statistics and gradients of all the
// cluster's rows are overwritten with NaN: what was finished in time cannot be
// told from what was not.
//
// Bound: HBM, with instruction issue close behind (loss and gradient: 4096 rows
// of 128256 bf16, k = 64, a tenth of weight 0: 344 us, 5.8 TB/s, 0.85 of the
// measured copy); the loss alone by the streaming warps' instructions and
// latency (2048 rows, 0.47 GB: 114 us, 0.61).  A slice of 64 KB in three stages
// fills an SM's shared memory, so a row of 128256 bf16 is 4 CTAs and 36 clusters
// are resident (144 of 152 SMs); 22 streaming warps of at most 6 vectors a
// thread and row leave 72 registers a thread (16 warps of 8: 483 us against 416
// at that step).
#pragma once

#include "sv_distill.cuh"

namespace sv {
namespace rows {

constexpr int kDpSt = 704;              // streaming threads
constexpr int kDpStWarps = kDpSt / 32;
constexpr int kDpLi = 64;               // most list threads of a group
constexpr int kDpLiE = 4;               // tokens a list thread
constexpr int kDpMaxK = kDpLiE * kDpLi; // the largest list
constexpr int kDpMaxThreads = kDpSt + 32 + 2 * kDpLi + 32;
constexpr int kDpSlice = 4096;          // most vectors per CTA and row
constexpr int kDpU = (kDpSlice + kDpSt - 1) / kDpSt;   // per streaming thread
constexpr int kDpStages = 3;
constexpr int kDpLists = 6;             // rows whose lists are alive
constexpr int kDpParts = 8;             // rows whose parts may arrive: a CTA's streams are at most 4 rows behind
                                        // another's statistics, and those at most 4 behind its own

// list threads of a group, and threads of a CTA, for lists of k tokens
__host__ __device__ constexpr int dp_list_threads(int k) { return k > 32 ? kDpLi : 32; }
__host__ __device__ constexpr int dp_threads(int k) { return kDpSt + 32 + 2 * dp_list_threads(k) + 32; }

struct DpList {
  int sid[kDpMaxK];                     // listed tokens (-1: ignored)
  float sw[kDpMaxK], sq[kDpMaxK];       // the teacher's and the student's weights
  float tm, km, ltail, wgt, sc;         // sc = wgt / temperature
  F2 Z, WK, E1, wt;
  int live;                             // 0: weight 0, 1: nothing to learn from, 2: a row
  int infinite, twice;
};
struct DpStat {
  float mt, A, M, invS, Es;
  F2 S;
  float st;
  int twice;
};
template <typename T>
struct DpSmem {
  uint4 ring[kDpStages][kDpSlice];
  uint32_t bits[3][kDpSlice * Tr<T>::VW / 32];
  uint2 dirty[3][kDpStWarps];           // a byte per (warp, u): some vector there holds a listed token
  DpList list[kDpLists];
  DpStat stat[kDpLists];
  float4 part[kDpParts][kDiMaxC];       // (maximum, sum, -, twice)
  float2 wpart[4][kDpStWarps];
  F2 lsum[2][kDpLi / 32][3];            // by group
  float2 lmax[2][kDpLi / 32];
  float tab[128];
  // mbarriers, each a ring over rows
  unsigned long long summed[4];         // streaming warps -> parts, list: row t is summed
  unsigned long long known[4];          // statistics -> streaming: row t's statistics
  unsigned long long listed[4];         // list -> streaming: row t's list
  unsigned long long written[4];        // streaming warps -> list: row t's dense gradient
  unsigned long long parts[kDpParts];   // parts warps of all CTAs -> statistics
  unsigned long long done[kDpLists];    // statistics -> list: row t's loss is written, its list may be reused
  uint32_t gave_up;                     // a wait somewhere in the cluster ran out
};
static_assert(sizeof(DpSmem<float>) <= 227 * 1024 && sizeof(DpSmem<__half>) <= 227 * 1024, "a CTA's shared memory");

// The meeting point of a list group (all of its warps wait, so a named
// barrier); returns whether all of them say yes.
__device__ __forceinline__ bool list_meet(int group, int n, bool yes) {
  uint32_t all;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\nbarrier.cta.red.and.pred q, %3, %1, p;\nselp.u32 %0, 1, 0, q;\n}"
               : "=r"(all) : "r"(n), "r"((uint32_t)yes), "r"(1 + group) : "memory");
  return all != 0u;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mb_init(unsigned long long* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
// One arrival for the calling warp, after everything its lanes did.
__device__ __forceinline__ void mb_arrive(unsigned long long* b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
// Wait for phase `phase` (0, 1, ...) of the barrier, all lanes; false: given
// up after about a second (a try that finds nothing lasts 3.9 us; a row takes
// microseconds).  The limit is a constant: read from the parameters it cost
// the fused call 1% (351 us against 347, 4096 rows of 128256 bf16, k 64).
constexpr int kDpPatience = 1 << 18;
template <bool CLUSTER = false>
__device__ __forceinline__ bool mb_wait(unsigned long long* b, int phase) {
  const uint32_t a = smem_addr(b), parity = phase & 1;
  uint32_t done = 0u;
#pragma unroll 1
  for (int i = 0; i < kDpPatience && !done; ++i) {
    if (CLUSTER)
      asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                   : "=r"(done) : "r"(a), "r"(parity) : "memory");
    else
      asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                   : "=r"(done) : "r"(a), "r"(parity) : "memory");
  }
  return __all_sync(0xffffffffu, done != 0u);
}
// A warp gives up: every CTA of the cluster will know (they all stay until the
// last barrier of the kernel).
__device__ __forceinline__ void dp_give_up(uint32_t* flag, int C) {
  const int lane = threadIdx.x & 31;
  if (lane < C) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_addr(flag)), "r"(lane));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(d), "r"(1u) : "memory");
  }
  __syncwarp();
}
// Arrive at the barrier that `b` is in CTA `rank` of the cluster, after this
// thread's writes to that CTA's shared memory.
__device__ __forceinline__ void mb_arrive_remote(unsigned long long* b, int rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_addr(b)), "r"(rank));
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(d) : "memory");
}

// The statistics of a row from the C parts (one warp; lane 0 writes).  The
// sum outside the list is float32 up to here: its error moves the loss by
// q_t - p_t of it.  The row's whole sum is two-float, it moves the loss fully.
__device__ __forceinline__ void dp_statistics(const float4* part, int C, const DpList& L, int k, F2 c, const float* tab,
                                              DpStat& out, float* stats) {
  const int lane = threadIdx.x & 31;
  const float4 v = lane < C ? part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
  const bool twice = __any_sync(0xffffffffu, v.w != 0.f);
  float mt = v.x;
#pragma unroll
  for (int o = kDiMaxC / 2; o >= 1; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
  float st = v.x == mt ? v.y : v.y * ex2_approx((v.x - mt) * c.hi);
#pragma unroll
  for (int o = kDiMaxC / 2; o >= 1; o >>= 1) st += __shfl_xor_sync(0xffffffffu, st, o);
  F2 WK = L.WK;
  if (twice) {                          // a token's weight counts once, whatever the list says
    // (float32 weights here, off by half a step each, as the gradient's are; their sum is two-float)
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
    // one of the two maxima is M
    const F2 E = mt == km ? F2{1.f, 0.f} : weight_f2(fminf(mt, km), M, c, tab);
    const bool outside = mt == M;
    const F2 S = f2_add(outside ? F2{st, 0.f} : f2_mul(F2{st, 0.f}, E), km == M ? WK : f2_mul(WK, E));
    const bool good = S.hi > 0.f && S.hi < INFINITY;
    const float nan = __uint_as_float(0x7fffffffu);
    const float invS = good ? __frcp_rn(S.hi) : nan;
    const float invZ = __frcp_rn(L.Z.hi);
    const float pt = L.wt.hi * invZ;
    out.mt = mt == -INFINITY || !good ? 0.f : mt;
    out.A = !good || pt != pt ? nan : !(st > 0.f) ? 0.f : (outside ? invS : E.hi * invS) - (pt == 0.f ? 0.f : pt * __frcp_rn(st));
    out.M = M;
    out.invS = invS;
    out.Es = km == M ? 1.f : E.hi;
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

// The loss of a row (one warp).
__device__ __forceinline__ void dp_loss(const DpList& L, const DpStat& s, F2 inv_t, const float* tab, float* loss) {
  float l = 0.f;
  if (L.live == 2)
    l = L.wgt * distill_loss(L.Z, s.S, F2{s.st, 0.f}, L.E1, L.wt, L.ltail, L.tm, s.mt, L.km, s.M, L.infinite, inv_t, tab);
  if ((threadIdx.x & 31) == 0) *loss = l;
}

// A wait of the cluster ran out: NaN for all of its rows (their order and
// division among the CTAs as in the kernel).
template <typename T, bool GRAD>
__device__ __noinline__ void dp_mark(void* grad, float* loss, float* stats, int V, int SV, int g, int NG, int n, int rank) {
  const float nan = __uint_as_float(0x7fffffffu);
  float x[Tr<T>::VW];
#pragma unroll
  for (int e = 0; e < Tr<T>::VW; ++e) x[e] = nan;
  const uint4 nans = Elem<T>::pack(x);
  for (int t = 0; t < n; ++t) {
    const int r = g + t * NG;
    if (GRAD) {
      const Window<T> gwin(static_cast<T*>(grad), (size_t)r, V);
      const int nv = gwin.vectors(), v0 = min(rank * SV, nv), v1 = min(v0 + SV, nv);
      for (int v = v0 + (int)threadIdx.x; v < v1; v += (int)blockDim.x) gwin.store(v, nans);
    }
    if (rank == 0 && threadIdx.x == 0) loss[r] = nan;
    if (!GRAD && rank == 0 && stats && threadIdx.x < 8) stats[(size_t)r * 8 + threadIdx.x] = nan;
  }
}

// WHOLE: V is a multiple of the vector width, so every row is whole vectors.
template <typename T, bool GRAD, bool WHOLE>
__global__ void __launch_bounds__(kDpMaxThreads, 1) distill_pipe_kernel(const DistillParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DpSmem<T>& sm = *reinterpret_cast<DpSmem<T>*>(smem_raw);
  const int lane = threadIdx.x & 31;
  const int C = p.C, rank = blockIdx.x % C;
  const int g = blockIdx.x / C, NG = gridDim.x / C;
  const int n = (p.R - g + NG - 1) / NG;            // rows of this cluster: g, g + NG, ...
  const int k = p.k;
  const int nl = dp_list_threads(k);                // list threads of a group
  // the roles, by warp: parts, list, statistics, streaming
  const int role = threadIdx.x < 32 ? 0 : threadIdx.x < 32 + 2 * nl ? 1 : threadIdx.x < 64 + 2 * nl ? 2 : 3;
  const F2 c{p.c, p.c_lo};
  const T* student = static_cast<const T*>(p.student);
  // the CTA's vectors of a row [v0, v1)
  auto slice = [&](int nv, int* v0, int* v1) {
    *v0 = min(rank * p.SV, nv);
    *v1 = min(*v0 + p.SV, nv);
  };

  for (int i = threadIdx.x; i < 128; i += blockDim.x) sm.tab[i] = i < 64 ? __ldg(kExp2Hi + i) : __ldg(kExp2Lo + i - 64);
  if (threadIdx.x == 0) {
    sm.gave_up = 0u;
    for (int i = 0; i < 4; ++i) {
      mb_init(&sm.summed[i], kDpStWarps);
      mb_init(&sm.known[i], 1);
      mb_init(&sm.written[i], kDpStWarps);
      mb_init(&sm.listed[i], 1);
    }
    for (int i = 0; i < kDpParts; ++i) mb_init(&sm.parts[i], C);
    for (int i = 0; i < kDpLists; ++i) mb_init(&sm.done[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();                                   // every CTA of the cluster runs, its barriers stand

  if (role == 3) {
    // ================================================================ streaming
    const int tid = threadIdx.x - 64 - 2 * nl, warp = tid >> 5;
    int v0 = 0, v1 = 0;
    if (WHOLE) slice(p.V / VW, &v0, &v1);
    int mine = (v1 - v0 - tid + kDpSt - 1) / kDpSt;  // vectors of this thread in a row (WHOLE)
    const size_t nvr = (size_t)(p.V / VW);           // vectors from row to row (WHOLE)
    float w_next = p.weight ? __ldg(p.weight + g) : 1.f;
    auto issue = [&](int i) {                       // row i of the cluster into its stage
      if (i < n) {
        const int r = g + i * NG;
        uint4* st = &sm.ring[i % kDpStages][tid];
        if (w_next != 0.f) {
          if (WHOLE) {
            const uint4* src = reinterpret_cast<const uint4*>(student) + (size_t)r * nvr + v0 + tid;
            const unsigned sa = (unsigned)__cvta_generic_to_shared(st);
#pragma unroll
            for (int u = 0; u < kDpU; ++u)
              if (u < mine)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa + u * kDpSt * 16), "l"(src + u * kDpSt) : "memory");
          } else {
            const Window<T, const T> win(student, (size_t)r, p.V);
            int w0, w1;
            slice(win.vectors(), &w0, &w1);
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
              const int v = w0 + u * kDpSt + tid;
              if (v < w1) {
                if (win.whole(v)) {
                  const unsigned sa = (unsigned)__cvta_generic_to_shared(st + u * kDpSt);
                  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa), "l"(win.base + (size_t)v * VW) : "memory");
                } else {
                  st[u * kDpSt] = win.load(v);
                }
              }
            }
          }
        }
        if (p.weight && i + 1 < n) w_next = __ldg(p.weight + r + NG);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (WHOLE) {                                    // a thread's last slot stays -inf where the slice ends before it
      for (int s = 0; s < kDpStages; ++s)
        for (int u = mine; u < kDpU && u * kDpSt + tid < kDpSlice; ++u)
          sm.ring[s][u * kDpSt + tid] = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
    }
    issue(0);
    issue(1);
    if (!GRAD) issue(2);

#pragma unroll 1
    for (int t = 0; t <= n; ++t) {
      if (t < n) {
        // ---- row t without its listed tokens
        asm volatile("cp.async.wait_group %0;" ::"n"(GRAD ? 1 : 2) : "memory");
        if (!mb_wait(&sm.listed[t & 3], t >> 2)) { dp_give_up(&sm.gave_up, C); break; }
        if (sm.list[t % kDpLists].live != 0) {
          const uint4* st = &sm.ring[t % kDpStages][tid];
          int m_t = mine;
          if (!WHOLE) {
            const Window<T, const T> win(student, (size_t)(g + t * NG), p.V);
            int w0, w1;
            slice(win.vectors(), &w0, &w1);
            m_t = (w1 - w0 - tid + kDpSt - 1) / kDpSt;
          }
          uint4 x[kDpU];
#pragma unroll
          for (int u = 0; u < kDpU; ++u) {
            if (WHOLE && (u + 1) * kDpSt <= kDpSlice) {
              x[u] = st[u * kDpSt];                 // -inf where this thread has no vector
            } else {
              x[u] = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
              if (u < m_t) x[u] = st[u * kDpSt];
            }
          }
          const uint2 dirty = sm.dirty[t % 3][warp];
          if (dirty.x | dirty.y) {
            const unsigned char* bits = reinterpret_cast<const unsigned char*>(sm.bits[t % 3]);
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
              if (((u < 4 ? dirty.x : dirty.y) >> (8 * (u & 3))) & 0xffu) {
                const int lv = u * kDpSt + tid;
                const uint32_t b = lv >= kDpSlice ? 0u : VW == 8 ? bits[lv] : (bits[lv >> 1] >> ((lv & 1) * 4)) & 15u;
#pragma unroll
                for (int e = 0; e < VW; ++e)
                  if ((b >> e) & 1u) TR::put(x[u], e, Elem<T>::kNegInf);
              }
            }
          }
          float m = -INFINITY;
#pragma unroll
          for (int u = 0; u < kDpU; ++u) m = fmaxf(m, TR::template vmax<false>(x[u]));
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float ref = m == -INFINITY ? 0.f : m, rho = ref * p.c;
          float s, fix = 1.f;
          if (fabsf(rho) < kNear) {
            fix = ex2_approx(-fmaf(ref, p.c, -rho));
            const Pair cc = pair_of(p.c, p.c), rr = pair_of(-rho, -rho);
            Pair a0 = pair_of(0.f, 0.f), a1 = a0;
#pragma unroll
            for (int u = 0; u < kDpU; ++u)
#pragma unroll
              for (int e = 0; e < VW; e += 4) {
                a0 = pair_add(a0, pair_terms<T>(x[u], e, cc, rr));
                a1 = pair_add(a1, pair_terms<T>(x[u], e + 2, cc, rr));
              }
            float s0, s1;
            unpair(pair_add(a0, a1), s0, s1);
            s = s0 + s1;
          } else {
            s = 0.f;
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
#pragma unroll 1
              for (int e = 0; e < VW; ++e) s += ex2_approx((TR::get(x[u], e) - ref) * p.c);
            }
          }
          // chains of 12 terms, then a tree
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) sm.wpart[t & 3][warp] = make_float2(m, s * fix);
        }
        mb_arrive(&sm.summed[t & 3]);
        if (!GRAD) issue(t + 3);
      }
      if (!GRAD) {
        // the ring of the warps' parts holds four rows
        if (t >= 3 && !mb_wait(&sm.known[(t - 3) & 3], (t - 3) >> 2)) { dp_give_up(&sm.gave_up, C); break; }
      } else if (t >= 1) {
        // ---- row t - 1's gradient
        const int i = t - 1;
        if (!mb_wait(&sm.known[i & 3], i >> 2)) { dp_give_up(&sm.gave_up, C); break; }
        {
          const int r = g + i * NG;
          const DpList& L = sm.list[i % kDpLists];
          const uint4* st = &sm.ring[i % kDpStages][tid];
          const bool row = L.live == 2;
          const float mt = sm.stat[i % kDpLists].mt, rho = mt * p.c;
          float gA = L.sc * sm.stat[i % kDpLists].A;
          const Window<T> gwin(static_cast<T*>(p.grad), (size_t)r, p.V);
          int w0 = v0, w1 = v1;
          if (!WHOLE) slice(gwin.vectors(), &w0, &w1);
          if (!row) {
            zero_slice_of(gwin, w0, w1, tid, kDpSt);
          } else if (fabsf(rho) < kNear) {
            gA *= ex2_approx(-fmaf(mt, p.c, -rho));
            uint4* dst = reinterpret_cast<uint4*>(p.grad) + (size_t)r * nvr + v0 + tid;
            const Pair cc = pair_of(p.c, p.c), rr = pair_of(-rho, -rho), gg = pair_of(gA, gA);
#pragma unroll
            for (int u = 0; u < kDpU; ++u) {
              if (WHOLE ? u < mine : w0 + u * kDpSt + tid < w1) {
                const uint4 x = st[u * kDpSt];
                float gr[VW];
#pragma unroll
                for (int e = 0; e < VW; e += 2)
                  unpair(pair_mul(gg, pair_terms<T>(x, e, cc, rr)), gr[e], gr[e + 1]);
                if (WHOLE) __stcs(dst + u * kDpSt, Elem<T>::pack(gr));
                else gwin.store(w0 + u * kDpSt + tid, Elem<T>::pack(gr));
              }
            }
          } else {
#pragma unroll 1
            for (int u = 0; u < kDpU; ++u) {
              const int v = w0 + u * kDpSt + tid;
              if (v < w1) {
                const uint4 x = st[u * kDpSt];
                float gr[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) gr[e] = gA * ex2_approx((TR::get(x, e) - mt) * p.c);
                gwin.store(v, Elem<T>::pack(gr));
              }
            }
          }
        }
        mb_arrive(&sm.written[i & 3]);
      }
      if (GRAD) issue(t + 2);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (role == 0) {
    // ================================================================ parts
    // (float32, a tree over 22 warps: the part outside the list, see dp_statistics)
    const int last = rank == 0 ? (int)min((unsigned)n, (unsigned)p.stop) : n;   // n for -1
#pragma unroll 1
    for (int t = 0; t < last; ++t) {
      // (a summed row's list stands too)
      if (!mb_wait(&sm.summed[t & 3], t >> 2)) { dp_give_up(&sm.gave_up, C); break; }
      const DpList& L = sm.list[t % kDpLists];
      if (L.live != 0) {
        const float2 v = lane < kDpStWarps ? sm.wpart[t & 3][lane] : make_float2(-INFINITY, 0.f);
        float m = v.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = v.x == m ? v.y : v.y * ex2_approx((v.x - m) * p.c);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane < C) push_f4(&sm.part[t % kDpParts][rank], lane, make_float4(m, s, 0.f, L.twice ? 1.f : 0.f));
      }
      if (lane < C) mb_arrive_remote(&sm.parts[t % kDpParts], lane);
      __syncwarp();
    }
    if (last < n) dp_give_up(&sm.gave_up, C);
  } else if (role == 2) {
    // ================================================================ statistics
    const F2 inv_t = f2_from(p.inv_t);
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      if (!mb_wait<true>(&sm.parts[t % kDpParts], t / kDpParts)) { dp_give_up(&sm.gave_up, C); break; }
      const DpList& L = sm.list[t % kDpLists];
      DpStat& s = sm.stat[t % kDpLists];
      dp_statistics(sm.part[t % kDpParts], C, L, k, c, sm.tab, s,
                    !GRAD && rank == 0 && p.stats ? p.stats + (size_t)(g + t * NG) * 8 : nullptr);
      mb_arrive(&sm.known[t & 3]);
      if (t % C == rank) dp_loss(L, s, inv_t, sm.tab, p.loss + g + t * NG);
      mb_arrive(&sm.done[t % kDpLists]);
    }
  } else {
    // ================================================================ list
    const int group = threadIdx.x - 32 >= nl;       // rows of this parity
    const int lt = threadIdx.x - 32 - group * nl, lw = lt >> 5;   // lt < nl
    const F2 inv_t = f2_from(p.inv_t);
    const F2 l2e{kLog2eHi, kLog2eLo};
    // Up to kDpLiE tokens a thread, nl apart.  What is loaded stays as it
    // comes until the iteration that needs it: the indices of the group's next
    // row, the student's values of this one.
    int id1[kDpLiE], id2[kDpLiE];
    float lp1[kDpLiE], lp2[kDpLiE];
    uint32_t s1[kDpLiE];
    float wg1 = 1.f, tl1 = -INFINITY;               // the row's weight and tail
    bool ok = true;
    auto load_list = [&](int i, int* id, float* lp) {
#pragma unroll
      for (int q = 0; q < kDpLiE; ++q) {
        id[q] = -1;
        lp[q] = -INFINITY;
        if (i < n && lt + q * nl < k) {
          const size_t at = ((size_t)g + (size_t)i * NG) * k + lt + q * nl;
          id[q] = __ldg(p.indices + at);
          lp[q] = __ldg(p.logprobs + at);
        }
      }
    };
    auto load_student = [&](int i, const int* id) {
#pragma unroll
      for (int q = 0; q < kDpLiE; ++q)
        if ((unsigned)id[q] < (unsigned)p.V) s1[q] = Elem<T>::raw(student + ((size_t)g + (size_t)i * NG) * p.V + id[q]);
    };
    auto load_row = [&](int i) {
      if (i < n) {
        const int r = g + i * NG;
        if (p.weight) wg1 = __ldg(p.weight + r);
        if (p.tail) tl1 = __ldg(p.tail + r);
      }
    };
    load_list(group, id1, lp1);
    load_student(group, id1);
    load_list(group + 2, id2, lp2);
    load_row(group);

#pragma unroll 1
    for (int j = group; j <= (GRAD ? n + 1 : n - 1); j += 2) {
      if (j < n) {
        // ---- the list of row j
        // (the bitmap was row j - 3's, the list row j - kDpLists's)
        if (j >= 3) ok = ok && mb_wait(&sm.summed[(j - 3) & 3], (j - 3) >> 2);
        if (j >= kDpLists) ok = ok && mb_wait(&sm.done[j % kDpLists], j / kDpLists - 1);
        DpList& L = sm.list[j % kDpLists];
        // a NaN makes the maximum +inf, and the row NaN
        float tm = -INFINITY, km = -INFINITY;
#pragma unroll
        for (int q = 0; q < kDpLiE; ++q) {
          const bool on = (unsigned)id1[q] < (unsigned)p.V;
          const float lp = on ? lp1[q] : -INFINITY, s = on ? Elem<T>::of_raw(s1[q]) : -INFINITY;
          tm = fmaxf(tm, lp != lp ? INFINITY : lp);
          km = fmaxf(km, s);
          L.sid[lt + q * nl] = on ? id1[q] : -1;    // this thread's own places, until the weights replace the values
          L.sw[lt + q * nl] = lp;
          L.sq[lt + q * nl] = s;
          id1[q] = id2[q];
          lp1[q] = lp2[q];
        }
        const float wgt = wg1, ltail = tl1;
        load_student(j + 2, id1);
        load_list(j + 4, id2, lp2);
        load_row(j + 2);
        uint32_t* bits = sm.bits[j % 3];
        unsigned char* dirty = reinterpret_cast<unsigned char*>(sm.dirty[j % 3]);
        for (int w = lt; w < kDpSlice * VW / 128; w += nl) reinterpret_cast<uint4*>(bits)[w] = make_uint4(0u, 0u, 0u, 0u);
        for (int w = lt; w < kDpStWarps * 2; w += nl) reinterpret_cast<uint32_t*>(dirty)[w] = 0u;
        if (lt == 0) L.infinite = L.twice = 0;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, m));
          km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, m));
        }
        if (lane == 0) sm.lmax[group][lw] = make_float2(tm, km);
        if (!list_meet(group, nl, ok)) break;              // one gave up: all do, here
        tm = ltail != ltail ? INFINITY : ltail;
        for (int w = 0; w < nl / 32; ++w) {
          tm = fmaxf(tm, sm.lmax[group][w].x);
          km = fmaxf(km, sm.lmax[group][w].y);
        }
        F2 w{0.f, 0.f}, ws{0.f, 0.f}, e1{0.f, 0.f};
        const Window<T, const T> win(student, (size_t)(g + j * NG), p.V);
        int v0, v1;
        slice(win.vectors(), &v0, &v1);
#pragma unroll 1
        for (int q = 0; q * nl < k; ++q) {
          const int at = lt + q * nl;
          const int id_q = L.sid[at];
          const float lp_q = L.sw[at], s_q = L.sq[at];
          F2 w_q{0.f, 0.f}, ws_q{0.f, 0.f};
          if (id_q >= 0) {
            const float kr = km == -INFINITY ? 0.f : km;
            w_q = weight_f2(lp_q, tm, l2e, sm.tab);
            ws_q = weight_f2(s_q, km, c, sm.tab);
            if (w_q.hi != 0.f) {
              // w (ln p_j - ln q_j), up to the row's constants
              if ((s_q - kr) * inv_t.hi < -kDiFar) L.infinite = 1;
              else e1 = f2_add(e1, distill_term(w_q, lp_q, tm, s_q, kr, inv_t));
            }
            const int o = id_q + win.a0 - v0 * VW;
            if (o >= 0 && o < (v1 - v0) * VW) {
              const uint32_t bit = 1u << (o & 31);
              if (atomicOr(&bits[o >> 5], bit) & bit) L.twice = 1;
              const int lv = o / VW;                // vector lv = u * kDpSt + thread
              dirty[(lv % kDpSt) / 32 * 8 + lv / kDpSt] = 1;
            }
            w = f2_add(w, w_q);
            ws = f2_add(ws, ws_q);
          }
          L.sw[at] = w_q.hi;
          L.sq[at] = ws_q.hi;
        }
        w = warp_sum_f2(w);
        ws = warp_sum_f2(ws);
        e1 = warp_sum_f2(e1);
        if (lane == 0) {
          sm.lsum[group][lw][0] = w;
          sm.lsum[group][lw][1] = ws;
          sm.lsum[group][lw][2] = e1;
        }
        list_meet(group, nl, true);
        if (lt < 3) {                               // one of the three sums each
          F2 a = sm.lsum[group][0][lt];
          for (int q = 1; q < nl / 32; ++q) a = f2_add(a, sm.lsum[group][q][lt]);
          if (lt == 0) {
            const F2 wt = p.tail ? weight_f2(ltail, tm, l2e, sm.tab) : F2{0.f, 0.f};
            L.Z = f2_add(a, wt);
            L.wt = wt;
            L.tm = tm;
            L.km = km;
            L.ltail = ltail;
            L.wgt = wgt;
            L.sc = wgt * inv_t.hi + wgt * inv_t.lo;
            L.live = wgt == 0.f ? 0 : tm > -INFINITY ? 2 : 1;
          } else if (lt == 1) {
            L.WK = a;
          } else {
            L.E1 = a;
          }
        }
        if (lw == 0) mb_arrive(&sm.listed[j & 3]);  // (the other list warps' part lies before the barrier above)
      }
      if (GRAD && j >= 2) {
        // ---- the listed tokens of row j - 2, on top of its dense gradient
        const int i = j - 2;
        ok &= mb_wait(&sm.written[i & 3], i >> 2);
        const DpList& L = sm.list[i % kDpLists];
        if (ok && L.live == 2) {
          const DpStat& s = sm.stat[i % kDpLists];
          const Window<T> gwin(static_cast<T*>(p.grad), (size_t)(g + i * NG), p.V);
          int v0, v1;
          slice(gwin.vectors(), &v0, &v1);
          for (int e = lt; e < k; e += nl) {
            const int id = L.sid[e];
            const int o = id + gwin.a0;
            if (id < 0 || o < v0 * VW || o >= v1 * VW) continue;
            float w = L.sw[e];
            if (s.twice) {
              w = 0.f;
              for (int q = 0; q < k; ++q)
                if (L.sid[q] == id) w += L.sw[q];
            }
            Elem<T>::store(gwin.base + o, L.sc * (L.sq[e] * (s.Es * s.invS) - w * __frcp_rn(L.Z.hi)));
          }
        }
      }
    }
    if (!ok) dp_give_up(&sm.gave_up, C);            // (a group that leaves together has one that knows why)
  }
  cluster_arrive();
  cluster_wait();                                   // nobody leaves while its shared memory may be written
  if (sm.gave_up != 0u) dp_mark<T, GRAD>(p.grad, p.loss, p.stats, p.V, p.SV, g, NG, n, rank);
}

}  // namespace rows
}  // namespace sv
