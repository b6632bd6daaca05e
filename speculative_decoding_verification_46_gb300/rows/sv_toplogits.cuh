// The record of a teacher's row: its k best log-probabilities and the log of
// the mass outside them.
//
// A row is cut into H slices of at most 256 * U vectors, one CTA each, held
// in registers from one read of HBM.  A CTA finds a lower bound tau of its
// slice's k-th largest value (the k-th largest of some of its group maxima),
// sets the few vectors that hold an element >= tau aside in shared memory,
// ranks their elements >= tau exactly by (value descending, index ascending),
// and sums 2^((x - m) c) over everything it did not list, m the
// largest of those.  So the mass outside is a sum of its own terms and not a
// difference, and stays accurate however small it is.  The slices' lists and
// sums go to the workspace; the last CTA of a row to arrive (an atomic
// ticket, nobody waits) selects the k best of the H lists by a radix select
// over the 64-bit keys (value, ~index), ranks them, and adds what the lists
// hold beyond them to the mass outside.
//
// top_row_kernel, further down, is the form for many rows (one CTA a row, no
// hand-over).  Both read a row once.  Few rows are bound by the selection's
// chain of barriers (one row of 152064 bf16, k = 64: 18 us; 20 rows of 1024
// float32, k = 8: 9 us), many by instruction issue: 2304 rows of 152064 bf16, k
// = 64: 220 us, 3.2 TB/s (0.47 of the measured copy; in slices 469 us).
#pragma once

#include "sv_rows.cuh"

namespace sv {
namespace rows {

constexpr int kTlThreads = 256;
constexpr int kTlWarps = kTlThreads / 32;
constexpr int kTlCap = 2048;      // candidates of a slice; more are selected exactly
constexpr int kTlVecs = 1280;     // vectors of a slice set aside
constexpr int kTlStage = 4096;    // list entries of a row staged in shared memory

struct TopParams {
  int R, V, k;
  int H, SV;                      // slices per row, vectors per slice
  int KP;                         // group maxima per thread that tau is chosen from
  float c, c_lo;                  // log2(e) / temperature
  F2 inv_t;                       // 1 / temperature
  const void* logits;
  int32_t* indices;
  float* logprobs;
  float* tail;
  int* ticket;                    // [R]
  float4* part;                   // [R][H] (largest, sum high, sum low, bad)
  unsigned long long* lists;      // [R][H][k] sorted keys; 0 = none
};

struct PickSmem {
  int hist[256];
  int digit, rank, count;
};

struct TopSmem {
  union {
    struct {                            // a slice's selection
      unsigned long long cand[kTlCap];
      uint4 vec[kTlVecs];               // the vectors that hold an element >= tau
      int vid[kTlVecs];                 // and their numbers in the window
    };
    struct {                            // a row's selection
      unsigned long long buf[kTlStage];
      unsigned long long sel[kMaxK];
    };
  };
  PickSmem pick;
  float tab[128];
  float fred[kTlWarps];
  F2 f2red[kTlWarps];
  int ired[kTlWarps];
  unsigned long long u64red[kTlWarps];
  F2 lns;
  unsigned long long kth;
  unsigned lmax;                        // okey of the largest candidate beyond the k best
  int count, nvec, flag;
};

// One digit of a radix select: with hist[] complete, the digit (0..255, from
// the top) that holds the rank-th largest, the rank inside it and its count.
// digit -1: fewer than rank keys.  Every thread returns the same values.
__device__ __forceinline__ int pick_digit(PickSmem& sm, int rank, int* rank_in, int* count) {
  __syncthreads();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int c[8], lsum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = sm.hist[255 - 8 * lane - e];
      lsum += c[e];
    }
    int inc = lsum;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    const int excl = inc - lsum;
    const bool mine = excl < rank && inc >= rank;
    if (mine) {
      int run = excl, dg = -1, cc = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (dg < 0 && run + c[e] >= rank) {
          dg = 255 - 8 * lane - e;
          cc = c[e];
        }
        if (dg < 0) run += c[e];
      }
      sm.digit = dg;
      sm.rank = rank - run;
      sm.count = cc;
    }
    if (__ballot_sync(0xffffffffu, mine) == 0u && lane == 0) sm.digit = -1;
  }
  __syncthreads();
  *rank_in = sm.rank;
  *count = sm.count;
  return sm.digit;
}

// The largest K, bits below LOW zero, such that at least k of the block's
// keys (U per thread, 0 = none) are >= K; 0 if there are fewer than k.
template <int LOW, int U>
__device__ __forceinline__ uint32_t kth_key(const uint32_t (&key)[U], int k, PickSmem& sm) {
  uint32_t prefix = 0u;
  int rank = k;
#pragma unroll
  for (int hi = 31; hi >= LOW; hi -= 8) {
    const int lo = hi - 7 > LOW ? hi - 7 : LOW;
    const uint32_t upper = hi == 31 ? 0u : ~((1u << (hi + 1)) - 1u);
    sm.hist[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (key[u] != 0u && (key[u] & upper) == prefix)
        atomicAdd(&sm.hist[(key[u] >> lo) & ((1u << (hi - lo + 1)) - 1u)], 1);
    int in, cnt;
    const int dg = pick_digit(sm, rank, &in, &cnt);
    if (dg < 0) return 0u;
    prefix |= (uint32_t)dg << lo;
    rank = in;
    if (cnt == rank) break;   // everything in the digit is wanted: the rest of the bits may stay 0
  }
  return prefix;
}

// The k-th largest of more than k distinct keys (value, ~index) that
// each(f) passes to f, every thread its own: a radix select from the top, up
// to the digit whose keys are all wanted (then the bits below stay 0).
template <typename T, typename Each>
__device__ __forceinline__ unsigned long long select_kth64(int k, int V, PickSmem& sm, Each each) {
  constexpr int LOW = Tr<T>::KEY_LOW_BIT;
  const int nidx = V > 1 ? 32 - __clz(V - 1) : 1;          // index bits that differ
  unsigned long long prefix = 0ull, known = 0ull;
  int rank = k, hi = 63;
#pragma unroll 1
  while (true) {
    const int lo = max(hi - 7, hi >= 32 ? 32 + LOW : 0);
    const unsigned dmask = (1u << (hi - lo + 1)) - 1u;
    __syncthreads();
    sm.hist[threadIdx.x] = 0;
    __syncthreads();
    each([&](unsigned long long key) {
      if ((key & known) == prefix) atomicAdd(&sm.hist[(unsigned)(key >> lo) & dmask], 1);
    });
    int in, cnt;
    const int dg = pick_digit(sm, rank, &in, &cnt);
    prefix |= (unsigned long long)(unsigned)dg << lo;
    known |= (unsigned long long)dmask << lo;
    rank = in;
    if (cnt == rank || lo == 0) return prefix;
    hi = lo - 1;
    if (lo == 32 + LOW) {
      // value bits below LOW copy the sign (all ones in a negative's key);
      // index bits above those that differ are ones (the index is complemented)
      const unsigned long long skip = ((1ull << (32 + LOW)) - 1ull) & ~((1ull << 32) - 1ull);
      if (!(prefix >> 63)) prefix |= skip;
      const unsigned long long ones = nidx >= 32 ? 0ull : ((1ull << 32) - 1ull) & ~((1ull << nidx) - 1ull);
      prefix |= ones;
      known |= skip | ones;
      hi = nidx - 1;
    }
  }
}

// (x - m) / temperature, x <= m; one float where it leaves the range that
// two-float products have.
__device__ __forceinline__ F2 top_scaled(float x, float m, F2 inv_t) {
  const float f = (x - m) * inv_t.hi;
  return f > -1.0e30f ? f2_mul(two_diff(x, m), inv_t) : F2{f, 0.f};
}

// The record of a row from its k best (keys sel[0 .. kk), any order; sorted
// here) and the rest's mass st relative to mt (0: none).  Logarithms and
// log-probabilities are formed in two-float numbers, some 40 bits, and rounded
// once: the float32 results need no more, and float64 arithmetic, at a small
// part of float32's rate, took 6 us of 228 (2304 rows of 152064, k 64).
template <int NW>
__device__ __forceinline__ void top_write(const TopParams& p, int r, unsigned long long* sel, int kk, float mt, F2 st,
                                          const float* tab, F2* f2red, F2* s_lns) {
  constexpr int NT = NW * 32, E = kMaxK / NT;
  const int tid = threadIdx.x, k = p.k;
  const F2 c{p.c, p.c_lo};
  unsigned long long mine[E];
  int rank[E];
#pragma unroll
  for (int q = 0; q < E; ++q) {
    const int e = tid + q * NT;
    rank[q] = -1;
    if (e < kk) {
      mine[q] = sel[e];
      rank[q] = 0;
      for (int j = 0; j < kk; ++j) rank[q] += sel[j] > mine[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < E; ++q)
    if (rank[q] >= 0) sel[rank[q]] = mine[q];
  __syncthreads();
  const float M = comp_val(sel[0]);
  F2 sk{0.f, 0.f};
  for (int j = tid; j < kk; j += NT) sk = f2_add(sk, weight_f2(comp_val(sel[j]), M, c, tab));
  sk = block_sum_f2_n<NW>(sk, f2red);
  // ln of the whole row's sum relative to M, and of the rest's relative to mt
  if (tid < 32) {
    const bool some = st.hi > 0.f;
    const F2 all = some ? f2_add(sk, f2_mul(st, weight_f2(mt, M, c, tab))) : sk;
    const F2 lg = f2_log(tid == 1 && some ? st : all, tab);
    const F2 lt{__shfl_sync(0xffffffffu, lg.hi, 1), __shfl_sync(0xffffffffu, lg.lo, 1)};
    if (tid == 0) {
      *s_lns = lg;
      const F2 d = top_scaled(mt, M, p.inv_t);
      p.tail[r] = some ? (d.hi > -1.0e30f ? f2_add(d, f2_add(lt, f2_neg(lg))).hi : d.hi) : -INFINITY;
    }
  }
  __syncthreads();
  const F2 lns = *s_lns;
  for (int e = tid; e < k; e += NT) {
    const bool on = e < kk;
    float lp = -INFINITY;
    if (on) {
      const F2 d = top_scaled(comp_val(sel[e]), M, p.inv_t);
      lp = d.hi > -1.0e30f ? f2_add(d, f2_neg(lns)).hi : d.hi;
    }
    p.indices[(size_t)r * k + e] = on ? comp_idx(sel[e]) : -1;
    p.logprobs[(size_t)r * k + e] = lp;
  }
}

// The record of a row that defines no distribution.
__device__ __forceinline__ void top_write_bad(const TopParams& p, int r) {
  const float nan = __uint_as_float(0x7fffffffu);
  if (threadIdx.x == 0) p.tail[r] = nan;
  for (int j = threadIdx.x; j < p.k; j += blockDim.x) {
    p.indices[(size_t)r * p.k + j] = -1;
    p.logprobs[(size_t)r * p.k + j] = nan;
  }
}

// The row's lists are in: select, rank and write the record.
template <typename T>
__device__ void top_finish_row(const TopParams& p, int r, TopSmem& sm) {
  const int tid = threadIdx.x, k = p.k;
  const int slots = p.H * k;
  unsigned long long* lists = p.lists + (size_t)r * slots;
  float4* part = p.part + (size_t)r * p.H;
  const bool staged = slots <= kTlStage;
  int have = 0, bad = 0;
  for (int e = tid; e < slots; e += kTlThreads) {
    const unsigned long long key = __ldcg(lists + e);
    if (staged) sm.buf[e] = key;
    have += key != 0ull;
  }
  float mt = -INFINITY;
  for (int h = tid; h < p.H; h += kTlThreads) {
    const float4 v = __ldcg(part + h);
    mt = fmaxf(mt, v.x);
    bad |= v.w != 0.f;
  }
  have = block_sum_int_w<kTlWarps>(have, sm.ired);
  bad = __syncthreads_or(bad);
  const bool ok = have > 0 && !bad;
  const int kk = min(k, have);
  if (ok) {
    // ---- K64: exactly kk keys are >= it
    const unsigned long long K64 = have > k ? select_kth64<T>(k, p.V, sm.pick, [&](auto f) {
      for (int e = tid; e < slots; e += kTlThreads) {
        const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
        if (key != 0ull) f(key);
      }
    }) : 1ull;
    // ---- the k best, in any order, then ranked
    if (tid == 0) sm.count = 0;
    __syncthreads();
    float lm = -INFINITY;
    for (int e = tid; e < slots; e += kTlThreads) {
      const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
      if (key >= K64) {
        const int pos = atomicAdd(&sm.count, 1);
        if (pos < kMaxK) sm.sel[pos] = key;
      } else if (key != 0ull) {
        lm = fmaxf(lm, comp_val(key));
      }
    }
    mt = block_max_n<kTlWarps>(fmaxf(mt, lm), sm.fred);
    const F2 c{p.c, p.c_lo};
    F2 st{0.f, 0.f};
    for (int h = tid; h < p.H; h += kTlThreads) {
      const float4 v = __ldcg(part + h);
      if (v.x > -INFINITY) st = f2_add(st, f2_mul(F2{v.y, v.z}, weight_f2(v.x, mt, c, sm.tab)));
    }
    for (int e = tid; e < slots; e += kTlThreads) {
      const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
      if (key < K64 && key != 0ull) st = f2_add(st, weight_f2(comp_val(key), mt, c, sm.tab));
    }
    st = block_sum_f2_n<kTlWarps>(st, sm.f2red);
    top_write<kTlWarps>(p, r, sm.sel, kk, mt, st, sm.tab, sm.f2red, &sm.lns);
  } else {
    top_write_bad(p, r);
  }
  // leave the workspace zero-filled
  __syncthreads();
  for (int e = tid; e < slots; e += kTlThreads)
    if (!staged || sm.buf[e] != 0ull) lists[e] = 0ull;
  for (int h = tid; h < p.H; h += kTlThreads) part[h] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Too many elements reach the bound (ties, or fewer groups than k): the exact
// k-th largest value of the slice by bisection over its key, of its ties the
// first ones.  Fills cand[0 .. k) and returns the largest and the sum of the
// rest.  Rare, so it reads the slice again (L2) in small loops instead of
// keeping a second unrolled copy of the work in the instruction cache.
template <typename T>
__device__ __noinline__ F2 top_slice_exact(const Window<T, const T>& win, int v0, int v1, int k, float c, TopSmem& sm,
                                           float* rest_max) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  const int tid = threadIdx.x;
  auto each = [&](auto f) {
    for (int v = v0 + tid; v < v1; v += kTlThreads) {
      const uint4 x = win.load(v);
#pragma unroll
      for (int t = 0; t < VW; ++t) f(TR::get(x, t), v * VW - win.a0 + t);
    }
  };
  uint32_t KV = 0u;
#pragma unroll 1
  for (int bit = 31; bit >= TR::KEY_LOW_BIT; --bit) {
    const uint32_t Kt = KV | (1u << bit);
    int mine = 0;
    each([&](float x, int) { mine += x > -INFINITY && okey(x) >= Kt; });
    if (block_sum_int_w<kTlWarps>(mine, sm.ired) >= k) KV = Kt;
  }
  // the value itself: bits below KEY_LOW_BIT are ones in a negative's key
  const float tau = key_to_float((KV & 0x80000000u) ? KV : KV | ((1u << TR::KEY_LOW_BIT) - 1u));
  int above = 0;
  each([&](float x, int) { above += x > tau; });
  const int need = k - block_sum_int_w<kTlWarps>(above, sm.ired);
  int lo = v0 * VW - win.a0, hi = v1 * VW - win.a0 - 1;   // the smallest index with `need` ties up to it
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int mine = 0;
    each([&](float x, int i) { mine += x == tau && i <= mid; });
    if (block_sum_int_w<kTlWarps>(mine, sm.ired) >= need) hi = mid; else lo = mid + 1;
  }
  __syncthreads();
  if (tid == 0) sm.count = 0;
  __syncthreads();
  float mr = -INFINITY;
  each([&](float x, int i) {
    if (x > tau || (x == tau && i <= lo)) {
      const int pos = atomicAdd(&sm.count, 1);
      if (pos < kTlCap) sm.cand[pos] = comp_key(x, i);
    } else {
      mr = fmaxf(mr, x);
    }
  });
  mr = block_max_n<kTlWarps>(mr, sm.fred);
  *rest_max = mr;
  F2 s{0.f, 0.f};
  if (mr > -INFINITY) {
    each([&](float x, int i) {
      if (!(x > tau || (x == tau && i <= lo))) s = f2_add(s, F2{ex2_approx((x - mr) * c), 0.f});
    });
  }
  return s;
}

template <typename T, int U>
__global__ void __launch_bounds__(kTlThreads, 4) top_slice_kernel(const TopParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  __shared__ __align__(16) TopSmem sm;
  const int tid = threadIdx.x, k = p.k;
  const int r = blockIdx.x / p.H;
  const int h = blockIdx.x - r * p.H;
  const Window<T, const T> win(static_cast<const T*>(p.logits), (size_t)r, p.V);
  const int v0 = h * p.SV, v1 = min(v0 + p.SV, win.vectors());

  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int v = v0 + u * kTlThreads + tid;
    x[u] = v < v1 ? win.load(v) : make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
  }
  load_exp2_table(sm.tab);
  if (tid == 0) {
    sm.count = sm.nvec = 0;
    sm.lmax = 0u;
    sm.kth = 0ull;
  }
  // ---- tau from the maxima of KP groups of vectors per thread
  float vm[U];
  int bad = 0;
  uint32_t key[U];
  {
    const int gs = U / min(U, p.KP);
    float g = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      vm[u] = TR::template vmax<true>(x[u]);
      bad |= !(vm[u] < INFINITY);                      // NaN or +inf
      g = (u & (gs - 1)) == 0 ? vm[u] : fmaxf(g, vm[u]);
      key[u] = (u & (gs - 1)) == gs - 1 && g > -INFINITY ? okey(g) : 0u;
    }
  }
  bad = __syncthreads_or(bad);
  F2 s{0.f, 0.f};
  float mr = -INFINITY;
  if (!bad) {
    const uint32_t K = kth_key<TR::KEY_LOW_BIT, U>(key, k, sm.pick);
    const float tau = K == 0u ? -INFINITY : key_to_float(K);
    // ---- the few vectors that reach tau go to shared memory, their elements
    // >= tau out of the registers
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (vm[u] >= tau && vm[u] > -INFINITY) {
        const int pos = atomicAdd(&sm.nvec, 1);
        if (pos < kTlVecs) {
          sm.vec[pos] = x[u];
          sm.vid[pos] = v0 + u * kTlThreads + tid;
        }
        clear_ge<T>(x[u], tau);
        vm[u] = TR::template vmax<false>(x[u]);
      }
      mr = fmaxf(mr, vm[u]);
    }
    __syncthreads();
    const int NE = sm.nvec * VW;
    bool exact = NE > kTlVecs * VW;
    // ---- their elements, one thread each: the candidates
    if (!exact) {
      for (int e = tid; e < NE; e += kTlThreads) {
        const float xv = Elem<T>::load(reinterpret_cast<const T*>(sm.vec) + e);
        if (xv >= tau && xv > -INFINITY) {
          const int pos = atomicAdd(&sm.count, 1);
          if (pos < kTlCap) sm.cand[pos] = comp_key(xv, sm.vid[e / VW] * VW - win.a0 + e % VW);
        }
      }
      __syncthreads();
      exact = sm.count > kTlCap;
    }
    if (exact) {
      __syncthreads();                                 // everyone has read the counts
      s = top_slice_exact(win, v0, v1, k, p.c, sm, &mr);
      __syncthreads();
    }
    const int N = min(sm.count, kTlCap);
    // ---- exact ranks: the k best to the row's list, the others to the rest
    unsigned long long* list = p.lists + ((size_t)r * p.H + h) * k;
    for (int e = tid; e < N; e += kTlThreads) {
      const unsigned long long me = sm.cand[e];
      int rank = 0;
      for (int j = 0; j < N; ++j) rank += sm.cand[j] > me;
      if (rank < k) list[rank] = me;
      if (rank == k - 1) sm.kth = me;
      if (rank == k) sm.lmax = okey(comp_val(me));     // the largest beyond the list
    }
    // ---- the mass of everything not listed, relative to its largest
    if (!exact) {
      mr = block_max_n<kTlWarps>(mr, sm.fred);         // its barriers publish kth and lmax too
      const float lmax = sm.lmax != 0u ? key_to_float(sm.lmax) : -INFINITY;
      mr = fmaxf(mr, lmax);
      if (mr > -INFINITY) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < VW; t += 2) {
            s0 += ex2_approx((TR::get(x[u], t) - mr) * p.c);
            s1 += ex2_approx((TR::get(x[u], t + 1) - mr) * p.c);
          }
        s = f2_add(F2{s0, 0.f}, F2{s1, 0.f});
      }
      s = block_sum_f2_n<kTlWarps>(s, sm.f2red);
      if (lmax > -INFINITY) {                          // candidates beyond the list, in whatever order they stand
        const unsigned long long kth = sm.kth;
        unsigned long long w = 0ull;
        for (int e = tid; e < N; e += kTlThreads) {
          const unsigned long long me = sm.cand[e];
          if (me < kth) w += weight_fixed(weight_f2(comp_val(me), lmax, F2{p.c, p.c_lo}, sm.tab).hi);
        }
        const F2 left = fixed_f2(block_sum_u64<kTlWarps>(w, sm.u64red));
        s = f2_add(s, f2_mul(left, weight_f2(lmax, mr, F2{p.c, p.c_lo}, sm.tab)));
      }
    } else {
      s = block_sum_f2_n<kTlWarps>(s, sm.f2red);
    }
  }
  if (tid == 0) p.part[(size_t)r * p.H + h] = make_float4(mr, s.hi, s.lo, bad ? 1.f : 0.f);
  if (arrive_last(p.ticket + r, p.H, &sm.flag)) top_finish_row<T>(p, r, sm);
}

// ---- one CTA per row
//
// For many rows the slices' selections are most of the work: ten per row of
// 150 thousand tokens.  Here a CTA streams a whole row through a ring of
// cp.async stages private to each thread and selects once.  `thr` is a lower
// bound of the row's k-th largest value at any time: from the first step's
// vector maxima, later from the candidates so far.  An element that reaches
// it leaves the registers (its vector's number goes to a list, and after the
// step's barrier one thread per element of those vectors, still in the ring,
// adds the candidates to theirs); everything else goes into the thread's
// running (maximum, sum) at once.  Raising thr costs a radix select over some
// hundred candidates, and is done when their number has grown by k; when they
// outgrow their buffer they are cut back to the k best.  An element equal to
// the k-th best that comes later in the row loses the tie, so a raised bound
// is strict, and rows of ties or of rising values cost more cuts but need no
// other path.
constexpr int kTrU = 3;                         // vectors per thread per step (four CTAs per SM)
constexpr int kTrStages = 3;                    // ring stages: one read, one or two in flight
constexpr int kTrStep = kTrU * kTlThreads;      // vectors per step

// Listed vectors a step that need no look at the buffer's end; candidates at
// which it is cut back; its size.
__host__ __device__ constexpr int tr_few(int k) { return k + k / 4 < 64 ? 64 : k + k / 4 < kTrStep ? k + k / 4 : kTrStep; }
__host__ __device__ constexpr int tr_trigger(int k) { return 4 * k + 64 < 512 ? 512 : 4 * k + 64; }
__host__ __device__ constexpr int tr_capacity(int k) { return tr_trigger(k) + 8 * tr_few(k); }

struct TopRowSmem {
  PickSmem pick;
  float tab[128];
  float fred[kTlWarps];
  F2 f2red[kTlWarps];
  int ired[kTlWarps];
  unsigned long long u64red[kTlWarps];
  F2 lns;
  int nvec[3];                                  // listed vectors of a step, by step % 3
  int nk, count;
  uint16_t list[2][kTrStep];                    // their places in the step, by step % 2
};

// A thread's running (maximum, sum) of the elements that are not set aside.
// The sum is relative to an integer rho next to m c in units of log2, so that
// a term costs one multiply-add and one exponential, and a risen maximum
// rescales the sum by a power of two, which the exponential instruction forms
// exactly: a row may raise it at every step, whatever its logits have in
// common (a reference that is not kept through a raise, m c itself, left the
// sum's logarithm off by 2e-4 at logits around 1e4, by 0.08 around 3e6).  What
// rho leaves of m c is taken back by scale().  Terms gather in short float32
// chains that take() adds to the two-float total, so a row of 2^24 tokens is
// summed as exactly as a short one.  Beyond kNear the difference is taken first.
struct RunningSum {
  float m = -INFINITY, rho = -kNear;   // below any reference: what is rescaled then is 0, or NaN
  F2 s{0.f, 0.f};
  bool far = false;
  __device__ __forceinline__ float scale(float c) const { return far || m == -INFINITY ? 1.f : ex2_approx(-fmaf(m, c, -rho)); }
  __device__ __forceinline__ void raise(float to, float c) {
    if (to > m) {
      const float r = rintf(to * c);
      const bool to_far = !(fabsf(r) < kNear);
      float f;
      if (!far && !to_far) f = ex2_approx(rho - r);   // the difference of integers below 2^23 is exact
      else f = m == -INFINITY ? 0.f : ex2_approx((m - to) * c) * scale(c) * (to_far ? 1.f : ex2_approx(fmaf(to, c, -r)));
      s.hi *= f;
      s.lo *= f;
      m = to;
      rho = r;
      far = to_far;
    }
  }
  // 2^((x - m) c), x <= m
  __device__ __forceinline__ float term(float x, float c) const { return ex2_approx(fmaf(x, c, -rho)); }
  __device__ __forceinline__ float term_far(float x, float c) const { return ex2_approx((x - m) * c); }
  __device__ __forceinline__ void take(float t) { s = f2_add(s, F2{t, 0.f}); }
};

// WHOLE: V is a multiple of the vector width, so every row is whole vectors.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kTlThreads, 4) top_row_kernel(const TopParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ TopRowSmem sm;
  const int tid = threadIdx.x, k = p.k, r = blockIdx.x;
  const int trig = tr_trigger(k), few = tr_few(k);
  uint4* ring = reinterpret_cast<uint4*>(smem_raw);                            // [kTrStages][kTrU][kTlThreads]
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(ring + kTrStages * kTrStep);   // [tr_capacity(k)] candidates
  const Window<T, const T> win(static_cast<const T*>(p.logits), (size_t)r, p.V);
  const int NV = win.vectors();
  const int steps = (NV + kTrStep - 1) / kTrStep;
  const uint4 pad = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);

  const T* src = win.base + (size_t)tid * VW;                                  // this thread's next vectors
  int v0 = tid;
  uint4* slot = ring + tid;                                                    // and where they go
  auto issue = [&](int step) {
#pragma unroll
    for (int u = 0; u < kTrU; ++u) {
      const int v = v0 + u * kTlThreads;
      if (v < NV && (WHOLE || win.whole(v))) {
        const unsigned sa = (unsigned)__cvta_generic_to_shared(slot + u * kTlThreads);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa), "l"(src + u * kTlThreads * VW) : "memory");
      } else if (step < steps) {
        slot[u * kTlThreads] = !WHOLE && v < NV ? win.load(v) : pad;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    src += kTrStep * VW;
    v0 += kTrStep;
    slot = slot == ring + (kTrStages - 1) * kTrStep + tid ? ring + tid : slot + kTrStep;
  };
  issue(0);
  issue(1);
  load_exp2_table(sm.tab);
  if (tid == 0) sm.nvec[0] = sm.nvec[1] = sm.nvec[2] = sm.nk = 0;
  __syncthreads();

  const float c = p.c;
  float thr = -INFINITY;
  int look = min(trig, k + max(k, 64));                              // candidates at which thr is raised next
  int flag = 0;
  RunningSum acc;
  auto all_keys = [&](int n, auto f) {
    for (int e = tid; e < n; e += kTlThreads) f(keys[e]);
  };
  // adds the mass of keys that leave the candidates (any order) to thread 0's sum; top: the largest of them
  auto leave = [&](float top, auto each) {
    top = block_max_n<kTlWarps>(top, sm.fred);
    if (top == -INFINITY) return;
    unsigned long long w = 0ull;
    each([&](unsigned long long key) { w += weight_fixed(weight_f2(comp_val(key), top, F2{p.c, p.c_lo}, sm.tab).hi); });
    w = block_sum_u64<kTlWarps>(w, sm.u64red);
    if (tid == 0) {
      acc.raise(top, c);
      const float f = acc.far ? acc.term_far(top, c) : acc.term(top, c);
      acc.s = f2_add(acc.s, f2_mul(fixed_f2(w), F2{f, 0.f}));
    }
  };
  // the smallest float above the value of K64 (which may have stopped early,
  // with zeros below the digits it needed: a smaller bound then); keys of
  // finite values start at 0x00800000
  auto above = [&](unsigned long long K64) { return key_to_float(max((uint32_t)(K64 >> 32), 0x007fffffu) + 1u); };

#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    uint4 x[kTrU];
    float vm[kTrU];
    const uint4* stage = ring + (step % kTrStages) * kTrStep;
#pragma unroll
    for (int u = 0; u < kTrU; ++u) {
      x[u] = stage[u * kTlThreads + tid];
      vm[u] = TR::template vmax<false>(x[u]);
    }
    if (step == 0) {
      uint32_t key[kTrU];
#pragma unroll
      for (int u = 0; u < kTrU; ++u) key[u] = vm[u] > -INFINITY ? okey(vm[u]) : 0u;
      const uint32_t K = kth_key<TR::KEY_LOW_BIT, kTrU>(key, k, sm.pick);
      if (K != 0u) thr = key_to_float(K);
    }
    float mc = -INFINITY;
#pragma unroll
    for (int u = 0; u < kTrU; ++u) {
      if (vm[u] >= thr && vm[u] > -INFINITY) {
        const int pos = atomicAdd(&sm.nvec[step % 3], 1);
        sm.list[step & 1][pos] = (uint16_t)(u * kTlThreads + tid);
        flag |= pos >= few;
        clear_ge<T>(x[u], thr);
        vm[u] = TR::template vmax<false>(x[u]);
      }
      mc = fmaxf(mc, vm[u]);
    }
    acc.raise(mc, c);
    {
      // (with nothing but -inf so far the terms are 0, or NaN)
      float s0 = 0.f, s1 = 0.f;
      if (!acc.far) {
        const Pair cc = pair_of(c, c), rr = pair_of(-acc.rho, -acc.rho);
        Pair a = pair_of(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kTrU; ++u)
#pragma unroll
          for (int t = 0; t < VW; t += 2) a = pair_add(a, pair_terms<T>(x[u], t, cc, rr));
        unpair(a, s0, s1);
      } else {
#pragma unroll
        for (int u = 0; u < kTrU; ++u) {
#pragma unroll 1
          for (int t = 0; t < VW; ++t) s0 += acc.term_far(TR::get(x[u], t), c);
        }
      }
      acc.take(s0 + s1);
    }
    if (tid == 0) sm.nvec[(step + 1) % 3] = 0;                       // last read two steps ago
    const bool slow = __syncthreads_or(flag);                        // a buffer may be near its end, or thr is due
    issue(step + 2);                                                 // into the stage that everyone has left
    const int nv = sm.nvec[step % 3];
    // every element of the listed vectors that reaches thr
    auto listed = [&](auto f) {
      for (int e = tid; e < nv * VW; e += kTlThreads) {
        const int at = sm.list[step & 1][e / VW];
        const float xv = Elem<T>::load(reinterpret_cast<const T*>(stage + at) + e % VW);
        if (xv >= thr && xv > -INFINITY) f(comp_key(xv, (step * kTrStep + at) * VW - win.a0 + e % VW));
      }
    };
    flag = 0;
    if (!slow) {
      listed([&](unsigned long long key) {
        const int pos = atomicAdd(&sm.nk, 1);
        keys[pos] = key;
        flag |= pos >= look;
      });
    } else {
      const int nk = sm.nk;
      int fresh = 0;
      listed([&](unsigned long long) { ++fresh; });
      fresh = block_sum_int_w<kTlWarps>(fresh, sm.ired);             // its barriers: everyone has read nk
      if (nk + fresh > trig && nk + fresh > k) {
        // cut back to the k best
        const unsigned long long K64 = select_kth64<T>(k, p.V, sm.pick, [&](auto f) {
          all_keys(nk, f);
          listed(f);
        });
        float top = -INFINITY;
        auto leaving = [&](auto f) {
          auto g = [&](unsigned long long key) { if (key < K64) f(key); };
          all_keys(nk, g);
          listed(g);
        };
        leaving([&](unsigned long long key) { top = fmaxf(top, comp_val(key)); });
        leave(top, leaving);
        __syncthreads();
        if (tid == 0) sm.nk = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < nk; e0 += kTlThreads) {
          const unsigned long long key = e0 + tid < nk ? keys[e0 + tid] : 0ull;
          __syncthreads();                                           // this round's keys are in registers
          if (key != 0ull && key >= K64) keys[atomicAdd(&sm.nk, 1)] = key;
        }
        __syncthreads();
        listed([&](unsigned long long key) { if (key >= K64) keys[atomicAdd(&sm.nk, 1)] = key; });
        __syncthreads();
        thr = above(K64);
        look = min(trig, k + max(k, 64));
      } else {
        listed([&](unsigned long long key) { keys[atomicAdd(&sm.nk, 1)] = key; });
        __syncthreads();
        if (nk + fresh > k) {
          thr = fmaxf(thr, above(select_kth64<T>(k, p.V, sm.pick, [&](auto f) { all_keys(nk + fresh, f); })));
          look = min(trig, nk + fresh + max(k, 64));
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  __syncthreads();                                                   // the last step's candidates are in

  // ---- the record
  // a NaN is in its thread's sum, +inf among the candidates
  const int have = sm.nk;
  int bad = acc.s.hi != acc.s.hi;
  for (int e = tid; e < have; e += kTlThreads) bad |= comp_val(keys[e]) == INFINITY;
  bad = __syncthreads_or(bad);
  if (bad || have == 0) {
    top_write_bad(p, r);
    return;
  }
  unsigned long long* sel = reinterpret_cast<unsigned long long*>(ring);
  if (tid == 0) sm.count = 0;
  const unsigned long long K64 = have > k ? select_kth64<T>(k, p.V, sm.pick, [&](auto f) { all_keys(have, f); }) : 1ull;
  __syncthreads();
  float top = -INFINITY;
  all_keys(have, [&](unsigned long long key) {
    if (key >= K64) sel[atomicAdd(&sm.count, 1)] = key;
    else top = fmaxf(top, comp_val(key));
  });
  leave(top, [&](auto f) {
    all_keys(have, [&](unsigned long long key) { if (key < K64) f(key); });
  });
  const float mt = block_max_n<kTlWarps>(acc.m, sm.fred);
  F2 st{0.f, 0.f};
  if (acc.m > -INFINITY)
    st = f2_mul(f2_mul(acc.s, F2{acc.scale(c), 0.f}), weight_f2(acc.m, mt, F2{p.c, p.c_lo}, sm.tab));
  st = block_sum_f2_n<kTlWarps>(st, sm.f2red);
  top_write<kTlWarps>(p, r, sel, min(k, have), mt, st, sm.tab, sm.f2red, &sm.lns);
}

}  // namespace rows
}  // namespace sv
