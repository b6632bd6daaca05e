// The record of a teacher's row: its k best log-probabilities and the log of
// the mass outside them.
//
// A row is cut into H slices of at most 256 * U vectors, one CTA each, held
// in registers from one read of HBM.  A CTA finds a lower bound tau of its
// slice's k-th largest value (the k-th largest of some of its group maxima),
// lists the elements >= tau, ranks them exactly by (value descending, index
// ascending), and sums 2^((x - m) c) over everything it did not list, m the
// largest of those.  So the mass outside is a sum of its own terms and not a
// difference, and stays accurate however small it is.  The slices' lists and
// sums go to the workspace; the last CTA of a row to arrive (an atomic
// ticket, nobody waits) selects the k best of the H lists by a radix select
// over the 64-bit keys (value, ~index), ranks them, and adds what the lists
// hold beyond them to the mass outside.
//
// The bound is HBM for many rows (each row is read once) and the chain of
// barriers of the selection for few.
#pragma once

#include "sv_rows.cuh"

namespace sv {
namespace rows {

constexpr int kTlThreads = 256;
constexpr int kTlWarps = kTlThreads / 32;
constexpr int kTlCap = 2048;      // candidates of a slice; more are selected exactly
constexpr int kTlStage = 4096;    // list entries of a row staged in shared memory

struct TopParams {
  int R, V, k;
  int H, SV;                      // slices per row, vectors per slice
  int KP;                         // group maxima per thread that tau is chosen from
  float c, c_lo;                  // log2(e) / temperature
  double inv_t;                   // 1 / temperature
  const void* logits;
  int32_t* indices;
  float* logprobs;
  float* tail;
  int* ticket;                    // [R]
  float4* part;                   // [R][H] (largest, sum high, sum low, bad)
  unsigned long long* lists;      // [R][H][k] sorted keys; 0 = none
};

struct TopSmem {
  unsigned long long buf[kTlStage];   // a slice's candidates; a row's list entries
  unsigned long long sel[kMaxK];
  int hist[256];
  float tab[128];
  float fred[kTlWarps];
  F2 f2red[kTlWarps];
  int ired[kTlWarps];
  double lns;
  unsigned long long kth;
  unsigned lmax;                      // okey of the largest candidate beyond the k best
  int count, flag, pick_digit, pick_rank, pick_count;
};

// One digit of a radix select: with hist[] complete, the digit (0..255, from
// the top) that holds the rank-th largest, the rank inside it and its count.
// digit -1: fewer than rank keys.  Every thread returns the same values.
__device__ __forceinline__ int pick_digit(TopSmem& sm, int rank, int* rank_in, int* count) {
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
      sm.pick_digit = dg;
      sm.pick_rank = rank - run;
      sm.pick_count = cc;
    }
    if (__ballot_sync(0xffffffffu, mine) == 0u && lane == 0) sm.pick_digit = -1;
  }
  __syncthreads();
  *rank_in = sm.pick_rank;
  *count = sm.pick_count;
  return sm.pick_digit;
}

// The largest K, bits below LOW zero, such that at least k of the block's
// keys (U per thread, 0 = none) are >= K; 0 if there are fewer than k.
template <int LOW, int U>
__device__ __forceinline__ uint32_t kth_key(const uint32_t (&key)[U], int k, TopSmem& sm) {
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
    // ---- K64: exactly kk keys are >= it (the keys are distinct)
    unsigned long long K64 = 1ull;
    if (have > k) {
      constexpr int LOW = Tr<T>::KEY_LOW_BIT;
      const int nidx = p.V > 1 ? 32 - __clz(p.V - 1) : 1;        // index bits that differ
      unsigned long long prefix = 0ull, known = 0ull;
      int rank = k;
      int hi = 63;
      while (true) {
        const int stop = hi >= 32 ? 32 + LOW : 0;
        const int lo = max(hi - 7, stop);
        const unsigned dmask = (1u << (hi - lo + 1)) - 1u;
        sm.hist[tid] = 0;
        __syncthreads();
        for (int e = tid; e < slots; e += kTlThreads) {
          const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
          if (key != 0ull && (key & known) == prefix) atomicAdd(&sm.hist[(unsigned)(key >> lo) & dmask], 1);
        }
        int in, cnt;
        const int dg = pick_digit(sm, rank, &in, &cnt);
        prefix |= (unsigned long long)(unsigned)dg << lo;
        known |= (unsigned long long)dmask << lo;
        rank = in;
        if (cnt == rank || lo == 0) break;
        hi = lo - 1;
        if (lo == 32 + LOW) {
          // value bits below LOW copy the sign (all ones in a negative's key);
          // index bits above those that differ are ones (the index is complemented)
          const unsigned long long skip = ((1ull << (32 + LOW)) - 1ull) & ~((1ull << 32) - 1ull);
          if (!(prefix >> 63)) prefix |= skip;
          known |= skip;
          const unsigned long long ones = nidx >= 32 ? 0ull : ((1ull << 32) - 1ull) & ~((1ull << nidx) - 1ull);
          prefix |= ones;
          known |= ones;
          hi = nidx - 1;
        }
      }
      K64 = prefix;
    }
    // ---- the k best, in any order, then ranked
    if (tid == 0) sm.count = 0;
    __syncthreads();
    float lm = -INFINITY, M = -INFINITY;
    for (int e = tid; e < slots; e += kTlThreads) {
      const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
      if (key >= K64) {
        const int pos = atomicAdd(&sm.count, 1);
        if (pos < kMaxK) sm.sel[pos] = key;
        M = fmaxf(M, comp_val(key));
      } else if (key != 0ull) {
        lm = fmaxf(lm, comp_val(key));
      }
    }
    mt = block_max_n<kTlWarps>(fmaxf(mt, lm), sm.fred);
    M = block_max_n<kTlWarps>(M, sm.fred);
    const F2 c{p.c, p.c_lo};
    // ---- the masses: of K relative to M, of the rest relative to mt
    F2 sk{0.f, 0.f}, st{0.f, 0.f};
    for (int j = tid; j < kk; j += kTlThreads) sk = f2_add(sk, weight_f2(comp_val(sm.sel[j]), M, c, sm.tab));
    for (int h = tid; h < p.H; h += kTlThreads) {
      const float4 v = __ldcg(part + h);
      if (v.x > -INFINITY) st = f2_add(st, f2_mul(F2{v.y, v.z}, weight_f2(v.x, mt, c, sm.tab)));
    }
    for (int e = tid; e < slots; e += kTlThreads) {
      const unsigned long long key = staged ? sm.buf[e] : __ldcg(lists + e);
      if (key < K64 && key != 0ull) st = f2_add(st, weight_f2(comp_val(key), mt, c, sm.tab));
    }
    sk = block_sum_f2_n<kTlWarps>(sk, sm.f2red);
    st = block_sum_f2_n<kTlWarps>(st, sm.f2red);
    if (tid == 0) {
      const bool some = st.hi > 0.f;
      const F2 tail_m = some ? f2_mul(st, weight_f2(mt, M, c, sm.tab)) : F2{0.f, 0.f};
      const double lns = log(f2_double(f2_add(sk, tail_m)));
      sm.lns = lns;
      p.tail[r] = some ? (float)(((double)mt - (double)M) * p.inv_t + log(f2_double(st)) - lns) : -INFINITY;
    }
    __syncthreads();
    const double lns = sm.lns;
    for (int e = tid; e < kk; e += kTlThreads) {
      const unsigned long long me = sm.sel[e];
      int rank = 0;
      for (int j = 0; j < kk; ++j) rank += sm.sel[j] > me;
      p.indices[(size_t)r * k + rank] = comp_idx(me);
      p.logprobs[(size_t)r * k + rank] = (float)(((double)comp_val(me) - (double)M) * p.inv_t - lns);
    }
  } else if (tid == 0) {
    p.tail[r] = __uint_as_float(0x7fffffffu);
  }
  for (int j = (ok ? kk : 0) + tid; j < k; j += kTlThreads) {
    p.indices[(size_t)r * k + j] = -1;
    p.logprobs[(size_t)r * k + j] = ok ? -INFINITY : __uint_as_float(0x7fffffffu);
  }
  // leave the workspace zero-filled
  __syncthreads();
  for (int e = tid; e < slots; e += kTlThreads)
    if (!staged || sm.buf[e] != 0ull) lists[e] = 0ull;
  for (int h = tid; h < p.H; h += kTlThreads) part[h] = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename T, int U>
__global__ void __launch_bounds__(kTlThreads, 4) top_slice_kernel(const TopParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  __shared__ TopSmem sm;
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
    sm.count = 0;
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
      g = (u % gs) == 0 ? vm[u] : fmaxf(g, vm[u]);
      key[u] = (u % gs) == gs - 1 && g > -INFINITY ? okey(g) : 0u;
    }
  }
  bad = __syncthreads_or(bad);
  F2 s{0.f, 0.f};
  float mr = -INFINITY;
  if (!bad) {
    const uint32_t K = kth_key<TR::KEY_LOW_BIT, U>(key, k, sm);
    float tau = K == 0u ? -INFINITY : key_to_float(K);
    const int i0 = v0 * VW - win.a0;                   // row index of the slice's first element
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (vm[u] > -INFINITY && vm[u] >= tau) {
#pragma unroll
        for (int t = 0; t < VW; ++t) {
          const float xv = TR::get(x[u], t);
          if (xv > -INFINITY && xv >= tau) {
            const int pos = atomicAdd(&sm.count, 1);
            if (pos < kTlCap) sm.buf[pos] = comp_key(xv, i0 + (u * kTlThreads + tid) * VW + t);
          }
        }
      }
    }
    __syncthreads();
    int N = sm.count;
    int tie_idx = 0x7fffffff;                          // of the elements equal to tau, those up to this index are listed
    if (N > kTlCap) {
      // Too many (ties at tau, or fewer groups than k): the exact k-th
      // largest value by bisection over its key, then of its ties the first.
      uint32_t KV = 0u;
      for (int bit = 31; bit >= TR::KEY_LOW_BIT; --bit) {
        const uint32_t Kt = KV | (1u << bit);
        int mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < VW; ++t) {
            const float xv = TR::get(x[u], t);
            mine += xv > -INFINITY && okey(xv) >= Kt;
          }
        if (block_sum_int_w<kTlWarps>(mine, sm.ired) >= k) KV = Kt;
      }
      // the value itself: bits below KEY_LOW_BIT are ones in a negative's key
      tau = key_to_float((KV & 0x80000000u) ? KV : KV | ((1u << TR::KEY_LOW_BIT) - 1u));
      int above = 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < VW; ++t) above += TR::get(x[u], t) > tau;
      const int need = k - block_sum_int_w<kTlWarps>(above, sm.ired);
      int lo = i0, hi = i0 + p.SV * VW - 1;            // the smallest index with `need` ties up to it
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        int mine = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < VW; ++t)
            mine += TR::get(x[u], t) == tau && i0 + (u * kTlThreads + tid) * VW + t <= mid;
        if (block_sum_int_w<kTlWarps>(mine, sm.ired) >= need) hi = mid; else lo = mid + 1;
      }
      tie_idx = lo;
      __syncthreads();
      if (tid == 0) sm.count = 0;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < VW; ++t) {
          const float xv = TR::get(x[u], t);
          const int idx = i0 + (u * kTlThreads + tid) * VW + t;
          if (xv > tau || (xv == tau && idx <= tie_idx)) {
            const int pos = atomicAdd(&sm.count, 1);
            if (pos < kTlCap) sm.buf[pos] = comp_key(xv, idx);
          }
        }
      __syncthreads();
      N = min(sm.count, kTlCap);
    }
    // ---- exact ranks: the k best to the row's list, the others to the rest
    unsigned long long* list = p.lists + ((size_t)r * p.H + h) * k;
    for (int e = tid; e < N; e += kTlThreads) {
      const unsigned long long me = sm.buf[e];
      int rank = 0;
      for (int j = 0; j < N; ++j) rank += sm.buf[j] > me;
      if (rank < k) list[rank] = me;
      if (rank == k - 1) sm.kth = me;
      if (rank == k) sm.lmax = okey(comp_val(me));     // the largest beyond the list
    }
    // ---- the mass of everything not listed
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (vm[u] < tau) {
        mr = fmaxf(mr, vm[u]);
      } else {
#pragma unroll
        for (int t = 0; t < VW; ++t) {
          const float xv = TR::get(x[u], t);
          if (xv < tau || (xv == tau && i0 + (u * kTlThreads + tid) * VW + t > tie_idx)) mr = fmaxf(mr, xv);
        }
      }
    }
    mr = block_max_n<kTlWarps>(mr, sm.fred);           // its barriers publish kth and lmax too
    if (sm.lmax != 0u) mr = fmaxf(mr, key_to_float(sm.lmax));
    if (mr > -INFINITY) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < VW; t += 2) {
          const float xa = TR::get(x[u], t), xb = TR::get(x[u], t + 1);
          const int ia = i0 + (u * kTlThreads + tid) * VW + t;
          const bool ra = xa < tau || (xa == tau && ia > tie_idx);
          const bool rb = xb < tau || (xb == tau && ia + 1 > tie_idx);
          s0 += ra ? ex2_approx((xa - mr) * p.c) : 0.f;
          s1 += rb ? ex2_approx((xb - mr) * p.c) : 0.f;
        }
      s = f2_add(F2{s0, 0.f}, F2{s1, 0.f});
      const unsigned long long kth = sm.kth;           // 0: the list holds all candidates
      for (int e = tid; e < N; e += kTlThreads) {
        const unsigned long long me = sm.buf[e];
        if (me < kth) s = f2_add(s, weight_f2(comp_val(me), mr, F2{p.c, p.c_lo}, sm.tab));
      }
      s = block_sum_f2_n<kTlWarps>(s, sm.f2red);
    }
  }
  if (tid == 0) p.part[(size_t)r * p.H + h] = make_float4(mr, s.hi, s.lo, bad ? 1.f : 0.f);
  if (arrive_last(p.ticket + r, p.H, &sm.flag)) top_finish_row<T>(p, r, sm);
}

}  // namespace rows
}  // namespace sv
