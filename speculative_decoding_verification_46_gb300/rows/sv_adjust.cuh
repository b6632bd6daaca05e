// Penalties for repeated tokens, biases and masks on logits rows.
//
// One CTA owns a tile of the vocabulary for all gamma + 1 rows of a sequence.
// It counts the sequence's history and drafts that fall into the tile in
// shared memory (a word per token: occurrences, and flags for prompt, draft
// and bias; integer atomics, so the order of arrival does not matter) and
// lists the tokens it met: some hundreds of a tile's thousands.  Only those
// are computed; everything else of a row is copied or masked in 16-byte
// vectors, so the pass that moves the bytes costs no more than a copy,
// whatever the history holds.  A row i differs from row 0 of its sequence
// only by the drafts before it: tokens with the draft flag add them up from
// the list of drafts.
//
//   adjust_staged_kernel   out is another tensor and there are listed tokens:
//       each row of the tile passes through shared memory (a ring of
//       cp.async stages, the next rows loading meanwhile), where its listed
//       tokens are changed before it is written.  Changing them in `out`
//       afterwards instead, with the kernel below, read and wrote their
//       sectors a second time: 304 MB read from DRAM for 175 MB of logits, 9
//       rows of 64 sequences after 8192 tokens.
//   adjust_direct_kernel   in place (only vectors that a mask changes and the
//       listed tokens are touched), or nothing is listed (a masked copy).
//
// The bound is HBM: every row is read and written once (vectors that a mask
// rules out altogether are not read).  256 sequences, gamma 8, V = 152064 bf16,
// histories of 8192: 241 us, 5.6 TB/s (0.82 of the measured copy); what is
// left is the tiles' preparation, which is instructions (at gamma 0, where it
// is most of the work, 70 us for 162 MB; issue slots were 0.67 busy at 87 us)
// and which three CTAs an SM hide in part.  A tile is 12 KB of a row and 384
// threads: 16 KB and 512 threads, two CTAs an SM, 255 us, and 72 at gamma 0;
// 8 KB and 256 threads, four, 256 and 86 (the history is counted more often).
// CTAs that stay and load the next tile's history ahead: 305 (two an SM; they
// prepare at the same time, where CTAs launched one by one drift apart).
#pragma once

#include "sv_rows.cuh"

namespace sv {
namespace rows {

constexpr int kAdThreads = 384;           // two vectors of 16 bytes each per row of a full tile
constexpr int kAdTileBytes = 32 * kAdThreads;   // bytes of a row in a tile
constexpr int kAdStages = 3;
constexpr uint32_t kAdPrompt = 1u << 31;  // the token stands in the prompt
constexpr uint32_t kAdDraft = 1u << 30;   // the token is one of the round's drafts
constexpr uint32_t kAdBias = 1u << 29;    // the token has a bias
constexpr uint32_t kAdCount = (1u << 24) - 1;

struct AdjustParams {
  int B, G1, V;
  int tile, tiles;            // tokens per tile (a multiple of 64), tiles per row
  const void* logits;
  void* out;
  int copy;                   // out is not logits
  int count;                  // penalties are given and there is something to count
  const int32_t* draft;       // [B][G1 - 1] or nullptr
  const int32_t* gamma_b;
  const int32_t* history;
  int H;
  const int32_t* history_len;
  const int32_t* prompt_len;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_tokens;
  const float* bias_values;
  int NB;
  const uint32_t* mask;
  int M, W;                   // mask rows, words of each
  const int32_t* mask_index;
};

// One more token of the sequence: note it if it falls into the tile.  Nothing
// waits for the atomic's result (with a list entry for the first to meet a
// token, a warp waited some 200 cycles for each of its tokens in the tile).
__device__ __forceinline__ void adjust_note(uint32_t* cnt, int token, int t0, int n, uint32_t flag) {
  const unsigned o = (unsigned)token - (unsigned)t0;   // a negative token is far out
  if (o < (unsigned)n) {
    if (flag) atomicOr(cnt + o, flag);
    else atomicAdd(cnt + o, 1u);
  }
}

// The same for tokens that are all in the prompt, or all behind it: four
// instructions a token, no branch.  cnt: a shared-memory address.
template <bool PROMPT>
__device__ __forceinline__ void adjust_note_all(unsigned cnt, int token, int t0, int n) {
  const unsigned o = (unsigned)token - (unsigned)t0;
  if (PROMPT)
    asm volatile("{\n\t.reg .pred in;\n\tsetp.lt.u32 in, %1, %2;\n\t@in red.shared.or.b32 [%0], %3;\n\t}"
                 ::"r"(cnt + 4u * o), "r"(o), "r"((unsigned)n), "r"(kAdPrompt) : "memory");
  else
    asm volatile("{\n\t.reg .pred in;\n\tsetp.lt.u32 in, %1, %2;\n\t@in red.shared.add.u32 [%0], 1;\n\t}"
                 ::"r"(cnt + 4u * o), "r"(o), "r"((unsigned)n) : "memory");
}

// What the CTA has in shared memory.
template <typename T>
struct AdjustTile {
  uint32_t* cnt;    // [tile]
  int2* blist;      // [NB] (offset, entry)
  uint16_t* list;   // [tile]
  int* draft;       // [gamma]
  int* mask;        // [gamma + 1] the rows' mask rows: -1 none, -2 nothing is allowed
  int* nlist;
  int* nb;
  int b, t0, n, gb;
};
constexpr int kAdNone = -1, kAdNothing = -2;

// The rows' mask rows; complete after the next barrier.
template <typename T>
__device__ __forceinline__ void adjust_masks(const AdjustParams& p, const AdjustTile<T>& s) {
  if ((int)threadIdx.x > s.gb) return;
  const size_t row = (size_t)s.b * p.G1 + threadIdx.x;
  int mi = -1;
  if (p.mask) mi = p.mask_index ? __ldg(p.mask_index + row) : (int)row;
  s.mask[threadIdx.x] = mi < 0 ? kAdNone : mi < p.M ? mi : kAdNothing;
}

// The tile's tokens of the sequence.  start() issues every load that depends
// on nothing (sixteen of the history's tokens a thread before its length is known,
// four tokens a load where its rows are 16-byte aligned), so that a tile's
// preparation is one round trip to memory and not one after another; finish()
// counts, and is complete after the next barrier.
template <typename T>
struct AdjustCollect {
  int4 tok[4];
  int len, np, quads, draft;
  __device__ __forceinline__ const int32_t* history(const AdjustParams& p, const AdjustTile<T>& s) const {
    return p.history + (size_t)s.b * p.H;
  }
  __device__ __forceinline__ void start(const AdjustParams& p, const AdjustTile<T>& s) {
    const int tid = threadIdx.x;
    len = np = quads = 0;
    draft = p.count && p.draft && tid < p.G1 - 1 ? __ldg(p.draft + (size_t)s.b * (p.G1 - 1) + tid) : -1;
    if (p.count && p.history) {
      len = __ldg(p.history_len + s.b);
      np = p.prompt_len ? __ldg(p.prompt_len + s.b) : 0;
      const int32_t* h = history(p, s);
      quads = (reinterpret_cast<uintptr_t>(h) & 15u) == 0 ? p.H >> 2 : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int q = tid + u * kAdThreads;
        tok[u] = q < quads ? __ldg(reinterpret_cast<const int4*>(h) + q) : make_int4(-1, -1, -1, -1);
      }
    }
    for (int i = tid; i < p.tile / 4; i += kAdThreads) reinterpret_cast<uint4*>(s.cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) *s.nlist = *s.nb = 0;
  }
  __device__ __forceinline__ void note(const AdjustTile<T>& s, int i, int token) const {
    if (i < len) adjust_note(s.cnt, token, s.t0, s.n, i < np ? kAdPrompt : 0u);
  }
  // four tokens from position 4 q on; a warp's lanes hold 128 in a row
  __device__ __forceinline__ void note(const AdjustTile<T>& s, int q, const int4& t) const {
    const int first = 4 * (q - (int)(threadIdx.x & 31)), last = first + 127;
    const unsigned cnt = (unsigned)__cvta_generic_to_shared(s.cnt);
    if (first >= len) return;
    if (first >= np && last < len) {
      adjust_note_all<false>(cnt, t.x, s.t0, s.n);
      adjust_note_all<false>(cnt, t.y, s.t0, s.n);
      adjust_note_all<false>(cnt, t.z, s.t0, s.n);
      adjust_note_all<false>(cnt, t.w, s.t0, s.n);
    } else if (last < np) {
      adjust_note_all<true>(cnt, t.x, s.t0, s.n);
      adjust_note_all<true>(cnt, t.y, s.t0, s.n);
      adjust_note_all<true>(cnt, t.z, s.t0, s.n);
      adjust_note_all<true>(cnt, t.w, s.t0, s.n);
    } else {
      note(s, 4 * q, t.x);
      note(s, 4 * q + 1, t.y);
      note(s, 4 * q + 2, t.z);
      note(s, 4 * q + 3, t.w);
    }
  }
  // a barrier lies between start and finish
  __device__ __forceinline__ void finish(const AdjustParams& p, const AdjustTile<T>& s) {
    const int tid = threadIdx.x;
    if (p.count && p.history) {
      len = min(max(len, 0), p.H);
      np = min(max(np, 0), len);
      const int32_t* h = history(p, s);
#pragma unroll
      for (int u = 0; u < 4; ++u) note(s, tid + u * kAdThreads, tok[u]);
      for (int q = tid + 4 * kAdThreads; 4 * q < len && q < quads; q += kAdThreads)
        note(s, q, __ldg(reinterpret_cast<const int4*>(h) + q));
      for (int i = 4 * quads + tid; i < len; i += kAdThreads) note(s, i, __ldg(h + i));
    }
    if (p.count && p.draft && tid < s.gb) {
      s.draft[tid] = draft;
      adjust_note(s.cnt, draft, s.t0, s.n, kAdDraft);
    }
    for (int i = tid; i < p.NB; i += kAdThreads) {
      const int tok_i = __ldg(p.bias_tokens + (size_t)s.b * p.NB + i);
      adjust_note(s.cnt, tok_i, s.t0, s.n, kAdBias);
      if (tok_i >= s.t0 && tok_i < s.t0 + s.n) s.blist[atomicAdd(s.nb, 1)] = make_int2(tok_i - s.t0, i);
    }
    __syncthreads();
    // the tokens met: sixteen words a thread, one reservation a warp
    static_assert(kAdTileBytes / 2 <= 16 * kAdThreads, "a tile is looked through once");
    uint32_t met = 0u;                                               // bit 4 u + t: word t of the thread's u-th four
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int w = tid + u * kAdThreads;
      if (w < p.tile / 4) {
        const uint4 c = reinterpret_cast<const uint4*>(s.cnt)[w];
        met |= (c.x != 0u ? 1u : 0u) << (4 * u) | (c.y != 0u ? 2u : 0u) << (4 * u) | (c.z != 0u ? 4u : 0u) << (4 * u) |
               (c.w != 0u ? 8u : 0u) << (4 * u);
      }
    }
    const int mine = __popc(met);
    int upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, m);
      if ((tid & 31) >= m) upto += v;
    }
    int at = 0;
    if ((tid & 31) == 31 && upto > 0) at = atomicAdd(s.nlist, upto);
    at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
    for (; met; met &= met - 1u) {
      const int k = __ffs(met) - 1;
      s.list[at++] = (uint16_t)(4 * (tid + (k >> 2) * kAdThreads) + (k & 3));
    }
  }
};

struct AdjustPenalties {
  float rep, freq, pres;
  __device__ __forceinline__ AdjustPenalties(const AdjustParams& p, int b)
      : rep(p.repetition ? __ldg(p.repetition + b) : 1.f), freq(p.frequency ? __ldg(p.frequency + b) : 0.f),
        pres(p.presence ? __ldg(p.presence + b) : 0.f) {}
};

// The mask bits of the VW tokens from v on.  WHOLE: v is a multiple of VW;
// otherwise it may lie up to VW - 1 before the row, and the bits in two words.
template <int VW, bool WHOLE>
__device__ __forceinline__ uint32_t adjust_bits(const uint32_t* mrow, int W, int v) {
  constexpr uint32_t kFull = (1u << VW) - 1u;
  if (WHOLE) return (__ldg(mrow + (v >> 5)) >> (v & 31)) & kFull;
  const int w = max(v, 0) >> 5, sh = v - (w << 5);
  const uint32_t lo = __ldg(mrow + w);
  const uint32_t hi = (sh + VW > 32 && w + 1 < W) ? __ldg(mrow + w + 1) : 0u;
  return (sh >= 0 ? __funnelshift_r(lo, hi, sh) : lo << -sh) & kFull;
}

// What row i does to the listed token at tile offset o (the row's mask aside).
struct AdjustChange {
  float less, bias;   // frequency and presence together; the bias
  bool seen, biased;
  __device__ __forceinline__ bool any() const { return seen || biased; }
  __device__ __forceinline__ float apply(float x, float rep) const {
    if (seen) {
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      x -= less;
    }
    return biased ? x + bias : x;
  }
};
template <typename T>
__device__ __forceinline__ AdjustChange adjust_change(const AdjustParams& p, const AdjustTile<T>& s,
                                                      const AdjustPenalties& pen, int i, int o) {
  const uint32_t w = s.cnt[o];
  int c = (int)(w & kAdCount);
  if (w & kAdDraft)
    for (int j = 0; j < i; ++j) c += (s.draft[j] == s.t0 + o);
  AdjustChange a;
  a.seen = (w & kAdPrompt) || c > 0;
  a.less = fmaf(pen.freq, (float)c, c > 0 ? pen.pres : 0.f);
  a.biased = w & kAdBias;
  a.bias = 0.f;
  if (a.biased) {
    int last = -1;
    for (int k = 0; k < *s.nb; ++k)
      if (s.blist[k].x == o) last = max(last, s.blist[k].y);
    a.bias = __ldg(p.bias_values + (size_t)s.b * p.NB + last);
  }
  return a;
}
// whether the mask row lets token v pass
__device__ __forceinline__ bool adjust_allowed(const uint32_t* mrow, int v) {
  return !mrow || ((__ldg(mrow + (v >> 5)) >> (v & 31)) & 1u);
}

template <typename T>
__device__ __forceinline__ AdjustTile<T> adjust_tile(const AdjustParams& p, unsigned char* smem, int* draft, int* mask, int* counters) {
  AdjustTile<T> s;
  s.cnt = reinterpret_cast<uint32_t*>(smem);
  s.blist = reinterpret_cast<int2*>(s.cnt + p.tile);
  s.list = reinterpret_cast<uint16_t*>(s.blist + p.NB);
  s.draft = draft;
  s.mask = mask;
  s.nlist = counters;
  s.nb = counters + 1;
  s.b = blockIdx.x / p.tiles;
  s.t0 = (blockIdx.x - s.b * p.tiles) * p.tile;
  s.n = min(p.tile, p.V - s.t0);
  s.gb = p.gamma_b ? min(max(__ldg(p.gamma_b + s.b), 0), p.G1 - 1) : p.G1 - 1;
  return s;
}

// A vector with what the mask rules out set to -inf.  Two 16-bit elements at a
// time: a product puts bit k at k and at k + 15, so one shift brings a pair's
// bits to 0 and 16, and a second product widens them to halves.
template <typename T>
__device__ __forceinline__ void adjust_masked(uint4& x, uint32_t bits) {
  constexpr uint32_t kOut = Tr<T>::kPadWord;
  uint32_t* w[4] = {&x.x, &x.y, &x.z, &x.w};
  if (sizeof(T) == 2) {
    const uint32_t two = bits * 0x8001u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t keep = ((two >> (2 * i)) & 0x10001u) * 0xffffu;
      *w[i] = (*w[i] & keep) | (kOut & ~keep);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) *w[i] = (bits >> i) & 1u ? *w[i] : kOut;
  }
}

// WHOLE: V is a multiple of the vector width, so every row is whole vectors.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kAdThreads, 3) adjust_staged_kernel(const AdjustParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ int sdraft[kMaxG1], smask[kMaxG1];
  __shared__ int counters[2];
  const int tid = threadIdx.x;
  const int SV = p.tile / VW + 1;                                  // vectors of a stage: a row may start inside one
  uint4* ring = reinterpret_cast<uint4*>(smem_raw);                // [kAdStages][SV]
  const AdjustTile<T> s = adjust_tile<T>(p, smem_raw + (size_t)kAdStages * SV * sizeof(uint4), sdraft, smask, counters);
  const size_t first = (size_t)s.b * p.G1 * (size_t)p.V + s.t0;    // row 0's first element in the tile
  const T* logits = static_cast<const T*>(p.logits);
  T* out = static_cast<T*>(p.out);

  auto issue = [&](int i) {                                        // row i of the sequence into its stage
    const int mi = i <= s.gb ? smask[i] : kAdNothing;
    if (mi != kAdNothing) {
      const uint32_t* mrow = mi >= 0 ? p.mask + (size_t)mi * p.W : nullptr;
      const size_t e0 = first + (size_t)i * p.V;
      const int a = WHOLE ? 0 : (int)(e0 % VW);
      const T* src = logits + (e0 - a);
      uint4* st = ring + (i % kAdStages) * SV;
      const int nv = (a + s.n + VW - 1) / VW;
      for (int j = tid; j < nv; j += kAdThreads) {
        const int o = j * VW - a;
        if (WHOLE || (o >= 0 && o + VW <= s.n)) {
          if (!mrow || adjust_bits<VW, WHOLE>(mrow, p.W, s.t0 + o) != 0u) {
            const unsigned sa = (unsigned)__cvta_generic_to_shared(st + j);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sa), "l"(src + (size_t)j * VW) : "memory");
          }
        } else {
          for (int t = 0; t < VW; ++t)
            if (o + t >= 0 && o + t < s.n)
              Elem<T>::store_raw(reinterpret_cast<T*>(st + j) + t, Elem<T>::raw(src + (size_t)j * VW + t));
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  AdjustCollect<T> collect;
  collect.start(p, s);
  const AdjustPenalties pen(p, s.b);
  adjust_masks(p, s);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAdStages - 1; ++i) issue(i);
  collect.finish(p, s);
  __syncthreads();
  // a thread's first listed token keeps what is done to it: the same in every
  // row, unless it is drafted
  const int nl = *s.nlist;
  int mine = -1;
  AdjustChange change{0.f, 0.f, false, false};
  if (tid < nl) {
    mine = s.list[tid];
    if (s.cnt[mine] & kAdDraft) mine = -1;
    else change = adjust_change(p, s, pen, 0, mine);
  }

  for (int i = 0; i <= s.gb; ++i) {
    issue(i + kAdStages - 1);                                      // its stage was written out an iteration ago
    asm volatile("cp.async.wait_group %0;" ::"n"(kAdStages - 1) : "memory");
    __syncthreads();                                               // row i is in
    const int mi = smask[i];
    const uint32_t* mrow = mi >= 0 ? p.mask + (size_t)mi * p.W : nullptr;
    const size_t e0 = first + (size_t)i * p.V;
    const int a = WHOLE ? 0 : (int)(e0 % VW);
    uint4* st = ring + (i % kAdStages) * SV;
    if (mi != kAdNothing) {
      T* elem = reinterpret_cast<T*>(st) + a;
      if (mine >= 0 && change.any() && adjust_allowed(mrow, s.t0 + mine))
        Elem<T>::store(elem + mine, change.apply(Elem<T>::load(elem + mine), pen.rep));
      for (int e = mine >= 0 ? tid + kAdThreads : tid; e < nl; e += kAdThreads) {
        const int o = s.list[e];
        const AdjustChange ch = adjust_change(p, s, pen, i, o);
        if (ch.any() && adjust_allowed(mrow, s.t0 + o))
          Elem<T>::store(elem + o, ch.apply(Elem<T>::load(elem + o), pen.rep));
      }
    }
    __syncthreads();
    T* dst = out + (e0 - a);
    const int nv = (a + s.n + VW - 1) / VW;
    for (int j = tid; j < nv; j += kAdThreads) {
      const int o = j * VW - a;
      uint4 x;
      if (mi == kAdNone) {
        x = st[j];
      } else {
        x = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
        const uint32_t bits = mrow ? adjust_bits<VW, WHOLE>(mrow, p.W, s.t0 + o) : 0u;
        if (bits != 0u) {
          x = st[j];
          if (bits != (1u << VW) - 1u) adjust_masked<T>(x, bits);
        }
      }
      if (WHOLE || (o >= 0 && o + VW <= s.n)) {
        __stcs(reinterpret_cast<uint4*>(dst + (size_t)j * VW), x);
      } else {
#pragma unroll
        for (int t = 0; t < VW; ++t)
          if (o + t >= 0 && o + t < s.n) Elem<T>::store_raw(dst + (size_t)j * VW + t, raw_of<T>(x, t));
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kAdThreads, 3) adjust_direct_kernel(const AdjustParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  constexpr uint32_t kFull = (1u << VW) - 1u;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ int sdraft[kMaxG1], smask[kMaxG1];
  __shared__ int counters[2];
  const int tid = threadIdx.x;
  const bool sparse = p.count || p.NB;
  const AdjustTile<T> s = adjust_tile<T>(p, smem_raw, sdraft, smask, counters);
  AdjustCollect<T> collect;
  if (sparse) collect.start(p, s);
  adjust_masks(p, s);
  __syncthreads();
  if (sparse) {
    collect.finish(p, s);
    __syncthreads();
  }

  // ---- the rows, masked: the tile's vectors of all rows, four at a time (a
  // vector waits for its mask before it is known whether it is read).  The
  // bound next to HBM is instruction issue, so the rows' vectors are counted
  // without divisions: 64 sequences, gamma 4, V = 128256 bf16, half of it
  // allowed, in place: 29 us (169 MB, 0.85 of the measured copy); 2% allowed: 26.
  const size_t first = (size_t)s.b * p.G1 * (size_t)p.V + s.t0;    // row 0's first element in the tile
  const T* logits = static_cast<const T*>(p.logits) + first;
  T* out = static_cast<T*>(p.out) + first;
  const int per = p.tile / VW + (WHOLE ? 0 : 1);                   // vectors of a row, at most
  const int step_i = kAdThreads / per, step_j = kAdThreads - step_i * per;
  int i = tid / per, j = tid - i * per;
  while (i <= s.gb) {
    uint4 x[4];
    uint32_t bits[4];
    long long e[4];                                                // the vector's first element, from `first`
    int at[4];                                                     // the same in the tile; at least s.n: no work
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      bits[u] = kFull;
      at[u] = s.n;
      if (i <= s.gb) {
        const int a = WHOLE ? 0 : (int)(((unsigned)first + (unsigned)i * (unsigned)p.V) % VW);
        at[u] = j * VW - a;
        e[u] = (long long)i * p.V + at[u];
        const int mi = smask[i];
        if (mi == kAdNothing) bits[u] = 0u;
        else if (mi >= 0 && at[u] < s.n) bits[u] = adjust_bits<VW, WHOLE>(p.mask + (size_t)mi * p.W, p.W, s.t0 + at[u]);
        if (!p.copy && bits[u] == kFull) at[u] = s.n;              // nothing changes
      }
      i += step_i;
      j += step_j;
      if (j >= per) {
        j -= per;
        ++i;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (bits[u] != 0u && at[u] < s.n && (WHOLE || (at[u] >= 0 && at[u] + VW <= s.n)))
        x[u] = *reinterpret_cast<const uint4*>(logits + e[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (at[u] >= s.n) continue;
      if (WHOLE || (at[u] >= 0 && at[u] + VW <= s.n)) {
        if (bits[u] == 0u) x[u] = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
        else adjust_masked<T>(x[u], bits[u]);
        *reinterpret_cast<uint4*>(out + e[u]) = x[u];
      } else {
        for (int t = 0; t < VW; ++t) {
          const int o = at[u] + t;
          if (o < 0 || o >= s.n) continue;
          const bool ok = (bits[u] >> t) & 1u;
          if (ok && !p.copy) continue;
          Elem<T>::store_raw(out + e[u] + t, ok ? Elem<T>::raw(logits + e[u] + t) : Elem<T>::kNegInf);
        }
      }
    }
  }
  if (!sparse) return;
  __syncthreads();   // the rows are masked

  // ---- the listed tokens of every row, in place
  const int nl = *s.nlist;
  const AdjustPenalties pen(p, s.b);
  for (int i = 0; i <= s.gb; ++i) {
    const size_t row = (size_t)s.b * p.G1 + i;
    const int mi = smask[i];
    const uint32_t* mrow = mi >= 0 ? p.mask + (size_t)mi * p.W : nullptr;
    if (mi == kAdNothing) continue;
    T* elem = static_cast<T*>(p.out) + row * (size_t)p.V + s.t0;
    for (int e = tid; e < nl; e += kAdThreads) {
      const int o = s.list[e];
      const AdjustChange ch = adjust_change(p, s, pen, i, o);
      if (ch.any() && adjust_allowed(mrow, s.t0 + o)) Elem<T>::store(elem + o, ch.apply(Elem<T>::load(elem + o), pen.rep));
    }
  }
}

}  // namespace rows
}  // namespace sv
