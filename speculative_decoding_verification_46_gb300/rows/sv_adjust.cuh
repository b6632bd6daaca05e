// Penalties for repeated tokens, biases and masks on logits rows.
//
// One CTA owns a tile of the vocabulary for all gamma + 1 rows of a sequence.
// It counts the sequence's history and drafts that fall into the tile in
// shared memory (a word per token: occurrences, and flags for prompt, draft
// and bias; integer atomics, so the order of arrival does not matter) and
// lists the tokens it met.  The rows then pass through in 16-byte vectors
// with the mask applied and nothing else done, and only the listed tokens,
// some hundreds of a tile's thousands, are computed and overwritten
// afterwards.  So the pass that moves the bytes costs no more than a copy,
// whatever the history holds, and an in-place call without a mask touches
// the listed tokens alone.
//
// A row i differs from row 0 of its sequence only by the drafts before it:
// tokens with the draft flag add them up from the list of drafts.
//
// The bound is HBM: every row is read and written once (vectors that a mask
// rules out altogether are not read).
#pragma once

#include "sv_rows.cuh"

namespace sv {
namespace rows {

constexpr int kAdThreads = 256;
constexpr int kAdMaxTile = 8192;          // tokens per tile: 48 KB of shared memory, four CTAs per SM
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

// One more token of the sequence: note it if it falls into the tile.
__device__ __forceinline__ void adjust_note(uint32_t* cnt, uint16_t* list, int* nlist, int token, int t0, int n,
                                            uint32_t flag) {
  const unsigned o = (unsigned)(token - t0);
  if (token >= 0 && o < (unsigned)n) {
    const uint32_t old = flag ? atomicOr(cnt + o, flag) : atomicAdd(cnt + o, 1u);
    if (old == 0u) list[atomicAdd(nlist, 1)] = (uint16_t)o;   // the first to meet it lists it
  }
}

template <typename T>
__global__ void __launch_bounds__(kAdThreads, 4) adjust_kernel(const AdjustParams p) {
  using TR = Tr<T>;
  constexpr int VW = TR::VW;
  constexpr uint32_t kFull = (1u << VW) - 1u;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint32_t* cnt = reinterpret_cast<uint32_t*>(smem_raw);                        // [tile]
  int2* blist = reinterpret_cast<int2*>(cnt + p.tile);                          // [NB] (offset, entry)
  uint16_t* list = reinterpret_cast<uint16_t*>(blist + p.NB);                   // [tile]
  __shared__ int sdraft[kMaxG1];
  __shared__ int nlist, nb;
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.tiles;
  const int t0 = (blockIdx.x - b * p.tiles) * p.tile;
  const int n = min(p.tile, p.V - t0);
  const int G = p.G1 - 1;
  const int gb = p.gamma_b ? min(max(__ldg(p.gamma_b + b), 0), G) : G;
  const bool sparse = p.count || p.NB;

  // ---- the tile's tokens of the sequence
  if (sparse) {
    for (int i = tid; i < p.tile; i += kAdThreads) cnt[i] = 0u;
    if (tid == 0) nlist = nb = 0;
    if (p.count && p.draft && tid < gb) sdraft[tid] = __ldg(p.draft + (size_t)b * G + tid);
    __syncthreads();
    if (p.count) {
      if (p.history) {
        const int len = min(max(__ldg(p.history_len + b), 0), p.H);
        const int np = p.prompt_len ? min(max(__ldg(p.prompt_len + b), 0), len) : 0;
        const int32_t* h = p.history + (size_t)b * p.H;
        for (int i0 = tid; i0 < len; i0 += 8 * kAdThreads) {
          int tok[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) tok[u] = i0 + u * kAdThreads < len ? __ldg(h + i0 + u * kAdThreads) : -1;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            adjust_note(cnt, list, &nlist, tok[u], t0, n, i0 + u * kAdThreads < np ? kAdPrompt : 0u);
        }
      }
      if (p.draft && tid < gb) adjust_note(cnt, list, &nlist, sdraft[tid], t0, n, kAdDraft);
    }
    for (int i = tid; i < p.NB; i += kAdThreads) {
      const int tok = __ldg(p.bias_tokens + (size_t)b * p.NB + i);
      adjust_note(cnt, list, &nlist, tok, t0, n, kAdBias);
      if (tok >= t0 && tok < t0 + n) blist[atomicAdd(&nb, 1)] = make_int2(tok - t0, i);
    }
  }

  // ---- the rows, masked
  for (int i = 0; i <= gb; ++i) {
    const size_t row = (size_t)b * p.G1 + i;
    int mi = -1;
    if (p.mask) mi = p.mask_index ? __ldg(p.mask_index + row) : (int)row;
    if (!p.copy && mi < 0) continue;
    const bool none = mi >= p.M;                                   // nothing is allowed
    const uint32_t* mrow = mi >= 0 && !none ? p.mask + (size_t)mi * p.W : nullptr;
    const size_t e0 = row * (size_t)p.V + t0;
    const int a = (int)(e0 % VW);
    const T* src = static_cast<const T*>(p.logits) + (e0 - a);
    T* dst = static_cast<T*>(p.out) + (e0 - a);
    const int nv = (a + n + VW - 1) / VW;
    for (int j0 = tid; j0 < nv; j0 += 4 * kAdThreads) {
      uint4 x[4];
      uint32_t bits[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * kAdThreads;
        const int o = j * VW - a;                                  // tile offset of the vector's first element
        bits[u] = none ? 0u : kFull;
        if (j < nv && mrow) {
          const int v = t0 + o;                                    // may reach VW - 1 before the row
          const int w = max(v, 0) >> 5, sh = v - (w << 5);
          uint32_t lo = __ldg(mrow + w);
          const uint32_t hi = (sh + VW > 32 && w + 1 < p.W) ? __ldg(mrow + w + 1) : 0u;
          bits[u] = (sh >= 0 ? __funnelshift_r(lo, hi, sh) : lo << -sh) & kFull;
        }
        const bool whole = o >= 0 && o + VW <= n;
        if (j < nv && whole && bits[u] != 0u && (p.copy || bits[u] != kFull))
          x[u] = __ldcs(reinterpret_cast<const uint4*>(src + (size_t)j * VW));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * kAdThreads;
        if (j >= nv || (!p.copy && bits[u] == kFull)) continue;
        const int o = j * VW - a;
        if (o >= 0 && o + VW <= n) {
          if (bits[u] == 0u) {
            x[u] = make_uint4(TR::kPadWord, TR::kPadWord, TR::kPadWord, TR::kPadWord);
          } else if (bits[u] != kFull) {
#pragma unroll
            for (int t = 0; t < VW; ++t)
              if (!((bits[u] >> t) & 1u)) TR::put(x[u], t, Elem<T>::kNegInf);
          }
          __stcs(reinterpret_cast<uint4*>(dst + (size_t)j * VW), x[u]);
        } else {
          for (int t = 0; t < VW; ++t) {
            if (o + t < 0 || o + t >= n) continue;
            const bool ok = (bits[u] >> t) & 1u;
            if (ok && !p.copy) continue;
            Elem<T>::store_raw(dst + (size_t)j * VW + t,
                               ok ? Elem<T>::raw(src + (size_t)j * VW + t) : Elem<T>::kNegInf);
          }
        }
      }
    }
  }
  if (!sparse) return;
  __syncthreads();   // the counts are complete, and the rows written

  // ---- the listed tokens of every row
  const int nl = nlist;
  if (nl == 0) return;
  const float rep = p.repetition ? __ldg(p.repetition + b) : 1.f;
  const float freq = p.frequency ? __ldg(p.frequency + b) : 0.f;
  const float pres = p.presence ? __ldg(p.presence + b) : 0.f;
  const long long items = (long long)nl * (gb + 1);
  for (long long it = tid; it < items; it += kAdThreads) {
    const int i = (int)(it / nl);
    const int o = list[(int)(it - (long long)i * nl)];
    const uint32_t w = cnt[o];
    int c = (int)(w & kAdCount);
    if (w & kAdDraft)
      for (int j = 0; j < i; ++j) c += (sdraft[j] == t0 + o);
    const bool seen = (w & kAdPrompt) || c > 0;
    if (!seen && !(w & kAdBias)) continue;
    const size_t row = (size_t)b * p.G1 + i;
    if (p.mask) {
      const int mi = p.mask_index ? __ldg(p.mask_index + row) : (int)row;
      const int v = t0 + o;
      if (mi >= p.M || (mi >= 0 && !((__ldg(p.mask + (size_t)mi * p.W + (v >> 5)) >> (v & 31)) & 1u))) continue;
    }
    const size_t e = row * (size_t)p.V + t0 + o;
    float x = Elem<T>::load(static_cast<const T*>(p.logits) + e);
    if (seen) {
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      x -= fmaf(freq, (float)c, c > 0 ? pres : 0.f);
    }
    if (w & kAdBias) {
      int last = -1;
      for (int k = 0; k < nb; ++k)
        if (blist[k].x == o) last = max(last, blist[k].y);
      x += __ldg(p.bias_values + (size_t)b * p.NB + last);
    }
    Elem<T>::store(static_cast<T*>(p.out) + e, x);
  }
}

}  // namespace rows
}  // namespace sv
