// Attention of a round's rows over the 4-bit cache (sv_attend_kv4).
//
// A head's block of a page gives a key as k = s n + o (codes n, scale s,
// offset o), a value as v = s' n' + o'.  Scale and offset belong to a whole
// row, so they never touch the codes:
//   q . k_t       = s_t (q . n_t) + o_t sum_d q_d
//   sum_t p_t v_t = sum_t (p_t s'_t) n'_t + sum_t p_t o'_t
// and both contractions run on the codes themselves.  Four bits of a word,
// masked where they lie, are a float16 subnormal: 0x000f of a half is n 2^-24,
// 0x00f0 is n 2^-20 (both exact, and the tensor cores take subnormals as they
// are), so a word of eight codes becomes four operand registers with one shift
// and four ANDs.  The factor 16 of every second register is taken out of q, or
// out of the sums at the end.  q is brought to float16 with a power of two per
// row, p_t s'_t with one per warp; the sums are float32.
//
// Work: the (sequence, head, row tile)s' tokens in units of 64 are one line of
// units; CTA i of W takes an equal part of it, finds its place from lengths
// and walks on.  Four warps of a CTA take 16 tokens of a unit each, with a
// softmax and sums of their own, and are joined at the end of the segment.  A
// segment that a CTA does not hold in full goes to the workspace;
// attend_join_kernel, which is launched right behind, joins these in order.
#pragma once

#include <float.h>

#include "sv_kv4.cuh"

namespace sv {
namespace cache {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kAtUnit = 64;               // tokens of a unit: 16 a warp
constexpr int kAtJoinThreads = 128;
constexpr float kAtSlack = 8.f;           // a row's reference may be 2^8 below its largest term
constexpr float kAtValueTop = 128.f;      // largest p s' 2^x / 2^slack: their product stays below float16's 65504

struct AttendParams {
  int B, rows, H, G, page, pages, N;      // rows: gamma + 1
  const void* q;
  long long qs[3];                        // strides: batch, row, head
  const unsigned char* cache;
  const int32_t *table, *lengths, *gamma_b;
  float scale;                            // softmax scale * log2(e)
  void* out;
  float* lse;
  int fill;
  float* part;                            // [2 W][TR * D sums, TR references, TR masses]
  int4* desc;                             // [W]: sequence, head, row tile, last CTA; -1: nothing to join
};

// Floats of a part of TR rows.
__host__ __device__ constexpr int part_floats(int TR, int D) { return TR * (D + 2); }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Tokens that rows of sequence b may see, its rows, and how they are cut.
struct Sequence {
  int rows, seen, tiles, chunks;          // row tiles; units a (head, row tile)
  int first;                              // tokens that row 0 sees, before the limit of the table
  __device__ __forceinline__ Sequence(const AttendParams& p, int b, int TR) {
    rows = p.gamma_b ? min(max(p.gamma_b[b], -1), p.rows - 1) + 1 : p.rows;
    first = (int)min((long long)max(p.lengths[b], 0) + 1, 0x7fffff00ll);
    seen = (int)min((long long)first + rows - 1, (long long)p.N * p.page);
    tiles = (rows * p.G + TR - 1) / TR;
    chunks = max(1, (seen + kAtUnit - 1) / kAtUnit);
  }
  __device__ __forceinline__ long long units(int H) const { return (long long)H * tiles * chunks; }
};

// 16 tokens of one head as a lane holds them (g = lane / 4, c = lane % 4), for
// the groups of eight tokens j = 0, 1: the key codes of token 8 j + g, quarter
// c; the value codes of tokens 8 j + 2 c and + 1, eighth g; those two tokens'
// numbers.
template <int KW>
struct Codes {
  uint32_t k[2][KW], v[2][KW];
  uint4 n[2];
};
template <int KW>
__device__ __forceinline__ void load_words(uint32_t (&w)[KW], const unsigned char* at) {
  if constexpr (KW == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(at));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(at));
  }
}
// block: the head's block of the page; t: the 16 tokens' first in the page
template <int D>
__device__ __forceinline__ void load_codes(Codes<D / 32>& x, const unsigned char* block, int t, int page, int g, int c) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    load_words(x.k[j], block + (t + 8 * j + g) * (D / 2) + c * (D / 8));
    load_words(x.v[j], block + page * (D / 2) + ((t >> 1) + 4 * j + c) * D + g * (D / 8));
    uint32_t n[4];
    load_words(n, block + page * D + (t + 8 * j + 2 * c) * 8);
    x.n[j] = make_uint4(n[0], n[1], n[2], n[3]);
  }
}

template <typename T, int D, int MT>
struct AttendShape {
  static constexpr int TR = 16 * MT;      // rows of a tile
  static constexpr int kSmem = kAtWarps * (TR * D + 2 * TR) * 4;
};

// Position of a group of four channels (dg) of row r in a warp's sums in
// shared memory: lanes that write at once go to different banks.
__device__ __forceinline__ int swizzled(int r, int dg) { return dg ^ ((dg >> 3) | (r & 1) << 2); }

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kAtThreads, MT == 1 ? 3 : 2) attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int KW = D / 32, TR = 16 * MT;
  extern __shared__ float at_sm[];
  __shared__ long long warp_units[kAtWarps];
  __shared__ long long found_base;
  __shared__ int found_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();

  // rows behind a sequence's last
  if (p.fill && p.gamma_b) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      const int from = min(max(p.gamma_b[b], -1), p.rows - 1) + 1;
      const long long r0 = (long long)b * p.rows + from, r1 = (long long)(b + 1) * p.rows;
      const int HG = p.H * p.G;
      for (long long x = r0 * HG * (D / 8) + tid; x < r1 * HG * (D / 8); x += kAtThreads)
        static_cast<uint4*>(p.out)[x] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (long long x = r0 * HG + tid; x < r1 * HG; x += kAtThreads) p.lse[x] = 0.f;
    }
  }

  // all units, and those of the sequences before each thread's run
  const int run = (p.B + kAtThreads - 1) / kAtThreads;
  const int b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += Sequence(p, b, TR).units(p.H);
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += x;
  }
  if (lane == 31) warp_units[warp] = upto;
  __syncthreads();
  long long U = 0;
#pragma unroll
  for (int w = 0; w < kAtWarps; ++w) {
    if (w < warp) upto += warp_units[w];
    U += warp_units[w];
  }
  const long long W = min((long long)gridDim.x, U);
  const int me = blockIdx.x;
  if (me >= W) {
    if (tid == 0) p.desc[me] = make_int4(-1, 0, 0, 0);
    return;
  }
  long long u = U * me / W;
  const long long end = U * (me + 1) / W;
  if (u >= upto - mine && u < upto) {
    long long base = upto - mine;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long n = Sequence(p, b, TR).units(p.H);
      if (u < base + n) break;
      base += n;
    }
    found_b = b;
    found_base = base;
  }
  __syncthreads();
  int b = found_b;
  long long base = found_base;
  if (tid == 0) p.desc[me] = make_int4(-1, 0, 0, 0);

  const long long block_bytes = (long long)p.page * kTokenBytes<D>;
  const int page_tiles = p.page / 16;
  while (u < end) {
    const Sequence s(p, b, TR);
    const long long n_units = s.units(p.H);
    if (u >= base + n_units) {
      base += n_units;
      ++b;
      continue;
    }
    const int at = (int)((u - base) / s.chunks), chunk0 = (int)(u - base - (long long)at * s.chunks);
    const int h = at / s.tiles, rt = at - h * s.tiles;
    const int chunks = (int)min((long long)(s.chunks - chunk0), end - u);

    // ---- the rows: q as float16 fragments, a power of two per row apart
    uint32_t qf[MT][2 * KW][4];
    float row_scale[MT][2], q_sum[MT][2], ref[MT][2], mass[MT][2], shift[MT][2];
    int limit[MT][2];                     // last position that the row sees
    float o[MT][4 * KW][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rt * TR + m * 16 + e * 8 + g, i = r / p.G;
        const bool there = i < s.rows;
        uint4 x[KW];
#pragma unroll
        for (int j = 0; j < KW; ++j) x[j] = make_uint4(0, 0, 0, 0);
        if (there) {
          const T* row = static_cast<const T*>(p.q) + b * p.qs[0] + i * p.qs[1] + (long long)(h * p.G + r - i * p.G) * p.qs[2];
#pragma unroll
          for (int j = 0; j < KW; ++j) x[j] = __ldg(reinterpret_cast<const uint4*>(row) + c * KW + j);
        }
        float f[KW][8], top = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            f[j][2 * t] = Kv<T>::lo(w[t]);
            f[j][2 * t + 1] = Kv<T>::hi(w[t]);
            top = fmaxf(top, fmaxf(fabsf(f[j][2 * t]), fabsf(f[j][2 * t + 1])));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^up * top in [2^13, 2^14)
        const int up = top > 0.f ? min(140 - (int)(__float_as_uint(top) >> 23), 126) : 0;
        const float raise = __uint_as_float((uint32_t)(up + 127) << 23);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            f[j][t] *= raise;
            sum += f[j][t];
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            qf[m][2 * j + t][e] = half2_bits(f[j][2 * t], f[j][2 * t + 4]);
            qf[m][2 * j + t][2 + e] = half2_bits(f[j][2 * t + 1] * 0.0625f, f[j][2 * t + 5] * 0.0625f);
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        q_sum[m][e] = sum * 0x1p-24f;       // in the units of the products with the codes
        row_scale[m][e] = p.scale * 0x1p24f * __uint_as_float((uint32_t)(127 - up) << 23);
        ref[m][e] = -FLT_MAX;
        mass[m][e] = shift[m][e] = 0.f;
        limit[m][e] = there ? min(s.first - 1 + i, s.seen - 1) : -1;
      }
#pragma unroll
      for (int t = 0; t < 4 * KW; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[m][t][x] = 0.f;
    }
    float value_scale = 0x1p126f;         // what p s' is multiplied by, a power of two

    // ---- this warp's groups of 16 tokens
    const int last = min((chunk0 + chunks) * (kAtUnit / 16), (s.seen + 15) / 16);
    const int first = chunk0 * (kAtUnit / 16) + warp;
    const int every = s.first;            // positions below it are seen by every row of the sequence
    int ahead = 0;                        // page of this lane's group of the next 32
    auto look = [&](int t) {
      const int mine_t = t + lane * kAtWarps;
      ahead = mine_t < last ? __ldg(p.table + (long long)b * p.N + mine_t / page_tiles) : -1;
      if (ahead >= p.pages) ahead = -1;
    };
    Codes<KW> next;
    int next_page = -1;
    if (first < last) {
      look(first);
      next_page = __shfl_sync(0xffffffffu, ahead, 0);
      if (next_page >= 0)
        load_codes<D>(next, p.cache + ((long long)next_page * p.H + h) * block_bytes, (first % page_tiles) * 16, p.page, g, c);
    }
    int turn = 0;
    for (int t = first; t < last; t += kAtWarps) {
      const Codes<KW> x = next;
      const int page = next_page;
      const int tn = t + kAtWarps;
      if (tn < last) {
        if (++turn == 32) {
          turn = 0;
          look(tn);
        }
        next_page = __shfl_sync(0xffffffffu, ahead, turn);
        if (next_page >= 0)
          load_codes<D>(next, p.cache + ((long long)next_page * p.H + h) * block_bytes, (tn % page_tiles) * 16, p.page, g, c);
      }
      if (page < 0) continue;

      // scores: q . n for 16 tokens
      float z[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[m][j][e] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t k = x.k[j][w] >> (8 * half);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(z[m][j], qf[m][2 * w + half], k & 0x000f000fu, k & 0x00f000f0u);
          }

      // the four tokens' numbers: [j][which of the two]
      float ks[2][2], ko[2][2], vs[2][2], vo[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ks[j][0] = Kv<T>::lo(x.n[j].x);
        ko[j][0] = Kv<T>::hi(x.n[j].x);
        vs[j][0] = Kv<T>::lo(x.n[j].y);
        vo[j][0] = Kv<T>::hi(x.n[j].y);
        ks[j][1] = Kv<T>::lo(x.n[j].z);
        ko[j][1] = Kv<T>::hi(x.n[j].z);
        vs[j][1] = Kv<T>::lo(x.n[j].w);
        vo[j][1] = Kv<T>::hi(x.n[j].w);
      }
      const bool masked = t * 16 + 16 > every;
      if (masked) {
        // numbers of tokens that nobody sees may be anything
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (t * 16 + 8 * j + 2 * c + e >= s.seen) ks[j][e] = ko[j][e] = vs[j][e] = vo[j][e] = 0.f;
      }
      float most = -FLT_MAX, largest = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) largest = fmaxf(largest, vs[j][e]);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = fmaf(z[m][j][e], ks[j][e & 1], ko[j][e & 1] * q_sum[m][e >> 1]);
            if (masked && t * 16 + 8 * j + 2 * c + (e & 1) > limit[m][e >> 1]) y = __int_as_float(0xff800000);
            z[m][j][e] = y;
            most = fmaxf(most, fmaf(y, row_scale[m][e >> 1], -ref[m][e >> 1]));
          }
      if (__any_sync(0xffffffffu, most > kAtSlack || largest * value_scale > kAtValueTop)) {
        // a row's terms outgrow its reference, or the values' scales theirs
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        float by = 1.f;
        if (largest * value_scale > kAtValueTop) {
          // largest < 2^(e - 126): 2^(133 - e) brings it below 2^7
          const int e = (int)(__float_as_uint(largest) >> 23);
          const float to = __uint_as_float((uint32_t)min(max(133 - e + 127, 1), 253) << 23);
          by = to / value_scale;
          value_scale = to;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(z[m][0][2 * e], z[m][0][2 * e + 1]), fmaxf(z[m][1][2 * e], z[m][1][2 * e + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float now = fmaxf(ref[m][e], top * row_scale[m][e]);
            const float f = ex2_approx(ref[m][e] - now);
            ref[m][e] = now;
            mass[m][e] *= f;
            shift[m][e] *= f;
            const float fv = f * by;
#pragma unroll
            for (int n = 0; n < 4 * KW; ++n) {
              o[m][n][2 * e] *= fv;
              o[m][n][2 * e + 1] *= fv;
            }
          }
      }
      float vn[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) vn[j][e] = vs[j][e] * value_scale;

      // weights, as the second product's left operand
      uint32_t pf[MT][4];
      uint32_t pl[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y = z[m][j][2 * r + e];
              const float w = ex2_approx(fmaf(y, row_scale[m][r], -ref[m][r]));
              mass[m][r] += w;
              if (masked) {
                const bool sees = t * 16 + 8 * j + 2 * c + e <= limit[m][r];
                shift[m][r] += sees ? w * vo[j][e] : 0.f;
                a[e] = sees ? w * vn[j][e] : 0.f;
              } else {
                shift[m][r] = fmaf(w, vo[j][e], shift[m][r]);
                a[e] = w * vn[j][e];
              }
            }
            pf[m][2 * j + r] = half2_bits(a[0], a[1]);
            if constexpr (std::is_same<T, __half>::value) {
              // a float16 result wants more than float16 weights: their rest
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&pf[m][2 * j + r]));
              pl[m][2 * j + r] = half2_bits(a[0] - back.x, a[1] - back.y);
            }
          }

      // sums over the 16 tokens, eight channels at a time
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t v0 = x.v[0][w] >> (8 * half), v1 = x.v[1][w] >> (8 * half);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma16816(o[m][4 * w + 2 * half], pf[m], v0 & 0x000f000fu, v1 & 0x000f000fu);
            mma16816(o[m][4 * w + 2 * half + 1], pf[m], v0 & 0x00f000f0u, v1 & 0x00f000f0u);
            if constexpr (std::is_same<T, __half>::value) {
              mma16816(o[m][4 * w + 2 * half], pl[m], v0 & 0x000f000fu, v1 & 0x000f000fu);
              mma16816(o[m][4 * w + 2 * half + 1], pl[m], v0 & 0x00f000f0u, v1 & 0x00f000f0u);
            }
          }
        }
    }

    // ---- the warps' sums side by side in shared memory
    float* sums = at_sm + warp * (TR * D + 2 * TR);
    const float down = 1.f / value_scale;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = m * 16 + e * 8 + g;
        float l = mass[m][e], f = shift[m][e];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        f += __shfl_xor_sync(0xffffffffu, f, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        f += __shfl_xor_sync(0xffffffffu, f, 2);
        if (c == 0) {
          sums[TR * D + r] = ref[m][e];
          sums[TR * D + TR + r] = l;
        }
#pragma unroll
        for (int col = 0; col < 2; ++col)
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const int dg = (2 * c + col) * KW + w;   // channels 4 dg ..
            float y[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              y[n] = fmaf(o[m][4 * w + n][2 * e + col] * (n & 1 ? 0x1p20f : 0x1p24f), down, f);
            reinterpret_cast<float4*>(sums)[r * (D / 4) + swizzled(r, dg)] = make_float4(y[0], y[1], y[2], y[3]);
          }
      }
    __syncthreads();
    const bool whole = chunk0 == 0 && chunks == s.chunks;
    float* part = p.part + (size_t)(2 * me + (chunk0 == 0)) * part_floats(TR, D);
    for (int x = tid; x < TR * (D / 4); x += kAtThreads) {
      const int r = x / (D / 4), dg = x % (D / 4), at_r = r * (D / 4) + swizzled(r, dg);
      float top = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float m = at_sm[w * (TR * D + 2 * TR) + TR * D + r];
        top = m > top || m != m ? m : top;
      }
      float l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float* sw = at_sm + w * (TR * D + 2 * TR);
        const float f = ex2_approx(sw[TR * D + r] - top);
        const float4 a = reinterpret_cast<const float4*>(sw)[at_r];
        l = fmaf(f, sw[TR * D + TR + r], l);
        y.x = fmaf(f, a.x, y.x);
        y.y = fmaf(f, a.y, y.y);
        y.z = fmaf(f, a.z, y.z);
        y.w = fmaf(f, a.w, y.w);
      }
      if (!whole) {
        reinterpret_cast<float4*>(part)[x] = y;
        if (dg == 0) {
          part[TR * D + r] = top;
          part[TR * D + TR + r] = l;
        }
        continue;
      }
      const int rr = rt * TR + r, i = rr / p.G;
      if (i >= s.rows) continue;
      const long long q_row = ((long long)b * p.rows + i) * p.H * p.G + (long long)h * p.G + (rr - i * p.G);
      const float over = l == 0.f ? 0.f : 1.f / l;
      reinterpret_cast<uint2*>(p.out)[q_row * (D / 4) + dg] =
          make_uint2(Kv<T>::pack(y.x * over, y.y * over), Kv<T>::pack(y.z * over, y.w * over));
      if (p.lse && dg == 0) p.lse[q_row] = l == 0.f ? __int_as_float(0xff800000) : (top + log2f(l)) * 6.931471805599453e-01f;
    }
    __syncthreads();
    if (!whole && chunk0 == 0 && tid == 0) {
      // the segment's last unit is CTA ((x + 1) W - 1) / U's
      const long long x = base + (long long)at * s.chunks + s.chunks - 1;
      p.desc[me] = make_int4(b, h, rt, (int)(((x + 1) * W - 1) / U));
    }
    u += chunks;
  }
}

// Joins the parts of the segment that begins in CTA blockIdx.x's range and
// ends behind it: its own second part, then the first parts of those behind.
template <typename T, int D, int TR>
__global__ void __launch_bounds__(kAtJoinThreads) attend_join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 0) return;
  const int b = d.x, h = d.y, rt = d.z, last = d.w;
  const Sequence s(p, b, TR);
  for (int x = blockIdx.y * kAtJoinThreads + threadIdx.x; x < TR * (D / 4); x += gridDim.y * kAtJoinThreads) {
    const int r = x / (D / 4), dg = x % (D / 4), rr = rt * TR + r, i = rr / p.G;
    if (i >= s.rows) continue;
    float top = -FLT_MAX;
    for (int a = blockIdx.x; a <= last; ++a) {
      const float m = p.part[(size_t)(2 * a + (a == (int)blockIdx.x)) * part_floats(TR, D) + TR * D + r];
      top = m > top || m != m ? m : top;
    }
    float l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int a = blockIdx.x; a <= last; ++a) {
      const float* part = p.part + (size_t)(2 * a + (a == (int)blockIdx.x)) * part_floats(TR, D);
      const float f = ex2_approx(part[TR * D + r] - top);
      const float4 v = reinterpret_cast<const float4*>(part)[x];
      l = fmaf(f, part[TR * D + TR + r], l);
      y.x = fmaf(f, v.x, y.x);
      y.y = fmaf(f, v.y, y.y);
      y.z = fmaf(f, v.z, y.z);
      y.w = fmaf(f, v.w, y.w);
    }
    const long long q_row = ((long long)b * p.rows + i) * p.H * p.G + (long long)h * p.G + (rr - i * p.G);
    const float over = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(p.out)[q_row * (D / 4) + dg] =
        make_uint2(Kv<T>::pack(y.x * over, y.y * over), Kv<T>::pack(y.z * over, y.w * over));
    if (p.lse && dg == 0) p.lse[q_row] = l == 0.f ? __int_as_float(0xff800000) : (top + log2f(l)) * 6.931471805599453e-01f;
  }
}

}  // namespace cache
}  // namespace sv
