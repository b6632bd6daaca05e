// The 4-bit cache's format (include/specverify_cache.h) and the kernels that
// write rows into it and read them back.
//
// Both move every byte once and are bound by HBM as long as a row costs few
// instructions.  D / 8 lanes (16 or 8) have eight channels each of two
// neighbouring rows of a head, so that a lane has four loads of 16 bytes on
// the way and, where the rows' slots are neighbours too, writes the two
// tokens' interleaved value codes as whole words.
//
// 8 x 4096 rows of 8 heads of 128, bf16, stored and read back: 59.6 us, 340 MB at
// 5.7 TB/s (85 % of a copy's rate); stored with a word for every two channels
// instead, 61.5; with a row at a time, one division and one reciprocal in every
// lane and float32 sums of codes, 90.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "../csrc/sv_device.cuh"

namespace sv {
namespace cache {

// Bytes of one token's key and value in a head's block: codes and numbers.
template <int D> constexpr int kTokenBytes = D + 8;

// The model's type: bits of an element to float32 and back.
template <typename T> struct Kv;
template <> struct Kv<__nv_bfloat16> {
  __device__ static __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  __device__ static __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  __device__ static __forceinline__ uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Kv<__half> {
  __device__ static __forceinline__ float lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
  __device__ static __forceinline__ float hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
  __device__ static __forceinline__ uint32_t bits(float x) { return __half_as_ushort(__float2half_rn(x)); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

struct StoreParams {
  int R, rows, H, page;          // rows: gamma + 1
  long long slots_end;           // pages * page
  const void *k, *v;             // append: inputs
  long long ks[3], vs[3];        // their strides: batch, row, head
  const int32_t* slots;
  unsigned char* cache;
  void *ko, *vo;                 // read: outputs
};

constexpr int kStoreThreads = 256;

// Elements two at a time.
template <typename T> struct Kv2;
template <> struct Kv2<__nv_bfloat16> {
  using V = __nv_bfloat162;
  // 128 + n for the codes n of 0x000f of both halves, less 128
  static constexpr uint32_t kMagic = 0x43004300u, kBase = 0x43004300u;
};
template <> struct Kv2<__half> {
  using V = __half2;
  static constexpr uint32_t kMagic = 0x64006400u, kBase = 0x64006400u;   // 1024 + n
};
template <typename V>
__device__ __forceinline__ V as_two(uint32_t x) { return *reinterpret_cast<const V*>(&x); }
template <typename V>
__device__ __forceinline__ uint32_t as_bits(V x) { return *reinterpret_cast<const uint32_t*>(&x); }

struct F2x {                         // two float32
  unsigned long long v;
};
__device__ __forceinline__ F2x f2x(float a, float b) {
  F2x p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void f2x_split(F2x p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ F2x f2x_add(F2x a, F2x b) {
  F2x d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2x f2x_fma(F2x a, F2x b, F2x c) {
  F2x d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

// The least element of a row and the least negative of one, side by side, in
// all of its LANES lanes; NaN stays.
template <typename T, int LANES>
__device__ __forceinline__ uint32_t ends_of(const uint4& x) {
  using V = typename Kv2<T>::V;
  const V lo2 = __hmin2_nan(__hmin2_nan(as_two<V>(x.x), as_two<V>(x.y)), __hmin2_nan(as_two<V>(x.z), as_two<V>(x.w)));
  const V hi2 = __hmax2_nan(__hmax2_nan(as_two<V>(x.x), as_two<V>(x.y)), __hmax2_nan(as_two<V>(x.z), as_two<V>(x.w)));
  const uint32_t a = as_bits(lo2), b = as_bits(hi2) ^ 0x80008000u;
  V both = __hmin2_nan(as_two<V>(__byte_perm(a, b, 0x5410)), as_two<V>(__byte_perm(a, b, 0x7632)));
#pragma unroll
  for (int m = LANES / 2; m >= 1; m >>= 1) both = __hmin2_nan(both, as_two<V>(__shfl_xor_sync(0xffffffffu, as_bits(both), m)));
  return as_bits(both);
}
// A row's scale and offset as bits, and what its elements are multiplied by;
// for a row that is held as NaN (an element is not finite, or the scale) NaN.
template <typename T>
__device__ __forceinline__ uint32_t numbers_of(uint32_t ends, float& inverse) {
  const float least = Kv<T>::lo(ends), most = -Kv<T>::hi(ends);
  const uint32_t sb = Kv<T>::bits(__fdiv_rn(most - least, 15.f));
  const float scale = Kv<T>::lo(sb);
  if (!(scale < __int_as_float(0x7f800000))) {
    const uint32_t nan = Kv<T>::bits(__int_as_float(0x7fffffff));
    inverse = 0.f;
    return nan | nan << 16;
  }
  inverse = scale < 1.17549435e-38f ? 0.f : __frcp_rn(scale);
  return sb | ends << 16;
}
// Codes of a lane's 8 elements, 4 bits each from the low end.
template <typename T>
__device__ __forceinline__ uint32_t codes_of(const uint4& x, uint32_t numbers, float inverse) {
  const float least = Kv<T>::hi(numbers);
  const F2x minus = f2x(-least, -least);
  // added and taken away again, 3 2^22 rounds to whole numbers, ties to even
  const F2x magic = f2x(12582912.f, 12582912.f), back = f2x(-12582912.f, -12582912.f);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  F2x c[4];                                      // codes i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = w[i >> 1], q = w[2 + (i >> 1)];
    const F2x f = i & 1 ? f2x(Kv<T>::hi(p), Kv<T>::hi(q)) : f2x(Kv<T>::lo(p), Kv<T>::lo(q));
    float y0, y1;
    f2x_split(f2x_add(f, minus), y0, y1);
    // (single products: paired ones are fused with the addition behind them,
    // which takes away their rounding)
    y0 = __fmul_rn(y0, inverse);
    y1 = __fmul_rn(y1, inverse);
    if (std::is_same<T, __half>::value) {
      // (a scale below the normal numbers may be rounded far down; others leave y below 15.5)
      y0 = fminf(y0, 15.f);
      y1 = fminf(y1, 15.f);
    }
    c[i] = f2x_add(f2x_add(f2x(y0, y1), magic), back);
  }
  const F2x k16 = f2x(16.f, 16.f);
  // (the sum of four codes' places stays exact)
  const F2x sum = f2x_add(f2x_fma(f2x_fma(f2x_fma(c[3], k16, c[2]), k16, c[1]), k16, c[0]), f2x(8388608.f, 8388608.f));
  float s0, s1;
  f2x_split(sum, s0, s1);
  return inverse > 0.f ? __byte_perm(__float_as_uint(s0), __float_as_uint(s1), 0x5410) : 0u;   // (0: NaN or constant rows)
}

// Bytes from a block's start to the 8 codes of channels 8 l .. of token t.
template <int D>
__device__ __forceinline__ int key_at(int t, int l) { return t * (D / 2) + 4 * l; }
// (its first two bytes; the other two are 4 bytes on)
template <int D>
__device__ __forceinline__ int value_at(int page, int t, int l) { return page * (D / 2) + (t >> 1) * D + 8 * l + 2 * (t & 1); }
template <int D>
__device__ __forceinline__ int numbers_at(int page, int t) { return page * D + 8 * t; }

// Where rows 2 i, 2 i + 1 of a lane group are.
struct RowPair {
  int r, h;                // first row, head
  int slot[2];             // -1: none
  int page[2], t[2];       // of the slots
  bool next;               // the second slot is the first one's odd neighbour
};
__device__ __forceinline__ RowPair row_pair(const StoreParams& p, uint32_t item) {
  RowPair x;
  const uint32_t i = item / (uint32_t)p.H;
  x.h = (int)(item - i * (uint32_t)p.H);
  x.r = 2 * (int)i;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int slot = x.r + j < p.R ? __ldg(p.slots + x.r + j) : -1;
    x.slot[j] = slot >= 0 && slot < p.slots_end ? slot : -1;
  }
  x.next = x.slot[0] >= 0 && (x.slot[0] & 1) == 0 && x.slot[1] == x.slot[0] + 1;
  x.page[0] = (int)((uint32_t)max(x.slot[0], 0) / (uint32_t)p.page);
  x.t[0] = x.slot[0] - x.page[0] * p.page;
  x.page[1] = x.page[0];
  x.t[1] = x.t[0] + 1;
  if (!x.next) {
    x.page[1] = (int)((uint32_t)max(x.slot[1], 0) / (uint32_t)p.page);
    x.t[1] = x.slot[1] - x.page[1] * p.page;
  }
  return x;
}
// (of a call's groups of D / 8 lanes, at most 2^31)
__device__ __forceinline__ uint32_t pair_items(const StoreParams& p) { return ((uint32_t)p.R + 1) / 2 * (uint32_t)p.H; }

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) append_kv4_kernel(const __grid_constant__ StoreParams p) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LANES;
  const uint32_t item = blockIdx.x * (kStoreThreads / LANES) + threadIdx.x / LANES;
  RowPair pair = row_pair(p, min(item, pair_items(p) - 1));
  if (item >= pair_items(p)) {
    pair.slot[0] = pair.slot[1] = -1;
    pair.next = false;
  }
  if (!__any_sync(0xffffffffu, pair.slot[0] >= 0 || pair.slot[1] >= 0)) return;
  uint4 x[4];                            // key, value of the first row, of the second
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = make_uint4(0, 0, 0, 0);
  {
    const int b = pair.r / p.rows, i = pair.r - b * p.rows;
    const long long ok = b * p.ks[0] + i * p.ks[1] + pair.h * p.ks[2], ov = b * p.vs[0] + i * p.vs[1] + pair.h * p.vs[2];
    const T *k = static_cast<const T*>(p.k) + ok + 8 * l, *v = static_cast<const T*>(p.v) + ov + 8 * l;
    if (pair.slot[0] >= 0) {
      x[0] = __ldcs(reinterpret_cast<const uint4*>(k));
      x[1] = __ldcs(reinterpret_cast<const uint4*>(v));
    }
    if (pair.slot[1] >= 0) {
      const bool same = i + 1 < p.rows;    // the sequence goes on
      k += same ? p.ks[1] : p.ks[0] - i * p.ks[1];
      v += same ? p.vs[1] : p.vs[0] - i * p.vs[1];
      x[2] = __ldcs(reinterpret_cast<const uint4*>(k));
      x[3] = __ldcs(reinterpret_cast<const uint4*>(v));
    }
  }
  uint32_t ends[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) ends[j] = ends_of<T, LANES>(x[j]);
  // the division and the reciprocal of row j in lanes j, j + 4 .. alone
  float inverse;
  const uint32_t numbers = numbers_of<T>((lane & 2) ? (lane & 1) ? ends[3] : ends[2] : (lane & 1) ? ends[1] : ends[0], inverse);
  uint32_t n[4], codes[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = __shfl_sync(0xffffffffu, numbers, (lane & ~3) | j);
    codes[j] = codes_of<T>(x[j], n[j], __shfl_sync(0xffffffffu, inverse, (lane & ~3) | j));
  }
  const int block_bytes = p.page * kTokenBytes<D>;
  if (pair.next) {
    const int t = pair.t[0];
    unsigned char* block = p.cache + (long long)((uint32_t)pair.page[0] * (uint32_t)p.H + pair.h) * block_bytes;
    uint32_t* key = reinterpret_cast<uint32_t*>(block + key_at<D>(t, l));
    key[0] = codes[0];
    key[D / 8] = codes[2];
    *reinterpret_cast<uint2*>(block + value_at<D>(p.page, t, l)) =
        make_uint2(__byte_perm(codes[1], codes[3], 0x5410), __byte_perm(codes[1], codes[3], 0x7632));
    if (l == 0) *reinterpret_cast<uint4*>(block + numbers_at<D>(p.page, t)) = make_uint4(n[0], n[1], n[2], n[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (pair.slot[j] < 0) continue;
    const int t = pair.t[j];
    unsigned char* block = p.cache + (long long)((uint32_t)pair.page[j] * (uint32_t)p.H + pair.h) * block_bytes;
    *reinterpret_cast<uint32_t*>(block + key_at<D>(t, l)) = codes[2 * j];
    unsigned char* at = block + value_at<D>(p.page, t, l);
    *reinterpret_cast<unsigned short*>(at) = (unsigned short)codes[2 * j + 1];
    *reinterpret_cast<unsigned short*>(at + 4) = (unsigned short)(codes[2 * j + 1] >> 16);
    if (l == 0) *reinterpret_cast<uint2*>(block + numbers_at<D>(p.page, t)) = make_uint2(n[2 * j], n[2 * j + 1]);
  }
}

// Eight elements from their codes; scale * code + offset rounds once.
template <typename T>
__device__ __forceinline__ uint4 held(uint32_t codes, uint32_t numbers) {
  using V = typename Kv2<T>::V;
  const V scale = as_two<V>(__byte_perm(numbers, numbers, 0x1010)), offset = as_two<V>(__byte_perm(numbers, numbers, 0x3232));
  uint32_t y[4];                                 // elements i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const V n = __hsub2(as_two<V>((codes >> (4 * i) & 0x000f000fu) | Kv2<T>::kMagic), as_two<V>(Kv2<T>::kBase));
    y[i] = as_bits(__hfma2(n, scale, offset));
  }
  return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                    __byte_perm(y[2], y[3], 0x7632));
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) read_kv4_kernel(const __grid_constant__ StoreParams p) {
  constexpr int LANES = D / 8;
  const int l = threadIdx.x % LANES;
  const uint32_t item = blockIdx.x * (kStoreThreads / LANES) + threadIdx.x / LANES;
  if (item >= pair_items(p)) return;
  const RowPair pair = row_pair(p, item);
  uint32_t ck[2] = {0, 0}, cv[2] = {0, 0};
  uint2 n[2] = {make_uint2(0, 0), make_uint2(0, 0)};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (pair.slot[j] < 0) continue;
    const int t = pair.t[j];
    const unsigned char* block = p.cache + ((long long)pair.page[j] * p.H + pair.h) * ((long long)p.page * kTokenBytes<D>);
    ck[j] = *reinterpret_cast<const uint32_t*>(block + key_at<D>(t, l));
    if (!pair.next) {
      const unsigned char* at = block + value_at<D>(p.page, t, l);
      cv[j] = *reinterpret_cast<const unsigned short*>(at) | (uint32_t) * reinterpret_cast<const unsigned short*>(at + 4) << 16;
    } else if (j == 0) {
      const uint2 x = *reinterpret_cast<const uint2*>(block + value_at<D>(p.page, t, l));
      cv[0] = __byte_perm(x.x, x.y, 0x5410);
      cv[1] = __byte_perm(x.x, x.y, 0x7632);
    }
    n[j] = *reinterpret_cast<const uint2*>(block + numbers_at<D>(p.page, t));
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (pair.r + j >= p.R) continue;
    // (without a slot: codes, scale and offset 0)
    const long long at = ((long long)(pair.r + j) * p.H + pair.h) * LANES + l;
    __stcs(static_cast<uint4*>(p.ko) + at, held<T>(ck[j], n[j].x));
    __stcs(static_cast<uint4*>(p.vo) + at, held<T>(cv[j], n[j].y));
  }
}

}  // namespace cache
}  // namespace sv
