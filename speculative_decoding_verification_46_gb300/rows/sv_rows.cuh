// Shared device code of the operators on logits rows (include/specverify_rows.h).
//
// A row of V elements at element offset r * V of a 16-byte aligned tensor
// starts at any element of a 16-byte vector when V is not a multiple of the
// vector width VW.  Every kernel here therefore walks a row through its
// window of aligned vectors: vector v of the window holds the row's elements
// v * VW - a0 .. v * VW - a0 + VW - 1, a0 = (r * V) % VW.  Whole vectors move
// as one 16-byte access; the first and the last, where they reach outside the
// row, element by element, so nothing outside the row is read or written.
#pragma once

#include "../csrc/sv_device.cuh"

namespace sv {
namespace rows {

// Bits of an element type's own lowest value: -inf.
template <typename T> struct Elem;
template <> struct Elem<float> {
  __device__ static __forceinline__ float of_raw(uint32_t r) { return __uint_as_float(r); }
  __device__ static __forceinline__ float load(const float* p) { return *p; }
  __device__ static __forceinline__ void store(float* p, float x) { *p = x; }
  __device__ static __forceinline__ uint32_t raw(const float* p) { return *reinterpret_cast<const uint32_t*>(p); }
  __device__ static __forceinline__ void store_raw(float* p, uint32_t x) { *reinterpret_cast<uint32_t*>(p) = x; }
  static constexpr uint32_t kNegInf = 0xff800000u;
  // VW rounded values packed into a vector
  __device__ static __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Elem<__nv_bfloat16> {
  __device__ static __forceinline__ float of_raw(uint32_t r) { return __uint_as_float(r << 16); }
  // the smallest value >= x, twice
  __device__ static __forceinline__ __nv_bfloat162 both_ru(float x) { return __bfloat162bfloat162(__float2bfloat16_ru(x)); }
  __device__ static __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
  __device__ static __forceinline__ uint32_t raw(const __nv_bfloat16* p) {
    return *reinterpret_cast<const unsigned short*>(p);
  }
  __device__ static __forceinline__ void store_raw(__nv_bfloat16* p, uint32_t x) {
    *reinterpret_cast<unsigned short*>(p) = (unsigned short)x;
  }
  static constexpr uint32_t kNegInf = 0xff80u;
  __device__ static __forceinline__ uint4 pack(const float* x) {
    uint4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * w], x[2 * w + 1]);
      set_word(v, w, *reinterpret_cast<const uint32_t*>(&h));
    }
    return v;
  }
};
template <> struct Elem<__half> {
  __device__ static __forceinline__ float of_raw(uint32_t r) { return __half2float(__ushort_as_half((unsigned short)r)); }
  __device__ static __forceinline__ __half2 both_ru(float x) { return __half2half2(__float2half_ru(x)); }
  __device__ static __forceinline__ float load(const __half* p) { return __half2float(*p); }
  __device__ static __forceinline__ void store(__half* p, float x) { *p = __float2half_rn(x); }
  __device__ static __forceinline__ uint32_t raw(const __half* p) { return *reinterpret_cast<const unsigned short*>(p); }
  __device__ static __forceinline__ void store_raw(__half* p, uint32_t x) {
    *reinterpret_cast<unsigned short*>(p) = (unsigned short)x;
  }
  static constexpr uint32_t kNegInf = 0xfc00u;
  __device__ static __forceinline__ uint4 pack(const float* x) {
    uint4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const __half2 h = __floats2half2_rn(x[2 * w], x[2 * w + 1]);
      set_word(v, w, *reinterpret_cast<const uint32_t*>(&h));
    }
    return v;
  }
};

// Element t (a compile-time index after unrolling) of a vector in float32.
template <typename T>
__device__ __forceinline__ uint32_t raw_of(const uint4& v, int t) {
  if (sizeof(T) == 4) return word_of(v, t);
  const uint32_t w = word_of(v, t >> 1);
  return (t & 1) ? (w >> 16) : (w & 0xffffu);
}

// A row's window of aligned vectors (P: T or const T).
template <typename T, typename P = T>
struct Window {
  P* base;   // first element of the window's first vector (16-byte aligned)
  int a0;    // elements of the window before the row
  int V;     // elements of the row
  __device__ __forceinline__ Window(P* tensor, size_t r, int V_) : V(V_) {
    const size_t e0 = r * (size_t)V_;
    a0 = (int)(e0 % Tr<T>::VW);
    base = tensor + (e0 - a0);
  }
  __device__ __forceinline__ int vectors() const { return (int)(((long long)a0 + V + Tr<T>::VW - 1) / Tr<T>::VW); }
  // whether vector v lies inside the row
  __device__ __forceinline__ bool whole(int v) const {
    const int t = v * Tr<T>::VW - a0;
    return t >= 0 && t + Tr<T>::VW <= V;
  }
  // vector v (0 <= v < vectors()); elements outside the row read as -inf.
  // Read once: the line is first in line to leave the caches.
  __device__ __forceinline__ uint4 load(int v) const {
    const T* p = base + (size_t)v * Tr<T>::VW;
    if (whole(v)) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint4 x = make_uint4(Tr<T>::kPadWord, Tr<T>::kPadWord, Tr<T>::kPadWord, Tr<T>::kPadWord);
#pragma unroll
    for (int t = 0; t < Tr<T>::VW; ++t) {
      const int e = v * Tr<T>::VW - a0 + t;
      if (e >= 0 && e < V) Tr<T>::put(x, t, Elem<T>::raw(p + t));
    }
    return x;
  }
  __device__ __forceinline__ void store(int v, const uint4& x) const {
    T* p = base + (size_t)v * Tr<T>::VW;
    if (whole(v)) {
      __stcs(reinterpret_cast<uint4*>(p), x);
      return;
    }
#pragma unroll
    for (int t = 0; t < Tr<T>::VW; ++t) {
      const int e = v * Tr<T>::VW - a0 + t;
      if (e >= 0 && e < V) Elem<T>::store_raw(p + t, raw_of<T>(x, t));
    }
  }
};

// ------------------------------------------------------------ paired float32
// Two float32 operations an instruction (add, multiply and multiply-add).

struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void unpair(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ Pair pair_fma(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
// Elements t and t + 1 of a vector (t even), and 2^(x c - rho) of both.
template <typename T>
__device__ __forceinline__ Pair pair_terms(const uint4& x, int t, Pair c, Pair minus_rho) {
  float a, b;
  unpair(pair_fma(pair_of(Tr<T>::get(x, t), Tr<T>::get(x, t + 1)), c, minus_rho), a, b);
  return pair_of(ex2_approx(a), ex2_approx(b));
}

// ------------------------------------------------------------ block reductions

template <int NW>
__device__ __forceinline__ float block_max_n(float v, float* sm) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = sm[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) t = fmaxf(t, sm[w]);
  return t;
}

__device__ __forceinline__ F2 warp_sum_f2(F2 v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v = f2_add(v, f2_shfl_xor(v, m));
  return v;
}

template <int NW>
__device__ __forceinline__ F2 block_sum_f2_n(F2 v, F2* sm) {
  v = warp_sum_f2(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  F2 t = sm[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) t = f2_add(t, sm[w]);
  return t;
}

template <int NW>
__device__ __forceinline__ int block_sum_int_w(int v, int* sm) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = sm[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) t += sm[w];
  return t;
}

// 2^((x - m) c) is formed as 2^(x c - rho), rho = m c rounded, one multiply-add
// and one exponential, where |rho| stays below this: rho is then off by at
// most half, which a factor common to all terms takes back (2^(rho - m c),
// its exponent from one multiply-add).  Beyond it
// (enormous logits or tiny temperatures) the difference is taken first.
constexpr float kNear = 8.0e6f;

// 2^((x - m) c) to about 44 bits, c = c.hi + c.lo; x <= m, either may be
// -inf (0 then).  The difference keeps its rounding error.
__device__ __forceinline__ F2 weight_f2(float x, float m, F2 c, const float* tab) {
  if (x == -INFINITY) return F2{0.f, 0.f};
  const float d = x - m;
  if (d * c.hi < -150.f) return F2{0.f, 0.f};   // also where the product leaves float32's range
  const float bb = d - x;
  const float de = (x - (d - bb)) + (-m - bb);
  const F2 y = exp2_f2(f2_mul(F2{d, de}, c), tab);
  return f2_norm(y.hi, y.lo);   // so that .hi alone is the rounded weight
}

// Sets the elements of x that are >= thr to -inf (thr may lie between two
// values of T; NaN stay).
template <typename T>
__device__ __forceinline__ void clear_ge(uint4& x, float thr) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (__uint_as_float(word_of(x, t)) >= thr) set_word(x, t, Elem<T>::kNegInf);
  } else {
    using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const P lim = Elem<T>::both_ru(thr);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t w = word_of(x, t);
      const uint32_t m = __hge2_mask(*reinterpret_cast<const P*>(&w), lim);
      set_word(x, t, (w & ~m) | (m & Tr<T>::kPadWord));
    }
  }
}

// Sums of weights 0 <= w <= 1 that come in any order: integers of 2^-50, so
// the sum does not depend on which thread met which term.
__device__ __forceinline__ unsigned long long weight_fixed(float w) { return (unsigned long long)(w * 1125899906842624.f); }
__device__ __forceinline__ F2 fixed_f2(unsigned long long s) {
  const float h = __ull2float_rz(s);
  const float l = __ull2float_rz(s - (unsigned long long)h);
  return F2{h * 8.8817841970012523e-16f, l * 8.8817841970012523e-16f};
}
template <int NW>
__device__ __forceinline__ unsigned long long block_sum_u64(unsigned long long v, unsigned long long* sm) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long t = sm[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) t += sm[w];
  return t;
}

__device__ __forceinline__ F2 f2_from(double d) {
  const float h = (float)d;
  return F2{h, (float)(d - (double)h)};
}

constexpr float kLog2eHi = 1.442695022e+00f, kLog2eLo = 1.925963033e-08f;

// ln a to about 40 bits, a a normalised two-float number >= 2^-100: a float
// logarithm y corrected by a e^-y - 1.
__device__ __forceinline__ F2 f2_log(F2 a, const float* tab) {
  const float y = logf(a.hi);
  const F2 e = exp2_f2(f2_mul(F2{-y, 0.f}, F2{kLog2eHi, kLog2eLo}), tab);
  const F2 r = f2_add(f2_mul(a, f2_norm(e.hi, e.lo)), F2{-1.f, 0.f});
  return f2_add(F2{y, 0.f}, f2_norm(r.hi, r.lo - 0.5f * r.hi * r.hi));
}

// a - b with its rounding error
__device__ __forceinline__ F2 two_diff(float a, float b) {
  const float d = a - b;
  const float bb = d - a;
  return F2{d, (a - (d - bb)) + (-b - bb)};
}

}  // namespace rows
}  // namespace sv
