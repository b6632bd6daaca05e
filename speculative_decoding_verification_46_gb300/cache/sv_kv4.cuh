// The 4-bit cache's format (include/specverify_cache.h) and the kernels that
// write rows into it and read them back.
//
// A row of D elements is 8 elements a lane: D / 8 lanes (16 or 8) of a warp
// take a row, so a warp has 2 or 4 of them.  Least and greatest element by
// shuffles, then every lane forms its 8 codes: one word.
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

// One row's codes (8 of a lane's elements, 4 bits each from the low end) and
// its scale and offset as bits; LANES lanes hold the row.
template <typename T, int LANES>
__device__ __forceinline__ uint32_t quantise(const uint4& x, uint32_t& numbers) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w;
    f[2 * j] = Kv<T>::lo(w);
    f[2 * j + 1] = Kv<T>::hi(w);
  }
  float least = f[0], most = f[0], bad = f[0] - f[0];   // 0, or NaN where an element is not finite
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    least = fminf(least, f[j]);
    most = fmaxf(most, f[j]);
    bad += f[j] - f[j];
  }
#pragma unroll
  for (int m = LANES / 2; m >= 1; m >>= 1) {
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, m));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
    bad += __shfl_xor_sync(0xffffffffu, bad, m);
  }
  const uint32_t sb = Kv<T>::bits(__fdiv_rn(most - least, 15.f));
  const float scale = Kv<T>::lo(sb);
  if (!(scale + bad < __int_as_float(0x7f800000))) {   // not finite, or a NaN
    const uint32_t nan = Kv<T>::bits(__int_as_float(0x7fffffff));
    numbers = nan | nan << 16;
    return 0;
  }
  numbers = sb | Kv<T>::bits(least) << 16;
  const float inverse = scale < 1.17549435e-38f ? 0.f : __frcp_rn(scale);
  uint32_t codes = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // (the product is at least 0)
    const uint32_t n = __float2uint_rn(__fmul_rn(__fadd_rn(f[j], -least), inverse));
    codes |= min(n, 15u) << (4 * j);
  }
  return codes;
}

// Bytes from a block's start to the 8 codes of channels 8 l .. of token t.
template <int D>
__device__ __forceinline__ int key_at(int t, int l) { return t * (D / 2) + 4 * l; }
// (its first two bytes; the other two are 4 bytes on)
template <int D>
__device__ __forceinline__ int value_at(int page, int t, int l) { return page * (D / 2) + (t >> 1) * D + 8 * l + 2 * (t & 1); }
template <int D>
__device__ __forceinline__ int numbers_at(int page, int t) { return page * D + 8 * t; }

// A lane group of D / 8 lanes per (row, head): its key, then its value.
template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) append_kv4_kernel(const __grid_constant__ StoreParams p) {
  constexpr int LANES = D / 8;
  const long long item = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) / LANES;
  const int l = threadIdx.x % LANES;
  const long long items = (long long)p.R * p.H;
  const int r = item < items ? (int)(item / p.H) : 0, h = item < items ? (int)(item % p.H) : 0;
  const int slot = item < items ? p.slots[r] : -1;
  const bool there = slot >= 0 && slot < p.slots_end;
  if (!__any_sync(0xffffffffu, there)) return;
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (there) {
    const int b = r / p.rows, i = r - b * p.rows;
    xk = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + b * p.ks[0] + i * p.ks[1] + h * p.ks[2]) + l);
    xv = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + b * p.vs[0] + i * p.vs[1] + h * p.vs[2]) + l);
  }
  uint32_t nk, nv;
  const uint32_t ck = quantise<T, LANES>(xk, nk), cv = quantise<T, LANES>(xv, nv);
  if (!there) return;
  const int page = slot / p.page, t = slot - page * p.page;
  unsigned char* block = p.cache + ((long long)page * p.H + h) * ((long long)p.page * kTokenBytes<D>);
  *reinterpret_cast<uint32_t*>(block + key_at<D>(t, l)) = ck;
  unsigned char* at = block + value_at<D>(p.page, t, l);
  *reinterpret_cast<unsigned short*>(at) = (unsigned short)cv;
  *reinterpret_cast<unsigned short*>(at + 4) = (unsigned short)(cv >> 16);
  if (l == 0) *reinterpret_cast<uint2*>(block + numbers_at<D>(p.page, t)) = make_uint2(nk, nv);
}

template <typename T>
__device__ __forceinline__ uint4 held(uint32_t codes, uint32_t numbers) {
  const float scale = Kv<T>::lo(numbers), offset = Kv<T>::hi(numbers);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __fmaf_rn((float)(codes >> (4 * j) & 15u), scale, offset);
  return make_uint4(Kv<T>::pack(f[0], f[1]), Kv<T>::pack(f[2], f[3]), Kv<T>::pack(f[4], f[5]), Kv<T>::pack(f[6], f[7]));
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) read_kv4_kernel(const __grid_constant__ StoreParams p) {
  constexpr int LANES = D / 8;
  const long long item = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) / LANES;
  const int l = threadIdx.x % LANES;
  if (item >= (long long)p.R * p.H) return;
  const int r = (int)(item / p.H), h = (int)(item % p.H);
  const int slot = p.slots[r];
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (slot >= 0 && slot < p.slots_end) {
    const int page = slot / p.page, t = slot - page * p.page;
    const unsigned char* block = p.cache + ((long long)page * p.H + h) * ((long long)p.page * kTokenBytes<D>);
    const uint32_t ck = *reinterpret_cast<const uint32_t*>(block + key_at<D>(t, l));
    const unsigned char* at = block + value_at<D>(p.page, t, l);
    const uint32_t cv = *reinterpret_cast<const unsigned short*>(at) |
                        (uint32_t) * reinterpret_cast<const unsigned short*>(at + 4) << 16;
    const uint2 n = *reinterpret_cast<const uint2*>(block + numbers_at<D>(p.page, t));
    xk = held<T>(ck, n.x);
    xv = held<T>(cv, n.y);
  }
  __stcs(static_cast<uint4*>(p.ko) + item * LANES + l, xk);
  __stcs(static_cast<uint4*>(p.vo) + item * LANES + l, xv);
}

}  // namespace cache
}  // namespace sv
