// Attention of many rows over the 4-bit cache: both contractions on the fifth
// generation tensor cores, with the codes as the operand in tensor memory.
//
// With R rows of a sequence and head (gamma + 1 times the query heads of a
// group), 128 tokens are one step:
//   scores^T [128 tokens x R] = codes of the keys [128 x D] . q^T
//   sums^T   [D x R]         += (codes of the values)^T [D x 128] . weights^T
// The codes are the left operand, so the tensor cores' time grows with R (a
// multiple of 16), not with a padded tile, and the codes go from registers to
// tensor memory: shared memory could not take them in and give them out again
// at this rate.  q and the weights, the small sides, are in shared memory.
// The formulas are those of sv_attend.cuh.  A tensor core cuts off what lies
// below its sum's last bits, so sums of n >= 0 would lose more and more over a
// long sequence: half of the tokens are taken as n - 15 (the sign bit and the
// complement, in the same AND and XOR), and their offset as o' + 15 s'.
//
// Eight warps do everything in turn, two CTAs per SM fill each other's waits.
// In a step (1) the step's value codes go to tensor memory; (2) the scores, whose
// product was issued a step ahead, become weights in shared memory against a
// reference per row; (3) the next step's key codes follow, then the one barrier,
// behind which one warp issues the next scores' product and another the sums'.
// Where a term outgrows its row's reference by 2^8 (a segment's first step,
// hardly ever later) the barrier says so to all, and the step's weights are
// formed again; a warp whose terms have not has formed its masses for good.
//
// Tensor memory, 256 columns a CTA: key codes, value codes, scores, sums.  With
// R = 80 and D = 128 the value codes take the place of the scores: then (1)
// follows (2)'s reading of them, at a barrier more, where the references are
// settled before the weights, and the next scores wait for this step's sums:
// scores, barrier, value codes and weights, barrier, sums follow one another.  (For
// fewer rows settling first took longer: 99, 112 and 123 us where 87, 100 and 114 at
// 32, 40 and 56 rows.)
//
// What bounds it: instructions, not bytes.  32 sequences of up to 8192 tokens, 8
// heads of 128 (32 us of bytes) take 88, 103, 121 and 145 us at 32, 40, 56 and 72
// rows (float16 results, with each value product and each store of weights twice:
// 93, 110, 129 and 169); the schedulers issue in 58 and 52 % of the cycles at 40
// and 72, with two CTAs of eight warps an SM, which wait for one another at the
// barrier, and no pipe is busy in more than 44 %.  Their 128 registers a thread do
// not hold 56 rows and more (72 to 200 bytes a thread are spilled).  A product of
// N <= 80 columns takes its issuing warp about 42 cycles, whatever N.  What was
// slower when it was tried:
// copies in bulk (a warp's lanes issue one in 75 cycles: 138 us where 116 at 32
// rows), a ninth warp for the products (96 registers a thread: 255 us where 222
// at 72 rows), a fourth step in the ring (97.5 us where 96.2 at 40 rows).
#pragma once

#include "sv_attend.cuh"

namespace sv {
namespace cache {

constexpr int kWdThreads = 256;
constexpr int kWdScoreWarp = 1, kWdSumWarp = 6;   // warps that also issue the first and the second product
constexpr int kWdAskWarp = 3;        // looks pages up
constexpr int kWdUnit = 128;         // tokens of a step
constexpr int kWdColumns = 256;      // of tensor memory
constexpr int kWdMostRows = 80;
constexpr int kWdPatience = 1 << 14; // tries of a wait, of up to 0.1 ms each

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 16 lanes: register 2 n + e of thread (g, c) goes to lane 8 e + g, column 4 n + c
__device__ __forceinline__ void tm_store_16x128(uint32_t at, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
      "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
      "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tm_store_16x128(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 lanes, 8 columns: thread (g, c) gets columns 2 c, 2 c + 1 of lane g, then of lane 8 + g
__device__ __forceinline__ void tm_load_16x256(float (&v)[4], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(at));
}
// 32 lanes, 8 columns: a thread has its lane's
__device__ __forceinline__ void tm_load_32x8(float (&v)[8], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(at));
}
__device__ __forceinline__ void tm_store_32x8(uint32_t at, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
// d [128 x N] (+)= a [128 x 16] . b [N x 16]^T, float16 in, float32 sums
__device__ __forceinline__ void tm_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tm_commit(uint32_t barrier) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(barrier) : "memory");
}
// A K-major operand in shared memory: rows of 128 bytes, 16-byte pieces
// exchanged by the row's number (the 128-byte swizzle), eight rows each 1 KB.
__device__ __forceinline__ uint64_t smem_operand(uint32_t at) {
  return (uint64_t)(at >> 4 & 0x3fff) | 1ull << 16 | 64ull << 32 | 1ull << 46 | 2ull << 61;
}

// A wait that ends: where the phase does not come, *gave_up is set for the
// whole CTA, whose later waits are short and whose rows become NaN.
__device__ __forceinline__ bool phase_there(uint32_t barrier, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(barrier), "r"(parity), "r"(100000u) : "memory");
  return done != 0;
}
static __device__ __noinline__ void wait_longer(uint32_t barrier, uint32_t parity, volatile int* gave_up) {
  bool done = false;
  for (int i = 0; i < kWdPatience && !done; ++i) {
    done = phase_there(barrier, parity);
    if (!done && i >= 64 && *gave_up) break;
  }
  if (!done) *gave_up = 1;
}
__device__ __forceinline__ void wait_phase(uint32_t barrier, uint32_t parity, volatile int* gave_up) {
  if (!__all_sync(0xffffffffu, phase_there(barrier, parity))) {
    wait_longer(barrier, parity, gave_up);
    __syncwarp();
  }
}

// The transposes of four 8 x 8 matrices of 16-bit elements: matrix i's row j
// goes to the address that lane 8 i + j gives.
__device__ __forceinline__ void store_transposed(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// NG: R / 16; each half of the warps (a warpgroup) has the softmax of NG
// groups of eight rows.
template <typename T, int D, int NG>
struct WideShape {
  static constexpr int R = 16 * NG;
  static constexpr bool kFine = std::is_same<T, __half>::value;   // the weights' rest is an operand too
  // a step in the ring: eight groups of 16 tokens (subs), their keys, their
  // values and their numbers; the padding sends subs to different banks
  static constexpr int kSubKeys = 8 * D, kSubValues = 8 * D + 16, kSubNumbers = 128 + 16;
  static constexpr int oValues = 8 * kSubKeys, oNumbers = oValues + 8 * kSubValues, kStage = oNumbers + 8 * kSubNumbers;
  static constexpr int kQ = R * D * 2, kP = R * kWdUnit * 2;
  // steps in the ring: three (a fourth gained nothing: 97.5 against 96.2 us for 40
  // rows), or the two that the CTAs have room for
  static constexpr int oP = kQ, oRing = oP + (kFine ? 2 : 1) * kP;
  static constexpr int kRoom = (112 * 1024 - 1024 - R * 19 * 4 - 8 - oRing) / kStage;
  static constexpr int kStages = kRoom < 3 ? kRoom : 3;
  static constexpr int oSmall = oRing + kStages * kStage;
  // row pairs' sums of q and references [4 R / 2], factor, tops [4], masses
  // [4], shifts [4], scales; limits; rows of the output
  static constexpr int kSmall = R * 19 * 4 + 8;
  static constexpr int kSmem = oSmall + kSmall + 1024;            // (aligned to 1 KB in the kernel)
  static constexpr bool kTight = D / 2 + 64 + 2 * R > kWdColumns;
  static constexpr int cV = D / 2, cS = kTight ? cV : cV + 64, cO = cS + R;
  static_assert(kStages >= (kTight ? 2 : 3), "a step's keys are read while the one before is at work");
  static_assert(!kTight || R >= 64, "value codes in the scores' place");
  static_assert(cO + R <= kWdColumns, "tensor memory");
  static_assert(R <= kWdMostRows, "rows");
  static_assert(2 * (kSmem + 2048) <= 228 * 1024, "two CTAs an SM");
};

template <typename T, int D, int NG>
__global__ void __launch_bounds__(kWdThreads, 2) attend_wide_kernel(const __grid_constant__ AttendParams p) {
  using S = WideShape<T, D, NG>;
  constexpr int R = S::R, KW = D / 32, RH = 8 * NG, LANES = D / 8;
  extern __shared__ unsigned char wd_raw[];
  __shared__ uint32_t tm_base;
  __shared__ __align__(8) unsigned long long bars[2];
  __shared__ unsigned long long places[2][32];
  __shared__ uint32_t place_subs[4];
  __shared__ int gave_up_flag, settled_flag;
  __shared__ float warp_top[8];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), w = warp & 3, wg = warp >> 2;   // (the compiler sees that a warp shares it)
  const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(wd_raw), sm = (sm0 + 1023u) & ~1023u;
  unsigned char* const sp = wd_raw + (sm - sm0);
  float4* const pairs = reinterpret_cast<float4*>(sp + S::oSmall);   // rows 2 i, 2 i + 1: sums of q, references below 0
  float* const factor = reinterpret_cast<float*>(pairs) + 2 * R;
  float* const tops = factor + R;
  float* const masses = tops + 4 * R;
  float* const shifts = masses + 4 * R;
  float* const row_scales = shifts + 4 * R;
  int* const limits = reinterpret_cast<int*>(row_scales + R);
  long long* const out_rows = reinterpret_cast<long long*>(limits + R);
  volatile int* const gave_up = &gave_up_flag;
  volatile int* const settled = &settled_flag;   // the segment's rows have their references
  // scores there, sums there
  const uint32_t bar_s = (uint32_t)__cvta_generic_to_shared(&bars[0]), bar_o = bar_s + 8;
  pdl_launch_dependents();

  fill_behind<T, D, kWdThreads>(p);
  const Part line = find_part(p, R, kWdUnit);
  if (!line.some()) return;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"((uint32_t)__cvta_generic_to_shared(&tm_base)),
                 "n"(kWdColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    gave_up_flag = 0;
    asm volatile("mbarrier.init.shared.b64 [%0], 1;\n\tmbarrier.init.shared.b64 [%1], 1;" ::"r"(bar_s), "r"(bar_o) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = tm_base, tm_w = tm + ((uint32_t)(32 * w) << 16);
  const uint32_t kind = 1u << 4 | (uint32_t)(R >> 3) << 17 | (128u >> 4) << 24;
  const uint64_t q_operand = smem_operand(sm), p_operand = smem_operand(sm + S::oP);
  uint32_t phase_s = 0, phase_o = 0;     // of the next wait
  int slot = 0, slot_to = 0;             // of the ring: the step's, the next to fill

  const long long block_bytes = (long long)p.page * kTokenBytes<D>;
  const int page_tiles = p.page / 16, me = blockIdx.x;
  long long u = line.u, base = line.base;
  int b = line.b;

  auto score_products = [&]() {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      tm_mma(tm + S::cS, tm + 8 * k, q_operand + (uint64_t)((k >> 2) * (R * 8) + (k & 3) * 2), kind, k > 0);
    tm_commit(bar_s);
  };
  auto first_product = [&]() {
    if (warp == kWdScoreWarp) {
      if (lane == 0) {
        tm_fence_after();
        score_products();
      }
      __syncwarp();
    }
  };
  // this thread's places in a step's keys and values
  const uint32_t keys_at = 2 * (g >> 1) * S::kSubKeys + (2 * (2 * w + wg) + (g & 1)) * (D / 2) + c * (D / 8);
  const uint32_t values_at = S::oValues + 2 * c * S::kSubValues + 4 * wg * D + 4 * (8 * w + g);
  // key codes of a step: the warpgroup's 16 lanes.  Lane 32 w + 16 bl + 8 e + g
  // is token 2 (2 w + bl) + g % 2 of sub 2 (g / 2) + e: the four pairs of tokens
  // of a piece of eight lanes are in four subs, in different banks
  auto keys = [&](int from_slot) {
    const uint32_t stage = sm + S::oRing + from_slot * S::kStage;
    uint32_t v[8 * KW];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t k[KW];
      shared_words(k, stage + keys_at + e * S::kSubKeys);
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        v[8 * j + e] = k[j] & 0x000f000fu;
        v[8 * j + 2 + e] = k[j] & 0x00f000f0u;
        v[8 * j + 4 + e] = k[j] >> 8 & 0x000f000fu;
        v[8 * j + 6 + e] = k[j] >> 8 & 0x00f000f0u;
      }
    }
    tm_store_16x128(tm_w + ((uint32_t)(16 * wg) << 16), v);
  };

  while (u < line.end) {
    const Sequence s(p, b, R, kWdUnit);
    const long long n_units = s.units(p.H);
    if (u >= base + n_units) {
      base += n_units;
      ++b;
      continue;
    }
    const Segment segment = segment_at(s, u, base, line.end);
    const int h = segment.h, rt = segment.rt, chunk0 = segment.chunk0, chunks = segment.chunks;
    u += segment.step;
    if (chunks == 0) continue;
    const int sub_end = (s.seen + 15) / 16;

    // ---- the ring: a warp copies a sub of a step.  Where a sub begins, its
    // number in the page in the low four bits (0: hidden), is looked up for
    // four steps (32 subs) at a time, by every warp for the first four, later by
    // one of them for all, two times four steps ahead.
    auto ask = [&](int q, int& sub) {
      const int mine = (chunk0 + 4 * q) * 8 + lane;
      if (mine >= sub_end) return -1;
      const int x = mine / page_tiles;
      sub = mine - x * page_tiles;
      return __ldg(p.table + (long long)b * p.N + x);
    };
    auto place_of = [&](int id, int sub) {
      return (uint32_t)id < (uint32_t)p.pages
                 ? reinterpret_cast<unsigned long long>(p.cache) +
                       (unsigned long long)(((long long)id * p.H + h) * block_bytes + sub * (8 * D + 1)) : 0ull;
    };
    auto tell = [&](int q, unsigned long long place) {
      places[q & 1][lane] = place;
      const uint32_t bits = __ballot_sync(0xffffffffu, place != 0);
      if (lane == 0) place_subs[q & 3] = bits;
    };
    int sub0 = 0, sub1 = 0, asked = -1, asked_sub = 0;
    const int id0 = ask(0, sub0);
    const int id1 = warp == kWdAskWarp ? ask(1, sub1) : -1;
    // q is on its way meanwhile: a thread's pieces of eight channels
    constexpr int PIECES = (R * LANES + kWdThreads - 1) / kWdThreads;
    uint4 qv[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const int x = tid + k * kWdThreads, rl = x / LANES, r = rt * R + rl, i = r / p.G;
      qv[k] = make_uint4(0, 0, 0, 0);
      if (rl < R && i < s.rows)
        qv[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + b * p.qs[0] + i * p.qs[1] +
                                                     (long long)(h * p.G + r - i * p.G) * p.qs[2]) + x % LANES);
    }
    auto copy_sub = [&](int x, unsigned long long from) {
      const bool here = from != 0;
      const int sub = (int)(from & 15);
      const unsigned char* codes = reinterpret_cast<const unsigned char*>(from - sub) + lane * 16;
      const uint32_t to = sm + S::oRing + slot_to * S::kStage + lane * 16;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        copy_ahead_if(here, to + x * S::kSubKeys + j * 512, codes + j * 512);
        copy_ahead_if(here, to + S::oValues + x * S::kSubValues + j * 512, codes + p.page * (D / 2) + j * 512);
      }
      copy_ahead_if(here && lane < 8, to + S::oNumbers + x * S::kSubNumbers, codes + p.page * D - sub * (8 * D - 128));
    };
    {
      const unsigned long long place = place_of(id0, sub0);
#pragma unroll
      for (int n = 0; n < S::kStages; ++n) {
        const unsigned long long from = __shfl_sync(0xffffffffu, place, 8 * n + warp);
        if (n < chunks) {
          copy_sub(warp, from);
          slot_to = slot_to + 1 == S::kStages ? 0 : slot_to + 1;
        }
        copies_end_group();
      }
      if (warp == kWdAskWarp) {
        tell(0, place);
        tell(1, place_of(id1, sub1));
      }
    }
    // (warps 1 and 6 are busy with the products; 2 and 5 take one sub more)
    auto copy_step = [&](int n) {
      if (n < chunks) {
        const unsigned long long* place = places[n >> 2 & 1] + (n & 3) * 8;
        if (warp != kWdScoreWarp && warp != kWdSumWarp) copy_sub(warp, place[warp]);
        if (warp == 2) copy_sub(kWdScoreWarp, place[kWdScoreWarp]);
        if (warp == 5) copy_sub(kWdSumWarp, place[kWdSumWarp]);
        slot_to = slot_to + 1 == S::kStages ? 0 : slot_to + 1;
      }
      copies_end_group();
    };

    if (S::kTight && tid == 0) *settled = 0;
    // ---- q: float16 with a power of two per row, channels in the order in
    // which the key codes come: element 2 (c + 4 (4 k + i)) + e is channel 8 (KW
    // c + k) + i + 4 e, halves e of pair i of word k
    {
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int x = tid + k * kWdThreads, rl = x / LANES, word = x % LANES;
        const uint32_t ww[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
        float f[8], top = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = Kv<T>::lo(ww[j]);
          f[2 * j + 1] = Kv<T>::hi(ww[j]);
          top = max3(top, fabsf(f[2 * j]), fabsf(f[2 * j + 1]));
          sum += f[2 * j] + f[2 * j + 1];
        }
#pragma unroll
        for (int m = LANES / 2; m >= 1; m >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, m);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        }
        if (rl >= R) continue;
        const int up = raised_by(top);
        const float raise = __uint_as_float((uint32_t)(up + 127) << 23);
        if (word == 0) {
          const int r = rt * R + rl, i = r / p.G;
          float* pair = reinterpret_cast<float*>(pairs + (rl >> 1)) + (rl & 1);
          pair[0] = sum * raise * 0x1p-24f;      // (the products' unit is 2^-24 of a code)
          pair[2] = 0.f;
          row_scales[rl] = times_power(p.scale, 24 - up);
          limits[rl] = i < s.rows ? min(s.first - 1 + i, s.seen - 1) : -1;
          out_rows[rl] = i < s.rows ? ((long long)b * p.rows + i) * p.H * p.G + (long long)h * p.G + (r - i * p.G) : -1;
        }
        const int cc = word / KW, kk = word % KW;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float t = j & 1 ? raise * 0.0625f : raise;
          const int piece = 4 * kk + j;
          *reinterpret_cast<uint32_t*>(sp + (piece >> 3) * (R * 128) + rl * 128 + (((piece & 7) ^ (rl & 7)) << 4) + 4 * cc) =
              half2_bits(f[j] * t, f[j + 4] * t);
        }
      }
    }
    copies_wait<S::kStages - 1>();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    keys(slot);
    tm_wait_st();
    copies_wait<S::kStages - 2>();
    tm_fence_before();
    __syncthreads();
    first_product();

    // this thread's rows, two at a time: 8 k + 2 c, + 1 of its warpgroup's
    Two mass[NG], shift[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) mass[k] = shift[k] = two(0.f, 0.f);
    float4* const my_pairs = pairs + wg * (RH / 2) + c;      // (+ 4 k)
    float value_scale = 0x1p126f;
    // No step so far had a sub that is there.  (With R = 80 and D = 128, where
    // registers are short, in shared memory: 141 us for 72 rows, and 149; for fewer
    // rows that takes longer, 87, 101 and 117 us where 85, 98 and 114.)
    bool none = true;
    const unsigned short half_range = w < 2 ? kMinusHalfRange : kHalfRange;

    for (int n = 0; n < chunks; ++n) {
      const uint32_t stage = sm + S::oRing + slot * S::kStage;
      const uint32_t subs = place_subs[n >> 2 & 3] >> ((n & 3) * 8) & 0xffu;
      const int slot_next = slot + 1 == S::kStages ? 0 : slot + 1;
      const bool fresh = S::kTight ? n == 0 || *settled == 0 : none;
      if (!S::kTight && n > 0) {
        wait_phase(bar_o, phase_o, gave_up);
        phase_o ^= 1;
        tm_fence_after();
      }

      // value codes: the warpgroup's 64 tokens.  Unit 8 w + g of a pair is
      // channels 4 (8 w + g) .., which go to lanes 16 (i / 2) + 8 (i % 2) + g
      auto values = [&](uint32_t column) {
        if (32 * w >= D) return;
        const uint32_t flip = wg ? 0x800f800fu : 0u, flip16 = wg ? 0x80f080f0u : 0u;
        uint32_t v0[16], v1[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t x;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x)
                       : "r"(stage + values_at + (i & 1) * S::kSubValues + (i >> 1) * D) : "memory");
          v0[2 * i] = (x & 0x000f000fu) ^ flip;
          v0[2 * i + 1] = (x & 0x00f000f0u) ^ flip16;
          v1[2 * i] = (x >> 8 & 0x000f000fu) ^ flip;
          v1[2 * i + 1] = (x >> 8 & 0x00f000f0u) ^ flip16;
        }
        tm_store_16x128(tm_w + column, v0);
        tm_store_16x128(tm_w + (16u << 16) + column, v1);
      };
      if (!S::kTight) values(S::cV + 32 * wg);
      wait_phase(bar_s, phase_s, gave_up);
      phase_s ^= 1;
      tm_fence_after();

      // (3) weights; the thread's tokens are those of lanes 16 bl + 8 e + g
      const int token0 = (chunk0 + n) * kWdUnit + 32 * (g >> 1) + 4 * w + (g & 1);      // + 16 e + 2 bl
      const uint32_t numbers_at = stage + S::oNumbers + 2 * (g >> 1) * S::kSubNumbers + (4 * w + (g & 1)) * 8;
      auto softmax = [&](auto masked_step) {
        constexpr bool kMasked = decltype(masked_step)::value;
        const bool unsettled = (kMasked || !S::kTight) && fresh;
        // whether rows 8 k + 2 c and + 1 see token (bl, e)
        auto sees = [&](int k, int bl, int e) {
          const int2 lim = *reinterpret_cast<const int2*>(limits + wg * RH + 8 * k + 2 * c);
          const int t = subs >> (2 * (g >> 1) + e) & 1 ? token0 + 16 * e + 2 * bl : 0x7fffffff;
          return make_int2(t <= lim.x, t <= lim.y);
        };
        uint32_t nk[2][2], nv[2][2];       // the tokens' numbers: key's, value's
#pragma unroll
        for (int bl = 0; bl < 2; ++bl)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t x[2];
            shared_words(x, numbers_at + e * S::kSubNumbers + bl * 16);
            // (those of tokens that nobody sees may be anything)
            if (kMasked && (token0 + 16 * e + 2 * bl >= s.seen || !(subs >> (2 * (g >> 1) + e) & 1))) x[0] = x[1] = 0;
            nk[bl][e] = x[0];
            nv[bl][e] = x[1];
          }
        float z[2][NG][4];
        auto exponents = [&]() {
#pragma unroll
          for (int bl = 0; bl < 2; ++bl)
#pragma unroll
            for (int k = 0; k < NG; ++k) tm_load_16x256(z[bl][k], tm_w + ((uint32_t)(16 * bl) << 16) + S::cS + wg * RH + 8 * k);
          tm_wait_ld();
          float most = -FLT_MAX;
          Two ks[2][2], ko[2][2];
#pragma unroll
          for (int bl = 0; bl < 2; ++bl)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = Kv<T>::lo(nk[bl][e]), o = Kv<T>::hi(nk[bl][e]);
              ks[bl][e] = two(a, a);
              ko[bl][e] = two(o, o);
            }
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            const float4 pair = my_pairs[4 * k];
            const float2 scale = *reinterpret_cast<const float2*>(row_scales + wg * RH + 8 * k + 2 * c);
            const Two q = two(pair.x, pair.y), r = two(pair.z, pair.w), f = two(scale.x, scale.y);
#pragma unroll
            for (int bl = 0; bl < 2; ++bl)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const Two y = fma2(fma2(two(z[bl][k][2 * e], z[bl][k][2 * e + 1]), ks[bl][e], mul2(ko[bl][e], q)), f, r);
                float y0, y1;
                split(y, y0, y1);
                if (kMasked) {
                  const int2 see = sees(k, bl, e);
                  if (!see.x) y0 = __int_as_float(0xff800000);
                  if (!see.y) y1 = __int_as_float(0xff800000);
                }
                most = max3(most, y0, y1);
                z[bl][k][2 * e] = y0;
                z[bl][k][2 * e + 1] = y1;
              }
          }
          return most;
        };
        // `by` times what weights() adds to the shifts for the middles of the
        // values' rows (not kFine): the weights of z as operands, times -+7.5
        auto centre = [&](float by) {
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            float c0 = 0.f, c1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int bl = j >> 1, e = j & 1;
              const float n_x = Kv<T>::lo(nv[bl][e]) * value_scale;
              float a0, a1;
              split(mul2(two(ex2_approx(z[bl][k][2 * e]), ex2_approx(z[bl][k][2 * e + 1])), two(n_x, n_x)), a0, a1);
              if (kMasked) {
                const int2 see = sees(k, bl, e);
                if (!see.x) a0 = 0.f;
                if (!see.y) a1 = 0.f;
              }
              add_product(c0, c1, half2_bits(a0, a1), half_range);
            }
            shift[k] = fma2(two(c0, c1), two(by, by), shift[k]);
          }
        };
        // (a warp whose terms have not outgrown their references has formed its
        // part of the masses for good: a reference that moves scales it)
        auto weights = [&](bool first) {
          // the weights of row r: 128 bytes for tokens 0 .. 63, and for the others
          const uint32_t to = sm + S::oP + (w >> 1) * (R * 128) + (wg * RH + (lane & 7)) * 128 +
                              ((((w & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
          Two vn[2][2], vo[2][2];
#pragma unroll
          for (int bl = 0; bl < 2; ++bl)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = Kv<T>::lo(nv[bl][e]), n_x = x * value_scale;
              const float o_x = fmaf(S::kFine ? w < 2 ? 0.f : 15.f : 7.5f, x, Kv<T>::hi(nv[bl][e]));
              vn[bl][e] = two(n_x, n_x);
              vo[bl][e] = two(o_x, o_x);
            }
          const float down = 1.f / value_scale;
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            uint32_t a[4], rest[4];
            float c0 = 0.f, c1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int bl = j >> 1, e = j & 1;
              const Two wt = two(ex2_approx(z[bl][k][2 * e]), ex2_approx(z[bl][k][2 * e + 1]));
              float a0, a1;
              split(mul2(wt, vn[bl][e]), a0, a1);
              if (kMasked) {
                // (a hidden token's numbers may be NaN)
                const int2 see = sees(k, bl, e);
                if (!see.x) a0 = 0.f;
                if (!see.y) a1 = 0.f;
                float f0, f1;
                split(mul2(wt, vo[bl][e]), f0, f1);
                if (!see.x) f0 = 0.f;
                if (!see.y) f1 = 0.f;
                if (first) {
                  mass[k] = add2(mass[k], wt);
                  shift[k] = add2(shift[k], two(f0, f1));
                }
              } else if (first) {
                mass[k] = add2(mass[k], wt);
                shift[k] = fma2(wt, vo[bl][e], shift[k]);
              }
              a[j] = half2_bits(a0, a1);
              if (S::kFine) {
                // a float16 result wants more than float16 weights: their rest
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&a[j]));
                rest[j] = half2_bits(a0 - back.x, a1 - back.y);
              } else {
                add_product(c0, c1, a[j], half_range);
              }
            }
            if (!S::kFine) shift[k] = fma2(two(c0, c1), two(down, down), shift[k]);
            store_transposed(to + k * 1024, a[0], a[1], a[2], a[3]);
            if (S::kFine) store_transposed(to + S::kP + k * 1024, rest[0], rest[1], rest[2], rest[3]);
          }
        };

        // everybody's operands are there, and the copies of a later step
        auto meet = [&](bool any) {
          tm_wait_st();
          copies_wait<S::kTight ? S::kStages - 2 : S::kStages - 3>();
          tm_fence_before();
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          return __syncthreads_or(any);
        };
        float largest = fmaxf(fmaxf(Kv<T>::lo(nv[0][0]), Kv<T>::lo(nv[0][1])), fmaxf(Kv<T>::lo(nv[1][0]), Kv<T>::lo(nv[1][1])));
        bool again = true, outgrown = true;
        if (n > 0 || S::kTight) {
          const float most = exponents();
          outgrown = unsettled || __any_sync(0xffffffffu, most > kAtSlack || largest * value_scale > kAtValueTop);
          if (!S::kTight) {
            if (!outgrown) weights(true);
            if (n + 1 < chunks) keys(slot_next);
          }
          again = meet(outgrown);
        }
        if (again) {
          // rows' references and the values' scale move; so do the sums.  The
          // first step with a sub that is there sets the references (they were
          // 0): a row that sees none of it sees none of the later ones, its mass
          // stays 0.
          if (S::kTight && unsettled && subs != 0 && tid == 0) *settled = 1;
          if (!S::kTight) {
            exponents();
            if (!S::kFine && !outgrown) centre(-1.f / value_scale);   // (they come with the weights formed again)
          }
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            float t0 = fmaxf(fmaxf(z[0][k][0], z[0][k][2]), fmaxf(z[1][k][0], z[1][k][2]));
            float t1 = fmaxf(fmaxf(z[0][k][1], z[0][k][3]), fmaxf(z[1][k][1], z[1][k][3]));
#pragma unroll
            for (int m = 4; m <= 16; m <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, m));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, m));
            }
            if (g == 0) *reinterpret_cast<float2*>(tops + w * R + wg * RH + 8 * k + 2 * c) = make_float2(t0, t1);
          }
          largest = fmaxf(largest, 0.f);
#pragma unroll
          for (int m = 16; m >= 1; m >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, m));
          if (lane == 0) warp_top[warp] = largest;
          __syncthreads();
#pragma unroll
          for (int j = 0; j < 8; ++j) largest = fmaxf(largest, warp_top[j]);
          float by = 1.f;
          if (largest * value_scale > kAtValueTop) {
            const int e = (int)(__float_as_uint(largest) >> 23);
            const float to = __uint_as_float((uint32_t)min(max(133 - e + 127, 1), 253) << 23);
            by = to / value_scale;
            value_scale = to;
          }
          // a row's terms move down by `up`
          auto rise = [&](float t) {
            return !unsettled ? fmaxf(t, 0.f) : t == __int_as_float(0xff800000) ? 0.f : t;
          };
#pragma unroll
          for (int k = 0; k < NG; ++k) {
            float up0 = __int_as_float(0xff800000), up1 = up0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 t = *reinterpret_cast<const float2*>(tops + j * R + wg * RH + 8 * k + 2 * c);
              up0 = fmaxf(up0, t.x);
              up1 = fmaxf(up1, t.y);
            }
            up0 = rise(up0);
            up1 = rise(up1);
            const float f0 = !unsettled ? ex2_approx(-up0) : 0.f, f1 = !unsettled ? ex2_approx(-up1) : 0.f;
            mass[k] = mul2(mass[k], two(f0, f1));
            shift[k] = mul2(shift[k], two(f0, f1));
#pragma unroll
            for (int bl = 0; bl < 2; ++bl)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                z[bl][k][2 * e] -= up0;
                z[bl][k][2 * e + 1] -= up1;
              }
            if (w == 0 && g == 0) {
              // (a warp of its own reads and writes these two rows' references here)
              *reinterpret_cast<float2*>(factor + wg * RH + 8 * k + 2 * c) = make_float2(f0 * by, f1 * by);
              my_pairs[4 * k].z -= up0;
              my_pairs[4 * k].w -= up1;
            }
          }
          __syncthreads();
          if (n > 0) {
            for (int k = 0; k < NG; ++k) {
              float o[8];
              const uint32_t col = tm_w + S::cO + wg * RH + 8 * k;
              tm_load_32x8(o, col);
              tm_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= factor[wg * RH + 8 * k + j];
              tm_store_32x8(col, o);
            }
          }
          if (!S::kTight) {
            weights(outgrown);
            if (n == 0 && n + 1 < chunks) keys(slot_next);
            meet(false);
          }
        }
        if (S::kTight) {
          values(S::cV + 32 * wg);
          weights(true);
          if (n + 1 < chunks) keys(slot_next);
          meet(false);
        }
        if (warp == kWdSumWarp) {
          if (lane == 0) {
            tm_fence_after();
#pragma unroll
            for (int k = 0; k < kWdUnit / 16; ++k) {
              const uint64_t at_p = p_operand + (uint64_t)((k >> 2) * (R * 8) + (k & 3) * 2);
              tm_mma(tm + S::cO, tm + S::cV + 8 * k, at_p, kind, n > 0 || k > 0);
              if (S::kFine) tm_mma(tm + S::cO, tm + S::cV + 8 * k, at_p + S::kP / 16, kind, true);
            }
            tm_commit(S::kTight && n + 1 == chunks ? bar_s : bar_o);
          }
          __syncwarp();
          if (S::kTight && n + 1 < chunks) {
            // the next scores take the value codes' place, once these are read
            wait_phase(bar_o, phase_o, gave_up);
            phase_o ^= 1;
            if (lane == 0) score_products();
            __syncwarp();
          }
        }
        if (!S::kTight && n + 1 < chunks) first_product();
        copy_step(n + S::kStages);         // (everybody has read this step's)
        if (warp == kWdAskWarp) {
          // (what was told for these four steps has been read when this is told)
          if ((n & 3) == 0) asked = ask((n >> 2) + 2, asked_sub);
          if ((n & 3) == 2) tell((n >> 2) + 2, place_of(asked, asked_sub));
        }
      };
      if ((S::kTight && fresh) || subs != 0xffu || (chunk0 + n) * kWdUnit + kWdUnit > s.first) softmax(std::true_type{});
      else softmax(std::false_type{});
      none = none && subs == 0;
      slot = slot_next;
    }

    // ---- the rows' totals over the warps
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      float m0, m1, f0, f1;
      split(mass[k], m0, m1);
      split(shift[k], f0, f1);
#pragma unroll
      for (int m = 4; m <= 16; m <<= 1) {
        m0 += __shfl_xor_sync(0xffffffffu, m0, m);
        m1 += __shfl_xor_sync(0xffffffffu, m1, m);
        f0 += __shfl_xor_sync(0xffffffffu, f0, m);
        f1 += __shfl_xor_sync(0xffffffffu, f1, m);
      }
      if (g == 0) {
        const int r = wg * RH + 8 * k + 2 * c;
        *reinterpret_cast<float2*>(masses + w * R + r) = make_float2(m0, m1);
        *reinterpret_cast<float2*>(shifts + w * R + r) = make_float2(f0, f1);
        if (w == 0) {
          *reinterpret_cast<float2*>(tops + r) = make_float2(-my_pairs[4 * k].z, -my_pairs[4 * k].w);
        }
      }
    }
    if (S::kTight) {
      wait_phase(bar_s, phase_s, gave_up);
      phase_s ^= 1;
    } else {
      wait_phase(bar_o, phase_o, gave_up);
      phase_o ^= 1;
    }
    tm_fence_after();
    __syncthreads();
    const bool failed = *gave_up;
    const bool whole = chunk0 == 0 && chunks == s.chunks;
    float* part = p.part + (size_t)(2 * me + (chunk0 == 0)) * part_floats(R, D);
    if (tid < R) {
      // (the first of the four keeps the sum)
      const float l = masses[tid] + masses[R + tid] + masses[2 * R + tid] + masses[3 * R + tid];
      const float f = shifts[tid] + shifts[R + tid] + shifts[2 * R + tid] + shifts[3 * R + tid];
      const float top = failed ? __int_as_float(0x7fffffff) : l == 0.f ? -FLT_MAX : tops[tid];
      if (!whole) {
        part[R * D + tid] = top;
        part[R * D + R + tid] = l;
        factor[tid] = 1.f;
      } else {
        factor[tid] = failed ? top : l == 0.f ? 0.f : 1.f / l;
        const long long row = out_rows[tid];
        if (p.lse && row >= 0)
          p.lse[row] = failed ? top : l == 0.f ? __int_as_float(0xff800000) : (top + log2f(l)) * 6.931471805599453e-01f;
      }
      shifts[tid] = f;
    }
    __syncthreads();
    const float down = (lane & 8 ? 0x1p20f : 0x1p24f), scale_down = 1.f / value_scale;
    // lane 16 bl + 8 e + g of warp w is channel 4 (8 w + g) + 2 bl + e
    const int channel = 32 * w + 4 * (lane & 7) + (lane >> 3);
#pragma unroll 1
    for (int k = 0; k < NG; ++k) {
      float o[8];
      tm_load_32x8(o, tm_w + S::cO + wg * RH + 8 * k);
      tm_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = wg * RH + 8 * k + j;
        const long long row = out_rows[r];
        if (row < 0 || channel >= D) continue;
        const float y = fmaf(o[j] * down, scale_down, shifts[r]) * factor[r];
        if (!whole) part[r * D + channel] = y;
        else static_cast<unsigned short*>(p.out)[row * D + channel] = (unsigned short)Kv<T>::bits(y);
      }
    }
    if (!whole && chunk0 == 0 && tid == 0)
      p.desc[me] = make_int4(b, h, rt, line.owner(segment.last(s, base)));
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(kWdColumns));
}

}  // namespace cache
}  // namespace sv
