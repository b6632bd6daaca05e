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
// row, p_t s'_t with one per warp; the sums are float32.  (The warp's power of two
// brings the largest s' so far to [2^6, 2^7): what float16's last bit, 2^-24, cuts
// off a weight is below 2^-25 15 s' / 2^6, about 2^-30 of the largest value.)
//
// A tensor core cuts off what lies below its sum's last bits, so sums of codes
// n >= 0 would lose more and more over a long sequence: every second group of
// eight tokens is taken as n - 15 (the sign bit and the complement, in the same
// AND and XOR), and its offset as o' + 15 s'.
//
// Rounding p s' to float16 would cost a bfloat16 result |n| or |n - 15| times
// the rounding, about 8 s' p, were its offset's term p o' formed from p as it
// is.  So the middle of the row, o' + 7.5 s', is taken with p, and the rest with
// the rounded weight r: r n' +- 7.5 r (-7.5 for n, 7.5 for n - 15), which leaves
// |n - 7.5|, about 3 (errors against 64 bits, 48 sequences of 6000 tokens:
// 0.001673 where 0.001751; rounding the exact result gives 0.001660).  A second
// operand for the weights' rest, as float16 results have it, would take out
// that too (0.001660), in 81 us where 67 for 20 rows and 219 where 182 for 16
// rows of 240,000 tokens; formed from p alone they took 63 and 174.
//
// Tokens and channels are the products' left side and the rows their right one,
// so that eight rows cost half of what sixteen do: scores^T [16 tokens x 8 rows]
// = codes . q^T, sums^T [16 channels x 8 rows] += (value codes)^T . weights^T.  A
// lane then has two tokens of every 16 and two rows of every eight: it reads two
// tokens' numbers and no others.  (When it was turned round: with the rows on the
// left, a lane has a row and numbers of four tokens, 8 rows took 60 us and 50 this
// way, 24 rows 88 and 79, 128 sequences of 4096 tokens 116 and 87.)
//
// Two ways to share the work out.  attend_joined (sv_attend_plan.h) chooses.
// Few segments, which are (sequence, head, row tile)s, over a short table: a
// cluster of eight CTAs a segment deals its 32-token groups out to its warps, and
// the CTAs read each other's sums from shared memory.  One launch: one request of
// 700 tokens, 8 heads of 128, takes 4.8 us, and 8.7 us the other way; a round of
// gamma 8 on 8 x 8 heads and up to 4096 tokens 13 us, and 25 in the kernel for
// many rows.
// Otherwise: the segments' tokens in units of 128 are one line of units; CTA i of
// W takes an equal part of it, finds its place from lengths and walks on.  A
// segment that a CTA does not hold in full goes to the workspace;
// attend_join_kernel, which is launched right behind, joins these in order.
// Either way the warps of a CTA take 32 tokens at a time each, with a softmax and
// sums of their own, and are joined at the end of the segment, in order.
//
// What bounds it.  Few rows over long sequences: the cache's bytes (128 sequences
// of 4096 tokens, 8 heads of 128, bf16: 84 us, 5.1 TB/s; 4 of 240,000: 182 us,
// 4.3 TB/s at 16 rows).  More rows: instructions.  A group of 32 tokens costs a
// warp about as much for masks, numbers, exponentials and the operands'
// exchange as for its products: 32 sequences of up to 8192 tokens take 46, 60 and
// 78 us at 8, 16 and 24 rows (32 us of bytes); at 16 rows the schedulers issue in
// half of the cycles and the tensor pipe is busy in 39 %, with 12 warps an SM and
// some registers spilled (52 bytes a thread).  float16 results, which form each
// value product twice, take 48, 70 and 93 us: the tensor pipe is busy in half of
// the cycles at 16 rows.  When they were tried, 16 tokens at a time with another
// CTA an SM took 206 us where 181, rings of three groups 49 us where 47 at 8 rows.
#pragma once

#include <float.h>

#include "sv_kv4.cuh"

namespace sv {
namespace cache {

constexpr int kAtUnit = 128;              // tokens of a unit
constexpr int kAtStart = 3;               // units that stand for a segment's start
constexpr int kAtStages = 2;              // groups of 32 tokens in a warp's ring
constexpr int kAtJoinThreads = 256;
constexpr int kAtCluster = 8;             // CTAs of a segment that is joined in one launch,
constexpr int kAtShort = 16640;           // which it may be up to this many positions of a table (16384 and a page)
constexpr float kAtSlack = 8.f;           // a row's reference may be 2^8 below its largest term
constexpr float kAtValueTop = 128.f;      // largest s' 2^x: p s' 2^x stays below 2^(7 + 8), float16 ends at 65504

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

// c [16 x 8] += a [16 x 16] . b [16 x 8]
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit elements, two of a row a lane, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// (a & b) ^ c
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr unsigned short kHalfRange = 0x4780, kMinusHalfRange = 0xc780;      // 7.5, -7.5 in float16
// c0 += half 0 of a * m, c1 += half 1 of a * m, in float32; m is a float16's bits
__device__ __forceinline__ void add_product(float& c0, float& c1, uint32_t a, unsigned short m) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tfma.rn.f32.f16 %0, x, %3, %0;\n\tfma.rn.f32.f16 %1, y, %3, %1;\n\t}"
      : "+f"(c0), "+f"(c1) : "r"(a), "h"(m));
}

// Tokens that rows of sequence b may see, its rows, and how they are cut.
struct Sequence {
  int rows, seen, tiles, chunks;          // row tiles; units a (head, row tile)
  int first;                              // tokens that row 0 sees, before the limit of the table
  __device__ __forceinline__ Sequence(const AttendParams& p, int b, int TR, int unit) {
    rows = p.gamma_b ? min(max(p.gamma_b[b], -1), p.rows - 1) + 1 : p.rows;
    first = (int)min((long long)max(p.lengths[b], 0) + 1, 0x7fffff00ll);
    seen = (int)min((long long)first + rows - 1, (long long)p.N * p.page);
    tiles = (rows * p.G + TR - 1) / TR;
    chunks = max(1, (seen + unit - 1) / unit);
  }
  // (a segment's start takes about as long as kAtStart of its units)
  __device__ __forceinline__ long long units(int H) const { return (long long)H * tiles * (chunks + kAtStart); }
};

// Rows behind a sequence's last become 0.
template <typename T, int D, int THREADS>
__device__ __forceinline__ void fill_behind(const AttendParams& p) {
  if (!p.fill || !p.gamma_b) return;
  const int HG = p.H * p.G;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int from = min(max(p.gamma_b[b], -1), p.rows - 1) + 1;
    const long long r0 = (long long)b * p.rows + from, r1 = (long long)(b + 1) * p.rows;
    for (long long x = r0 * HG * (D / 8) + threadIdx.x; x < r1 * HG * (D / 8); x += THREADS)
      static_cast<uint4*>(p.out)[x] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (long long x = r0 * HG + threadIdx.x; x < r1 * HG; x += THREADS) p.lse[x] = 0.f;
  }
}

// Four channels of a row: sums y and mass l, both relative to 2^top.
template <typename T, int D>
__device__ __forceinline__ void finish_row(const AttendParams& p, long long q_row, int dg, float4 y, float top, float l) {
  const float over = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(p.out)[q_row * (D / 4) + dg] =
      make_uint2(Kv<T>::pack(y.x * over, y.y * over), Kv<T>::pack(y.z * over, y.w * over));
  if (p.lse && dg == 0) p.lse[q_row] = l == 0.f ? __int_as_float(0xff800000) : (top + log2f(l)) * 6.931471805599453e-01f;
}

// A CTA's part of the line of units: [u, end), u in sequence b, whose first
// unit is `base`; U units in all, W CTAs have one at least.  Every warp finds
// it on its own.
struct Part {
  long long U = 0, W = 0, u = 0, end = 0, base = 0;
  int b = 0;
  __device__ __forceinline__ bool some() const { return blockIdx.x < W; }
  // the CTA that unit x belongs to
  __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * W - 1) / U); }
};
__device__ __forceinline__ Part find_part(const AttendParams& p, int TR, int unit) {
  const int lane = threadIdx.x & 31;
  Part x;
  // each lane takes a run of sequences
  const int run = (p.B + 31) / 32;
  const int b0 = min(lane * run, p.B), b1 = min(b0 + run, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += Sequence(p, b, TR, unit).units(p.H);
  long long upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += y;
  }
  x.U = __shfl_sync(0xffffffffu, upto, 31);
  x.W = min((long long)gridDim.x, x.U);
  if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (!x.some()) return x;
  x.u = x.U * blockIdx.x / x.W;
  x.end = x.U * (blockIdx.x + 1) / x.W;
  x.base = upto - mine;
  x.b = b0;
  const bool here = x.u >= upto - mine && x.u < upto;
  if (here) {
    for (; x.b < b1 - 1; ++x.b) {
      const long long n = Sequence(p, x.b, TR, unit).units(p.H);
      if (x.u < x.base + n) break;
      x.base += n;
    }
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  x.b = __shfl_sync(0xffffffffu, x.b, from);
  x.base = __shfl_sync(0xffffffffu, x.base, from);
  return x;
}

// The segment that unit u is in: head, row tile, and those of its units from u
// on that are this CTA's; the line goes on `step` units behind u.  The first
// kAtStart units of a segment are its start alone: who has no others of it
// (chunks = 0) does nothing.
struct Segment {
  int h, rt, at, chunk0, chunks, step;
  // its last unit
  __device__ __forceinline__ long long last(const Sequence& s, long long base) const {
    return base + (long long)(at + 1) * (s.chunks + kAtStart) - 1;
  }
};
__device__ __forceinline__ Segment segment_at(const Sequence& s, long long u, long long base, long long end) {
  Segment x;
  const int all = s.chunks + kAtStart;
  int begin;
  if (u - base < 0x7fffffffll) {          // (a 64-bit division takes longer)
    x.at = (int)(u - base) / all;
    begin = (int)(u - base) - x.at * all;
  } else {
    x.at = (int)((u - base) / all);
    begin = (int)(u - base - (long long)x.at * all);
  }
  x.h = x.at / s.tiles;
  x.rt = x.at - x.h * s.tiles;
  x.step = (int)min((long long)(all - begin), end - u);
  x.chunk0 = max(begin - kAtStart, 0);
  x.chunks = max(begin + x.step - kAtStart, 0) - x.chunk0;
  return x;
}

// 32 tokens of one head in a warp's ring: two subs of 16, each its keys, then
// its values, then (behind both) its numbers, as they lie in the cache.  As
// operands, lane (g, c) = (lane / 4, lane % 4) takes the key codes of tokens g
// and 8 + g of a sub, quarter c; the value codes of its tokens 2 c, 2 c + 1 and 8
// more, eighth g; the numbers of tokens g and 8 + g.
template <int D>
struct Stage {
  static constexpr int kCodes = 8 * D;                       // bytes of a sub's keys, and of its values
  static constexpr int kNumbers = 4 * kCodes;                // where the numbers begin
  static constexpr int kBytes = kNumbers + 2 * 128;
};
// 16 bytes, where `here`
__device__ __forceinline__ void copy_ahead_if(bool here, uint32_t to, const unsigned char* from) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(to), "l"(from),
               "r"((uint32_t)here) : "memory");
}
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <int WORDS>
__device__ __forceinline__ void shared_words(uint32_t (&w)[WORDS], uint32_t at) {
  if constexpr (WORDS == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
}

// Two float32 operations an instruction.
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void split(Two p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Shared memory of CTA k of the cluster.
__device__ __forceinline__ uint32_t cluster_address(uint32_t at, int k) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(at), "r"(k));
  return y;
}
__device__ __forceinline__ float cluster_load(uint32_t at) {
  float y;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(at) : "memory");
  return y;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t at) {
  float4 y;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(at) : "memory");
  return y;
}

// The power of two (its exponent) that brings a row's largest element to
// [2^13, 2^14), or as near as 2^126 does: a row of zeros, whose scores any scale
// leaves at 0, then has a small one.
__device__ __forceinline__ int raised_by(float top) { return top > 0.f ? min(140 - (int)(__float_as_uint(top) >> 23), 126) : 126; }
// x 2^e, |e| <= 252, in two steps: neither leaves float32's range where the result does not.
__device__ __forceinline__ float times_power(float x, int e) {
  const int a = e >> 1, b = e - a;
  return x * __uint_as_float((uint32_t)(a + 127) << 23) * __uint_as_float((uint32_t)(b + 127) << 23);
}

// NT: groups of eight rows
template <typename T, int D, int NT>
struct AttendShape {
  static constexpr int TR = 8 * NT;       // rows of a tile
  static constexpr int kCtas = NT == 1 ? 4 : NT == 2 ? 3 : 2;   // an SM
  static constexpr int kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kQ = NT * (D / 32) * 512;             // q as operands
  // a warp's ring, which its sums take the place of at the end of a segment
  static constexpr int kRing = kAtStages * Stage<D>::kBytes;
  static constexpr int kSums = (TR * D + 2 * TR) * 4;
  static constexpr int kWarp = kRing > kSums ? kRing : kSums;
  static constexpr int kSmem = kQ + kWarps * kWarp;
  static constexpr int kJoinedSmem = kSmem + kSums;          // with the CTA's own sums, which others read
  static_assert(kCtas * (kJoinedSmem + 2048) <= 228 * 1024, "shared memory of an SM");
};

// Position of a group of four channels (dg) of row r in a warp's sums in
// shared memory: lanes that write at once go to different banks.
template <int D>
__device__ __forceinline__ int swizzled(int r, int dg) { return dg ^ ((r >> 1 & 3) << (D == 128 ? 0 : 2)); }

// kJoined: a cluster of kAtCluster CTAs per sequence, head and row tile
template <typename T, int D, int NT, bool kJoined>
__global__ void __launch_bounds__(AttendShape<T, D, NT>::kThreads, AttendShape<T, D, NT>::kCtas) attend_kernel(const __grid_constant__ AttendParams p) {
  using S = AttendShape<T, D, NT>;
  constexpr int KW = D / 32, TR = S::TR, kWarpFloats = S::kWarp / 4, LANES = D / 8;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr bool kFine = std::is_same<T, __half>::value;     // the weights' rest is an operand too
  extern __shared__ __align__(16) float at_sm[];
  __shared__ float q_sums[TR], row_scales[TR];
  __shared__ int limits[TR];
  __shared__ long long out_rows[TR];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);    // (the compiler sees that a warp shares it)
  float* const all_sums = at_sm + S::kQ / 4;
  pdl_launch_dependents();

  fill_behind<T, D, kThreads>(p);
  Part line;
  int b, rank = 0, head = 0, tile = 0;
  if constexpr (kJoined) {
    rank = (int)cluster_rank();
    const int x = blockIdx.x / kAtCluster, tiles = (p.rows * p.G + TR - 1) / TR;
    tile = x % tiles;
    head = x / tiles % p.H;
    b = x / tiles / p.H;
  } else {
    line = find_part(p, TR, kAtUnit);
    if (!line.some()) return;
    b = line.b;
  }
  long long u = line.u, base = line.base;
  const int me = blockIdx.x;

  const long long block_bytes = (long long)p.page * kTokenBytes<D>;
  const int page_tiles = p.page / 16;
  const uint32_t zero = (uint32_t)p.page >> 16;              // which the compiler does not know
  const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(at_sm) + lane * 16;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(all_sums + warp * kWarpFloats);
  while (kJoined || u < line.end) {
    const Sequence s(p, b, TR, kAtUnit);
    Segment segment;
    if constexpr (kJoined) {
      if (tile >= s.tiles) return;
      segment = Segment{head, tile, 0, 0, s.chunks, 0};
    } else {
      const long long n_units = s.units(p.H);
      if (u >= base + n_units) {
        base += n_units;
        ++b;
        continue;
      }
      segment = segment_at(s, u, base, line.end);
      u += segment.step;
      if (segment.chunks == 0) continue;
    }
    const int h = segment.h, rt = segment.rt, chunk0 = segment.chunk0, chunks = segment.chunks;

    // ---- this warp's groups of 32 tokens, number `first` + kStep n
    constexpr int kStep = kJoined ? kAtCluster * kWarps : kWarps;
    const int sub_end = (s.seen + 15) / 16;
    const int first = chunk0 * (kAtUnit / 32) + rank * kWarps + warp;
    const int groups = max(0, (min((chunk0 + chunks) * (kAtUnit / 32), (sub_end + 1) / 2) - first + kStep - 1) / kStep);
    // A lane knows where sub lane % 2 of group lane / 2 of the next 16 begins
    // in the cache, its number in the page in the low four bits; 0: hidden.
    // The 16 behind them are asked for ahead of time.
    int ask_id = -1, ask_sub = 0;
    auto ask = [&](int n) {
      const int mine = 2 * (first + kStep * (n + (lane >> 1))) + (lane & 1);
      ask_id = -1;
      if (n + (lane >> 1) < groups && mine < sub_end) {
        const int x = mine / page_tiles;
        ask_id = __ldg(p.table + (long long)b * p.N + x);
        ask_sub = mine - x * page_tiles;
      }
    };
    unsigned long long ahead = 0;
    auto learn = [&]() {
      ahead = 0;
      if (ask_id >= 0 && ask_id < p.pages)
        ahead = reinterpret_cast<unsigned long long>(p.cache) +
                (unsigned long long)(((long long)ask_id * p.H + h) * block_bytes + ask_sub * (8 * D) + ask_sub);
    };
    ask(0);
    // q is on its way meanwhile: a thread's pieces of eight channels
    constexpr int PIECES = (TR * LANES + kThreads - 1) / kThreads;
    uint4 qv[PIECES];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      const int x = tid + k * kThreads, rl = x / LANES, r = rt * TR + rl, i = r / p.G;
      qv[k] = make_uint4(0, 0, 0, 0);
      if (rl < TR && i < s.rows)
        qv[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + b * p.qs[0] + i * p.qs[1] +
                                                     (long long)(h * p.G + r - i * p.G) * p.qs[2]) + x % LANES);
    }
    uint32_t to = ring;                   // where the next group goes
    uint32_t there = 0;                   // bits 2 (n % 8), + 1: which subs of group n are there
    auto copy_group = [&](int n) {
      if (n < groups) {
        if ((n & 15) == 0) {
          learn();
          ask(n + 16);
        }
        const unsigned long long from0 = __shfl_sync(0xffffffffu, ahead, 2 * (n & 15));
        const unsigned long long from1 = __shfl_sync(0xffffffffu, ahead, 2 * (n & 15) + 1);
        const int bit = 2 * (n & 7);
        there = (there & ~(3u << bit)) | (uint32_t)(from0 != 0) << bit | (uint32_t)(from1 != 0) << (bit + 1);
        constexpr int C = Stage<D>::kCodes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned long long from = i ? from1 : from0;
          const bool here = from != 0;
          const int sub = (int)(from & 15);
          const unsigned char* codes = reinterpret_cast<const unsigned char*>(from - sub) + lane * 16;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            copy_ahead_if(here, to + lane * 16 + i * 2 * C + j * 512, codes + j * 512);
            copy_ahead_if(here, to + lane * 16 + i * 2 * C + C + j * 512, codes + p.page * (D / 2) + j * 512);
          }
          copy_ahead_if(here && lane < 8, to + lane * 16 + Stage<D>::kNumbers + i * 128,
                        codes + p.page * D - sub * (8 * D - 128));
        }
        to = to == ring + (kAtStages - 1) * Stage<D>::kBytes ? ring : to + Stage<D>::kBytes;
      }
      copies_end_group();
    };
#pragma unroll
    for (int n = 0; n < kAtStages - 1; ++n) copy_group(n);

    // ---- q as operands: float16 with a power of two per row
    {
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int x = tid + k * kThreads, rl = x / LANES, word = x % LANES;
        const uint32_t w[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
        float top = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float f0 = Kv<T>::lo(w[j]), f1 = Kv<T>::hi(w[j]);
          top = max3(top, fabsf(f0), fabsf(f1));
          sum += f0 + f1;
        }
#pragma unroll
        for (int m = LANES / 2; m >= 1; m >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, m);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        }
        if (rl >= TR) continue;
        const int up = raised_by(top);
        const float raise = __uint_as_float((uint32_t)(up + 127) << 23);
        if (word == 0) {
          const int r = rt * TR + rl, i = r / p.G;
          q_sums[rl] = sum * raise * 0x1p-24f;   // (the products' unit is 2^-24 of a code)
          row_scales[rl] = times_power(p.scale, 24 - up);
          limits[rl] = i < s.rows ? min(s.first - 1 + i, s.seen - 1) : -1;
          out_rows[rl] = i < s.rows ? ((long long)b * p.rows + i) * p.H * p.G + (long long)h * p.G + (r - i * p.G) : -1;
        }
        // word j of quarter cc: halves t; channels 2 t, 2 t + 4 as they are,
        // 2 t + 1, 2 t + 5 for codes of 16 times their size
        const int cc = word / KW, j = word % KW;
        uint32_t y[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          y[2 * t] = half2_bits(Kv<T>::lo(w[t]) * raise, Kv<T>::lo(w[t + 2]) * raise);
          y[2 * t + 1] = half2_bits(Kv<T>::hi(w[t]) * raise * 0.0625f, Kv<T>::hi(w[t + 2]) * raise * 0.0625f);
        }
        reinterpret_cast<uint4*>(at_sm)[((rl >> 3) * KW + j) * 32 + (rl & 7) * 4 + cc] = make_uint4(y[0], y[1], y[2], y[3]);
      }
      __syncthreads();
    }

    // rows 8 m + 2 c and + 1
    Two q_sum[NT], row_scale[NT], minus_ref[NT], mass[NT], shift[NT];
    float o[NT][2 * KW][4];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const float2 q = *reinterpret_cast<const float2*>(q_sums + 8 * m + 2 * c);
      const float2 f = *reinterpret_cast<const float2*>(row_scales + 8 * m + 2 * c);
      q_sum[m] = two(q.x, q.y);
      row_scale[m] = two(f.x, f.y);
      minus_ref[m] = mass[m] = shift[m] = two(0.f, 0.f);
#pragma unroll
      for (int t = 0; t < 2 * KW; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[m][t][x] = 0.f;
    }
    float value_scale = 0x1p126f;         // what p s' is multiplied by, a power of two
    // The first group sets the references.  A row that sees none of it sees
    // none of the later ones: its mass stays 0.
    bool fresh = true;
    const uint32_t flip = 0x800f800fu + zero, flip16 = 0x80f080f0u + zero;   // (registers: an instruction takes one constant)

    auto group = [&](auto masked_group, int token0, uint32_t subs, uint32_t from) {
      constexpr bool kMasked = decltype(masked_group)::value;
      // scores: q . n for 32 tokens; z[i][m]: tokens g, 8 + g of sub i, two rows each
      float z[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[i][m][e] = 0.f;
      {
        uint32_t kw[2][2][KW];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            shared_words(kw[i][e], from + i * 2 * Stage<D>::kCodes + (8 * e + g) * (D / 2) + c * (D / 8));
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t qf[NT][4];
#pragma unroll
          for (int m = 0; m < NT; ++m) shared_words(qf[m], q_at + (m * KW + w) * 512);
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = kw[i][0][w] >> (8 * half), y = kw[i][1][w] >> (8 * half);
              const uint32_t a0 = x & 0x000f000fu, a1 = y & 0x000f000fu, a2 = x & 0x00f000f0u, a3 = y & 0x00f000f0u;
#pragma unroll
              for (int m = 0; m < NT; ++m) mma16816(z[i][m], a0, a1, a2, a3, qf[m][2 * half], qf[m][2 * half + 1]);
            }
        }
      }
      // whether rows 8 m + 2 c and + 1 see token 8 e + g of sub i
      auto sees = [&](int m, int i, int e) {
        const int2 lim = *reinterpret_cast<const int2*>(limits + 8 * m + 2 * c);
        const int t = subs >> i & 1 ? token0 + 16 * i + 8 * e + g : 0x7fffffff;
        return make_int2(t <= lim.x, t <= lim.y);
      };
      uint32_t nv[2][2];                  // the values' numbers
      float most = -FLT_MAX, largest = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t x[2];
          shared_words(x, from + Stage<D>::kNumbers + (16 * i + 8 * e + g) * 8);
          // (those of tokens that nobody sees may be anything)
          if (kMasked && (!(subs >> i & 1) || token0 + 16 * i + 8 * e + g >= s.seen)) x[0] = x[1] = 0;
          nv[i][e] = x[1];
          const float k_scale = Kv<T>::lo(x[0]), k_offset = Kv<T>::hi(x[0]);
          const Two ks = two(k_scale, k_scale), ko = two(k_offset, k_offset);
          largest = fmaxf(largest, Kv<T>::lo(x[1]));
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            float y0, y1;
            split(fma2(fma2(two(z[i][m][2 * e], z[i][m][2 * e + 1]), ks, mul2(ko, q_sum[m])), row_scale[m], minus_ref[m]), y0, y1);
            if (kMasked) {
              const int2 see = sees(m, i, e);
              if (!see.x) y0 = __int_as_float(0xff800000);
              if (!see.y) y1 = __int_as_float(0xff800000);
            }
            z[i][m][2 * e] = y0;
            z[i][m][2 * e + 1] = y1;
            most = max3(most, y0, y1);
          }
        }
      if (__any_sync(0xffffffffu, fresh || most > kAtSlack || largest * value_scale > kAtValueTop)) {
        // a row's terms outgrow its reference, or the values' scales theirs
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, x));
        float by = 1.f;
        if (largest * value_scale > kAtValueTop) {
          // largest < 2^(e - 126): 2^(133 - e) brings it below 2^7
          const int e = (int)(__float_as_uint(largest) >> 23);
          const float to_scale = __uint_as_float((uint32_t)min(max(133 - e + 127, 1), 253) << 23);
          by = to_scale / value_scale;
          value_scale = to_scale;
        }
        // a row's terms move down by `up`
        auto rise = [&](float up) {
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, x));
          return fresh ? (up == __int_as_float(0xff800000) ? 0.f : up) : fmaxf(up, 0.f);
        };
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const float up0 = rise(fmaxf(fmaxf(z[0][m][0], z[0][m][2]), fmaxf(z[1][m][0], z[1][m][2])));
          const float up1 = rise(fmaxf(fmaxf(z[0][m][1], z[0][m][3]), fmaxf(z[1][m][1], z[1][m][3])));
          minus_ref[m] = add2(minus_ref[m], two(-up0, -up1));
          const float f0 = fresh ? 0.f : ex2_approx(-up0), f1 = fresh ? 0.f : ex2_approx(-up1);
          mass[m] = mul2(mass[m], two(f0, f1));
          shift[m] = mul2(shift[m], two(f0, f1));
#pragma unroll
          for (int n = 0; n < 2 * KW; ++n) {
            o[m][n][0] *= f0 * by;
            o[m][n][1] *= f1 * by;
            o[m][n][2] *= f0 * by;
            o[m][n][3] *= f1 * by;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            z[i][m][0] -= up0;
            z[i][m][1] -= up1;
            z[i][m][2] -= up0;
            z[i][m][3] -= up1;
          }
        }
        fresh = false;
      }

      // weights and sums, 16 tokens at a time: their first eight as codes n,
      // the others as n - 15
      [[maybe_unused]] float centre[NT][2];
      if constexpr (!kFine) {
#pragma unroll
        for (int m = 0; m < NT; ++m) centre[m][0] = centre[m][1] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t pb[NT][2];
        [[maybe_unused]] uint32_t pl[NT][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float scale = Kv<T>::lo(nv[i][e]), n_scale = scale * value_scale;
          // (not kFine: the middle of the row, and the rest with the rounded weights)
          const float offset = fmaf(kFine ? e ? 15.f : 0.f : 7.5f, scale, Kv<T>::hi(nv[i][e]));
          const Two vn = two(n_scale, n_scale), vo = two(offset, offset);
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const Two w = two(ex2_approx(z[i][m][2 * e]), ex2_approx(z[i][m][2 * e + 1]));
            mass[m] = add2(mass[m], w);
            float a0, a1;
            split(mul2(w, vn), a0, a1);
            if (kMasked) {
              // (a hidden token's numbers may be NaN)
              const int2 see = sees(m, i, e);
              float f0, f1;
              split(mul2(w, vo), f0, f1);
              if (!see.x) a0 = f0 = 0.f;
              if (!see.y) a1 = f1 = 0.f;
              shift[m] = add2(shift[m], two(f0, f1));
            } else {
              shift[m] = fma2(w, vo, shift[m]);
            }
            const uint32_t x = half2_bits(a0, a1);
            pb[m][e] = transposed(x);
            if constexpr (kFine) {
              // a float16 result wants more than float16 weights: their rest
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&x));
              pl[m][e] = transposed(half2_bits(a0 - back.x, a1 - back.y));
            } else {
              add_product(centre[m][0], centre[m][1], x, e ? kHalfRange : kMinusHalfRange);
            }
          }
        }
        uint32_t vw[2][KW];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          shared_words(vw[e], from + (2 * i + 1) * Stage<D>::kCodes + (4 * e + c) * D + g * (D / 8));
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x = vw[0][w] >> (8 * half), y = vw[1][w] >> (8 * half);
            const uint32_t a0 = x & 0x000f000fu, a1 = x & 0x00f000f0u;
            const uint32_t a2 = and_xor(y, 0x000f000fu, flip), a3 = and_xor(y, 0x00f000f0u, flip16);
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              mma16816(o[m][2 * w + half], a0, a1, a2, a3, pb[m][0], pb[m][1]);
              if constexpr (kFine) mma16816(o[m][2 * w + half], a0, a1, a2, a3, pl[m][0], pl[m][1]);
            }
          }
      }
      if constexpr (!kFine) {
        const float down = 1.f / value_scale;
#pragma unroll
        for (int m = 0; m < NT; ++m) shift[m] = fma2(two(centre[m][0], centre[m][1]), two(down, down), shift[m]);
      }
    };

    uint32_t from = ring;
    for (int n = 0; n < groups; ++n) {
      copies_wait<kAtStages - 2>();
      __syncwarp();                       // every lane's copies are there, and everybody is done with the group before
      const uint32_t subs = there >> (2 * (n & 7)) & 3u;
      copy_group(n + kAtStages - 1);
      const int token0 = 32 * (first + kStep * n);
      if (subs == 3u && token0 + 32 <= s.first) group(std::false_type{}, token0, subs, from);
      else if (subs) group(std::true_type{}, token0, subs, from);
      from = from == ring + (kAtStages - 1) * Stage<D>::kBytes ? ring : from + Stage<D>::kBytes;
    }
    copies_wait<0>();
    __syncwarp();

    // ---- the warps' sums side by side in shared memory
    float* sums = all_sums + warp * kWarpFloats;
    const float down = 1.f / value_scale;
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      float l[2], f[2], ref[2];
      split(mass[m], l[0], l[1]);
      split(shift[m], f[0], f[1]);
      split(minus_ref[m], ref[0], ref[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * m + 2 * c + e;
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) {
          l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
          f[e] += __shfl_xor_sync(0xffffffffu, f[e], x);
        }
        if (g == 0) {
          sums[TR * D + r] = l[e] == 0.f ? -FLT_MAX : -ref[e];
          sums[TR * D + TR + r] = l[e];
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {     // channels 4 (KW g + w) ..
          float y[4];
#pragma unroll
          for (int n = 0; n < 4; ++n)
            y[n] = fmaf(o[m][2 * w + (n >> 1)][2 * (n & 1) + e] * (n & 1 ? 0x1p20f : 0x1p24f), down, f[e]);
          reinterpret_cast<float4*>(sums)[r * (D / 4) + swizzled<D>(r, g * KW + w)] = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    }
    __syncthreads();
    const bool whole = !kJoined && chunk0 == 0 && chunks == s.chunks;
    float* part = kJoined ? at_sm + S::kSmem / 4 : p.part + (size_t)(2 * me + (chunk0 == 0)) * part_floats(TR, D);
#pragma unroll
    for (int x0 = 0; x0 < TR * (D / 4); x0 += kThreads) {
      const int x = x0 + tid;
      if (TR * (D / 4) % kThreads != 0 && x >= TR * (D / 4)) break;
      const int r = x / (D / 4), dg = x % (D / 4), at_r = r * (D / 4) + swizzled<D>(r, dg);
      const long long q_row = out_rows[r];
      if (q_row < 0) continue;
      float top = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = all_sums[w * kWarpFloats + TR * D + r];
        top = m > top || m != m ? m : top;
      }
      float l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* sw = all_sums + w * kWarpFloats;
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
      } else {
        finish_row<T, D>(p, q_row, dg, y, top, l);
      }
    }
    if constexpr (kJoined) {
      // each CTA finishes an eighth of the channels' fours from all CTAs' sums
      cluster_barrier();
      constexpr int kMine = TR * (D / 4) / kAtCluster;
      const uint32_t sums_at = (uint32_t)__cvta_generic_to_shared(part);
      for (int x = rank * kMine + tid; x < (rank + 1) * kMine; x += kThreads) {
        const int r = x / (D / 4), dg = x % (D / 4);
        const long long q_row = out_rows[r];
        if (q_row < 0) continue;
        float m[kAtCluster], mass_k[kAtCluster], top = -FLT_MAX, l = 0.f;
        float4 y_k[kAtCluster], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kAtCluster; ++k) {
          const uint32_t there_at = cluster_address(sums_at, k);
          m[k] = cluster_load(there_at + (TR * D + r) * 4);
          mass_k[k] = cluster_load(there_at + (TR * D + TR + r) * 4);
          y_k[k] = cluster_load4(there_at + x * 16);
        }
#pragma unroll
        for (int k = 0; k < kAtCluster; ++k) top = m[k] > top || m[k] != m[k] ? m[k] : top;
#pragma unroll
        for (int k = 0; k < kAtCluster; ++k) {
          const float f = ex2_approx(m[k] - top);
          l = fmaf(f, mass_k[k], l);
          y.x = fmaf(f, y_k[k].x, y.x);
          y.y = fmaf(f, y_k[k].y, y.y);
          y.z = fmaf(f, y_k[k].z, y.z);
          y.w = fmaf(f, y_k[k].w, y.w);
        }
        finish_row<T, D>(p, q_row, dg, y, top, l);
      }
      cluster_barrier();                  // (the others have read this CTA's sums)
      return;
    } else {
      __syncthreads();
      if (!whole && chunk0 == 0 && tid == 0)
        p.desc[me] = make_int4(b, h, rt, line.owner(segment.last(s, base)));
    }
  }
}

// Joins the parts of the segment that begins in CTA blockIdx.x's range and
// ends behind it: its own second part, then the first parts of those behind.
// A warp has a row; a lane four channels, and the reference and the mass of
// one of 32 parts at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kAtJoinThreads) attend_join_kernel(const __grid_constant__ AttendParams p, const int TR) {
  pdl_wait();
  const int own = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * (kAtJoinThreads / 32) + (threadIdx.x >> 5);
  const int4 d = p.desc[own];
  if (d.x < 0) return;
  const int b = d.x, h = d.y, rt = d.z, count = d.w - own + 1;
  const int rows = p.gamma_b ? min(max(p.gamma_b[b], -1), p.rows - 1) + 1 : p.rows;
  const int rr = rt * TR + r, i = rr / p.G;
  if (i >= rows) return;
  const int floats = part_floats(TR, D);
  float top = -FLT_MAX, l = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int a0 = 0; a0 < count; a0 += 32) {
    const int a = a0 + lane, n = min(count - a0, 32);
    float m = -FLT_MAX, mass = 0.f;
    if (a < count) {
      const float* part = p.part + (size_t)(2 * (own + a) + (a == 0)) * floats + TR * D + r;
      m = part[0];
      mass = part[TR];
    }
    float now = m;
    bool bad = m != m;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, x));
    now = fmaxf(now, top);
    if (__any_sync(0xffffffffu, bad)) now = __int_as_float(0x7fffffff);
    const float f = ex2_approx(m - now), back = ex2_approx(top - now);
    top = now;
    float sum = f * mass;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = fmaf(l, back, sum);
    y.x *= back;
    y.y *= back;
    y.z *= back;
    y.w *= back;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float g = __shfl_sync(0xffffffffu, f, k);
      if (lane < D / 4) {
        const float4 v = reinterpret_cast<const float4*>(p.part + (size_t)(2 * (own + a0 + k) + (a0 + k == 0)) * floats)[r * (D / 4) + lane];
        y.x = fmaf(g, v.x, y.x);
        y.y = fmaf(g, v.y, y.y);
        y.z = fmaf(g, v.z, y.z);
        y.w = fmaf(g, v.w, y.w);
      }
    }
  }
  if (lane < D / 4)
    finish_row<T, D>(p, ((long long)b * p.rows + i) * p.H * p.G + (long long)h * p.G + (rr - i * p.G), lane, y, top, l);
}

}  // namespace cache
}  // namespace sv
