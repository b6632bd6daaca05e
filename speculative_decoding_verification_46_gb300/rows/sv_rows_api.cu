// Host side of the operators on logits rows: argument validation and launches
// for the C ABI declared in include/specverify_rows.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "specverify_rows.h"
#include "sv_adjust.cuh"
#include "sv_distill.cuh"
#include "sv_distill_pipe.cuh"
#include "sv_toplogits.cuh"

namespace {

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(sv_dtype dt) { return dt == SV_DTYPE_F32 || dt == SV_DTYPE_BF16 || dt == SV_DTYPE_F16; }
int vec_width(sv_dtype dt) { return dt == SV_DTYPE_F32 ? 4 : 8; }
size_t elem_size(sv_dtype dt) { return dt == SV_DTYPE_F32 ? 4 : 2; }
bool rows_ok(long long R, int V) { return R >= 0 && R <= SV_MAX_ROWS && V >= 1 && V <= SV_MAX_VOCAB; }
bool temperature_ok(float t) { return t > 0.f && std::isfinite(t) && std::isfinite((float)(1.4426950408889634 / (double)t)); }

// a is b, or the n bytes at a and at b have nothing in common
bool same_or_apart(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x == y || x + n <= y || y + n <= x;
}

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  return n;
}

// Opt in to `most` bytes of dynamic shared memory, the most that any launch of
// the kernel asks for, once per kernel (`set`: a static of the launch site)
// and device.  One size for all calls: threads that come here together set the
// same limit, and none lowers another's between its opt-in and its launch.
bool allow_smem(std::atomic<bool> (&set)[64], const void* kern, size_t most) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (set[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  set[dev].store(true, std::memory_order_release);
  return true;
}

sv_status launched() {
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv::F2 two_float(double d) {
  const float hi = (float)d;
  return sv::F2{hi, (float)(d - (double)hi)};
}

// log2(e) / temperature as a float pair
void exponent_scale(float temperature, float* hi, float* lo) {
  const double c = 1.4426950408889634 / (double)temperature;
  *hi = (float)c;
  *lo = (float)(c - (double)*hi);
}

// ---------------------------------------------------------------- adjust

// Tokens per tile: 12 KB of a row, fewer for small calls, as long as every CTA
// is resident at once (three an SM) and down to 256 tokens; the tiles of a row
// are then made equal.
void choose_tile(sv::rows::AdjustParams& p, int elem) {
  const long long at_once = 3ll * sm_count() / p.B;
  const long long tiles =
      std::max<long long>(ceil_div(p.V, sv::rows::kAdTileBytes / elem), std::min<long long>(at_once, ceil_div(p.V, 256)));
  p.tile = (int)(ceil_div(ceil_div(p.V, tiles), 64) * 64);
  p.tiles = (int)ceil_div(p.V, p.tile);
}

// Dynamic shared memory of an adjust kernel: the listed tokens' part and, where
// rows pass through shared memory, the stages.
template <typename T>
size_t adjust_smem(int tile, int NB, bool sparse, bool staged) {
  size_t smem = sparse ? (size_t)tile * 6 + (size_t)NB * 8 : 0;
  if (staged) smem += (size_t)sv::rows::kAdStages * (tile / sv::Tr<T>::VW + 1) * 16;
  return smem;
}

template <typename T>
sv_status launch_adjust(sv::rows::AdjustParams p, cudaStream_t stream) {
  choose_tile(p, (int)sizeof(T));
  const long long grid = (long long)p.B * p.tiles;
  if (grid > 0x7fffffffll) return SV_ERR_UNSUPPORTED;
  const bool sparse = p.count || p.NB, staged = p.copy && sparse;
  const bool whole = p.V % sv::Tr<T>::VW == 0;
  auto kern = staged ? whole ? sv::rows::adjust_staged_kernel<T, true> : sv::rows::adjust_staged_kernel<T, false>
              : whole ? sv::rows::adjust_direct_kernel<T, true> : sv::rows::adjust_direct_kernel<T, false>;
  const size_t smem = adjust_smem<T>(p.tile, p.NB, sparse, staged);
  // (the kernel's static shared memory counts toward the 48 KB that need no opt-in)
  static std::atomic<bool> set[4][64];
  if (smem > 32 * 1024 && !allow_smem(set[2 * staged + whole], (const void*)kern,
                                      adjust_smem<T>(sv::rows::kAdTileBytes / (int)sizeof(T), SV_MAX_BIAS, true, staged)))
    return SV_ERR_CUDA;
  kern<<<(unsigned)grid, sv::rows::kAdThreads, smem, stream>>>(p);
  return launched();
}

// ---------------------------------------------------------------- top logits

// SPECVERIFY_PATH=toprow / =topslice overrides the choice between rows and slices (tests cover both).
int top_override() {
  const char* e = std::getenv("SPECVERIFY_PATH");
  return !e ? 0 : std::strcmp(e, "toprow") == 0 ? 1 : std::strcmp(e, "topslice") == 0 ? 2 : 0;
}

// A CTA per row from as many rows as SMs on, slices of rows for fewer.  In us,
// slices and one CTA each, bf16:
//   152064 tokens   k 8        k 64       k 256
//     100 rows      26   28    33   39    72   56
//     152 rows      33   29    44   39    97   58
//     608 rows      104  50    135  65    299  125
//   32000 tokens
//     100 rows      15   14    17   20    34   32
//     152 rows      15   15    17   22    31   32
//     608 rows      34   23    42   31    87   65
bool top_by_rows(long long R) {
  const int o = top_override();
  return o == 1 || (o == 0 && R >= sm_count());
}

struct TopLayout {
  size_t ticket, part, lists, total;
  int H, SV;
};

// Slices of at most 2048 vectors; more, smaller ones where the rows alone
// would leave SMs without work, as long as a slice holds 8 k elements (its
// candidates are then a small part of it) and the slices' lists stay a short
// piece of work for the CTA that joins them (one row of 152064 bf16, k 64: 74
// slices 40 us, 32 slices 18).
TopLayout top_layout(long long R, int V, int k, int VW, int sms) {
  TopLayout L{};
  const long long nv = ceil_div((long long)V + (V % VW ? VW - 1 : 0), VW);
  long long H = ceil_div(nv, sv::rows::kTlThreads * 8);
  const long long most =
      std::max<long long>(H, std::min<long long>(nv / std::max(sv::rows::kTlThreads, 8 * k / VW), 2048 / k));
  if (R > 0) H = std::max(H, std::min(most, (2ll * sms) / R));
  L.SV = (int)ceil_div(nv, H);
  L.H = (int)ceil_div(nv, L.SV);
  size_t o = 0;
  L.ticket = o; o += up(sizeof(int) * (size_t)R);
  L.part = o;   o += up(sizeof(float4) * (size_t)R * L.H);
  L.lists = o;  o += up(sizeof(unsigned long long) * (size_t)R * L.H * k);
  L.total = o;
  return L;
}

template <typename T, int U>
sv_status launch_top_u(const sv::rows::TopParams& p, cudaStream_t stream) {
  sv::rows::top_slice_kernel<T, U><<<(unsigned)((long long)p.R * p.H), sv::rows::kTlThreads, 0, stream>>>(p);
  return launched();
}
template <typename T>
sv_status launch_top_rows(const sv::rows::TopParams& p, cudaStream_t stream) {
  auto kern = p.V % sv::Tr<T>::VW == 0 ? sv::rows::top_row_kernel<T, true> : sv::rows::top_row_kernel<T, false>;
  const auto smem = [](int k) {
    return (size_t)sv::rows::kTrStages * sv::rows::kTrStep * sizeof(uint4) +
           (size_t)sv::rows::tr_capacity(k) * sizeof(unsigned long long);
  };
  static std::atomic<bool> set[2][64];
  if (!allow_smem(set[p.V % sv::Tr<T>::VW == 0], (const void*)kern, smem(SV_MAX_TOP_K))) return SV_ERR_CUDA;
  kern<<<(unsigned)p.R, sv::rows::kTlThreads, smem(p.k), stream>>>(p);
  return launched();
}

template <typename T>
sv_status launch_top(const sv::rows::TopParams& p, cudaStream_t stream) {
  if (top_by_rows(p.R)) return launch_top_rows<T>(p, stream);
  const int u = (int)ceil_div(p.SV, sv::rows::kTlThreads);
  if (u <= 1) return launch_top_u<T, 1>(p, stream);
  if (u <= 2) return launch_top_u<T, 2>(p, stream);
  if (u <= 4) return launch_top_u<T, 4>(p, stream);
  return launch_top_u<T, 8>(p, stream);
}

// ---------------------------------------------------------------- distill

template <typename T, int U, bool GRAD>
sv_status launch_distill_u(sv::rows::DistillParams p, cudaStream_t stream) {
  p.NCK = (int)ceil_div(p.SV, sv::rows::kDiThreads * U);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.R * p.C));
  cfg.blockDim = dim3(sv::rows::kDiThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, sv::rows::distill_kernel<T, U, GRAD>, p) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return launched();
}

// SPECVERIFY_PATH=distillrow takes a cluster per row everywhere (tests cover both).
int distill_override() {
  const char* e = std::getenv("SPECVERIFY_PATH");
  return e && std::strcmp(e, "distillrow") == 0 ? 2 : 0;
}

// SPECVERIFY_PATH=distillstopN: in the persistent form, one warp of each
// cluster leaves at the cluster's row N, so that the other warps' waits run out
// (tests see what is left then).
int distill_stop() {
  const char* e = std::getenv("SPECVERIFY_PATH");
  return e && std::strncmp(e, "distillstop", 11) == 0 ? std::atoi(e + 11) : -1;
}

// The persistent form (sv_distill_pipe.cuh): as many clusters as fit at once.
// Returns SV_ERR_UNSUPPORTED where it does not apply.
template <typename T, bool GRAD>
sv_status launch_distill_pipe(sv::rows::DistillParams p, cudaStream_t stream) {
  constexpr int VW = sv::Tr<T>::VW;
  const long long nv = ceil_div((long long)p.V + (p.V % VW ? VW - 1 : 0), VW);
  const long long C = ceil_div(nv, sv::rows::kDpSlice);
  if (C > sv::rows::kDiMaxC || p.k > sv::rows::kDpMaxK) return SV_ERR_UNSUPPORTED;
  p.C = (int)C;
  p.SV = (int)ceil_div(nv, C);
  p.stop = distill_stop();
  auto kern = p.V % VW == 0 ? sv::rows::distill_pipe_kernel<T, GRAD, true> : sv::rows::distill_pipe_kernel<T, GRAD, false>;
  const size_t smem = sizeof(sv::rows::DpSmem<T>);
  static std::atomic<bool> set[2][64];
  if (!allow_smem(set[p.V % VW == 0], (const void*)kern, smem)) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.C);
  cfg.blockDim = dim3((unsigned)sv::rows::dp_threads(p.k));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> fit[64][sv::rows::kDiMaxC + 1];   // clusters at once, by device and size
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SV_ERR_CUDA;
  int clusters = fit[dev][p.C].load(std::memory_order_relaxed);
  if (clusters == 0) {
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) {
      cudaGetLastError();
      return SV_ERR_UNSUPPORTED;   // no room for such a cluster: the other form
    }
    fit[dev][p.C].store(clusters, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(std::min<long long>(clusters, p.R) * p.C));
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return launched();
}

// The persistent form wherever it applies: with few rows it is as fast as a
// cluster per row (the loss of 20 rows of 1024 float32: 9.2 us against 9.0; 64
// of 128256 bf16: 11.5 against 15.2), with many it is far ahead (4000 rows of
// 1024 bf16: 66 us against 130; 500 of 50001 f16: 25 against 48).  A cluster per row
// remains for longer lists and larger vocabularies.  CTAs per row there: as
// few as hold the row in registers (8 vectors per thread), more where the
// rows alone would leave SMs without work, at most 8.
template <typename T, bool GRAD>
sv_status launch_distill(sv::rows::DistillParams p, cudaStream_t stream) {
  constexpr int VW = sv::Tr<T>::VW;
  if (distill_override() != 2) {
    const sv_status st = launch_distill_pipe<T, GRAD>(p, stream);
    if (st != SV_ERR_UNSUPPORTED) return st;
  }
  const long long nv = ceil_div((long long)p.V + (p.V % VW ? VW - 1 : 0), VW);
  int C = (int)std::min<long long>(sv::rows::kDiMaxC, ceil_div(nv, sv::rows::kDiThreads * 8));
  while (C < sv::rows::kDiMaxC && (long long)p.R * C < sm_count() && ceil_div(nv, C) > sv::rows::kDiThreads) ++C;
  p.C = C;
  p.SV = (int)ceil_div(nv, C);
  const int u = (int)ceil_div(p.SV, sv::rows::kDiThreads);
  if (u <= 1) return launch_distill_u<T, 1, GRAD>(p, stream);
  if (u <= 2) return launch_distill_u<T, 2, GRAD>(p, stream);
  if (u <= 4) return launch_distill_u<T, 4, GRAD>(p, stream);
  return launch_distill_u<T, 8, GRAD>(p, stream);
}

template <typename T>
sv_status launch_distill_backward(sv::rows::DistillParams p, cudaStream_t stream) {
  constexpr int VW = sv::Tr<T>::VW;
  const long long nv = ceil_div((long long)p.V + (p.V % VW ? VW - 1 : 0), VW);
  p.C = (int)ceil_div(nv, sv::rows::kDiBwThreads * sv::rows::kDiBwU);
  p.SV = sv::rows::kDiBwThreads * sv::rows::kDiBwU;
  const long long grid = (long long)p.R * p.C;
  if (grid > 0x7fffffffll) return SV_ERR_UNSUPPORTED;
  sv::rows::distill_backward_kernel<T><<<(unsigned)grid, sv::rows::kDiBwThreads, 0, stream>>>(p);
  return launched();
}

// What the three distillation calls check alike.
sv_status check_distill(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                        const float* logprobs, int k, float temperature) {
  if (!rows_ok(R, V) || !dtype_ok(dtype) || k < 1 || k > SV_MAX_TOP_K || !temperature_ok(temperature))
    return SV_ERR_INVALID_ARG;
  if (R == 0) return SV_OK;
  if (!student || !indices || !logprobs || !aligned16(student)) return SV_ERR_INVALID_ARG;
  return SV_OK;
}

sv::rows::DistillParams distill_params(int R, int V, const void* student, const int32_t* indices,
                                       const float* logprobs, const float* tail, int k, float temperature,
                                       const float* weight) {
  sv::rows::DistillParams p{};
  p.R = R;
  p.V = V;
  p.k = k;
  exponent_scale(temperature, &p.c, &p.c_lo);
  p.inv_t = 1.0 / (double)temperature;
  p.student = student;
  p.indices = indices;
  p.logprobs = logprobs;
  p.tail = tail;
  p.weight = weight;
  return p;
}

}  // namespace

extern "C" sv_status sv_adjust_logits(int B, int gamma, int V, const void* logits, sv_dtype dtype, void* out,
                                      const int32_t* draft_tokens, const int32_t* gamma_b, const int32_t* history,
                                      int H, const int32_t* history_len, const int32_t* prompt_len,
                                      const float* repetition, const float* frequency, const float* presence,
                                      const int32_t* bias_tokens, const float* bias_values, int NB,
                                      const uint32_t* mask, int M, const int32_t* mask_index, sv_stream_t stream) {
  if (B < 0 || gamma < 0 || gamma > SV_MAX_GAMMA || !rows_ok((long long)B * (gamma + 1), V) || !dtype_ok(dtype) ||
      H < 0 || H > SV_MAX_HISTORY || NB < 0 || NB > SV_MAX_BIAS || M < 0 || M > SV_MAX_MASKS)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  const size_t bytes = (size_t)B * (gamma + 1) * (size_t)V * elem_size(dtype);
  if (!logits || !out || !aligned16(logits) || !aligned16(out) || !same_or_apart(logits, out, bytes))
    return SV_ERR_INVALID_ARG;
  if (history && H > 0 && !history_len) return SV_ERR_INVALID_ARG;
  if (NB > 0 && (!bias_tokens || !bias_values)) return SV_ERR_INVALID_ARG;
  if (mask && !mask_index && (long long)M != (long long)B * (gamma + 1)) return SV_ERR_INVALID_ARG;
  sv::rows::AdjustParams p{};
  p.B = B;
  p.G1 = gamma + 1;
  p.V = V;
  p.logits = logits;
  p.out = out;
  p.copy = out != logits;
  p.draft = gamma > 0 ? draft_tokens : nullptr;
  p.gamma_b = gamma_b;
  p.history = H > 0 ? history : nullptr;
  p.H = H;
  p.history_len = history_len;
  p.prompt_len = prompt_len;
  p.repetition = repetition;
  p.frequency = frequency;
  p.presence = presence;
  p.count = (repetition || frequency || presence) && (p.history || p.draft);
  p.bias_tokens = bias_tokens;
  p.bias_values = bias_values;
  p.NB = NB;
  p.mask = mask;
  p.M = M;
  p.W = (V + 31) / 32;
  p.mask_index = mask_index;
  if (!p.copy && !p.count && !p.NB && !p.mask) return SV_OK;   // nothing to do in place
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SV_DTYPE_F32: return launch_adjust<float>(p, s);
    case SV_DTYPE_BF16: return launch_adjust<__nv_bfloat16>(p, s);
    default: return launch_adjust<__half>(p, s);
  }
}

extern "C" size_t sv_top_logits_workspace_bytes(int R, int V, int k) {
  if (!rows_ok(R, V) || k < 1 || k > SV_MAX_TOP_K) return 0;
  if (top_by_rows(R)) return kAlign;   // nothing passes between CTAs
  // one size for every type: a float32 row has the most slices
  const size_t a = top_layout(R, V, k, 4, sm_count()).total, b = top_layout(R, V, k, 8, sm_count()).total;
  return std::max<size_t>(std::max(a, b), kAlign);
}

extern "C" sv_status sv_top_logits(int R, int V, const void* logits, sv_dtype dtype, int k, float temperature,
                                   int32_t* indices, float* logprobs, float* tail, void* workspace,
                                   size_t workspace_bytes, sv_stream_t stream) {
  if (!rows_ok(R, V) || !dtype_ok(dtype) || k < 1 || k > SV_MAX_TOP_K || !temperature_ok(temperature))
    return SV_ERR_INVALID_ARG;
  if (R == 0) return SV_OK;
  if (!logits || !aligned16(logits) || !indices || !logprobs || !tail) return SV_ERR_INVALID_ARG;
  const TopLayout L = top_layout(R, V, k, vec_width(dtype), sm_count());
  if (!workspace || !aligned16(workspace) || workspace_bytes < sv_top_logits_workspace_bytes(R, V, k))
    return SV_ERR_WORKSPACE;
  if ((long long)R * L.H > 0x7fffffffll) return SV_ERR_UNSUPPORTED;
  sv::rows::TopParams p{};
  p.R = R;
  p.V = V;
  p.k = k;
  p.H = L.H;
  p.SV = L.SV;
  // tau from one maximum per thread, or from more where k is near the number
  // of threads (a slice then lists about 1.4 k elements)
  p.KP = 1;
  while (p.KP < 8 && sv::rows::kTlThreads * p.KP < 2 * k) p.KP *= 2;
  exponent_scale(temperature, &p.c, &p.c_lo);
  p.inv_t = two_float(1.0 / (double)temperature);
  p.logits = logits;
  p.indices = indices;
  p.logprobs = logprobs;
  p.tail = tail;
  unsigned char* w = static_cast<unsigned char*>(workspace);
  p.ticket = reinterpret_cast<int*>(w + L.ticket);
  p.part = reinterpret_cast<float4*>(w + L.part);
  p.lists = reinterpret_cast<unsigned long long*>(w + L.lists);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SV_DTYPE_F32: return launch_top<float>(p, s);
    case SV_DTYPE_BF16: return launch_top<__nv_bfloat16>(p, s);
    default: return launch_top<__half>(p, s);
  }
}

extern "C" sv_status sv_distill_forward(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                                        const float* logprobs, const float* tail, int k, float temperature,
                                        const float* weight, float* loss, float* stats, sv_stream_t stream) {
  const sv_status st = check_distill(R, V, student, dtype, indices, logprobs, k, temperature);
  if (st != SV_OK || R == 0) return st;
  if (!loss || (stats && !aligned16(stats))) return SV_ERR_INVALID_ARG;
  sv::rows::DistillParams p = distill_params(R, V, student, indices, logprobs, tail, k, temperature, weight);
  p.loss = loss;
  p.stats = stats;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SV_DTYPE_F32: return launch_distill<float, false>(p, s);
    case SV_DTYPE_BF16: return launch_distill<__nv_bfloat16, false>(p, s);
    default: return launch_distill<__half, false>(p, s);
  }
}

extern "C" sv_status sv_distill_backward(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                                         const float* logprobs, int k, float temperature, const float* weight,
                                         const float* stats, const float* grad_loss, int grad_loss_stride, void* grad,
                                         sv_stream_t stream) {
  const sv_status st = check_distill(R, V, student, dtype, indices, logprobs, k, temperature);
  if (st != SV_OK || R == 0) return st;
  if (!stats || !aligned16(stats) || !grad_loss || grad_loss_stride < 0 || grad_loss_stride > 1 || !grad ||
      !aligned16(grad) ||
      !same_or_apart(student, grad, (size_t)R * V * elem_size(dtype)))
    return SV_ERR_INVALID_ARG;
  sv::rows::DistillParams p = distill_params(R, V, student, indices, logprobs, nullptr, k, temperature, weight);
  p.stats = const_cast<float*>(stats);
  p.grad_loss = grad_loss;
  p.up_stride = grad_loss_stride;
  p.grad = grad;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SV_DTYPE_F32: return launch_distill_backward<float>(p, s);
    case SV_DTYPE_BF16: return launch_distill_backward<__nv_bfloat16>(p, s);
    default: return launch_distill_backward<__half>(p, s);
  }
}

extern "C" sv_status sv_distill_loss_grad(int R, int V, const void* student, sv_dtype dtype, const int32_t* indices,
                                          const float* logprobs, const float* tail, int k, float temperature,
                                          const float* weight, float* loss, void* grad, sv_stream_t stream) {
  const sv_status st = check_distill(R, V, student, dtype, indices, logprobs, k, temperature);
  if (st != SV_OK || R == 0) return st;
  if (!loss || !grad || !aligned16(grad) || !same_or_apart(student, grad, (size_t)R * V * elem_size(dtype)))
    return SV_ERR_INVALID_ARG;
  sv::rows::DistillParams p = distill_params(R, V, student, indices, logprobs, tail, k, temperature, weight);
  p.loss = loss;
  p.grad = grad;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SV_DTYPE_F32: return launch_distill<float, true>(p, s);
    case SV_DTYPE_BF16: return launch_distill<__nv_bfloat16, true>(p, s);
    default: return launch_distill<__half, true>(p, s);
  }
}
