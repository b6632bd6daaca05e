// Host side of the operators on the paged 4-bit cache: argument validation and
// launches for the C ABI declared in include/specverify_cache.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "specverify_cache.h"
#include "sv_attend_plan.h"
#include "sv_kv4.cuh"
#include "sv_plan.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool model_type(sv_dtype dt) { return dt == SV_DTYPE_BF16 || dt == SV_DTYPE_F16; }
bool page_ok(int page) { return page >= 16 && page <= SV_MAX_CACHE_PAGE && page % 16 == 0; }
bool rows_ok(int B, int gamma) {
  return B >= 0 && gamma >= 0 && gamma < SV_MAX_CACHE_ROWS && (long long)B * (gamma + 1ll) <= SV_MAX_CACHE_ROWS;
}
bool cache_ok(int heads, int D, int page, int pages) {
  return heads >= 1 && heads <= SV_MAX_CACHE_HEADS && (D == 64 || D == 128) && page_ok(page) && pages >= 0 &&
         (long long)pages * page <= SV_MAX_CACHE_SLOTS;
}
bool strides_ok(const int64_t* s) {
  if (!s) return false;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] % 8) return false;
  return true;
}

// The bytes from x on of [B][rows][heads][D] 16-bit elements through strides.
size_t extent(const int64_t* strides, int B, int rows, int heads, int D) {
  return 2 * ((size_t)(B - 1) * strides[0] + (size_t)(rows - 1) * strides[1] + (size_t)(heads - 1) * strides[2] + D);
}
// a's na bytes and b's nb have nothing in common
bool apart(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + na <= y || y + nb <= x;
}
size_t cache_bytes(int pages, int heads, int page, int D) { return (size_t)pages * heads * page * (D + 8); }

using sv::cache::allow_smem;
using sv::cache::launched;

// ---------------------------------------------------------------- store

sv::cache::StoreParams store_params(int R, int rows, int heads, int page, int pages, const int32_t* slots) {
  sv::cache::StoreParams p{};
  p.R = R;
  p.rows = rows;
  p.H = heads;
  p.page = page;
  p.slots_end = (long long)pages * page;
  p.slots = slots;
  return p;
}

// CTAs for a group of D / 8 lanes per (two rows, head); 0: more groups than an
// int counts (whose rows no card holds)
unsigned store_grid(int R, int heads, int D) {
  const long long groups = ((long long)R + 1) / 2 * heads;
  const int per_cta = sv::cache::kStoreThreads / (D / 8);
  return groups > 0x7fffffffll ? 0u : (unsigned)((groups + per_cta - 1) / per_cta);
}

bool attend_sizes_ok(int gamma, int heads, int G, int D) {
  return gamma >= 0 && gamma <= SV_MAX_GAMMA && heads >= 1 && heads <= SV_MAX_CACHE_HEADS && G >= 1 &&
         G <= SV_MAX_CACHE_GROUP && (D == 64 || D == 128);
}

}  // namespace

extern "C" sv_status sv_plan_round(int B, int gamma, int page, int N, int pool, int32_t* lengths, const int32_t* kept,
                                   const int32_t* gamma_b, int32_t* block_table, int32_t* blocks, int32_t* free_blocks,
                                   int32_t* free_count, int32_t* slots, int32_t* positions, int32_t* status,
                                   sv_stream_t stream) {
  if (!rows_ok(B, gamma) || B > SV_MAX_PLAN_SEQUENCES || !page_ok(page) || N < 0 || pool < 0 ||
      (long long)B * N > SV_MAX_CACHE_SLOTS || (long long)N * page > SV_MAX_CACHE_SLOTS ||
      (long long)pool * page > SV_MAX_CACHE_SLOTS)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!lengths || !blocks || !free_count || !slots || !positions || !status || (N > 0 && !block_table) ||
      (pool > 0 && !free_blocks))
    return SV_ERR_INVALID_ARG;
  sv::cache::PlanParams p{};
  p.B = B;
  p.rows = gamma + 1;
  p.page = page;
  p.N = N;
  p.pool = pool;
  p.whole = aligned16(slots) && aligned16(positions);
  p.lengths = lengths;
  p.kept = kept;
  p.gamma_b = gamma_b;
  p.table = block_table;
  p.blocks = blocks;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.slots = slots;
  p.positions = positions;
  p.status = status;
  static std::atomic<bool> set[64];
  if (!allow_smem(set, (const void*)sv::cache::plan_round_kernel, sv::cache::plan_smem(SV_MAX_PLAN_SEQUENCES)))
    return SV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.ids = SV_MAX_CACHE_SLOTS / page;
  p.slots_here = (long long)B * p.rows <= sv::cache::kPlanFew;
  cudaLaunchAttribute attr[1];
  sv_status st;
  if ((long long)B * p.rows <= sv::cache::kPlanMany) {
    sv::cache::plan_round_kernel<<<1, sv::cache::kPlanThreads, sv::cache::plan_smem(B), s>>>(p);
    st = launched();
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = sv::cache::kPlanCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    st = launch(sv::cache::plan_round_kernel, dim3(sv::cache::kPlanCtas), sv::cache::kPlanThreads, sv::cache::plan_smem(B), s, p,
                attr);
  }
  if (st != SV_OK || p.slots_here) return st;
  const long long groups = (long long)B * ((p.rows + 3) / 4);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return launch(sv::cache::plan_slots_kernel,
                dim3((unsigned)((groups + sv::cache::kPlanSlotThreads - 1) / sv::cache::kPlanSlotThreads)),
                sv::cache::kPlanSlotThreads, 0, s, p, attr);
}

extern "C" sv_status sv_append_kv4(int B, int gamma, int heads, int D, int page, int pages, const void* k,
                                   const int64_t* k_strides, const void* v, const int64_t* v_strides, sv_dtype dtype,
                                   const int32_t* slots, void* cache, sv_stream_t stream) {
  if (!rows_ok(B, gamma) || !cache_ok(heads, D, page, pages) || !model_type(dtype) || !strides_ok(k_strides) ||
      !strides_ok(v_strides))
    return SV_ERR_INVALID_ARG;
  if (B == 0 || pages == 0) return SV_OK;
  if (!k || !v || !slots || !cache || !aligned16(k) || !aligned16(v) || !aligned16(cache)) return SV_ERR_INVALID_ARG;
  if (!apart(k, extent(k_strides, B, gamma + 1, heads, D), cache, cache_bytes(pages, heads, page, D)) ||
      !apart(v, extent(v_strides, B, gamma + 1, heads, D), cache, cache_bytes(pages, heads, page, D)))
    return SV_ERR_INVALID_ARG;
  sv::cache::StoreParams p = store_params(B * (gamma + 1), gamma + 1, heads, page, pages, slots);
  p.k = k;
  p.v = v;
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = k_strides[i];
    p.vs[i] = v_strides[i];
  }
  p.cache = static_cast<unsigned char*>(cache);
  const unsigned grid = store_grid(p.R, heads, D);
  if (grid == 0) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using namespace sv::cache;
  if (dtype == SV_DTYPE_BF16) {
    if (D == 64) append_kv4_kernel<__nv_bfloat16, 64><<<grid, kStoreThreads, 0, s>>>(p);
    else append_kv4_kernel<__nv_bfloat16, 128><<<grid, kStoreThreads, 0, s>>>(p);
  } else {
    if (D == 64) append_kv4_kernel<__half, 64><<<grid, kStoreThreads, 0, s>>>(p);
    else append_kv4_kernel<__half, 128><<<grid, kStoreThreads, 0, s>>>(p);
  }
  return launched();
}

extern "C" sv_status sv_read_kv4(int R, int heads, int D, int page, int pages, const void* cache, sv_dtype dtype,
                                 const int32_t* slots, void* k, void* v, sv_stream_t stream) {
  if (R < 0 || R > SV_MAX_CACHE_ROWS || !cache_ok(heads, D, page, pages) || !model_type(dtype))
    return SV_ERR_INVALID_ARG;
  if (R == 0) return SV_OK;
  if (!slots || !k || !v || !aligned16(k) || !aligned16(v) || (pages > 0 && (!cache || !aligned16(cache))))
    return SV_ERR_INVALID_ARG;
  const size_t bytes = (size_t)R * heads * D * 2;
  if (!apart(k, bytes, v, bytes) || !apart(k, bytes, cache, cache_bytes(pages, heads, page, D)) ||
      !apart(v, bytes, cache, cache_bytes(pages, heads, page, D)))
    return SV_ERR_INVALID_ARG;
  sv::cache::StoreParams p = store_params(R, 1, heads, page, pages, slots);
  p.cache = static_cast<unsigned char*>(const_cast<void*>(cache));
  p.ko = k;
  p.vo = v;
  const unsigned grid = store_grid(R, heads, D);
  if (grid == 0) return SV_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using namespace sv::cache;
  if (dtype == SV_DTYPE_BF16) {
    if (D == 64) read_kv4_kernel<__nv_bfloat16, 64><<<grid, kStoreThreads, 0, s>>>(p);
    else read_kv4_kernel<__nv_bfloat16, 128><<<grid, kStoreThreads, 0, s>>>(p);
  } else {
    if (D == 64) read_kv4_kernel<__half, 64><<<grid, kStoreThreads, 0, s>>>(p);
    else read_kv4_kernel<__half, 128><<<grid, kStoreThreads, 0, s>>>(p);
  }
  return launched();
}

extern "C" size_t sv_attend_kv4_workspace_bytes(int gamma, int heads, int G, int D) {
  if (!attend_sizes_ok(gamma, heads, G, D)) return 0;
  return sv::cache::attend_layout(sv::cache::attend_tile_rows((gamma + 1) * G), D).total;
}

extern "C" sv_status sv_attend_kv4(int B, int gamma, int heads, int G, int D, int page, int pages, int N, const void* q,
                                   const int64_t* q_strides, sv_dtype dtype, const void* cache,
                                   const int32_t* block_table, const int32_t* lengths, const int32_t* gamma_b,
                                   float scale, void* out, float* lse, int fill, void* workspace,
                                   size_t workspace_bytes, sv_stream_t stream) {
  if (!rows_ok(B, gamma) || !attend_sizes_ok(gamma, heads, G, D) || !cache_ok(heads, D, page, pages) || N < 0 ||
      (long long)B * N > SV_MAX_CACHE_SLOTS || (long long)N * page > SV_MAX_CACHE_SLOTS || !model_type(dtype) ||
      !strides_ok(q_strides) || !(scale > 0.f) || !std::isfinite(scale * 1.44269504f))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!q || !lengths || !out || !aligned16(q) || !aligned16(out) || (N > 0 && !block_table) ||
      (pages > 0 && (!cache || !aligned16(cache))))
    return SV_ERR_INVALID_ARG;
  // (a CTA may write a row while another still reads q)
  const size_t out_bytes = (size_t)B * (gamma + 1) * heads * G * D * 2;
  if (!apart(out, out_bytes, q, extent(q_strides, B, gamma + 1, heads * G, D)) ||
      !apart(out, out_bytes, cache, cache_bytes(pages, heads, page, D)))
    return SV_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) || workspace_bytes < sv_attend_kv4_workspace_bytes(gamma, heads, G, D))
    return SV_ERR_WORKSPACE;
  sv::cache::AttendParams p{};
  p.B = B;
  p.rows = gamma + 1;
  p.H = heads;
  p.G = G;
  p.page = page;
  p.pages = pages;
  p.N = N;
  p.q = q;
  for (int i = 0; i < 3; ++i) p.qs[i] = q_strides[i];
  p.cache = static_cast<const unsigned char*>(cache);
  p.table = block_table;
  p.lengths = lengths;
  p.gamma_b = gamma_b;
  p.scale = scale * 1.44269504f;
  p.out = out;
  p.lse = lse;
  p.fill = fill;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == SV_DTYPE_BF16 ? sv::cache::launch_attend_bf16(p, D, workspace, s)
                                : sv::cache::launch_attend_f16(p, D, workspace, s);
}
