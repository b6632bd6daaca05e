// The attention kernels' launches, for the translation unit of each element type.
#pragma once

#include "sv_attend_plan.h"

namespace sv {
namespace cache {

template <typename T, int D, int TR>
sv_status launch_attend(AttendParams p, void* workspace, cudaStream_t stream) {
  const int ctas = attend_ctas(TR);
  const AttendLayout L = attend_layout(TR, D);
  p.desc = reinterpret_cast<int4*>(static_cast<unsigned char*>(workspace) + L.desc);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + L.part);
  static std::atomic<bool> set[64];
  if constexpr (TR <= 24) {
    using Shape = AttendShape<T, D, TR / 8>;
    auto kern = attend_kernel<T, D, TR / 8, false>;
    if (!allow_smem(set, (const void*)kern, Shape::kSmem)) return SV_ERR_CUDA;
    kern<<<ctas, Shape::kThreads, Shape::kSmem, stream>>>(p);
  } else {
    auto kern = attend_wide_kernel<T, D, TR / 16>;
    if (!allow_smem(set, (const void*)kern, WideShape<T, D, TR / 16>::kSmem)) return SV_ERR_CUDA;
    kern<<<ctas, kWdThreads, WideShape<T, D, TR / 16>::kSmem, stream>>>(p);
  }
  const sv_status st = launched();
  if (st != SV_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, TR * 32 / kAtJoinThreads);
  cfg.blockDim = dim3(kAtJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D>, p, TR) != cudaSuccess) {
    cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return launched();
}

template <typename T, int D, int TR>
sv_status launch_joined(const AttendParams& p, int segments, cudaStream_t stream) {
  using Shape = AttendShape<T, D, TR / 8>;
  auto kern = attend_kernel<T, D, TR / 8, true>;
  static std::atomic<bool> set[64];
  if (!allow_smem(set, (const void*)kern, Shape::kJoinedSmem)) return SV_ERR_CUDA;
  cudaLaunchAttribute cluster[1];
  cluster[0].id = cudaLaunchAttributeClusterDimension;
  cluster[0].val.clusterDim.x = kAtCluster;
  cluster[0].val.clusterDim.y = 1;
  cluster[0].val.clusterDim.z = 1;
  return launch(kern, dim3(segments * kAtCluster), Shape::kThreads, Shape::kJoinedSmem, stream, p, cluster);
}

template <typename T, int D>
sv_status launch_attend_rows(const AttendParams& p, void* workspace, cudaStream_t stream) {
  const AttendJoined joined = attend_joined(p);
  if (joined.segments > 0) switch (joined.rows) {
      case 8: return launch_joined<T, D, 8>(p, joined.segments, stream);
      case 16: return launch_joined<T, D, 16>(p, joined.segments, stream);
      default: return launch_joined<T, D, 24>(p, joined.segments, stream);
    }
  switch (attend_tile_rows(p.rows * p.G)) {
    case 8: return launch_attend<T, D, 8>(p, workspace, stream);
    case 16: return launch_attend<T, D, 16>(p, workspace, stream);
    case 24: return launch_attend<T, D, 24>(p, workspace, stream);
    case 32: return launch_attend<T, D, 32>(p, workspace, stream);
    case 48: return launch_attend<T, D, 48>(p, workspace, stream);
    case 64: return launch_attend<T, D, 64>(p, workspace, stream);
    default: return launch_attend<T, D, 80>(p, workspace, stream);
  }
}

}  // namespace cache
}  // namespace sv
