#include "sv_attend_launch.cuh"

sv_status sv::cache::launch_attend_bf16(const AttendParams& p, int D, void* workspace, cudaStream_t stream) {
  return D == 64 ? launch_attend_rows<__nv_bfloat16, 64>(p, workspace, stream) : launch_attend_rows<__nv_bfloat16, 128>(p, workspace, stream);
}
