#include "sv_attend_launch.cuh"

sv_status sv::cache::launch_attend_f16(const AttendParams& p, int D, void* workspace, cudaStream_t stream) {
  return D == 64 ? launch_attend_rows<__half, 64>(p, workspace, stream) : launch_attend_rows<__half, 128>(p, workspace, stream);
}
