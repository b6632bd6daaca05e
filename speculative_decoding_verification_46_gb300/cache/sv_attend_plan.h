// How an attention call is cut into tiles of rows, CTAs and workspace.
#pragma once

#include <algorithm>

#include "sv_attend.cuh"
#include "sv_attend_wide.cuh"
#include "sv_cache_host.h"

namespace sv {
namespace cache {

inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of a tile: up to 24 go to attend_kernel; more to attend_wide_kernel, in
// as few tiles as its 80 rows allow, of equal size.
inline int attend_tile_rows(int rows) {
  if (rows <= 24) return (std::max(rows, 1) + 7) / 8 * 8;
  const int tiles = (rows + kWdMostRows - 1) / kWdMostRows;
  return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}
inline int attend_ctas(int TR) { return sm_count() * (TR == 8 ? 4 : TR == 16 ? 3 : 2); }

struct AttendLayout {
  size_t desc, part, total;
};
inline AttendLayout attend_layout(int TR, int D) {
  AttendLayout L;
  const size_t ctas = attend_ctas(TR);
  L.desc = 0;
  L.part = align_up(ctas * sizeof(int4));
  L.total = L.part + align_up(2 * ctas * part_floats(TR, D) * sizeof(float));
  return L;
}

// The launches of one element type (sv_attend_bf16.cu, sv_attend_f16.cu: they
// take the longest to compile).
sv_status launch_attend_bf16(const AttendParams& p, int D, void* workspace, cudaStream_t stream);
sv_status launch_attend_f16(const AttendParams& p, int D, void* workspace, cudaStream_t stream);

}  // namespace cache
}  // namespace sv
