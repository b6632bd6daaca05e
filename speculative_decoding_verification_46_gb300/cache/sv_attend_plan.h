// How an attention call is cut into tiles of rows, CTAs and workspace.
#pragma once

#include <algorithm>

#include "sv_attend.cuh"
#include "sv_attend_wide.cuh"
#include "sv_cache_host.h"

namespace sv {
namespace cache {

inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

// Rows of a tile where the call is not joined in one launch: up to 24 go to attend_kernel; more to attend_wide_kernel, in
// as few tiles as its 80 rows allow, of equal size.  At 32 sequences of up to
// 8192 tokens, 8 heads of 128, attend_kernel takes 74 us for 24 rows, and took
// 100 for 32; attend_wide_kernel takes 85
// us for 32, and for fewer, which it pads, no less.
inline int attend_tile_rows(int rows) {
  if (rows <= 24) return (std::max(rows, 1) + 7) / 8 * 8;
  const int tiles = (rows + kWdMostRows - 1) / kWdMostRows;
  return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}
inline int attend_ctas(int TR) { return sm_count() * (TR == 8 ? 4 : TR == 16 ? 3 : 2); }

// Whether a call is joined in one launch, by a cluster of eight CTAs a segment
// (tiles of 8, 16 or 24 rows, as few as there can be, of equal size): the table
// is short enough for eight, and all clusters are on the GPU at once (with 3 or 2
// CTAs an SM some SMs' places do not make up a cluster: 57 segments of 16 rows
// would take two turns).  Rows beyond 24 read the cache once a tile, from L2 for
// the most part.  us with the workspace -> joined, 8 heads of 128 (2 in the last
// line), tables and up to all of their tokens:
//   sequences, rows   1024          8192          12200         16384
//        1,   1        8.8 ->  5.2  20.8 ->  9.8  24.5 -> 11.4  24.9 -> 14.4
//        9,   1       11.7 ->  6.9  20.7 -> 15.8  26.7 -> 22.1  29.9 -> 24.7
//        6,  16       13.0 ->  8.9  20.9 -> 17.3  26.5 -> 24.7  29.9 -> 28.6
//        7,  16       13.5 -> 12.9  21.3 -> 21.7                31.1 -> 34.7
//        3,  24       13.2 ->  9.3  19.4 -> 17.6  23.8 -> 22.4  25.4 -> 26.9
//        2,  40       14.8 ->  9.4  24.5 -> 18.5  27.3 -> 23.1  30.2 -> 29.3
//        1,  72       17.1 ->  9.8  29.8 -> 19.3  32.6 -> 24.0  35.5 -> 30.0
//        1, 256       15.0 ->  9.6  27.5 -> 19.2  29.9 -> 23.8  32.0 -> 30.1
struct AttendJoined {
  int rows, segments;                     // of a tile; 0 segments: not joined
};
inline AttendJoined attend_joined(const AttendParams& p) {
  const int rows = p.rows * p.G, tiles = (rows + 23) / 24;
  const int TR = ((rows + tiles - 1) / tiles + 7) / 8 * 8;
  const int places = TR == 8 ? attend_ctas(TR) : attend_ctas(TR) / 8 * 7;
  const long long segments = (long long)p.B * p.H * tiles;
  const bool few = segments * kAtCluster <= places && (long long)p.N * p.page <= kAtShort;
  return AttendJoined{TR, few ? (int)segments : 0};
}

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
