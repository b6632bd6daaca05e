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
// 8192 tokens, 8 heads of 128, attend_kernel takes 78 us for 24 rows, and took
// 100 for 32; attend_wide_kernel takes 88 us for 32, and for fewer, which it pads,
// no less.
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
// the most part.  us with the workspace -> joined, heads of 128, sequences of half
// to all of the tokens above them (all of them for a single one), tables as wide:
//   segments, rows            700          4096          8192         12200         16384
//   8 (8 heads),  1    8.7 ->  4.8  13.1 ->  7.1  20.0 ->  9.8  23.6 -> 12.5  23.8 -> 15.2
//  72 (8 heads),  1   10.6 ->  6.7  15.9 -> 11.2  20.7 -> 16.0  25.8 -> 20.9  29.7 -> 24.7
//  48 (8 heads), 16   11.9 ->  8.4  17.1 -> 13.2  21.5 -> 18.8  25.0 -> 24.1  31.9 -> 31.8
//  24 (8 heads), 24   12.7 ->  8.8  17.0 -> 13.2  20.4 -> 17.3  22.0 -> 21.6  28.1 -> 28.2
//  33 (11 heads), 24  13.0 ->  9.0  17.8 -> 13.3  21.6 -> 17.4  26.0 -> 21.7  31.8 -> 28.3
//  32 (8 heads), 40   13.5 ->  8.8  22.9 -> 12.7  26.0 -> 18.4  27.8 -> 23.9  31.7 -> 29.3
//  24 (8 heads), 72   17.1 ->  8.9  25.0 -> 13.2  30.9 -> 18.8  34.2 -> 24.3  36.7 -> 29.8
//  33 (3 heads), 256  15.6 ->  9.1  25.7 -> 13.3  27.9 -> 19.0  30.6 -> 24.5  34.4 -> 29.8
// The lengths are on the device; a table that is wider than its sequences need is
// taken for what it could hold.
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
