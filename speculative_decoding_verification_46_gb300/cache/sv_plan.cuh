// The bookkeeping between two rounds (sv_plan_round).
//
// One cluster of CTAs, so that its steps are separated by the hardware's
// cluster barrier in one launch: (1) every CTA forms the same prefix sums of
// the pages that the sequences give and take, in its own shared memory; (2)
// what is given goes onto the free list; (3) what is taken comes off it; (4)
// slots and positions, where there are few; a second kernel has those of many.
// Steps 2 to 4 are spread over all threads by flat indices, which the prefix sums
// lead back to their sequence.
//
// It is all latency: the bytes (8.5 at most of each row, 4 of each page) take less
// than a microsecond, the launch, the loads of a sequence's numbers, the sums
// over the CTA and the barriers behind one another the rest.  A round and the
// next: 5.8 us for one sequence, 12.1 for 1024 of 9 rows, 12.5 for 64 prompts of
// 4096 tokens.  Every sequence's number in shared memory (five of 8192: 160 KB) is
// what limits a call to 8192.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sv_kv4.cuh"

namespace sv {
namespace cache {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;        // of a cluster with many rows
// Rows whose slots the first kernel forms; those of more are a kernel of their
// own.  (Two rounds, one kernel against two: 8.1 and 9.3 us for 64 sequences of 9
// rows, 8.6 and 9.0 for one of 2048, 11.2 and 9.9 for 256 of 9, 19 and 12 for 1024.)
constexpr int kPlanFew = 2048;
// Rows whose pages are moved by more CTAs than one.  (Two rounds, one CTA against
// eight: 11.6 and 12.3 us for 1024 sequences of 9 rows, 9.1 and 10.1 for 4 prompts
// of 4096, 12.5 and 10.3 for 16, 27.6 and 12.7 for 64.)
constexpr int kPlanMany = 32768;
constexpr int kPlanSlotThreads = 256;
constexpr int kNoPages = 1, kTooLong = 2;

struct PlanParams {
  int B, rows, page, N, pool;       // rows: gamma + 1
  int ids;                          // page ids below it give slots below 2^30
  bool slots_here;                  // plan_round_kernel forms the slots too
  bool whole;                       // slots and positions are 16-byte aligned
  int32_t* lengths;
  const int32_t *kept, *gamma_b;
  int32_t *table, *blocks, *free_blocks, *free_count, *slots, *positions, *status;
};

// Shared memory of the kernel: five integers a sequence.
constexpr size_t plan_smem(int B) { return (size_t)B * 5 * sizeof(int); }

// The sequence that flat index x belongs to: the last one whose sum of those
// before it is at most x.
__device__ __forceinline__ int sequence_of(const int* before, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_round_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int plan_sm[];
  __shared__ int2 warp_sum[kPlanThreads / 32];
  __shared__ int taken;
  int* gives = plan_sm;            // pages given by the sequences before
  int* takes = gives + p.B;        // pages wanted by the sequences before
  int* held = takes + p.B;         // pages that it had
  int* length = held + p.B;        // its new length
  int* part = length + p.B;        // its rows, and its status << 28
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  const unsigned rank = cluster_rank();
  unsigned ctas;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));

  // (1) each thread takes a run of sequences
  const int run = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
  const int count0 = min(max(*p.free_count, 0), p.pool);
  int2 mine = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    const long long len = max(0ll, (long long)p.lengths[b] + (p.kept ? p.kept[b] : 0));
    const int n = p.gamma_b ? min(max(p.gamma_b[b], -1), p.rows - 1) + 1 : p.rows;
    const int has = min(max(p.blocks[b], 0), p.N);
    const long long need = (len + n + p.page - 1) / p.page;
    const bool too_long = need > p.N;
    const int wants = too_long ? has : (int)need;
    gives[b] = max(has - wants, 0);
    takes[b] = max(wants - has, 0);
    held[b] = has;
    length[b] = (int)min(len, 0x7fffffffll);
    part[b] = n | (too_long ? kTooLong << 28 : 0);
    mine.x += gives[b];
    mine.y += takes[b];
  }
  int2 upto = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto.x, m), y = __shfl_up_sync(0xffffffffu, upto.y, m);
    if (lane >= m) {
      upto.x += x;
      upto.y += y;
    }
  }
  if (lane == 31) warp_sum[warp] = upto;
  if (tid == 0) taken = 0;
  __syncthreads();
  if (warp == 0) {
    int2 s = warp_sum[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s.x, m), y = __shfl_up_sync(0xffffffffu, s.y, m);
      if (lane >= m) {
        s.x += x;
        s.y += y;
      }
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int given = warp_sum[kPlanThreads / 32 - 1].x;
  const int there = (int)min((long long)count0 + given, (long long)p.pool);
  int2 before = make_int2(upto.x - mine.x, upto.y - mine.y);
  if (warp > 0) {
    before.x += warp_sum[warp - 1].x;
    before.y += warp_sum[warp - 1].y;
  }
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    const int g = gives[b], t = takes[b];
    gives[b] = before.x;
    takes[b] = before.y;
    before.x += g;
    before.y += t;
    if (t > 0) {
      if (before.y <= there) most = before.y;
      else part[b] |= kNoPages << 28;
    }
  }
  if (most > 0) atomicMax(&taken, most);
  cluster_barrier();   // the state is read, and the sums are there
  const int coming = taken;
  const int NT = kPlanThreads * (int)ctas, at = (int)rank * kPlanThreads + tid;

  // (2) the last page of the last sequence goes onto the list first
  for (int x = at; x < given; x += NT) {
    const int b = sequence_of(gives, p.B, x);
    const int last = b + 1 < p.B ? gives[b + 1] : given;
    int32_t* entry = p.table + (long long)b * p.N + (held[b] - (last - x));
    const long long to = (long long)count0 + given - 1 - x;
    if (to < p.pool) p.free_blocks[to] = __ldcg(entry);
    *entry = -1;
  }
  if (rank == 0) {
    for (int b = tid; b < p.B; b += kPlanThreads) {
      const int st = part[b] >> 28, n = part[b] & 0x0fffffff;
      p.lengths[b] = length[b];
      p.status[b] = st;
      p.blocks[b] = st ? held[b] : (length[b] + n + p.page - 1) / p.page;
    }
    if (tid == 0) *p.free_count = there - coming;
  }
  if (given > 0) cluster_barrier();

  // (3) the first page of the first sequence is the last of the list
  for (int x = at; x < coming; x += NT) {
    const int b = sequence_of(takes, p.B, x);
    p.table[(long long)b * p.N + held[b] + (x - takes[b])] = __ldcg(p.free_blocks + (there - 1 - x));
  }
  if (!p.slots_here) return;
  cluster_barrier();

  // (4)
  const int cells = p.B * p.rows;
#pragma unroll 4
  for (int x = at; x < cells; x += NT) {
    const int b = x / p.rows, i = x - b * p.rows;
    int slot = -1, position = 0;
    if (i < (part[b] & 0x0fffffff)) {
      position = (int)min((long long)length[b] + i, 0x7fffffffll);
      if (part[b] >> 28 == 0) {
        const int c = position / p.page;
        const int id = __ldcg(p.table + (long long)b * p.N + c);
        if (id >= 0 && id < p.ids) slot = id * p.page + (position - c * p.page);
      }
    }
    p.slots[x] = slot;
    p.positions[x] = position;
  }
}

// Slots and positions of many rows, behind the kernel above (which then leaves
// them out): a thread has four neighbouring rows of one sequence, which lie in
// two pages at most.
__global__ void __launch_bounds__(kPlanSlotThreads) plan_slots_kernel(const __grid_constant__ PlanParams p) {
  const int groups = (p.rows + 3) / 4;      // of a sequence
  const long long x = (long long)blockIdx.x * kPlanSlotThreads + threadIdx.x;
  const int b = (int)(x / groups), i = 4 * (int)(x - (long long)b * groups);
  pdl_wait();
  if (b >= p.B) return;
  const int n = p.gamma_b ? min(max(p.gamma_b[b], -1), p.rows - 1) + 1 : p.rows;
  const long long first = (long long)p.lengths[b] + i;
  const bool fine = p.status[b] == 0 && i < n;
  const int c = fine ? (int)(first / p.page) : 0, t = fine ? (int)first - c * p.page : 0;
  int id[2] = {-1, -1};
  if (fine) {
    id[0] = p.table[(long long)b * p.N + c];
    if (t + min(n - i, 4) > p.page) id[1] = p.table[(long long)b * p.N + c + 1];
  }
  int slot[4], position[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int over = t + j >= p.page;
    const int page = id[over];
    slot[j] = fine && i + j < n && page >= 0 && page < p.ids ? page * p.page + t + j - over * p.page : -1;
    position[j] = i + j < n ? (int)min(first + j, 0x7fffffffll) : 0;
  }
  const long long to = (long long)b * p.rows + i;
  if (p.rows % 4 == 0 && p.whole) {
    *reinterpret_cast<int4*>(p.slots + to) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.positions + to) = make_int4(position[0], position[1], position[2], position[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < p.rows) {
        p.slots[to + j] = slot[j];
        p.positions[to + j] = position[j];
      }
  }
}

}  // namespace cache
}  // namespace sv
