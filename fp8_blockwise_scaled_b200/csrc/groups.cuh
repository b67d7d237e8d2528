// Row ranges of groups (experts) given by a device array of offsets: group e
// owns the rows offsets[e] .. offsets[e + 1] - 1 of a matrix of `rows` rows.
//
// The offsets come from a router that ran on the device, so the host cannot
// check them: every range is clamped to [0, rows) and counts as empty when it
// is not increasing, so that a bad array gives wrong results but no access out
// of range.
#pragma once

#include <stdint.h>

namespace fp8blk {

constexpr int kMaxGroups = 1024;     // the kernels keep one word a group in shared memory
constexpr int kGroupBlock = 128;     // rows of a block: tiles and token groups start anew in every group

__device__ __forceinline__ int clamp_row(int r, int rows) { return min(max(r, 0), rows); }

// First row of group e; *size = its number of rows.
__device__ __forceinline__ int group_rows(const int* offsets, int e, int rows, int* size) {
  const int begin = clamp_row(__ldg(offsets + e), rows);
  *size = max(clamp_row(__ldg(offsets + e + 1), rows) - begin, 0);
  return begin;
}

// The whole block (`threads` threads, this one `t`): ends[e] = number of
// `block`-row blocks of groups 0 .. e together (never above rows / block + groups,
// which offsets in order cannot exceed), and, unless null, ranges[e] = (first row,
// number of rows).  All offsets are read at once, one warp adds up.  The caller
// synchronises the block before it reads the result.
__device__ __forceinline__ void build_block_ends(int* ends, int2* ranges, const int* offsets, int groups, int rows, int t,
                                                 int threads, int block = kGroupBlock) {
  for (int e = t; e < groups; e += threads) {
    int size;
    const int begin = group_rows(offsets, e, rows, &size);
    ends[e] = (size + block - 1) / block;
    if (ranges) ranges[e] = make_int2(begin, size);
  }
  __syncthreads();
  if (t >= 32) return;
  const int most = rows / block + groups;
  int before = 0;
  for (int base = 0; base < groups; base += 32) {
    const int e = base + t;
    int n = e < groups ? ends[e] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, n, o);
      if (t >= o) n = min(n + v, most);
    }
    n = min(n + before, most);
    if (e < groups) ends[e] = n;
    before = __shfl_sync(0xFFFFFFFFu, n, 31);
  }
}

// The group that owns block b < ends[groups - 1], given that it is group e or a
// later one (callers walk the blocks upwards).
__device__ __forceinline__ int find_group(const int* ends, int groups, int b, int e) {
  if (b < ends[e]) return e;
  int lo = e + 1, hi = groups - 1;     // ends[lo - 1] <= b < ends[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b < ends[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The same by a whole warp, without a first guess: how many groups end at or before b.
__device__ __forceinline__ int find_group_warp(const int* ends, int groups, int b, int lane) {
  int e = 0;
  for (int base = 0; base < groups; base += 32) {
    const int i = base + lane;
    const unsigned before = __ballot_sync(0xFFFFFFFFu, i < groups && ends[i] <= b);
    e += __popc(before);
    if (before != 0xFFFFFFFFu) break;
  }
  return e;
}

}  // namespace fp8blk
