// Where a thread's elements of a row lie, and which 16-byte pieces of the row its loads ask
// for: the norm's index arithmetic, plain C++ so that a host program can go through it.
#pragma once

#ifdef __CUDACC__
#define FSDP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FSDP_HOST_DEVICE inline
#endif

namespace fsdp {

// Where a thread's 8 kV elements of a row lie.
//   kVector: groups of 8 consecutive elements, read and written as vectors: cols is a
//     multiple of 8 and every row of every array starts on a 16-byte boundary. (A group
//     is whole or absent: one predicate and no branch around a load, so that all of
//     a thread's loads are in flight together.)
//   kShifted: the same groups moved back by the row's own distance from a 16-byte
//     boundary (`phase` elements, the same for all arrays), so that rows of any
//     length are read and written as aligned vectors too; the first and the last group
//     of a row are partly outside, where a load's surplus is dropped (it lies in
//     a 16-byte piece that holds an element of the row) and stores go one by one.
//     (43633 x 769 bf16 with the residual, 268 MB: 224 us strided, see below.)
//   kGroups: 8 consecutive elements from any place, put together from the aligned vectors
//     that hold them (8-bit outputs of other rows: 33520 x 1001 bf16 with the residual, groups
//     of 128: 72 us, 139 one by one; 8194 x 4095 with one scale a row 74 us, 277 strided).
//   kSingles: the same one by one, for rows that a warp holds: all of it would wait for the
//     last, partial group, which goes one by one anyway (260111 x 129: 121 us, 170 by vectors).
//   kStrided: element by element across the row's threads, so that a warp's
//     accesses stay contiguous (other rows).
enum RowMap { kVector, kShifted, kGroups, kSingles, kStrided };

// The row's threads: `t` of `n` (n up to 32: part of a warp or a warp; else the block).
struct RowThreads {
  int t, n;
  int phase;  // kShifted: elements from the last 16-byte boundary to the row's first
};

// First element of group v, or element (v, e) in the strided map.
template <RowMap kMap>
FSDP_HOST_DEVICE int place(const RowThreads& r, int v, int e) {
  const int j = kMap == kStrided ? (v * 8 + e) * r.n + r.t : (v * r.n + r.t) * 8 + e;
  return kMap == kShifted ? j - r.phase : j;
}

// Whether some of the `count` places from j on hold an element of a row of `cols`: what a
// vector load asks for. A row that is not there (cols = 0) has none, whatever its phase.
template <RowMap kMap>
FSDP_HOST_DEVICE bool holds_some(int j, int count, int cols) {
  if (kMap == kVector) return j < cols;  // j >= 0, and a group is whole or absent
  return j < cols && j + count > 0 && cols > 0;
}

}  // namespace fsdp
