// norm_rows.hpp -- how the norm's backward kernels share out rows: arithmetic on counts alone,
// for the host and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// How the rows are shared out among slots, ranges of rows that one workgroup or one of its
// `streams` walks over.  A slot has whole groups (rows that share a gate row), or, where
// groups are fewer than the slots wanted, an even part of one group; the streams of a
// workgroup then have parts of the same group.
struct Split {
  int64_t rows, groups, slots;
  int parts;        // slots per group; 0: a slot has whole groups
  int streams;      // slots per workgroup, whose sums leave it as one
  int64_t sums;     // workgroups: rows of each result's sums in the workspace
};

__host__ __device__ inline Split split_rows(int64_t rows, int64_t groups, int streams, int64_t workgroups) {
  Split s = {rows, groups, 0, 0, streams, 0};
  int64_t want = workgroups * streams;
  if (want > rows) want = rows;
  if (groups >= want) {
    s.slots = want;
  } else {
    const int64_t per = rows / groups;
    // (rounded down: a few workgroups more than the CUs hold at once take twice as long)
    int64_t parts = workgroups / groups * streams;
    if (parts < streams) parts = streams;
    if (parts > per) parts = per;
    s.parts = (int)((parts + streams - 1) / streams * streams);   // (the last may be empty)
    s.slots = groups * s.parts;
  }
  s.sums = (s.slots + streams - 1) / streams;
  return s;
}

__host__ __device__ inline void slot_rows(const Split &s, int64_t slot, int64_t &r0, int64_t &r1) {
  const int64_t per = s.rows / s.groups;
  if (slot >= s.slots) {
    r0 = r1 = s.rows;
  } else if (s.parts == 0) {
    r0 = slot * s.groups / s.slots * per;
    r1 = (slot + 1) * s.groups / s.slots * per;
  } else {
    const int64_t g = slot / s.parts, i = slot % s.parts;
    r0 = g * per + i * per / s.parts;
    r1 = g * per + (i + 1) * per / s.parts;
  }
}

// Whether the form of the kernel that closes one group per slot, whether or not the slot has
// rows, may be taken: where groups are in parts, whose sums all go through the workspace.
// Slots of whole groups write the gate's gradient themselves, and where one row is all there is,
// its workgroup also has slots without rows, which must not write (zero) in its place.
__host__ __device__ inline bool one_group(const Split &s) { return s.parts > 0; }

}  // namespace nvfp4
