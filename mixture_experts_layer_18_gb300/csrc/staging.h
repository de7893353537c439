// staging.h - turns of a warp's two staging buffers, which bulk copies drain.
// No CUDA header, so that the order can be checked without a GPU.
#pragma once

#ifdef __CUDACC__
#define STAGING_HD __host__ __device__ __forceinline__
#else
#define STAGING_HD inline
#endif

namespace moe {

// Boxes go to the first buffer and the second in turn, one copy group each
// (an empty one for a box that is left out), so that all but the newest group
// read means that the buffer whose turn it is may be written.  A block that
// takes both buffers waits for every group, and commits an empty group behind
// its own: whatever follows, the newest group never reads the first buffer.
// `Copies` has wait_read<N>() (all but the newest N groups have been read) and
// commit(); the calls are one thread's.
template <class Copies>
struct StagingTurns {
  Copies copies;
  STAGING_HD void before_box() { copies.template wait_read<1>(); }
  STAGING_HD void after_box() { copies.commit(); }
  STAGING_HD void before_both() { copies.template wait_read<0>(); }
  STAGING_HD void after_both() {
    copies.commit();
    copies.commit();
  }
};

}  // namespace moe
