// Page copies of a state pool (state_copy.cu).
#pragma once

#include <cuda_runtime.h>

namespace gdr {

// Pairs of one launch, passed by value: 4 KB of kernel arguments.
constexpr int kMaxCopyPairs = 480;
struct CopyPairs {
  int n;
  int src[kMaxCopyPairs];   // -1: zeros
  int dst[kMaxCopyPairs];
};
// Up to these go as 256 bytes (8 pages forked: 10.5 us a call, with 4 KB of arguments 11.7).
constexpr int kFewCopyPairs = 31;

}  // namespace gdr

// No pair's destination may be another pair's source or destination.  The
// largest launch has 2^31 - 1 blocks of 32 KB.
cudaError_t gdr_launch_state_copy(float *pool, size_t page_floats, int layers, int pages, const gdr::CopyPairs &pairs,
                                  cudaStream_t s);
