// Tensor-core runs of the linear attention (linear_chunk.cu).
#pragma once

#include <cuda.h>

#include "linear.cuh"

namespace gdr {

struct LinChunkMaps {
  CUtensorMap m[4];   // of LinProblem::t
};

}  // namespace gdr

// Tensor maps of the tensors the runs use; false if the driver refuses one.
bool gdr_linear_chunk_maps(const gdr::LinProblem &p, gdr::LinChunkMaps *maps);
cudaError_t gdr_launch_linear_chunk(const gdr::LinProblem &p, const gdr::LinChunkMaps &maps, bool phase1, bool pdl,
                                    cudaStream_t s);
// Read and clear this file's device error word; synchronises `s`; -1 on a CUDA error.
int gdr_linear_read_device_error(cudaStream_t s);
