// cross_kernels.h -- the attention kernels of pa_cross_attention and the rule
// that chooses among them.
#pragma once

#include <cstddef>

namespace pa {

struct CrossKernel {
  const void* fn;        // __global__ void fn(CrossArgs)
  int threads, ctas_per_sm, workers_per_cta;
  size_t smem;           // dynamic shared memory of a CTA
  int cols, keys;        // columns of an item, keys of a tile
  int min_tiles;         // a worker's share is at least this long
};

CrossKernel cross_kernel(int num_seqs, int num_rows, int group, int head_dim, int elem_bytes);

// fp32 arithmetic on the CUDA cores (cross_simt.cu)
CrossKernel cross_simt_kernel_info(int head_dim, int elem_bytes);

// bf16, many columns: tcgen05 tensor cores (cross_tc.cu)
CrossKernel cross_tc_kernel_info(int head_dim);

}  // namespace pa
