// Internal interface between the C-ABI layer (abi.cu) and the block-scaled
// 8-bit operators.  Argument structs are passed to kernels by value.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "block_plan.h"

namespace gbf {

// ------------------------------------- add + RMSNorm + block-scaled FP8
struct AddRmsNormBlockArgs {
  const void* x;
  const void* res_in;
  void* res_out;
  const void* gate;       // nullable
  const void* weight;     // kNormWeight
  const void* ada_scale;  // kNormAda
  const void* ada_shift;  // kNormAda
  uint8_t* q_out;
  float* scales;          // [rows, block_count(hidden)]
  int64_t rows;
  int64_t hidden;
  float eps;
  int mode;
  int tpr;                // threads per row (set by the launcher)
};

cudaError_t launch_add_rmsnorm_block(AddRmsNormBlockArgs a, cudaStream_t stream);

// --------------------------- (gated activation or copy) + block-scaled FP8
struct QuantBlockArgs {
  const void* x;          // bf16 [rows, d], or [rows, 2d] (gate | up) with an activation
  uint8_t* q_out;         // [rows, d]
  float* scales;          // [rows, block_count(d)], or one row for every 128 rows
  int64_t rows, d;
  int act;                // kActNone: quantise x itself
  int64_t step_rows;      // one grid stride, in whole rows and blocks (set by the launcher)
  int step_blocks;
};

cudaError_t launch_quant_rows(QuantBlockArgs a, cudaStream_t stream);
cudaError_t launch_quant_tiles(const QuantBlockArgs& a, cudaStream_t stream);

// ---------------------------------------------- Linear on block-scaled codes
struct LinearBlockArgs {
  const uint8_t* x;       // [m, k] E4M3 codes
  const float* x_scales;  // [m, block_count(k)]
  const uint8_t* w;       // [n, k] E4M3 codes
  const float* w_scales;  // [block_count(n), block_count(k)]
  const void* bias;       // bf16 [n], nullable
  void* y;                // bf16 [m, n]
  unsigned int* err;
  int64_t m, n, k;
  int act;
};

// What a call of these sizes (m > 0) launches on the current device.
cudaError_t linear_block_plan(int64_t m, int64_t n, int64_t k, LinearBlockPlan* plan, LinearBlockRoom* room);
cudaError_t launch_linear_block(const LinearBlockArgs& a, cudaStream_t stream, const char** why);
cudaError_t launch_linear_block_pair(const LinearBlockArgs& a, const LinearBlockPlan& plan, int clusters,
                                     cudaStream_t stream, const char** why);
// Clusters of 1 to kBpMaxSplit pairs that fit on the current device at once (0 where it
// does not say); raises the pair kernel's shared memory limit.
void linear_block_clusters(int (&clusters)[kBpMaxSplit + 1]);

}  // namespace gbf
