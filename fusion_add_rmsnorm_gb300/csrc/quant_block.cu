// quantize_fp8_block and gated_act_fp8_block: bf16 rows, or act(gate) * up of
// [gate | up] rows, to E4M3 codes with a scale for every 128 columns (or, of a
// weight, for every 128 x 128 block), in one read and one write.  The scale's
// definition is in block_scale.cuh.
//
// Bound: HBM.  An element is 2 bytes read (4 with a gate) and 1 written, a
// block 4 bytes more.
//
// Rows: eight lanes hold a block, so its maximum is three shuffles and no
// block waits for another.  The blocks of all rows are one list that groups of
// eight lanes walk with the grid's stride; a group's place in the row moves on
// by a stride that the host has split into rows and blocks, so nothing is
// divided in the loop.
#include "block_scale.cuh"
#include "kernels.h"

namespace gbf {
namespace {

constexpr int kQbThreads = 128;
constexpr int kQbGroups = kQbThreads / kSegLanes;

// act(g) in float32.  SiLU and the tanh GELU (g times the logistic function of
// g, or of 2u with the GELU's inner polynomial u) take the exponential of a
// negative argument only, so nothing overflows on the way; the scale is a
// float32 that the activation's error reaches, so the 11-bit hardware tanh is
// not used here.  The erf GELU by erfcf, whose small values are exact to
// their own size.
template <int ACT>
GBF_DEVICE float gate_of(float g) {
  if (ACT == kActGeluErf) return 0.5f * g * erfcf(g * -0.70710678118654752f);
  const float z = ACT == kActGeluTanh ? 2.0f * 0.7978845608f * fmaf(0.044715f * g, g * g, g) : g;
  const float e = __expf(-fabsf(z));
  return g * __fdividef(z >= 0.0f ? 1.0f : e, 1.0f + e);
}

template <int ACT>
__global__ void __launch_bounds__(kQbThreads) quant_rows_kernel(const QuantBlockArgs a) {
  constexpr bool GATED = ACT != kActNone;
  const int l = threadIdx.x & (kSegLanes - 1);
  const int blocks = static_cast<int>(block_count(a.d));
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQbGroups + threadIdx.x / kSegLanes;
  int64_t row = first / blocks;
  int block = static_cast<int>(first - row * blocks);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
  pdl_wait();
  pdl_launch_dependents();
  // a warp's four groups leave together: its first one is the last to run out
  const int64_t total = a.rows * blocks, stride = static_cast<int64_t>(gridDim.x) * kQbGroups;
  for (int64_t at = first; at - ((threadIdx.x & 31) / kSegLanes) < total; at += stride) {
    const bool live = at < total;
    const __nv_bfloat16* g = x + row * a.d * (GATED ? 2 : 1);
    uint4 v[kSegVecs] = {}, u[kSegVecs] = {};
    int64_t col[kSegVecs];
    bool in[kSegVecs];
#pragma unroll
    for (int k = 0; k < kSegVecs; ++k) {
      col[k] = static_cast<int64_t>(block) * kBlockCols + (l + k * kSegLanes) * 8;
      in[k] = live && col[k] < a.d;
      if (in[k]) {
        v[k] = ld_stream(g + col[k]);
        if (GATED) u[k] = ld_stream(g + a.d + col[k]);
      }
    }
    float y[kSegVecs][8], m = 0.0f;
#pragma unroll
    for (int k = 0; k < kSegVecs; ++k) {
      bf16x8_to_f32(v[k], y[k]);
      if (GATED) {
        float up[8];
        bf16x8_to_f32(u[k], up);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[k][i] = gate_of<ACT>(y[k][i]) * up[i];
      }
      m = amax8(y[k], m);                                     // a vector behind the row's end is zeros
    }
    const float s = scale_of(seg_max(m)), r = __frcp_rn(s);
#pragma unroll
    for (int k = 0; k < kSegVecs; ++k)
      if (in[k]) *reinterpret_cast<uint2*>(a.q_out + row * a.d + col[k]) = codes8(y[k], r);
    if (live && l == 0) a.scales[row * blocks + block] = s;
    row += a.step_rows;
    block += a.step_blocks;
    if (block >= blocks) {
      block -= blocks;
      ++row;
    }
  }
}

// A weight's 128 x 128 blocks, one a CTA: 256 threads hold the block (eight
// vectors each, 16 rows apart), so it is read once.
constexpr int kQtThreads = 256;
constexpr int kQtRows = kQtThreads / (kBlockCols / 8);        // rows of one pass
constexpr int kQtVecs = kBlockCols / kQtRows;

__global__ void __launch_bounds__(kQtThreads) quant_tiles_kernel(const QuantBlockArgs a) {
  __shared__ float part[kQtThreads / 32];
  const int64_t across = block_count(a.d);
  const int64_t up = blockIdx.x / across, over = blockIdx.x - up * across;
  const int64_t col = over * kBlockCols + (threadIdx.x % (kBlockCols / 8)) * 8;
  const int64_t row0 = up * kBlockCols + threadIdx.x / (kBlockCols / 8);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
  pdl_wait();
  pdl_launch_dependents();
  uint4 v[kQtVecs] = {};
#pragma unroll
  for (int k = 0; k < kQtVecs; ++k)
    if (row0 + k * kQtRows < a.rows && col < a.d) v[k] = ld_stream(x + (row0 + k * kQtRows) * a.d + col);
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < kQtVecs; ++k) {
    float y[8];
    bf16x8_to_f32(v[k], y);
    m = amax8(y, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQtThreads / 32; ++w) m = max_nan(m, part[w]);
  const float s = scale_of(m), r = __frcp_rn(s);
#pragma unroll
  for (int k = 0; k < kQtVecs; ++k)
    if (row0 + k * kQtRows < a.rows && col < a.d) {
      float y[8];
      bf16x8_to_f32(v[k], y);
      *reinterpret_cast<uint2*>(a.q_out + (row0 + k * kQtRows) * a.d + col) = codes8(y, r);
    }
  if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
}

template <int ACT>
cudaError_t launch_rows(QuantBlockArgs a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t blocks = block_count(a.d), need = (a.rows * blocks + kQbGroups - 1) / kQbGroups;
  // at most 16 CTAs per SM; what fewer registers would allow is not needed to fill HBM
  const int64_t grid = need < 16LL * sms ? need : 16LL * sms;
  a.step_rows = grid * kQbGroups / blocks;
  a.step_blocks = static_cast<int>(grid * kQbGroups % blocks);
  return launch_pdl(quant_rows_kernel<ACT>, dim3(static_cast<unsigned>(grid)), dim3(kQbThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_quant_rows(QuantBlockArgs a, cudaStream_t stream) {
  switch (a.act) {
    case kActNone: return launch_rows<kActNone>(a, stream);
    case kActGeluTanh: return launch_rows<kActGeluTanh>(a, stream);
    case kActGeluErf: return launch_rows<kActGeluErf>(a, stream);
    case kActSilu: return launch_rows<kActSilu>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_quant_tiles(const QuantBlockArgs& a, cudaStream_t stream) {
  const int64_t tiles = block_count(a.rows) * block_count(a.d);
  return launch_pdl(quant_tiles_kernel, dim3(static_cast<unsigned>(tiles)), dim3(kQtThreads), 0, stream, a);
}

}  // namespace gbf
