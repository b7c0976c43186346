// quantize_fp8_block and gated_act_fp8_block: bf16 rows, or act(gate) * up of
// [gate | up] rows, to E4M3 codes with a scale for every 128 columns (or, of a
// weight, for every 128 x 128 block), in one read and one write.  The scale's
// definition is in block_scale.cuh.
//
// Bound: HBM.  An element is 2 bytes read (4 with a gate) and 1 written, a
// block 4 bytes more.
//
// Rows: eight lanes hold a block, two neighbouring vectors each (one 32-byte load
// and one 16-byte store), so its maximum is three shuffles and no block waits for
// another.  The blocks of all rows are one list that groups of
// eight lanes walk with the grid's stride; a group's place in the row moves on
// by a stride that the host has split into rows and blocks, so nothing is
// divided in the loop.  CTAs are persistent.  With an activation the next block's
// vectors are on their way while this one's are reduced and written (five CTAs an
// SM: 4096 x 2 x 11008 37.3 us, without 38.0); without one, more CTAs are worth
// more (eight: 4096 x 4096 9.6 us, four with the loads ahead 10.2).
#include "block_scale.cuh"
#include "kernels.h"

namespace gbf {
namespace {

constexpr int kQbThreads = 256;
constexpr int kQbGroups = kQbThreads / kSegLanes;

// act(g) in float32, to (10 + 4 |z|) 2^-23 of itself, z the logistic function's
// argument, or (10 + g^2) 2^-23 (erf): the exponential's argument is rounded, and its
// error grows with it.  The scale is a float32 that the activation's error reaches,
// so neither the 11-bit hardware tanh nor an approximation with an absolute error
// only is used here.  SiLU and the tanh GELU are g times the logistic function of
// g, or of 2u with the GELU's inner polynomial u, by the exponential of a negative
// argument, so that nothing overflows on the way.
//
// The erf GELU is g Phi(g), Phi(g) = erfc(-g / sqrt 2) / 2.  With z = |g| / sqrt 2
// and t = 1 / (1 + z / 2), erfc(z) = t exp(-z^2 + P(t)) (the form of Press et al.,
// Numerical Recipes, 6.2; the fit is this library's), where P is a polynomial
// of degree 8 fitted to log(erfc(z) exp(z^2) / t) at Chebyshev nodes of t for z up
// to 9.6 (relative error 2.4e-7, 3.8e-7 with the coefficients and Horner's steps
// in float32; from z = 9.4 on the exponential is below float32's range).
// erfcf took 99 us where this takes 62 (4096 x 2 x 11008; the tanh GELU 43, SiLU 37).
GBF_DEVICE float gelu_erf_of(float g) {
  const float t = rcp_approx(fmaf(fabsf(g), 0.353553391f, 1.0f));
  float p = 0.0844842046f;
  p = fmaf(p, t, -0.583680928f);
  p = fmaf(p, t, 1.53390813f);
  p = fmaf(p, t, -1.84880638f);
  p = fmaf(p, t, 0.89813441f);
  p = fmaf(p, t, -0.255226195f);
  p = fmaf(p, t, 0.444004029f);
  p = fmaf(p, t, 0.992339432f);
  p = fmaf(p, t, -1.26515687f);
  const float erfc = t * __expf(fmaf(-0.5f * g, g, p));
  const float h = 0.5f * erfc * (g >= 0.0f ? fminf(g, 16.0f) : g);      // an infinite g is not multiplied by 0
  return g >= 0.0f ? g - h : h;
}

template <int ACT>
GBF_DEVICE float gate_of(float g) {
  if (ACT == kActGeluErf) return gelu_erf_of(g);
  const float z = ACT == kActGeluTanh ? 2.0f * 0.7978845608f * fmaf(0.044715f * g, g * g, g) : g;
  const float e = __expf(-fabsf(z));
  return g * __fdividef(z >= 0.0f ? 1.0f : e, 1.0f + e);
}

// 32 contiguous bytes that stay out of L1: one load where they are aligned to
// their size (WIDE), else two.
template <bool WIDE>
GBF_DEVICE void ld_stream32(const void* p, uint4 (&v)[2]) {
  if (WIDE) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                 : "l"(p));
  } else {
    v[0] = ld_stream(p);
    v[1] = ld_stream(static_cast<const uint4*>(p) + 1);
  }
}

template <int ACT, bool WIDE>
__global__ void __launch_bounds__(kQbThreads, ACT == kActNone ? 8 : 5) quant_rows_kernel(const QuantBlockArgs a) {
  constexpr bool GATED = ACT != kActNone;
  const int l = threadIdx.x & (kSegLanes - 1);
  const int blocks = static_cast<int>(block_count(a.d));
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQbGroups + threadIdx.x / kSegLanes;
  int64_t row = first / blocks;
  int block = static_cast<int>(first - row * blocks);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t total = a.rows * blocks, stride = static_cast<int64_t>(gridDim.x) * kQbGroups;
  // column of vector k of a block (a width is whole pairs of vectors)
  auto column = [&](int b, int k) { return static_cast<int64_t>(b) * kBlockCols + (l * kSegVecs + k) * 8; };
  uint4 v[kSegVecs] = {}, u[kSegVecs] = {};
  auto load = [&](int64_t at, int64_t r, int b) {
    const __nv_bfloat16* g = x + r * a.d * (GATED ? 2 : 1);
    if (at < total && column(b, 0) < a.d) {
      ld_stream32<WIDE>(g + column(b, 0), v);
      if (GATED) ld_stream32<WIDE>(g + a.d + column(b, 0), u);
    } else {                                                  // behind the row's end: zeros
#pragma unroll
      for (int k = 0; k < kSegVecs; ++k) v[k] = u[k] = uint4{};
    }
  };
  load(first, row, block);
  // a warp's groups go on together, as long as its first one has a block
  for (int64_t at = first; at - (threadIdx.x & 31) / kSegLanes < total; at += stride) {
    float y[kSegVecs][8], m = 0.0f;
    uint4 own[kSegVecs], up[kSegVecs];
#pragma unroll
    for (int k = 0; k < kSegVecs; ++k) {
      own[k] = v[k];
      up[k] = u[k];
    }
    int64_t next_row = row + a.step_rows;
    int next = block + a.step_blocks;
    if (next >= blocks) {
      next -= blocks;
      ++next_row;
    }
    if (GATED) load(at + stride, next_row, next);
#pragma unroll
    for (int k = 0; k < kSegVecs; ++k) {
      bf16x8_to_f32(own[k], y[k]);
      if (GATED) {
        float w[8];
        bf16x8_to_f32(up[k], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[k][i] = gate_of<ACT>(y[k][i]) * w[i];
      }
      m = GATED ? amax8(y[k], m) : amax8(own[k], m);
    }
    const float s = scale_of(seg_max(m)), r = __frcp_rn(s);
    if (at < total && column(block, 0) < a.d) {
      const uint2 c0 = codes8(y[0], r), c1 = codes8(y[1], r);
      st_16(a.q_out + row * a.d + column(block, 0), make_uint4(c0.x, c0.y, c1.x, c1.y));
    }
    if (at < total && l == 0) a.scales[row * blocks + block] = s;
    row = next_row;
    block = next;
    if (!GATED) load(at + stride, row, block);
  }
}

// A weight's 128 x 128 blocks, one a CTA: 256 threads hold the block (16 columns
// of four rows each, 32 rows apart), so it is read once.
constexpr int kQtThreads = 256;
constexpr int kQtRows = kQtThreads / kSegLanes;               // rows of one pass
constexpr int kQtPasses = kBlockCols / kQtRows;

template <bool WIDE>
__global__ void __launch_bounds__(kQtThreads, 4) quant_tiles_kernel(const QuantBlockArgs a) {
  __shared__ float part[kQtThreads / 32];
  const int64_t across = block_count(a.d);
  const int64_t up = blockIdx.x / across, over = blockIdx.x - up * across;
  const int64_t col = over * kBlockCols + threadIdx.x % kSegLanes * 16;
  const int64_t row0 = up * kBlockCols + threadIdx.x / kSegLanes;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
  pdl_wait();
  pdl_launch_dependents();
  uint4 v[kQtPasses][kSegVecs] = {};
#pragma unroll
  for (int k = 0; k < kQtPasses; ++k)
    if (row0 + k * kQtRows < a.rows && col < a.d) ld_stream32<WIDE>(x + (row0 + k * kQtRows) * a.d + col, v[k]);
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < kQtPasses; ++k) m = amax8(v[k][0], amax8(v[k][1], m));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQtThreads / 32; ++w) m = max_nan(m, part[w]);
  const float s = scale_of(m), r = __frcp_rn(s);
#pragma unroll
  for (int k = 0; k < kQtPasses; ++k)
    if (row0 + k * kQtRows < a.rows && col < a.d) {
      float y0[8], y1[8];
      bf16x8_to_f32(v[k][0], y0);
      bf16x8_to_f32(v[k][1], y1);
      const uint2 c0 = codes8(y0, r), c1 = codes8(y1, r);
      st_16(a.q_out + (row0 + k * kQtRows) * a.d + col, make_uint4(c0.x, c0.y, c1.x, c1.y));
    }
  if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
}

template <int ACT, bool WIDE>
cudaError_t launch_wide(QuantBlockArgs a, cudaStream_t stream) {
  const int64_t blocks = block_count(a.d), need = (a.rows * blocks + kQbGroups - 1) / kQbGroups;
  const int64_t fit = resident<quant_rows_kernel<ACT, WIDE>>(kQbThreads), grid = need < fit ? need : fit;
  a.step_rows = grid * kQbGroups / blocks;
  a.step_blocks = static_cast<int>(grid * kQbGroups % blocks);
  return launch_pdl(quant_rows_kernel<ACT, WIDE>, dim3(static_cast<unsigned>(grid)), dim3(kQbThreads), 0, stream, a);
}

template <int ACT>
cudaError_t launch_rows(const QuantBlockArgs& a, cudaStream_t stream) {
  return reinterpret_cast<uintptr_t>(a.x) % 32 == 0 ? launch_wide<ACT, true>(a, stream) : launch_wide<ACT, false>(a, stream);
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
  auto kern = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 ? quant_tiles_kernel<true> : quant_tiles_kernel<false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles)), dim3(kQtThreads), 0, stream, a);
}

}  // namespace gbf
