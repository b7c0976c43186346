// Scales found from the data: one float32 for every 128 columns of a row (or
// 128 x 128 block of a weight), E4M3 codes of the values over it.
//
//   scale = max(amax * RN(1 / 448), 2^-100),  code = e4m3_rne_sat(y * RN(1 / scale))
//
// in binary32.  448 is E4M3's largest value, so a block's largest element
// lands there; 2^-100 keeps the reciprocal finite where a block holds only
// zeros (or values below 448 * 2^-100).  The maximum passes NaN on: a block
// that holds one gets scale NaN and NaN codes, one that holds an infinity gets
// scale infinity, NaN codes at the infinities and zeros elsewhere, so that
// code * scale is never a finite number that stands for neither.
#pragma once

#include <atomic>

#include "block.h"
#include "common.cuh"

namespace gbf {

constexpr int kSegLanes = 8;              // lanes that hold a block of 128 columns, two 8-column vectors each
constexpr int kSegVecs = 2;               // which two of the block's sixteen, each kernel says

// The larger of two values, NaN if either is.
GBF_DEVICE float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

GBF_DEVICE float amax8(const float (&v)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

// The same of eight packed bf16, in bf16: exact, and without widening them.
GBF_DEVICE float amax8(uint4 v, float m) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 a = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
  return max_nan(max_nan(__low2float(a), __high2float(a)), m);
}

// Maximum over the aligned eight lanes of a block; every lane of the warp takes part.
GBF_DEVICE float seg_max(float m) {
#pragma unroll
  for (int o = kSegLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

GBF_DEVICE float scale_of(float amax) { return max_nan(amax * (1.0f / 448.0f), 0x1p-100f); }

// Eight codes of v over the scale whose reciprocal is r.
GBF_DEVICE uint2 codes8(const float (&v)[8], float r) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * r;
  return f32x8_to_e4m3x8(q);
}

// CTAs of KERNEL with `threads` threads (a multiple of 32, at most 1024) that fit
// on the GPU at once: a persistent grid's size.  Asked for once on each device.
template <auto KERNEL>
int64_t resident(int threads) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][33];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool keep = dev >= 0 && dev < kDevices;
  int n = keep ? known[dev][threads / 32].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    int sms = 0, per_sm = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, threads, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
    cudaGetLastError();
    n = (sms < 1 ? 1 : sms) * per_sm;
    if (keep) known[dev][threads / 32].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace gbf
