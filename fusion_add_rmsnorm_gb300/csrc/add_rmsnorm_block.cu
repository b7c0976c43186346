// add_rmsnorm_fp8_block: (gated) residual add -> RMSNorm / _noweight /
// AdaRMSNorm -> E4M3 codes with a scale for every 128 columns of the row, one
// read and one write per element.  The arithmetic up to the norm's output y is
// add_rmsnorm_fp8's; the scale's definition is in block_scale.cuh.
//
// Bound: HBM; an element is 4 bytes read and 3 written, a block 4 bytes more.
//
// Layout: eight lanes hold a block of 128 columns (two 16-byte vectors each),
// TPR threads a row, NS blocks a lane group; a thread's columns are the same in
// every row, so its factors (weight, gate, AdaRMSNorm scale and shift) stay
// packed in registers for the whole launch.  A row needs two sums over its
// threads: the mean square (shuffles, then per-warp partials and one barrier
// where a row has several warps) and each block's maximum (three shuffles).
// CTAs are persistent and hold the next row's x and res in registers while
// they reduce and write the current one.
#include "block_scale.cuh"
#include "kernels.h"

namespace gbf {
namespace {

constexpr int kNbThreads = 512;           // most threads of a CTA

// Factors per column: the gate (GATED) first, then the weight (WEIGHT) or the
// scale and the shift (ADA).
template <int MODE, bool GATED>
constexpr int factors() { return (GATED ? 1 : 0) + (MODE == kNormWeight ? 1 : 0) + (MODE == kNormAda ? 2 : 0); }

// One rounding: x + r, or g * x + r, of eight bf16.
template <bool GATED>
GBF_DEVICE uint4 residual(uint4 g, uint4 x, uint4 r) {
  uint4 o;
  const __nv_bfloat162* pg = reinterpret_cast<const __nv_bfloat162*>(&g);
  const __nv_bfloat162* px = reinterpret_cast<const __nv_bfloat162*>(&x);
  const __nv_bfloat162* pr = reinterpret_cast<const __nv_bfloat162*>(&r);
  __nv_bfloat162* po = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) po[i] = GATED ? __hfma2(pg[i], px[i], pr[i]) : __hadd2(px[i], pr[i]);
  return o;
}

// NS blocks a lane group.  One or two: the next row's loads are in flight while
// this one is reduced and written; four: they begin with the row.  The factors
// are held in registers but for AdaRMSNorm's at two blocks and all at four, which
// are read from L1 where they are used (16384 x 8192 gated AdaRMSNorm: 149 us, held
// and spilled 181).  CTAS: an SM's at one block a lane group, three for streaming
// (32768 x 4096: 143 us, two 150), two for fewer rows (777 x 2736: 3.8 us, three 4.4).
// What four cost above 16,384 columns, against a floor of 141: 4096 x 32768 weighted
// 172 us, gated AdaRMSNorm 222 (8192 x 16384 weighted, two blocks: 143).
template <int MODE, bool GATED, int NS, int CTAS>
__global__ void __launch_bounds__(NS == 1 ? kNbThreads / 2 : kNbThreads, CTAS)
add_rmsnorm_block_kernel(const AddRmsNormBlockArgs a) {
  constexpr bool AHEAD = NS <= 2, HELD = NS == 1 || (NS == 2 && MODE != kNormAda);
  constexpr int NV = NS * kSegVecs, NF = factors<MODE, GATED>();
  const int tpr = a.tpr, rows_per_cta = blockDim.x / tpr;
  const int t = threadIdx.x % tpr;
  const int groups = tpr / kSegLanes;
  const int hidden = static_cast<int>(a.hidden), blocks = static_cast<int>(block_count(a.hidden));
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(a.res_in);
  __nv_bfloat16* res_out = static_cast<__nv_bfloat16*>(a.res_out);
  const void* source[3] = {GATED ? a.gate : (MODE == kNormWeight ? a.weight : a.ada_scale),
                           GATED ? (MODE == kNormWeight ? a.weight : a.ada_scale) : a.ada_shift, a.ada_shift};
  pdl_wait();

  // column of vector k: block t / 8 + (k / 2) * groups, vector t % 8 or 8 further
  auto column = [&](int k) {
    return (t / kSegLanes + k / kSegVecs * groups) * kBlockCols + (t % kSegLanes + k % kSegVecs * kSegLanes) * 8;
  };
  auto factor = [&](int j, int k) { return ld_cached(static_cast<const __nv_bfloat16*>(source[j]) + column(k)); };

  const int64_t stride = static_cast<int64_t>(gridDim.x) * rows_per_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + threadIdx.x / tpr;
  uint4 xr[NV] = {}, rr[NV] = {};
  auto load_row = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (r < a.rows && column(k) < hidden) {
        xr[k] = ld_stream(x + r * hidden + column(k));
        rr[k] = ld_stream(res + r * hidden + column(k));
      }
  };
  if (AHEAD) load_row(row);
  uint4 held[HELD ? NV : 1][NF > 0 ? NF : 1] = {};
  if (HELD)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        if (column(k) < hidden) held[HELD ? k : 0][j] = factor(j, k);
  pdl_launch_dependents();

  // Partial sums of a row's warps, two copies by trip parity: a warp that
  // writes trip n + 2's has passed the barrier of trip n + 1, which every warp
  // reaches after it has read trip n's.
  __shared__ float part[2][kNbThreads / 32];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_cta;
  int parity = 0;
  for (int64_t base = first; base < a.rows; base += stride, row += stride, parity ^= 1) {
    if (!AHEAD) load_row(row);
    uint4 h[NV];
    float sum = 0.0f;
    const bool live = row < a.rows;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = live && column(k) < hidden;
      const uint4 g = !GATED ? uint4{} : HELD ? held[HELD ? k : 0][0] : in ? factor(0, k) : uint4{};
      h[k] = in ? residual<GATED>(g, xr[k], rr[k]) : uint4{};
      if (in) st_16(res_out + row * hidden + column(k), h[k]);
      float f[8];
      bf16x8_to_f32(h[k], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
    }
    if (AHEAD) load_row(row + stride);
    sum = group_sum(sum, tpr < 32 ? tpr : 32);
    if (tpr > 32) {                                           // one row a CTA
      if ((threadIdx.x & 31) == 0) part[parity][threadIdx.x >> 5] = sum;
      __syncthreads();
      sum = 0.0f;
      for (int w = 0; w < tpr / 32; ++w) sum += part[parity][w];
    }
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(hidden) + a.eps);
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float y[kSegVecs][8], m = 0.0f;
#pragma unroll
      for (int v = 0; v < kSegVecs; ++v) {
        const int k = n * kSegVecs + v;
        const bool in = column(k) < hidden;
        bf16x8_to_f32(h[k], y[v]);
        constexpr int F = GATED ? 1 : 0;
        float f0[8], f1[8];
        if (MODE != kNormNoWeight) {
          const int j1 = MODE == kNormAda ? F + 1 : F;
          bf16x8_to_f32(HELD ? held[HELD ? k : 0][F] : in ? factor(F, k) : uint4{}, f0);
          bf16x8_to_f32(HELD ? held[HELD ? k : 0][j1] : in ? factor(j1, k) : uint4{}, f1);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[v][i] *= inv;
          if (MODE == kNormWeight) y[v][i] *= f0[i];
          if (MODE == kNormAda) y[v][i] = fmaf(y[v][i], 1.0f + f0[i], f1[i]);
        }
        if (in) m = amax8(y[v], m);
      }
      const float s = scale_of(seg_max(m)), r = __frcp_rn(s);
#pragma unroll
      for (int v = 0; v < kSegVecs; ++v) {
        const int c = column(n * kSegVecs + v);
        if (live && c < hidden) *reinterpret_cast<uint2*>(a.q_out + row * hidden + c) = codes8(y[v], r);
      }
      const int block = t / kSegLanes + n * groups;
      if (live && t % kSegLanes == 0 && block < blocks) a.scales[row * blocks + block] = s;
    }
  }
}

template <int MODE, bool GATED, int NS, int CTAS>
cudaError_t launch(const AddRmsNormBlockArgs& a, int threads, cudaStream_t stream) {
  auto kern = add_rmsnorm_block_kernel<MODE, GATED, NS, CTAS>;
  const int rows_per_cta = threads / a.tpr;
  const int64_t need = (a.rows + rows_per_cta - 1) / rows_per_cta, fit = resident<add_rmsnorm_block_kernel<MODE, GATED, NS, CTAS>>(threads);
  return launch_pdl(kern, dim3(static_cast<unsigned>(need < fit ? need : fit)), dim3(threads), 0, stream, a);
}

template <int MODE, bool GATED>
cudaError_t launch_plan(AddRmsNormBlockArgs a, cudaStream_t stream) {
  // One block a lane group, two where a row then still fits a warp or would not
  // fit 256 threads, four (without loads ahead) where it would not fit 512.
  const int64_t blocks = block_count(a.hidden);
  const int ns = blocks > 2 * kNbThreads / kSegLanes ? 4 : blocks > 256 / kSegLanes || (blocks > 4 && blocks <= 8) ? 2 : 1;
  const int64_t need = (blocks + ns - 1) / ns * kSegLanes;
  int tpr = kSegLanes;
  while (tpr < need && tpr < 32) tpr *= 2;
  if (need > 32) tpr = static_cast<int>((need + 31) / 32 * 32);
  a.tpr = tpr;
  const int threads = tpr > 32 ? tpr : 128;
  if (ns == 4) return launch<MODE, GATED, 4, 1>(a, threads, stream);
  if (ns == 2) return launch<MODE, GATED, 2, 1>(a, threads, stream);
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const bool streaming = a.rows / (threads / tpr) > 8LL * sms;          // over eight CTAs an SM
  return streaming ? launch<MODE, GATED, 1, 3>(a, threads, stream) : launch<MODE, GATED, 1, 2>(a, threads, stream);
}

}  // namespace

cudaError_t launch_add_rmsnorm_block(AddRmsNormBlockArgs a, cudaStream_t stream) {
  const bool gated = a.gate != nullptr;
  switch (a.mode) {
    case kNormWeight: return gated ? launch_plan<kNormWeight, true>(a, stream) : launch_plan<kNormWeight, false>(a, stream);
    case kNormNoWeight:
      return gated ? launch_plan<kNormNoWeight, true>(a, stream) : launch_plan<kNormNoWeight, false>(a, stream);
    case kNormAda: return gated ? launch_plan<kNormAda, true>(a, stream) : launch_plan<kNormAda, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gbf
