// linear_fp8_block: Y = act(X W^T + bias) on E4M3 codes with one float32 scale
// for every 128 columns of an X row and every 128 x 128 block of W, on the
// 5th-generation tensor cores:
//
//   y[m, n] = act(sum_b (sx[m, b] sw[n / 128, b]) sum_{k in block b} x[m, k] w[n, k] + bias[n])
//
// The scales change with every 128 columns of K, so the sum over K cannot stay
// in the tensor core's accumulator: each block's product (one 128-byte K row
// of codes, four MMAs) is a product of its own in tensor memory, which the
// epilogue warps read back and add, times its scale, to float32 registers,
// while the tensor core goes on with the next ones in further accumulators.
//
// linear_block_kernel: the 128 rows of a W block are the MMA's rows (TMEM
// lanes), NX rows of X its columns, so a decode batch of a few rows wastes no
// MMA rows and all of W's bytes are spread over the CTAs.  A thread holds one
// output channel and its NX rows' sums.
//   warp 0     TMA producer: W's 128 and X's NX rows of a K block into a ring
//   warp 1     MMA issuer: four MMAs of 32 K into the next accumulator
//   warp 2     tensor memory
//   warps 4-7  epilogue: accumulators of 32 channels each; the X scales of a
//              block, times W's, go through shared memory one block ahead
// With few output tiles, a cluster of up to eight CTAs cuts K between them and
// adds its partial sums through distributed shared memory, in the order of K,
// so that a result has the same bits in every run.
//
// Every mbarrier wait is bounded, as in gemm_tcgen05.cu: one that gives up
// sets the device error word and an abort flag, every role leaves its loop,
// the MMAs and copies in flight are waited for (bounded), all CTAs of a cluster
// reach its barriers and TMEM is freed.
#include <atomic>

#include "block.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace gbf {
namespace {

constexpr int kLbThreads = 256;
constexpr int kLbRows = 128;              // W rows of a tile: one scale block
constexpr int kLbEpilogue = 4;            // first epilogue warp
constexpr int kLbMaxSplit = 8;            // portable cluster size

// Shared memory of a CTA with NX rows of X: two CTAs an SM up to 64 of them, so
// that one's start and end hide behind the other's loads.
template <int NX>
struct Lb {
  static constexpr int kPerSm = NX <= 64 ? 2 : 1;
  static constexpr int kStageBytes = (kLbRows + NX) * BK_BYTES;
  static constexpr int kStages = NX == 16 ? 6 : NX == 32 ? 5 : NX == 64 ? 4 : 6;
  static constexpr int kAccs = NX == 16 ? 8 : (kPerSm == 2 ? 256 : 512) / NX;     // accumulators in TMEM
  static constexpr int kTmemCols = kAccs * NX;
  static constexpr int kScaleBytes = 4 * 2 * NX * 4;                              // [epilogue warp][2][NX]
};

template <int NX>
struct __align__(8) LbCtl {
  uint64_t full[Lb<NX>::kStages];
  uint64_t empty[Lb<NX>::kStages];
  uint64_t acc_full[Lb<NX>::kAccs];
  uint64_t acc_empty[Lb<NX>::kAccs];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int NX>
constexpr size_t lb_smem() {
  return 1024 /* alignment */ + Lb<NX>::kStages * Lb<NX>::kStageBytes + Lb<NX>::kScaleBytes + sizeof(LbCtl<NX>);
}

struct LinearBlockParams {
  const float* x_scales;
  const float* w_scales;
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;
  unsigned int* err;
  int m, n, blocks;          // blocks: of K
  int m_tiles, n_tiles, split;
  int act;
};

// 16 float32 columns of this warp's 32 TMEM lanes, one lane per thread.
GBF_DEVICE void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

GBF_DEVICE float ld_cluster_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

GBF_DEVICE void sts32f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

template <int NX>
__global__ void __launch_bounds__(kLbThreads, Lb<NX>::kPerSm)
linear_block_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const LinearBlockParams p) {
  using L = Lb<NX>;
  constexpr int S = L::kStages, A = L::kAccs;
  constexpr uint32_t kIdesc = idesc(true, kLbRows, NX);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_w = smem;                                   // S x 128 rows of 128 bytes
  uint8_t* smem_x = smem + S * kLbRows * BK_BYTES;          // S x NX rows of 128 bytes
  uint8_t* smem_s = smem + S * L::kStageBytes;
  LbCtl<NX>* ctl = reinterpret_cast<LbCtl<NX>*>(smem_s + L::kScaleBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.split;
  const int m0 = tile % p.m_tiles * NX, nt = tile / p.m_tiles, n0 = nt * kLbRows;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < A; ++b) {
      mbar_init(&ctl->acc_full[b], 1);
      mbar_init(&ctl->acc_empty[b], 4);                     // one arrive per epilogue warp
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
  }
  if (warp == 2) tmem_alloc<false>(&ctl->tmem_base, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  pdl_wait();
  pdl_launch_dependents();

  float acc[NX];
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        const int s = issued % S;
        if (!mbar_wait<false, false>(&ctl->empty[s], ((issued / S) & 1) ^ 1u, &ctl->abort, p.err)) break;
        mbar_arrive_expect_tx(&ctl->full[s], L::kStageBytes);
        tma_load_2d(smem_w + s * kLbRows * BK_BYTES, &map_w, &ctl->full[s], kb * BK_BYTES, n0);
        tma_load_2d(smem_x + s * NX * BK_BYTES, &map_x, &ctl->full[s], kb * BK_BYTES, m0);
      }
      // every copy has landed before the CTA may go on to leave (at once but after an abort)
      int own = 0;
      for (int i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_wait(&ctl->full[i % S], (i / S) & 1, &own, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      for (int i = 0; i < kb1 - kb0; ++i) {
        const int s = i % S, b = i % A;
        if (!mbar_wait<false, false>(&ctl->acc_empty[b], ((i / A) & 1) ^ 1u, &ctl->abort, p.err)) break;
        if (!mbar_wait<false, false>(&ctl->full[s], (i / S) & 1, &ctl->abort, p.err)) break;
        tc_fence_after();
        const uint32_t w_addr = smem_u32(smem_w + s * kLbRows * BK_BYTES), x_addr = smem_u32(smem_x + s * NX * BK_BYTES);
#pragma unroll
        for (int kk = 0; kk < BK_BYTES / UMMA_K_BYTES; ++kk)
          tc_mma<true, false>(tmem_base + b * NX, smem_desc_sw128(w_addr + kk * UMMA_K_BYTES),
                              smem_desc_sw128(x_addr + kk * UMMA_K_BYTES), kIdesc, kk != 0);
        tc_commit<false>(&ctl->empty[s]);
        tc_commit<false>(&ctl->acc_full[b]);
      }
      tc_commit_self<false>(&ctl->drain);
      int own = 0;
      mbar_wait(&ctl->drain, 0, &own, p.err);
    }
  } else if (warp >= kLbEpilogue) {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp - kLbEpilogue;                 // TMEM lanes 32 * quarter .. + 31
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t sbuf = smem_u32(smem_s) + quarter * 2 * NX * 4;
    constexpr int PER = NX < 32 ? 1 : NX / 32;              // scales a lane fetches
    float next[PER], w_next;                                // multiplied where they are used: no wait here
    auto fetch = [&](int kb) {
      w_next = kb < kb1 ? p.w_scales[static_cast<int64_t>(nt) * p.blocks + kb] : 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int row = m0 + lane + i * 32;
        next[i] = (NX >= 32 || lane < NX) && kb < kb1 && row < p.m
                      ? p.x_scales[static_cast<int64_t>(row) * p.blocks + kb]
                      : 0.0f;
      }
    };
#pragma unroll
    for (int j = 0; j < NX; ++j) acc[j] = 0.0f;
    fetch(kb0);
    for (int i = 0; i < kb1 - kb0; ++i) {
      const int b = i % A;
      const uint32_t sc = sbuf + (i & 1) * NX * 4;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (NX >= 32 || lane < NX) sts32f(sc + (lane + j * 32) * 4, next[j] * w_next);
      fetch(kb0 + i + 1);
      __syncwarp();
      if (!mbar_wait_warp<false>(&ctl->acc_full[b], (i / A) & 1, &ctl->abort, p.err)) break;
      tc_fence_after();
      constexpr int STEP = NX < 32 ? 16 : 32;
#pragma unroll
      for (int c = 0; c < NX; c += STEP) {
        uint32_t r[STEP];
        if constexpr (STEP == 16) tmem_ld_16cols(taddr + b * NX + c, r);
        else tmem_ld_32cols(taddr + b * NX + c, r);
#pragma unroll
        for (int j = 0; j < STEP; j += 4) {
          const float4 f = lds128f(sc + (c + j) * 4);
          const float2 lo = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                       make_float2(f.x, f.y), make_float2(acc[c + j], acc[c + j + 1]));
          const float2 hi = __ffma2_rn(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                                       make_float2(f.z, f.w), make_float2(acc[c + j + 2], acc[c + j + 3]));
          acc[c + j] = lo.x;
          acc[c + j + 1] = lo.y;
          acc[c + j + 2] = hi.x;
          acc[c + j + 3] = hi.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->acc_empty[b]);
    }
    const int ch = quarter * 32 + lane;                     // this thread's row of the W tile
    if (p.split > 1) {
      // the ring is free: the last accumulator came after every copy and MMA
#pragma unroll
      for (int j = 0; j < NX; ++j) sts32f(smem_u32(smem) + (j * kLbRows + ch) * 4, acc[j]);
    } else if (n0 + ch < p.n) {
      const float bias = p.bias ? __bfloat162float(p.bias[n0 + ch]) : 0.0f;
#pragma unroll
      for (int j = 0; j < NX; ++j)
        if (m0 + j < p.m)
          p.y[static_cast<int64_t>(m0 + j) * p.n + n0 + ch] = __float2bfloat16(fast_act(acc[j] + bias, p.act));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, L::kTmemCols);
  }
  if (p.split > 1) {
    cluster_sync();                                         // every CTA's partial sums are in its shared memory
    const int per = NX / p.split, ch = threadIdx.x & (kLbRows - 1);
    for (int j = rank * per + threadIdx.x / kLbRows; j < (rank + 1) * per; j += kLbThreads / kLbRows) {
      const uint32_t at = smem_u32(smem) + (j * kLbRows + ch) * 4;
      float part[kLbMaxSplit], sum = 0.0f;
#pragma unroll
      for (int r = 0; r < kLbMaxSplit; ++r) part[r] = r < p.split ? ld_cluster_f32(map_cluster(at, r)) : 0.0f;
#pragma unroll
      for (int r = 0; r < kLbMaxSplit; ++r) sum += part[r];
      if (m0 + j < p.m && n0 + ch < p.n) {
        const float bias = p.bias ? __bfloat162float(p.bias[n0 + ch]) : 0.0f;
        p.y[static_cast<int64_t>(m0 + j) * p.n + n0 + ch] = __float2bfloat16(fast_act(sum + bias, p.act));
      }
    }
    cluster_sync();                                         // no CTA leaves while another reads its sums
  }
}

// Raises the kernel's shared memory limit once on each device.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int NX>
cudaError_t launch_lb(const LinearBlockArgs& a, LinearBlockParams p, int sms, cudaStream_t stream, const char** why) {
  CUtensorMap map_x, map_w;
  if (!make_map(&map_x, a.x, a.m, a.k, NX, true) || !make_map(&map_w, a.w, a.n, a.k, kLbRows, true)) {
    *why = "cuTensorMapEncodeTiled is unavailable or rejected the operands";
    return cudaErrorInvalidValue;
  }
  auto kern = linear_block_kernel<NX>;
  cudaError_t e = allow_smem<linear_block_kernel<NX>>(lb_smem<NX>());
  if (e != cudaSuccess) {
    *why = "could not reserve shared memory";
    return e;
  }
  p.m_tiles = (p.m + NX - 1) / NX;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  // K is cut while the CTAs still fit the GPU at once and each keeps four blocks
  p.split = 1;
  while (p.split < kLbMaxSplit && tiles * p.split * 2 <= static_cast<int64_t>(sms) * Lb<NX>::kPerSm &&
         p.blocks >= p.split * 2 * 4)
    p.split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
  cfg.blockDim = dim3(kLbThreads);
  cfg.dynamicSmemBytes = lb_smem<NX>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, p);
}

}  // namespace

cudaError_t launch_linear_block(const LinearBlockArgs& a, cudaStream_t stream, const char** why) {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (a.m > 128) return launch_linear_block_pair(a, stream, why);
  LinearBlockParams p = {};
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.err = a.err;
  p.m = static_cast<int>(a.m);
  p.n = static_cast<int>(a.n);
  p.blocks = static_cast<int>(block_count(a.k));
  p.n_tiles = static_cast<int>(block_count(a.n));
  p.act = a.act;
  return a.m <= 16   ? launch_lb<16>(a, p, sms, stream, why)
         : a.m <= 32 ? launch_lb<32>(a, p, sms, stream, why)
         : a.m <= 64 ? launch_lb<64>(a, p, sms, stream, why)
                     : launch_lb<128>(a, p, sms, stream, why);
}

}  // namespace gbf
