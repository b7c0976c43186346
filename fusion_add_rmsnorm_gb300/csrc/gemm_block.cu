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
// output channel and the sums of some of the NX rows.
//   warp 0     TMA producer: W's 128 and X's NX rows of a K block into a ring
//   warp 1     MMA issuer: four MMAs of 32 K into the next accumulator (the whole
//              warp walks the loop, which keeps the descriptors in uniform
//              registers; one lane issues)
//   warps 2-3  the X scales of 8 K blocks ahead, times W's; warp 2 tensor memory
//   warps 4...  epilogue, 32 channels and 16 or 32 rows of X each
// With few output tiles, a cluster of up to eight CTAs cuts K between them.  Each
// owns NX / split of the tile's rows of X, gets the others' sums of them by remote
// stores and adds them in the order of K, so that a result has the same bits in
// every run.
//
// Every mbarrier wait is bounded, as in gemm_tcgen05.cu: one that gives up
// sets the device error word and an abort flag, every role leaves its loop,
// the MMAs and copies in flight are waited for (bounded), all CTAs of a cluster
// reach its barriers and TMEM is freed.
#include <atomic>

#include "gemm_block.cuh"

namespace gbf {
namespace {

constexpr int kLbRows = 128;              // W rows of a tile: one scale block
constexpr int kLbEpilogue = 4;            // first epilogue warp

constexpr int kLbChunk = 8;               // K blocks whose scales are filled at a time

// Shared memory of a CTA with NX rows of X, alone on K or one of a cluster
// (SPLIT): two CTAs an SM up to 32 rows, so that the next call's comes beside
// this one's; from 64 on a deeper ring is worth more.  No more accumulators than
// stages: the epilogue then waits for a stage's MMAs before that stage can be
// through twice.
template <int NX, bool SPLIT>
struct Lb {
  static constexpr int kPerSm = NX <= 32 ? 2 : 1;
  static constexpr int kGroups = NX <= 32 ? 1 : NX / 32;                            // groups of four epilogue warps
  static constexpr int kCols = NX / kGroups;                                      // rows of X of a group
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kStageBytes = (kLbRows + NX) * BK_BYTES;
  static constexpr int kPartBytes = SPLIT ? NX * kLbRows * 4 : 0;                 // [part][owned row][channel]
  static constexpr int kScaleRow = NX + 4;                                        // read as 16-byte vectors
  static constexpr int kScaleBytes = 2 * kLbChunk * kScaleRow * 4;
  static constexpr int kRoom = (kPerSm == 2 ? 115712 : 232448) - 2048;            // of a CTA, less alignment and barriers
  static constexpr int kFit = (kRoom - kPartBytes - kScaleBytes) / kStageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kAccs = kStages < 512 / kPerSm / NX ? kStages : 512 / kPerSm / NX;
  static constexpr int kTmemCols = kAccs * NX <= 32 ? 32 : kAccs * NX <= 64 ? 64 : kAccs * NX <= 128 ? 128 : kAccs * NX <= 256 ? 256 : 512;
  static_assert(kStages >= 3 && kAccs >= 3, "stages and accumulators in flight");
  // A CTA that waits for tensor memory while one of its cluster waits for it could wait for ever, where
  // two clusters each hold what the other asks for.  So an SM's shared memory never admits CTAs whose
  // columns sum to more than 512: two of these at most, and none beside a Linear on its own SM (180 KB or more).
  static constexpr int kSmem = kStages * kStageBytes + kPartBytes + kScaleBytes;
  static_assert(kPerSm * kTmemCols <= 512 && kSmem > (kPerSm == 2 ? 228 * 1024 / 3 : 228 * 1024 / 2), "tensor memory for all CTAs of an SM");
};

template <int S, int A>
struct __align__(8) LbCtl {
  uint64_t full[S];
  uint64_t done[S];          // a K block's MMAs: its stage is free, its accumulator full
  uint64_t acc_empty[A];
  uint64_t scales_full[2];
  uint64_t scales_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int NX, bool SPLIT>
constexpr size_t lb_smem() {
  using L = Lb<NX, SPLIT>;
  return 1024 /* alignment */ + L::kStages * L::kStageBytes + L::kPartBytes + L::kScaleBytes +
         sizeof(LbCtl<L::kStages, L::kAccs>);
}

struct LinearBlockParams {
  const float* x_scales;
  const float* w_scales;
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;
  unsigned int* err;
  int m, n, blocks;          // blocks: of K
  int m_tiles, n_tiles;
  int split;                 // CTAs (a cluster) that cut K: a power of two, at most kLbMaxSplit
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

GBF_DEVICE void st_cluster_f32(uint32_t a, float v) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

template <int NX, bool SPLIT>
__global__ void __launch_bounds__(Lb<NX, SPLIT>::kThreads, Lb<NX, SPLIT>::kPerSm)
linear_block_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const LinearBlockParams p) {
  using L = Lb<NX, SPLIT>;
  constexpr int S = L::kStages, A = L::kAccs, COLS = L::kCols;
  constexpr uint32_t kIdesc = idesc(true, kLbRows, NX);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_w = smem;                                   // S x 128 rows of 128 bytes
  uint8_t* smem_x = smem + S * kLbRows * BK_BYTES;          // S x NX rows of 128 bytes
  float* part = reinterpret_cast<float*>(smem + S * L::kStageBytes);
  float* scales = reinterpret_cast<float*>(smem + S * L::kStageBytes + L::kPartBytes);
  LbCtl<S, A>* ctl = reinterpret_cast<LbCtl<S, A>*>(smem + S * L::kStageBytes + L::kPartBytes + L::kScaleBytes);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.split;
  const int m0 = tile % p.m_tiles * NX, nt = tile / p.m_tiles, n0 = nt * kLbRows;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->done[s], 1);
    }
    for (int b = 0; b < A; ++b) mbar_init(&ctl->acc_empty[b], 4 * L::kGroups);     // one arrive per epilogue warp
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->scales_full[b], 2);                   // the two warps that fill them
      mbar_init(&ctl->scales_empty[b], 4 * L::kGroups);
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
  // every CTA of the cluster runs before its shared memory is written to (waited for below)
  if (SPLIT) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_launch_dependents();

  float acc[COLS];
  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        const int s = issued % S;
        if (!mbar_wait<false, false>(&ctl->done[s], ((issued / S) & 1) ^ 1u, &ctl->abort, p.err)) break;
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
    const bool elected = elect_one();
    bool ok = true;
    for (int i = 0; i < kb1 - kb0 && ok; ++i) {
      const int s = i % S, b = i % A;
      const uint64_t w_desc = smem_desc_sw128(smem_u32(smem_w) + s * kLbRows * BK_BYTES);
      const uint64_t x_desc = smem_desc_sw128(smem_u32(smem_x) + s * NX * BK_BYTES);
      ok = mbar_wait<false, false>(&ctl->acc_empty[b], ((i / A) & 1) ^ 1u, &ctl->abort, p.err) &&
           mbar_wait<false, false>(&ctl->full[s], (i / S) & 1, &ctl->abort, p.err);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (ok && elected) {
#pragma unroll
        for (int kk = 0; kk < BK_BYTES / UMMA_K_BYTES; ++kk)         // 32 bytes on inside the swizzled row
          tc_mma<true, false>(tmem_base + b * NX, w_desc + kk * (UMMA_K_BYTES >> 4), x_desc + kk * (UMMA_K_BYTES >> 4),
                              kIdesc, kk != 0);
        tc_commit<false>(&ctl->done[s]);
      }
    }
    if (elected) {
      tc_commit_self<false>(&ctl->drain);
      int own = 0;
      mbar_wait(&ctl->drain, 0, &own, p.err);
    }
  } else if (warp < kLbEpilogue) {
    // ---------------------------------------------------------------- scales
    const int at = lane % kLbChunk, first = (warp - 2) * 4 + lane / kLbChunk;     // a lane's K block, every eighth row
    for (int kb = kb0, chunk = 0; kb < kb1; kb += kLbChunk, ++chunk) {
      if (!mbar_wait_warp(&ctl->scales_empty[chunk & 1], ((chunk >> 1) & 1) ^ 1u, &ctl->abort, p.err)) break;
      float* to = scales + (chunk & 1) * kLbChunk * L::kScaleRow + at * L::kScaleRow;
      const bool in = kb + at < kb1;
      const float w = in ? p.w_scales[static_cast<int64_t>(nt) * p.blocks + kb + at] : 0.0f;
      float v[NX / 8];
#pragma unroll
      for (int i = 0; i < NX / 8; ++i) {                    // rows behind the last have no scales, and are not stored
        const int row = m0 + first + 8 * i;
        v[i] = in && row < p.m ? p.x_scales[static_cast<int64_t>(row) * p.blocks + kb + at] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NX / 8; ++i) to[first + 8 * i] = v[i] * w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->scales_full[chunk & 1]);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3, col0 = (warp - kLbEpilogue) / 4 * COLS;     // TMEM lanes 32 * quarter .. + 31
    const uint32_t taddr = tmem_base + col0 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
    for (int j = 0; j < COLS; ++j) acc[j] = 0.0f;
    bool ok = true;
    int i = 0;
    for (int kb = kb0, chunk = 0; kb < kb1 && ok; kb += kLbChunk, ++chunk) {
      uint32_t sc = smem_u32(scales + (chunk & 1) * kLbChunk * L::kScaleRow + col0);
      ok = mbar_wait_warp<false>(&ctl->scales_full[chunk & 1], (chunk >> 1) & 1, &ctl->abort, p.err);
      for (const int end = min(kb1 - kb0, i + kLbChunk); i < end && ok; ++i, sc += L::kScaleRow * 4) {
        const int b = i % A;
        ok = mbar_wait<false, false>(&ctl->done[i % S], (i / S) & 1, &ctl->abort, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        constexpr int STEP = COLS < 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < COLS; c += STEP) {
          uint32_t r[STEP];
          if constexpr (STEP == 16) tmem_ld_16cols(taddr + b * NX + c, r);
          else tmem_ld_32cols(taddr + b * NX + c, r);
          if (c + STEP == COLS) {                             // all read: the accumulator goes back before the sums
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->acc_empty[b]);
          }
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
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->scales_empty[chunk & 1]);
    }
    const int ch = quarter * 32 + lane;                     // this thread's row of the W tile
    if constexpr (SPLIT) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      const int owned = NX / p.split, log = __ffs(owned) - 1;      // a power of two
      const uint32_t to = smem_u32(part) + (rank * owned * kLbRows + ch) * 4;
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        st_cluster_f32(map_cluster(to + ((col0 + j) & (owned - 1)) * kLbRows * 4, (col0 + j) >> log), acc[j]);
    } else if (n0 + ch < p.n) {
      const float bias = p.bias ? __bfloat162float(p.bias[n0 + ch]) : 0.0f;
      with_act(p.act, [&](auto ACT) {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (m0 + col0 + j < p.m)
            p.y[static_cast<int64_t>(m0 + col0 + j) * p.n + n0 + ch] = __float2bfloat16(fast_act(acc[j] + bias, ACT.value));
      });
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, L::kTmemCols);
  }
  if constexpr (SPLIT) {
    if (warp < kLbEpilogue) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    cluster_sync();                                         // every CTA's sums are where they are added
    const int owned = NX / p.split, ch = threadIdx.x & (kLbRows - 1);
    const float bias = p.bias && n0 + ch < p.n ? __bfloat162float(p.bias[n0 + ch]) : 0.0f;
    for (int j = threadIdx.x / kLbRows; j < owned; j += L::kThreads / kLbRows) {
      const int row = m0 + rank * owned + j;
      float v[kLbMaxSplit], sum = 0.0f;
#pragma unroll
      for (int r = 0; r < kLbMaxSplit; ++r)
        v[r] = r < p.split ? part[(r * owned + j) * kLbRows + ch] : 0.0f;
#pragma unroll
      for (int r = 0; r < kLbMaxSplit; ++r) sum += v[r];
      if (row < p.m && n0 + ch < p.n)
        p.y[static_cast<int64_t>(row) * p.n + n0 + ch] = __float2bfloat16(fast_act(sum + bias, p.act));
    }
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

template <int NX, bool SPLIT>
cudaError_t launch_split(const LinearBlockArgs& a, const LinearBlockParams& p, cudaStream_t stream, const char** why) {
  CUtensorMap map_x, map_w;
  if (!make_map(&map_x, a.x, a.m, a.k, NX, true) || !make_map(&map_w, a.w, a.n, a.k, kLbRows, true)) {
    *why = "cuTensorMapEncodeTiled is unavailable or rejected the operands";
    return cudaErrorInvalidValue;
  }
  auto kern = linear_block_kernel<NX, SPLIT>;
  cudaError_t e = allow_smem<linear_block_kernel<NX, SPLIT>>(lb_smem<NX, SPLIT>());
  if (e != cudaSuccess) {
    *why = "could not reserve shared memory";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.m_tiles) * p.n_tiles * p.split);
  cfg.blockDim = dim3(Lb<NX, SPLIT>::kThreads);
  cfg.dynamicSmemBytes = lb_smem<NX, SPLIT>();
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

template <int NX>
cudaError_t launch_lb(const LinearBlockArgs& a, const LinearBlockParams& p, cudaStream_t stream, const char** why) {
  return p.split > 1 ? launch_split<NX, true>(a, p, stream, why) : launch_split<NX, false>(a, p, stream, why);
}

}  // namespace

cudaError_t linear_block_plan(int64_t m, int64_t n, int64_t k, LinearBlockPlan* plan, LinearBlockRoom* room) {
  int dev = 0;
  *room = {};
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&room->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (m > 32) linear_block_clusters(room->clusters);
  *plan = plan_linear_block(m, n, k, *room);
  return cudaSuccess;
}

cudaError_t launch_linear_block(const LinearBlockArgs& a, cudaStream_t stream, const char** why) {
  LinearBlockPlan plan;
  LinearBlockRoom room;
  const cudaError_t e = linear_block_plan(a.m, a.n, a.k, &plan, &room);
  if (e != cudaSuccess) return e;
  if (plan.rows == kBpTile) return launch_linear_block_pair(a, plan, room.clusters[plan.split], stream, why);
  LinearBlockParams p = {};
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.err = a.err;
  p.m = static_cast<int>(a.m);
  p.n = static_cast<int>(a.n);
  p.blocks = static_cast<int>(block_count(a.k));
  p.m_tiles = static_cast<int>((a.m + plan.rows - 1) / plan.rows);
  p.n_tiles = static_cast<int>(block_count(a.n));
  p.split = plan.split;
  p.act = a.act;
  switch (plan.rows) {
    case 16: return launch_lb<16>(a, p, stream, why);
    case 32: return launch_lb<32>(a, p, stream, why);
    case 64: return launch_lb<64>(a, p, stream, why);
    default: return launch_lb<128>(a, p, stream, why);
  }
}

}  // namespace gbf
