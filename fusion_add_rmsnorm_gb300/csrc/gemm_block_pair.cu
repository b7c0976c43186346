// linear_fp8_block on CTA pairs: the products of gemm_block.cu's operator that the
// tensor core, and not the reading of W, bounds.
//
// Two CTAs on adjacent 128-row tiles of X run as one tcgen05 pair
// (cta_group::2) on a 256 x 256 tile of Y, as in gemm_tcgen05.cu; X's rows are
// the MMA's rows, so a thread of the epilogue holds one row, and a K block's
// scale is one number a thread: sx[row, b] * sw[channels / 128, b].  The tile's
// two halves of 128 channels (a scale block of W each) are products of their
// own: either has two accumulators of 128 columns in turn, an issuer and half of
// the epilogue, so that neither waits for the other.
//   warp 0      TMA producer: the CTA's 128 X rows and 64 W rows of either half,
//               a K block at a time, into a four-stage ring
//   warps 1-2   one a half.  Even CTA: MMA issuers, four M256 N128 K32 MMAs a K
//               block (the whole warp walks the loop, which keeps the descriptors
//               in uniform registers: 25 cycles an MMA, 120 from a lane's own).
//               Odd CTA: tell the even one's issuer that an accumulator was read
//   warp 3      tensor memory; the scales of 16 K blocks ahead, and the bias
//   warps 4-11  epilogue, 32 rows x 128 channels each: a K block's accumulator is
//               read back, given back, and added, scaled, to 128 float32 registers;
//               after the last block bias, activation, one bf16 rounding, and bulk
//               tensor stores
// The registers that the first four warps do not need go to the epilogue
// (setmaxnreg: 128 x 72 + 256 x 216 = 384 x 168).
// What bounds it: an accumulator's way round (MMAs, completion, read back, given
// back in both CTAs), as 512 TMEM columns hold two K blocks.  So that way is kept
// short: an SM's epilogue gives back through a hardware barrier, not an mbarrier,
// scales come from shared memory, nothing in the loop acquires or releases at
// cluster scope (an acquire there empties L1, a release waits for loads in flight;
// see mbar_arrive_relaxed), and the next accumulator is asked about while this one's
// last columns are added.  8192 x 16384 x 4096: 418 to 426 us with the tanh GELU on
// several GPUs (461 in a run of eager calls), 390 to 410 without an activation.
//
// CTAs are persistent and walk the tiles.  With few of them, up to four pairs of
// a cluster cut K, and add their partial sums through distributed shared memory,
// in the order of K.
//
// mbarrier waits are bounded, as in gemm_tcgen05.cu.  After one that gave up, the
// producers leave; issuers, relays and epilogue walk the rest of their K blocks
// without working, in step (see wait_taken), so that the hardware barriers' phases
// still are K blocks, and all CTAs of a cluster leave together.
#include <atomic>

#include "gemm_block.cuh"

namespace gbf {
namespace {

constexpr int kBpThreads = 384;
constexpr int kBpRows = kBpTile / 2;            // X rows of a CTA
constexpr int kBpCols = kBpTile;                // channels of a pair's tile
constexpr int kBpHalf = kBpCols / 2;
constexpr int kBpStages = 4;
constexpr int kBpStageBytes = (kBpRows + kBpHalf) * BK_BYTES;
constexpr int kBpEpilogue = 4;                  // first epilogue warp
constexpr int kBpEpilogueWarps = 8;
constexpr int kBpWarpCols = 128;                // channels of an epilogue warp: a half
constexpr int kBpBoxCols = 64;                  // an epilogue warp's stores: 32 rows x 64 columns of bf16
constexpr int kBpBoxBytes = 32 * kBpBoxCols * 2;
// Scales of 16 K blocks, one copy in use and one being filled: X's as
// [K block][row], two words more a row than needed so that both the filling (16
// K blocks of two rows) and the reading (32 rows of one) meet every bank once.
constexpr int kBpChunk = 16;
constexpr int kBpChunkRow = kBpRows + 2;

struct __align__(16) BpScales {
  float x[kBpChunk * kBpChunkRow];
  float w[2][kBpChunk];
};
// The biases of this tile's channels and of the next one's, by the tile's parity:
// they are written with a tile's first scales and read at its end, when its first
// scales' place may already hold the next tile's.
struct __align__(16) BpBias {
  __nv_bfloat16 of[2][kBpCols];
};

struct __align__(8) BpCtl {
  uint64_t full[kBpStages];
  uint64_t empty[kBpStages];
  uint64_t acc_full[4];                         // [K block's parity][half]
  uint64_t peer_gave[4];                        // even CTA: the odd one has read its accumulator
  uint64_t scales_full[2];
  uint64_t scales_empty[2];
  uint64_t drain[2];
  uint32_t tmem_base;
  uint32_t peer_issued;                         // even CTA: K blocks whose copies the odd CTA issued
  uint32_t taken[2];                            // K blocks whose accumulators a half's issuer or relay took back
  int abort;
};

constexpr size_t kBpSmem = 1024 /* alignment */ + kBpStages * kBpStageBytes + kBpEpilogueWarps * 2 * kBpBoxBytes +
                           2 * sizeof(BpScales) + sizeof(BpBias) + sizeof(BpCtl);
static_assert(kBpSmem <= 232448, "227 KB a CTA");
static_assert(kBpRows * kBpCols * 4 <= kBpStages * kBpStageBytes, "partial sums fit the ring");
static_assert(kBpChunk * kBpRows % 32 == 0 && kBpChunk == 16, "a lane's share of the scales");

struct BlockPairParams {
  const float* x_scales;
  const float* w_scales;
  const __nv_bfloat16* bias;
  __nv_bfloat16* y;
  unsigned int* err;
  int m, n, blocks;
  int m_units, n_tiles;                         // tiles of 256 x 256
  int group_n;                                  // tile columns that are walked together
  int split;                                    // pairs (a cluster) that cut K
  int act;
};

// First row (of this CTA) and column of a pair's tile: groups of group_n tile
// columns, inside a group column by column, so that the pairs at work share a
// group's W in L2 while X goes past.
GBF_DEVICE void bp_origin(const BlockPairParams& p, int odd, int tile, int& m0, int& n0) {
  const int per_group = p.group_n * p.m_units, g = tile / per_group, i = tile - g * per_group;
  const int width = min(p.group_n, p.n_tiles - g * p.group_n);
  m0 = (i / width * 2 + odd) * kBpRows;
  n0 = (g * p.group_n + i % width) * kBpCols;
}

// The hardware barrier of accumulator b ([parity][half]): the half's epilogue
// warps arrive once they have read it, the half's issuer (odd CTA: relay) waits
// for all of them.
constexpr int kBpGivers = (kBpEpilogueWarps / 2 + 1) * 32;
GBF_DEVICE void give_back(int b) { asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(1 + b), "n"(kBpGivers) : "memory"); }
GBF_DEVICE void take_back(int b) { asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(1 + b), "n"(kBpGivers) : "memory"); }
GBF_DEVICE void set_taken(uint32_t* taken, uint32_t blocks) { *reinterpret_cast<volatile uint32_t*>(taken) = blocks; }

// The barrier counts arrivals, whoever they are from, so a warp may not arrive for
// K block i before block i - 2's phase is over: two arrivals in one phase, and a
// later phase stays short of one for ever.  While the waits succeed, acc_full says
// so (block i's MMAs go out behind that phase).  A warp whose wait gave up has only
// the issuer's (relay's) own count to go by.  That count moves on: every warp
// arrives for a block, and the issuer's other waits are bounded.
GBF_DEVICE void wait_taken(const uint32_t* taken, uint32_t blocks) {
  for (uint32_t i = 0; i < 4 * kWaitMaxPolls && *reinterpret_cast<const volatile uint32_t*>(taken) < blocks; ++i) __nanosleep(256);
  __syncwarp();
}

// An accumulator goes from CTA to CTA: the odd one's relay arrives on the even one's
// mbarrier, and the even one's commit on the odd one's.  What goes over is tensor
// memory alone, so arrival and wait are relaxed, at the scope that holds both CTAs,
// and the order is the tcgen05 fences': loads waited for, before_thread_sync, the
// half's hardware barrier, after_ and before_thread_sync in the relay, this arrival,
// wait_accumulator, after_thread_sync, the MMAs that write it again.  With a
// release and an acquire instead 8192 x 16384 x 4096 takes 741 us, not 418.
GBF_DEVICE void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

GBF_DEVICE bool wait_accumulator(uint64_t* bar, uint32_t parity, int* abort, unsigned int* err) {
  return mbar_wait<true, false, true>(bar, parity, abort, err);
}

// Arrives on `bar` of both CTAs of the pair whose even one this is, once the
// MMAs that this thread issued are done.
GBF_DEVICE void commit_pair(uint64_t* bar, int rank) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(0x3 << rank))
      : "memory");
}

// A copy of N bytes to shared memory that nobody waits for (zeros where `has` is
// false, and nothing is read), and an arrival on `bar` when all of this thread's
// copies before it have landed.
template <int N>
GBF_DEVICE void async_copy(void* dst, const void* src, bool has) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(has ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(has ? 4 : 0) : "memory");
}
GBF_DEVICE void async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// X's scales of a tile's rows and of kBpChunk K blocks from kb on, by `threads`
// threads (a multiple of kBpChunk) of which this is `t`.  Rows and K blocks outside
// have none: zeros, and what they sum is not stored.
GBF_DEVICE void fill_x(const BlockPairParams& p, BpScales& sc, int m0, int kb, int kb_end, int t, int threads) {
  const int at = t % kBpChunk;
#pragma unroll 8
  for (int r = t / kBpChunk; r < kBpRows; r += threads / kBpChunk) {
    const bool has = kb + at < kb_end && m0 + r < p.m;
    async_copy<4>(&sc.x[at * kBpChunkRow + r], p.x_scales + (has ? static_cast<int64_t>(m0 + r) * p.blocks + kb + at : 0), has);
  }
}

// 32 float32 columns of this warp's TMEM lanes, not waited for.
GBF_DEVICE void tmem_ld_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// Waits for the loads above.  The registers pass through, so that no use of
// them is moved ahead of the wait.
GBF_DEVICE void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// Whether an accumulator's phase with this parity is over, without waiting.
GBF_DEVICE uint32_t test_accumulator(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok;
}
GBF_DEVICE void add_scaled(float (&acc)[kBpWarpCols], int at, const uint32_t (&r)[32], float2 s) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float2 v = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), s,
                                make_float2(acc[at + j], acc[at + j + 1]));
    acc[at + j] = v.x;
    acc[at + j + 1] = v.y;
  }
}

GBF_DEVICE float4 ld_cluster_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Eight outputs from their sums: bias, activation, one rounding.
GBF_DEVICE uint4 finish8(const float (&a)[8], uint4 bias, int act) {
  float z[8], v[8];
  bf16x8_to_f32(bias, z);
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 o = fast_act2(__fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(z[e], z[e + 1])), act);
    v[e] = o.x;
    v[e + 1] = o.y;
  }
  return f32x8_to_bf16x8(v);
}

__global__ void __launch_bounds__(kBpThreads, 1)
linear_block_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_y, const BlockPairParams p) {
  constexpr int S = kBpStages;
  constexpr uint32_t kIdesc = idesc(true, 2 * kBpRows, kBpHalf);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offsets in all CTAs of a cluster: MMAs and remote accesses use one CTA's for another's
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smem_x = smem;
  uint8_t* smem_w = smem + S * kBpRows * BK_BYTES;
  uint8_t* smem_out = smem + S * kBpStageBytes;
  BpScales* scales = reinterpret_cast<BpScales*>(smem_out + kBpEpilogueWarps * 2 * kBpBoxBytes);
  BpBias* biases = reinterpret_cast<BpBias*>(scales + 2);
  BpCtl* ctl = reinterpret_cast<BpCtl*>(biases + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), odd = rank & 1, part = rank >> 1;
  const int first = blockIdx.x / (2 * p.split), stride = gridDim.x / (2 * p.split);
  const int kb_begin = static_cast<int>(static_cast<int64_t>(p.blocks) * part / p.split);
  const int kb_end = static_cast<int>(static_cast<int64_t>(p.blocks) * (part + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 2);                         // both halves' MMAs
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&ctl->acc_full[b], 1);
      mbar_init(&ctl->peer_gave[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->drain[b], 1);
      mbar_init(&ctl->scales_full[b], 32);                  // the lanes that fill them
      mbar_init(&ctl->scales_empty[b], kBpEpilogueWarps);
    }
    ctl->peer_issued = 0;
    ctl->taken[0] = ctl->taken[1] = 0;
    ctl->abort = 0;
    mbar_fence_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_y)) : "memory");
  }
  if (warp == 3) tmem_alloc<true>(&ctl->tmem_base, 2 * kBpCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                           // the barriers and TMEM of all CTAs are there
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  // all of TMEM is allocated, so both bases are column 0; a pair that finds otherwise does no work
  const bool usable = ld_cluster_u32(map_cluster(smem_u32(&ctl->tmem_base), rank ^ 1)) == tmem_base;
  if (!usable && threadIdx.x == 0) raise_error(p.err, DEV_ERR_PAIR_TMEM);
  const int tiles = usable ? p.m_units * p.n_tiles : 0;
  pdl_wait();
  pdl_launch_dependents();

  uint32_t issued = 0;                                      // producer: K blocks whose copies it issued
  if (warp < kBpEpilogue) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      if (lane == 0) {
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += stride) {
          int m0, n0;
          bp_origin(p, odd, tile, m0, n0);
          for (int kb = kb_begin; kb < kb_end; ++kb, ++issued) {
            const uint32_t s = issued % S;
            ok = mbar_wait<false, false>(&ctl->empty[s], ((issued / S) & 1) ^ 1u, &ctl->abort, p.err);
            if (!ok) break;
            if (!odd) mbar_arrive_expect_tx(&ctl->full[s], 2 * kBpStageBytes);
            const uint32_t bar = map_cluster(smem_u32(&ctl->full[s]), rank & ~1);
            tma_load_2d_pair(smem_x + s * kBpRows * BK_BYTES, &map_x, bar, kb * BK_BYTES, m0);
            // 64 rows of either scale block of W, so that a half's MMA covers one of them
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d_pair(smem_w + (s * 2 + h) * (kBpHalf / 2) * BK_BYTES, &map_w, bar, kb * BK_BYTES,
                               n0 + h * kBpHalf + odd * (kBpHalf / 2));
          }
        }
        if (odd)                                            // the even CTA waits for the odd one's copies too
          st_cluster_u32(map_cluster(smem_u32(&ctl->peer_issued), rank ^ 1), issued);
      }
    } else if (warp < 3) {
      const uint32_t h = warp - 1;                          // half of the tile's channels
      const bool elected = elect_one();
      uint32_t it = 0;
      if (!odd) {
        // ---------------------------------------------------------- MMA issuer
        bool ok = true;
        for (int tile = first; tile < tiles; tile += stride) {
          for (int kb = kb_begin; kb < kb_end; ++kb, ++it) {
            const uint32_t s = it % S, b = (it & 1) * 2 + h;
            const uint64_t x_desc = smem_desc_sw128(smem_u32(smem_x) + s * kBpRows * BK_BYTES);
            const uint64_t w_desc = smem_desc_sw128(smem_u32(smem_w) + (s * 2 + h) * (kBpHalf / 2) * BK_BYTES);
            // the operands first: they are there early, the accumulator (from K block it - 2) is not
            ok = ok && mbar_wait<false, false>(&ctl->full[s], (it / S) & 1, &ctl->abort, p.err);
            if (it >= 2) {
              __syncwarp();
              take_back(b);
              set_taken(&ctl->taken[h], it - 1);
              ok = ok && wait_accumulator(&ctl->peer_gave[b], ((it >> 1) & 1) ^ 1u, &ctl->abort, p.err);
            }
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (ok && elected) {
#pragma unroll
              for (int kk = 0; kk < BK_BYTES / UMMA_K_BYTES; ++kk)   // 32 bytes on inside the swizzled row
                tc_mma<true, true>(tmem_base + b * kBpHalf, x_desc + kk * (UMMA_K_BYTES >> 4),
                                   w_desc + kk * (UMMA_K_BYTES >> 4), kIdesc, kk != 0);
              commit_pair(&ctl->acc_full[b], rank);
              commit_pair(&ctl->empty[s], rank);
            }
          }
        }
        __syncwarp();
        for (uint32_t i = it > 2 ? it - 2 : 0; i < it; ++i) {
          take_back((i & 1) * 2 + h);
          set_taken(&ctl->taken[h], i + 1);
        }
        if (elected) {
          tc_commit_self<true>(&ctl->drain[h]);
          int own = 0;
          mbar_wait(&ctl->drain[h], 0, &own, p.err);
        }
      } else {
        // --------------------------------------------------------------- relay
        const uint32_t peer = map_cluster(smem_u32(&ctl->peer_gave[h]), rank ^ 1);
        for (int tile = first; tile < tiles; tile += stride)
          for (int kb = kb_begin; kb < kb_end; ++kb, ++it) {
            take_back((it & 1) * 2 + h);
            tc_fence_after();
            tc_fence_before();
            if (elected) mbar_arrive_relaxed(peer + (it & 1) * 16);
            set_taken(&ctl->taken[h], it + 1);
            __syncwarp();
          }
      }
    } else {
      // ---------------------------------------------------------------- scales
      const int at = lane % kBpChunk, second = lane / kBpChunk;   // a lane's K block, and which rows
      uint32_t chunk = 0, turn = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += stride, turn ^= 1) {
        int m0, n0;
        bp_origin(p, odd, tile, m0, n0);
        for (int kb = kb_begin; kb < kb_end; kb += kBpChunk, ++chunk) {
          BpScales& sc = scales[chunk & 1];
          ok = mbar_wait_warp(&ctl->scales_empty[chunk & 1], ((chunk >> 1) & 1) ^ 1u, &ctl->abort, p.err);
          if (!ok) break;
          const bool in = kb + at < kb_end;
          const int n = n0 + second * kBlockCols;
          const bool has = in && n < p.n;
          async_copy<4>(&sc.w[second][at], p.w_scales + (has ? static_cast<int64_t>(n / kBlockCols) * p.blocks + kb + at : 0), has);
          if (kb == kb_begin) {
            const bool some = p.bias && n0 + lane * 8 < p.n;
            async_copy<16>(&biases->of[turn][lane * 8], some ? static_cast<const void*>(p.bias + n0 + lane * 8) : p.y, some);
          }
          if (chunk > 0) fill_x(p, sc, m0, kb, kb_end, lane, 32);   // the first is the epilogue's
          async_arrive(&ctl->scales_full[chunk & 1]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");   // none in flight when the CTA leaves
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int quarter = warp & 3;                           // TMEM lanes 32 * quarter .. + 31
    const int col_at = (warp - kBpEpilogue) / 4 * kBpWarpCols, half = col_at / kBpHalf;
    const uint32_t taddr = tmem_base + col_at + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* box = smem_out + (warp - kBpEpilogue) * 2 * kBpBoxBytes;
    uint32_t it = 0, chunk = 0, ready = 0, turn = 0;
    bool ok = true;
    if (first < tiles) {
      // The first scales of X are filled here, by eight warps that have nothing to do yet: one warp takes
      // 2,000 cycles longer, later ones are filled ahead.
      int m0, n0;
      bp_origin(p, odd, first, m0, n0);
      fill_x(p, scales[0], m0, kb_begin, kb_end, threadIdx.x - kBpEpilogue * 32, kBpEpilogueWarps * 32);
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("barrier.cta.sync.aligned 5, %0;" ::"n"(kBpEpilogueWarps * 32) : "memory");
    }
    for (int tile = first; tile < tiles; tile += stride, turn ^= 1) {
      const __nv_bfloat16* bias = biases->of[turn] + col_at;
      float acc[kBpWarpCols];
#pragma unroll
      for (int j = 0; j < kBpWarpCols; ++j) acc[j] = 0.0f;
      for (int kb0 = kb_begin; kb0 < kb_end; kb0 += kBpChunk, ++chunk) {
        const BpScales& sc = scales[chunk & 1];
        const float* sx = sc.x + quarter * 32 + lane;
        const float* sw = sc.w[half];
        const int end = min(kBpChunk, kb_end - kb0);
        ok = ok && mbar_wait_warp(&ctl->scales_full[chunk & 1], (chunk >> 1) & 1, &ctl->abort, p.err);
        float s_next = sx[0] * sw[0];
        for (int kb = 0; kb < end; ++kb, ++it) {
          const uint32_t b = (it & 1) * 2 + half;
          const float s = s_next;
          if (!ready) ok = ok && wait_accumulator(&ctl->acc_full[b], (it >> 1) & 1, &ctl->abort, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const float2 ss = make_float2(s, s);
          const uint32_t at = taddr + (it & 1) * kBpCols;
          uint32_t r0[32], r1[32];
          tmem_ld_async(at, r0);
          tmem_ld_wait(r0);
          tmem_ld_async(at + 32, r1);
          add_scaled(acc, 0, r0, ss);
          tmem_ld_wait(r1);
          tmem_ld_async(at + 64, r0);
          add_scaled(acc, 32, r1, ss);
          tmem_ld_wait(r0);
          tmem_ld_async(at + 96, r1);
          add_scaled(acc, 64, r0, ss);
          tmem_ld_wait(r1);
          tc_fence_before();
          give_back(b);
          ready = test_accumulator(&ctl->acc_full[b ^ 2], ((it + 1) >> 1) & 1);
          const int after = min(kb + 1, end - 1);           // the next one's scale, ahead of its wait
          s_next = sx[after * kBpChunkRow] * sw[after];
          add_scaled(acc, 96, r1, ss);
        }
        if (!ok) break;
        // the last chunk goes back once the tile's bias has been read: with one chunk a tile, the
        // next but one's bias takes this one's place
        if (kb0 + kBpChunk < kb_end && lane == 0) mbar_arrive(&ctl->scales_empty[chunk & 1]);
      }
      if (!ok) {                                            // a wait gave up: the K blocks of all tiles that are left
        const uint32_t all = ((tiles - 1 - first) / stride + 1u) * (kb_end - kb_begin);
        for (; it < all; ++it) {
          if (it >= 2) wait_taken(&ctl->taken[half], it - 1);
          give_back((it & 1) * 2 + half);
        }
        if (p.split > 1) asm volatile("barrier.cta.sync.aligned 5, %0;" ::"n"(kBpEpilogueWarps * 32) : "memory");
        break;
      }
      if (p.split > 1) {
        // One tile a cluster.  The ring is free once both halves' last accumulators have come: they came
        // after every copy and MMA of the pair.
        asm volatile("barrier.cta.sync.aligned 5, %0;" ::"n"(kBpEpilogueWarps * 32) : "memory");
        // 16-byte piece c of a row sits at c ^ (row % 8), so that a warp's rows meet every bank once.
        const int row = quarter * 32 + lane;
#pragma unroll
        for (int c = 0; c < kBpWarpCols / 4; ++c)
          sts128f(smem_u32(smem) + row * kBpCols * 4 + (((col_at / 4 + c) ^ (row & 7)) << 4), acc[c * 4], acc[c * 4 + 1],
                  acc[c * 4 + 2], acc[c * 4 + 3]);
        break;
      }
      int m0, n0;
      bp_origin(p, odd, tile, m0, n0);
      const int row0 = m0 + quarter * 32, col0 = n0 + col_at;
      if (lane == 0) bulk_wait_read_all();                  // the tile before has left the boxes
      __syncwarp();
      with_act(p.act, [&](auto ACT) {
        uint4 z[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) z[g] = reinterpret_cast<const uint4*>(bias)[g];
#pragma unroll
        for (int c = 0; c < kBpWarpCols / 8; c += 2) {
          uint4 next[2], o[2];                          // the next biases are asked for ahead of the stores
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (c + 2 < kBpWarpCols / 8) next[g] = reinterpret_cast<const uint4*>(bias)[c + 2 + g];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float a[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = acc[(c + g) * 8 + e];
            o[g] = finish8(a, z[g], ACT.value);
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            // piece c of a row sits at c ^ (row % 8): the TMA 128-byte swizzle
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                         ::"r"(smem_u32(box) + (c + g) / 8 * kBpBoxBytes + lane * 128 + ((((c + g) & 7) ^ (lane & 7)) << 4)),
                         "r"(o[g].x), "r"(o[g].y), "r"(o[g].z), "r"(o[g].w)
                         : "memory");
            z[g] = next[g];
          }
          if (c % 8 == 8 - 2) {                            // a box is whole
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && col0 + c / 8 * kBpBoxCols < p.n && row0 < p.m) {
              tma_store_2d(&map_y, box + c / 8 * kBpBoxBytes, col0 + c / 8 * kBpBoxCols, row0);
              bulk_commit();
            }
          }
        }
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->scales_empty[(chunk - 1) & 1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                                           // issue counts and partial sums are in place
  if (warp >= kBpEpilogue && lane == 0) bulk_wait_all();    // the stores have left shared memory
  if (warp == 0 && lane == 0 && !odd && *reinterpret_cast<volatile int*>(&ctl->abort)) {
    // Every copy to either CTA has landed before they leave: its MMAs are done, or,
    // after an abort, it is waited for.  The producers may then stand one K block
    // apart on a stage: the phase that only one of them filled is completed by hand.
    int own = 0;
    for (int s = 0; s < S; ++s) {
      const uint32_t mine = (issued + S - 1 - s) / S, theirs = (ctl->peer_issued + S - 1 - s) / S;   // on this stage
      if (theirs > mine)
        mbar_arrive_expect_tx(&ctl->full[s], kBpStageBytes);
      else if (mine > theirs)
        mbar_complete_tx(&ctl->full[s], kBpStageBytes);
      const uint32_t last = mine > theirs ? mine : theirs;
      if (last) mbar_wait(&ctl->full[s], (last - 1) & 1u, &own, nullptr);
    }
  }
  if (p.split > 1 && usable) {
    int m0, n0;
    bp_origin(p, odd, first, m0, n0);
    const int col = n0 + lane * 8;                          // a warp sums a row, a lane eight channels
    const uint4 bias = p.bias && col < p.n ? ld_cached(p.bias + col) : make_uint4(0, 0, 0, 0);
    const int end = min(kBpRows * (part + 1) / p.split, p.m - m0);
    for (int row = kBpRows * part / p.split + warp; row < end; row += kBpThreads / 32) {
      float4 v[kBpMaxSplit][2];                             // all parts' loads are on their way together
#pragma unroll
      for (int r = 0; r < kBpMaxSplit; ++r)
        if (r < p.split) {
          const uint32_t base = map_cluster(smem_u32(smem) + row * kBpCols * 4, 2 * r + odd);
#pragma unroll
          for (int h = 0; h < 2; ++h) v[r][h] = ld_cluster_f32x4(base + (((lane * 2 + h) ^ (row & 7)) << 4));
        }
      float a[8] = {};
#pragma unroll
      for (int r = 0; r < kBpMaxSplit; ++r)
        if (r < p.split)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[h * 4] += v[r][h].x;
            a[h * 4 + 1] += v[r][h].y;
            a[h * 4 + 2] += v[r][h].z;
            a[h * 4 + 3] += v[r][h].w;
          }
      if (col < p.n) st_16(p.y + static_cast<int64_t>(m0 + row) * p.n + col, finish8(a, bias, p.act));
    }
  }
  __syncthreads();
  cluster_sync();                                           // nothing is in flight between the CTAs
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc<true>(tmem_base, 2 * kBpCols);
  }
}

// Clusters of 2 * split CTAs that fit on the GPU at once, by device: a GPC's SMs
// that do not fill a cluster stay out.  Raises the kernel's shared memory limit
// the first time.
cudaError_t resident_clusters(int split, int* clusters) {
  static std::atomic<int> known[64][kBpMaxSplit + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*clusters = known[dev][split].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(linear_block_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kBpSmem));
  if (e != cudaSuccess) return e;
  int sms = 0, n = 0;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(sms / (2 * split) * 2 * split));
  cfg.blockDim = dim3(kBpThreads);
  cfg.dynamicSmemBytes = kBpSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, linear_block_pair_kernel, &cfg) != cudaSuccess || n < 1) n = 1;
  cudaGetLastError();
  if (dev < 64) known[dev][split].store(n, std::memory_order_relaxed);
  *clusters = n;
  return cudaSuccess;
}

}  // namespace

void linear_block_clusters(int (&clusters)[kBpMaxSplit + 1]) {
  for (int split = 1; split <= kBpMaxSplit; ++split)
    if (resident_clusters(split, &clusters[split]) != cudaSuccess) clusters[split] = 0;
}

cudaError_t launch_linear_block_pair(const LinearBlockArgs& a, const LinearBlockPlan& plan, int fit, cudaStream_t stream,
                                     const char** why) {
  CUtensorMap map_x, map_w, map_y;
  if (!make_map(&map_x, a.x, a.m, a.k, kBpRows, true) || !make_map(&map_w, a.w, a.n, a.k, kBpHalf / 2, true) ||
      !make_map(&map_y, a.y, a.m, a.n, 32, false)) {
    *why = "cuTensorMapEncodeTiled is unavailable or rejected the operands";
    return cudaErrorInvalidValue;
  }
  BlockPairParams p = {};
  p.x_scales = a.x_scales;
  p.w_scales = a.w_scales;
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.err = a.err;
  p.m = static_cast<int>(a.m);
  p.n = static_cast<int>(a.n);
  p.blocks = static_cast<int>(block_count(a.k));
  p.m_units = static_cast<int>((a.m + 2 * kBpRows - 1) / (2 * kBpRows));
  p.n_tiles = static_cast<int>((a.n + kBpCols - 1) / kBpCols);
  p.split = plan.split;
  p.act = a.act;
  const int clusters = static_cast<int>(plan.tiles < fit ? plan.tiles : fit);
  // as in gemm_tcgen05.cu: the divisor of the clusters at work nearest 16 within 12..24
  p.group_n = 16;
  for (int d = 0; d <= 8; ++d) {
    if (16 + d <= 24 && clusters % (16 + d) == 0) { p.group_n = 16 + d; break; }
    if (d > 0 && 16 - d >= 12 && clusters % (16 - d) == 0) { p.group_n = 16 - d; break; }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * p.split));
  cfg.blockDim = dim3(kBpThreads);
  cfg.dynamicSmemBytes = kBpSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(2 * p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_block_pair_kernel, map_x, map_w, map_y, p);
}

}  // namespace gbf
