// Internal interface of the decode-step operators (paged slots, paged
// attention, sampling) between the C-ABI layer and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gbf {

// Lets `Kernel` use `bytes` of dynamic shared memory on the current device, and
// asks for the largest shared-memory share of the L1 (the default one holds a
// single CTA of these kernels); done once per device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// How many clusters of 2^log_ranks CTAs (1 to 8) of `Kernel` the current device holds at once; asked once per device.
// (Fewer than SMs would hold: those of a GPC are not a multiple of 8.)
template <auto Kernel>
cudaError_t resident_clusters(int log_ranks, int threads, int smem, int* out) {
  static std::atomic<int> known[64][4];              // how many, and one; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>& k = known[dev & 63][log_ranks];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    e = allow_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << log_ranks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(1u << log_ranks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg);
    if (e != cudaSuccess) return e;
    k.store(++n, std::memory_order_relaxed);
  }
  *out = n - 1;
  return cudaSuccess;
}

// Further bits of the device error word (bits 0..2 are common.cuh's).
enum : unsigned int {
  DEV_ERR_BLOCK_RANGE = 1u << 3,   // a block id outside the cache, or a length outside its block-table row
  DEV_ERR_BLOCK_POOL = 1u << 4,    // the ring of free blocks ran out, or its state is inconsistent
  DEV_ERR_SAMPLING = 1u << 5,      // a sampling parameter outside its range, or a row without a candidate
};

// ---------------------------------------------------------- paged attention
struct PagedAttnArgs {
  const void* q;            // bf16 [batch, hq, d]
  const void* k;            // bf16 [cache_rows, hkv, d]
  const void* v;
  const int32_t* table;     // [batch, max_blocks], rows table_stride apart
  const int32_t* lens;      // [batch]
  void* out;                // bf16 [batch, hq, d], or E4M3 codes when out_fp8
  float* lse;               // [batch, hq], nullable
  float* ws;                // partial results
  unsigned int* err;
  int64_t table_stride;
  int64_t num_blocks;
  int batch, hq, hkv, d;
  int max_blocks, block_size;
  int window;               // 0: the whole length
  int out_fp8;
  float scale_log2;         // softmax scale * log2(e)
  float inv_out_scale;
  // set by the launcher
  int room;                 // longest length: max_blocks * block_size, and positions of a tile stay below 2^31
  int block_shift;          // log2(block_size), or -1
  int group, chunks;        // query heads per KV head; row tiles they are cut into
  int min_units;            // least token tiles per CTA
  int ctas;
  int log_ranks;            // CTAs of an item's cluster, where items are clusters; -1: items are warps
};

int64_t paged_attention_workspace(int hq, int hkv, int d);
cudaError_t launch_paged_attention(PagedAttnArgs a, cudaStream_t stream);

// --------------------------------------------------------------- paged slots
constexpr int kSlotsMaxBatch = 8192;

struct PagedSlotsArgs {
  const int32_t* ctx;       // [batch]
  const int32_t* add;       // [batch]
  int32_t* table;           // [batch, max_blocks], rows table_stride apart
  int32_t* free_ring;       // [num_blocks]
  const int32_t* ring;      // [2] head, count
  int32_t* seq;             // [batch] (may equal ctx)
  int32_t* ring_out;        // [2] (may equal ring)
  int32_t* slots;           // [tokens]
  int32_t* pos;             // [tokens]
  int32_t* start;           // [batch + 1], nullable
  unsigned int* err;
  int64_t table_stride;
  int32_t num_blocks, tokens;
  int batch, max_blocks, block_size;
  // set by the launcher
  int wide;                 // slots and pos are 16-byte aligned
  int room;                 // longest length of a table row: few and large blocks may hold more tokens than an int32 can say
};

cudaError_t launch_paged_slots(PagedSlotsArgs a, cudaStream_t stream);

// ----------------------------------------------------------------- sampling
struct SampleArgs {
  const void* logits;       // [batch, vocab], rows `stride` elements apart
  const float* uniform;     // [batch]
  const float* temperature; // [batch], nullable: 1
  const int32_t* top_k;     // [batch], nullable: off
  const float* top_p;       // [batch], nullable: off
  const float* min_p;       // [batch], nullable: off
  int32_t* tokens;          // [batch]
  float* logprob;           // [batch], nullable
  unsigned int* err;
  int64_t stride;
  int64_t batch;
  int vocab;
  int f32;                  // logits are float32 (else bf16)
};

cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t stream);

}  // namespace gbf
