// paged_slots: block tables, slot maps and positions of a serving step, built
// on the GPU from the requests' lengths.
//
//   have_b = ceil(ctx_b / bs), want_b = ceil((ctx_b + add_b) / bs)
//   the want_b - have_b blocks a request lacks come from the front of a ring of
//   free blocks, in request order; the blocks of an ended request (add_b < 0)
//   go back behind its end
//   token i of request b: p = ctx_b + i, slot = table[b, p / bs] * bs + p % bs
//
// Everything follows from three prefix sums over the batch (tokens, blocks
// taken, blocks given back).  They are some hundred integers: what bounds the
// call is latency, so each CTA scans the whole batch by itself and keeps the
// sums in shared memory, and every write after that is independent.  Tokens
// and blocks find their request by bisection of the sums, which costs the same
// for a batch of decode rows and for one long prompt.  A call with many tokens
// runs as one cluster of eight CTAs that share the writes (one barrier between
// the last read of ctx and ring and the first write, so that both may be
// updated in place); a small one as a single CTA.
#include "common.cuh"
#include "decode.h"

#include <cooperative_groups.h>

namespace gbf {
namespace {

namespace cg = cooperative_groups;

constexpr int kSlotThreads = 1024;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr int kPerThread = kSlotsMaxBatch / kSlotThreads;
constexpr int kSlotsCluster = 8;
constexpr int kSlotsClusterTokens = 4096;   // more tokens than this: a cluster

GBF_DEVICE int clamp31(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v); }

// The last index i in [0, n) with first[i] <= x, for a non-decreasing `first`.
GBF_DEVICE int find_last(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

GBF_DEVICE int ceil_div(int64_t n, int d) { return static_cast<int>((n + d - 1) / d); }

template <bool CLUSTER>
__global__ void __launch_bounds__(kSlotThreads) paged_slots_kernel(const PagedSlotsArgs a) {
  extern __shared__ int dyn[];
  const int n = a.batch;
  int* first_tok = dyn;                 // [n + 1] tokens of the requests before
  int* first_new = first_tok + n + 1;   // [n + 1] blocks they take
  int* first_old = first_new + n + 1;   // [n + 1] blocks they give back
  int* ctx = first_old + n + 1;         // [n] cached length; ~length when the request is refused
  __shared__ int64_t sums[3][kSlotWarps];
  __shared__ int s_taken;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = a.block_size;
  const int64_t room = static_cast<int64_t>(a.max_blocks) * bs;
  int head = a.ring[0], count = a.ring[1];
  if (head < 0 || head >= a.num_blocks || count < 0 || count > a.num_blocks) {
    if (tid == 0) raise_error(a.err, DEV_ERR_BLOCK_POOL);
    head = count = 0;
  }
  if (tid == 0) s_taken = 0;

  // this thread's requests, a contiguous run of them
  const int per = (n + kSlotThreads - 1) / kSlotThreads;
  const int b0 = tid * per < n ? tid * per : n, b1 = b0 + per < n ? b0 + per : n;
  int c_[kPerThread], fresh[kPerThread], need[kPerThread], back[kPerThread];
  int64_t sum[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    c_[i] = fresh[i] = need[i] = back[i] = 0;
    if (b >= b1) continue;
    int len = a.ctx[b];
    const int more = a.add[b];
    bool refuse = false;
    if (len < 0 || len > room) {
      raise_error(a.err, DEV_ERR_BLOCK_RANGE);
      len = len < 0 ? 0 : static_cast<int>(room);
      refuse = true;
    }
    fresh[i] = more > 0 ? more : 0;
    if (static_cast<int64_t>(len) + fresh[i] > room) {
      raise_error(a.err, DEV_ERR_BLOCK_RANGE);
      refuse = true;
    }
    if (!refuse) {
      const int have = ceil_div(len, bs);
      if (more < 0) back[i] = have;
      else need[i] = ceil_div(static_cast<int64_t>(len) + more, bs) - have;
    }
    c_[i] = refuse ? ~len : len;
    sum[0] += fresh[i];
    sum[1] += need[i];
    sum[2] += back[i];
  }
  int64_t incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += up;
    }
  if (lane == 31)
    for (int k = 0; k < 3; ++k) sums[k][warp] = incl[k];
  __syncthreads();
  int64_t at[3], total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int64_t mine = sums[k][lane];
    int64_t before = lane < warp ? mine : 0, all = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    at[k] = before + incl[k] - sum[k];
    total[k] = all;
  }
  int taken = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    if (b >= b1) continue;
    first_tok[b] = clamp31(at[0]);
    first_new[b] = clamp31(at[1]);
    first_old[b] = clamp31(at[2]);
    at[0] += fresh[i];
    at[1] += need[i];
    at[2] += back[i];
    // requests are served in order while the ring lasts: this one and all later
    // ones that need blocks are refused once the sum passes its count
    if (need[i] > 0) {
      if (at[1] <= count) taken = static_cast<int>(at[1]);
      else {
        c_[i] = ~c_[i];
        raise_error(a.err, DEV_ERR_BLOCK_POOL);
      }
    }
    ctx[b] = c_[i];
  }
  if (tid == 0) {
    first_tok[n] = clamp31(total[0]);
    first_new[n] = clamp31(total[1]);
    first_old[n] = clamp31(total[2]);
  }
  // every read of ctx, add and ring is done
  if (taken > 0) atomicMax(&s_taken, taken);
  unsigned rank = 0, ranks = 1;
  if (CLUSTER) {
    cg::cluster_group cluster = cg::this_cluster();
    rank = cluster.block_rank();
    ranks = cluster.num_blocks();
    cluster.sync();
  } else {
    __syncthreads();
  }
  taken = s_taken;
  int given = first_old[n];
  if (static_cast<int64_t>(count) + given > a.num_blocks) {     // more blocks than there are: nothing goes back
    if (tid == 0) raise_error(a.err, DEV_ERR_BLOCK_POOL);
    given = 0;
  }
  const int64_t worker = static_cast<int64_t>(rank) * kSlotThreads + tid;
  const int64_t workers = static_cast<int64_t>(ranks) * kSlotThreads;
  auto ring_at = [&](int64_t i) {               // i < 2 * num_blocks
    const int64_t j = head + i;
    return j >= a.num_blocks ? (j - a.num_blocks >= a.num_blocks ? j - 2LL * a.num_blocks : j - a.num_blocks) : j;
  };

  if (worker == 0) {
    const int64_t h = ring_at(taken);
    a.ring_out[0] = static_cast<int32_t>(h);
    a.ring_out[1] = count - taken + given;
  }
  for (int64_t b = worker; b < n; b += workers) {
    const int c = ctx[b];
    const int tokens = first_tok[b + 1] - first_tok[b];
    const bool ended = c >= 0 && first_old[b + 1] != first_old[b];
    a.seq[b] = c < 0 ? ~c : ended ? 0 : c + tokens;
    if (a.start) a.start[b] = first_tok[b];
  }
  if (worker == 0 && a.start) a.start[n] = first_tok[n];

  // blocks taken
  for (int64_t i = worker; i < taken; i += workers) {
    const int b = find_last(first_new, n, static_cast<int>(i));
    const int j = ceil_div(ctx[b], bs) + static_cast<int>(i) - first_new[b];
    a.table[b * a.table_stride + j] = a.free_ring[ring_at(i)];
  }
  // blocks given back
  for (int64_t i = worker; i < given; i += workers) {
    const int b = find_last(first_old, n, static_cast<int>(i));
    const int32_t id = a.table[b * a.table_stride + (i - first_old[b])];
    if (id < 0 || id >= a.num_blocks) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
    a.free_ring[ring_at(static_cast<int64_t>(count) + i)] = id;
  }
  // tokens: a new block's id is read from the ring, not from the table entry that another thread writes
  const int tokens = first_tok[n] < a.tokens ? first_tok[n] : a.tokens;
  if (worker == 0 && first_tok[n] > a.tokens) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
  for (int64_t t = worker; t < tokens; t += workers) {
    const int b = find_last(first_tok, n, static_cast<int>(t));
    const int c = ctx[b];
    const int64_t p = static_cast<int64_t>(c < 0 ? ~c : c) + (t - first_tok[b]);
    int32_t slot = -1;
    if (c >= 0) {
      const int blk = static_cast<int>(p / bs), have = ceil_div(c, bs);
      const int32_t id = blk < have ? a.table[b * a.table_stride + blk]
                                    : a.free_ring[ring_at(static_cast<int64_t>(first_new[b]) + blk - have)];
      if (id >= 0 && id < a.num_blocks) slot = id * bs + static_cast<int>(p - static_cast<int64_t>(blk) * bs);
      else raise_error(a.err, DEV_ERR_BLOCK_RANGE);
    }
    a.slots[t] = slot;
    a.pos[t] = clamp31(p);
  }
}

}  // namespace

cudaError_t launch_paged_slots(const PagedSlotsArgs& a, cudaStream_t stream) {
  const size_t smem = (4 * static_cast<size_t>(a.batch) + 3) * sizeof(int);
  const bool cluster = a.tokens > kSlotsClusterTokens;
  auto kernel = cluster ? paged_slots_kernel<true> : paged_slots_kernel<false>;
  constexpr int most = (4 * kSlotsMaxBatch + 3) * static_cast<int>(sizeof(int));
  const cudaError_t e = cluster ? allow_smem<paged_slots_kernel<true>>(most) : allow_smem<paged_slots_kernel<false>>(most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster ? kSlotsCluster : 1);
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSlotsCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace gbf
