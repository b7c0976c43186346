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
// for a batch of decode rows and for one long prompt.  A small call is a single
// CTA.  In one with many tokens a thread takes four of them in a row for one
// bisection, and several CTAs share the writes: as many as the tokens fill,
// independent of one another, when seq_lens and ring_out have memory of their
// own; one cluster of eight, with a barrier between the last read of ctx and
// ring and the first write, when one of them is updated in place.
//
// Measured (device time, back to back): 32 decode rows 3.7 us, of which a launch
// alone is some 2; 300 rows beside 24 prompts, 50,000 tokens, 7.3 us (14.8 in
// place, 202 on one CTA).
#include "common.cuh"
#include "decode.h"

#include <cooperative_groups.h>

namespace gbf {
namespace {

namespace cg = cooperative_groups;

constexpr int kSlotsCluster = 8;
constexpr int kSlotsGrid = 152;
// A batch of up to 512 requests is scanned by 256 threads (32 decode rows 3.9 us, 6.5 by 1024), a larger one by 1024.
constexpr int kSlotsSmall = 512;
// Up to two tokens per thread are one CTA's: 1000 decode rows 8.8 us, 10.2 shared; some 1500 tokens on 256 threads 5.2
// shared, 8.1 alone; 32 rows 3.9 alone, 5.3 shared.
constexpr int kAlonePerThread = 2;

__host__ GBF_DEVICE int clamp31(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v); }

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

enum Share { kAlone, kCluster, kGrid };      // one CTA; a cluster with a barrier; CTAs that do not wait for one another

// THREADS per CTA, each with up to PER requests of the scan.
template <int THREADS, int PER, Share SHARE>
__global__ void __launch_bounds__(THREADS) paged_slots_kernel(const PagedSlotsArgs a) {
  constexpr int kSlotThreads = THREADS, kSlotWarps = THREADS / 32, kPerThread = PER;
  constexpr int kRow = SHARE == kAlone ? 1 : 4;          // tokens in a row per thread
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
  int head = a.ring[0], count = a.ring[1];
  if (head < 0 || head >= a.num_blocks || count < 0 || count > a.num_blocks) {
    if (tid == 0) raise_error(a.err, DEV_ERR_BLOCK_POOL);
    head = 0;
    count = -1;                                  // a bad ring: nothing to take
  }
  if (tid == 0) s_taken = 0;

  unsigned rank = 0, ranks = 1;                  // (the cluster is the whole grid)
  if (SHARE != kAlone) {
    rank = blockIdx.x;
    ranks = gridDim.x;
  }
  const int64_t worker = static_cast<int64_t>(rank) * kSlotThreads + tid;
  const int64_t workers = static_cast<int64_t>(ranks) * kSlotThreads;

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
    if (len < 0 || len > a.room) {
      raise_error(a.err, DEV_ERR_BLOCK_RANGE);
      len = len < 0 ? 0 : a.room;
      refuse = true;
    }
    fresh[i] = more > 0 ? more : 0;
    if (fresh[i] > a.room - len) {
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
    const int64_t mine = lane < kSlotWarps ? sums[k][lane] : 0;
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
  if (SHARE == kCluster) cg::this_cluster().sync();
  else __syncthreads();
  taken = s_taken;
  int given = first_old[n];
  // more blocks than there are, or a bad ring: nothing goes back, and the ended requests keep their blocks and lengths
  const bool returns = count >= 0 && static_cast<int64_t>(count) + given <= a.num_blocks;
  if (!returns) {
    if (given > 0 && tid == 0) raise_error(a.err, DEV_ERR_BLOCK_POOL);
    given = 0;
  }
  auto ring_at = [&](int64_t i) {               // i < 2 * num_blocks
    const int64_t j = head + i;
    return j >= a.num_blocks ? (j - a.num_blocks >= a.num_blocks ? j - 2LL * a.num_blocks : j - a.num_blocks) : j;
  };

  if (worker == 0) {
    // (a bad ring stays as it is, so that the next call reports it again)
    a.ring_out[0] = count < 0 ? a.ring[0] : static_cast<int32_t>(ring_at(taken));
    a.ring_out[1] = count < 0 ? a.ring[1] : count - taken + given;
  }
  // (by the workers that have the fewest tokens, which would wait for the read of add: 0.2 us of 3.8, 0.3 in place; of CTAs
  // that do not wait for one another, by those that start first: 0.3 of 6.4)
  for (int64_t b = SHARE == kGrid ? worker : workers - 1 - worker; b < n; b += workers) {
    // (by its own new tokens: the prefix sums stop at 2^31 - 1, which a refused request's new length may reach)
    const int c = ctx[b], more = a.add[b];
    a.seq[b] = c < 0 ? ~c : more >= 0 ? c + more : returns ? 0 : c;
    if (a.start) a.start[b] = first_tok[b];
  }
  if (worker == 0 && a.start) a.start[n] = first_tok[n];

  // blocks taken
  for (int64_t i = worker; i < taken; i += workers) {
    const int b = find_last(first_new, n, static_cast<int>(i));
    const int j = ceil_div(ctx[b], bs) + static_cast<int>(i) - first_new[b];
    a.table[b * a.table_stride + j] = a.free_ring[ring_at(i)];
  }
  // blocks given back (a bad id too: leaving it out would move all behind it, which CTAs that do not wait for one another
  // cannot agree on; the tokens of whoever takes it get slot -1)
  for (int64_t i = worker; i < given; i += workers) {
    const int b = find_last(first_old, n, static_cast<int>(i));
    const int32_t id = a.table[b * a.table_stride + (i - first_old[b])];
    if (id < 0 || id >= a.num_blocks) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
    a.free_ring[ring_at(static_cast<int64_t>(count) + i)] = id;
  }
  // tokens: a new block's id is read from the ring, not from the table entry that another thread writes
  const int tokens = first_tok[n] < a.tokens ? first_tok[n] : a.tokens;
  if (worker == 0 && first_tok[n] > a.tokens) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
  for (int64_t t0 = worker * kRow; t0 < tokens; t0 += workers * kRow) {
    int b = find_last(first_tok, n, static_cast<int>(t0)), last_blk = -1, last_b = -1;
    int32_t id = -1;
    int32_t slot[kRow], pos[kRow];
#pragma unroll
    for (int i = 0; i < kRow; ++i) {
      slot[i] = pos[i] = -1;
      if (t0 + i >= tokens) continue;
      const int t = static_cast<int>(t0 + i);
      while (first_tok[b + 1] <= t) ++b;                 // (requests without tokens are passed over)
      const int c = ctx[b];
      const int64_t p = static_cast<int64_t>(c < 0 ? ~c : c) + (t - first_tok[b]);
      pos[i] = clamp31(p);
      if (c < 0) continue;
      const int blk = static_cast<int>(p / bs);
      if (blk != last_blk || b != last_b) {
        const int have = ceil_div(c, bs);
        id = blk < have ? a.table[b * a.table_stride + blk]
                        : a.free_ring[ring_at(static_cast<int64_t>(first_new[b]) + blk - have)];
        last_blk = blk;
        last_b = b;
        if (id < 0 || id >= a.num_blocks) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
      }
      if (id >= 0 && id < a.num_blocks) slot[i] = id * bs + static_cast<int>(p - static_cast<int64_t>(blk) * bs);
    }
    if (kRow == 4 && t0 + kRow <= tokens && a.wide) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1 % kRow], slot[2 % kRow], slot[3 % kRow]);
      *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1 % kRow], pos[2 % kRow], pos[3 % kRow]);
    } else {
#pragma unroll
      for (int i = 0; i < kRow; ++i)
        if (t0 + i < tokens) {
          a.slots[t0 + i] = slot[i];
          a.pos[t0 + i] = pos[i];
        }
    }
  }
}

template <int THREADS, int PER, Share SHARE>
cudaError_t launch(const PagedSlotsArgs& a, size_t smem, cudaStream_t stream) {
  constexpr int most = (4 * THREADS * PER + 3) * static_cast<int>(sizeof(int));
  const cudaError_t e = allow_smem<paged_slots_kernel<THREADS, PER, SHARE>>(most);
  if (e != cudaSuccess) return e;
  const int fill = static_cast<int>((static_cast<int64_t>(a.tokens) + 4 * THREADS - 1) / (4 * THREADS));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(SHARE == kAlone ? 1 : SHARE == kCluster ? kSlotsCluster : fill < kSlotsGrid ? fill : kSlotsGrid);
  cfg.blockDim = dim3(THREADS);
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
  cfg.numAttrs = SHARE == kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, paged_slots_kernel<THREADS, PER, SHARE>, a);
}

}  // namespace

cudaError_t launch_paged_slots(PagedSlotsArgs a, cudaStream_t stream) {
  const size_t smem = (4 * static_cast<size_t>(a.batch) + 3) * sizeof(int);
  a.room = clamp31(static_cast<int64_t>(a.max_blocks) * a.block_size);
  a.wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
  const bool in_place = a.seq == a.ctx || a.ring_out == a.ring, small = a.batch <= kSlotsSmall;
  if (a.tokens <= kAlonePerThread * (small ? 256 : 1024))
    return small ? launch<256, 2, kAlone>(a, smem, stream) : launch<1024, 8, kAlone>(a, smem, stream);
  if (in_place) return launch<1024, 8, kCluster>(a, smem, stream);
  return small ? launch<256, 2, kGrid>(a, smem, stream) : launch<1024, 8, kGrid>(a, smem, stream);
}

}  // namespace gbf
