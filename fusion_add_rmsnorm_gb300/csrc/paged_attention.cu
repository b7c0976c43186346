// paged_attention: attention of one new token per request over the paged K/V
// cache that the QKV kernels write, split over the length and joined.
//
//   s_j = scale q . k_j  for the cached positions j in [max(0, len - window), len)
//   out = sum_j softmax(s)_j v_j,   lse = ln sum_j exp(s_j)
//
// The query heads of one KV head (a group) share its K and V, so up to 16 of them
// read each once: per token and KV head 4 d bytes for 4 d group flops, far on HBM's
// side.  A larger group is cut into row tiles of 16 heads, items of their own, each
// of which reads K and V again, from L2 at best: 32 requests of 4096 on one KV head
// of 128 (67 MB) take 12.1 us with 8 heads, 14.2 with 16, 28.7 with 32 and 42.3 with 64.
//
// Work split: the unit is a tile of 16 cached tokens of one (request, KV head)
// item, and kOwn units per item for what an item costs by itself.  All
// items' units in a row (requests, then KV heads, then tokens) are cut into
// equal contiguous ranges, one per CTA of a grid that just fills the GPU, so a
// ragged batch loads every SM alike and no length needs to be known on the
// host.  Each CTA finds its range itself: a scan over the lengths.  An item
// whose tiles lie in one CTA is finished there; one that a range border cuts
// leaves a partial (max, sum, unnormalised output, float32) per CTA in the
// workspace, and a second small kernel joins the partials in CTA order, so
// results do not depend on timing.
//
// A call whose lengths cannot be long (by the block table's width, or the
// window) takes another split: an item is one warp's, or, where all items find
// room at once, a cluster's of 1 to 8 CTAs, joined through distributed shared
// memory; with no scan, no workspace and no second launch.
//
// Inside a CTA the warps take a range's tiles in turn and never wait for one
// another within an item: each has its own ring of stages (16 K rows and 16 V
// rows) filled by 16-byte cp.async, its own running maximum and sum, and its
// own accumulators; the ring runs on across item borders, so the next item's
// rows are on their way while the warps' results are joined through shared
// memory.  A short item is one warp's alone: the warps take such items in turn
// and finish them without a barrier.  Scores are mma.m16n8k16 with the group's heads as the 16 rows and
// the tokens as columns; the score accumulators are then, element for
// element, the A operand of the product with V.
//
// What bounds it: HBM, from the first tile's arrival to the last one's.  In front of that lie the reads that follow one
// from another (lengths, table, rows: 3.5 us of the 36 to 50 us of a batch), behind it the join.  Device time, back to
// back: 32 requests up to 4096, 32 heads on 8 of 128, 49 us (277 MB: 5.6 TB/s); 256 such requests 326 us (2.16 GB: 6.6
// TB/s); two documents of 131072 on 8 KV heads 126 us (806 MB: 6.4 TB/s); 48 requests on one KV head of 256, window 4096,
// 35.8 us (158 MB: 4.4 TB/s; at that width the loop takes 255 registers and spills 184 bytes, with one warp per scheduler);
// one request of 700 tokens 5.5 us (a launch, and reads that wait for one another) behind a table of up to 4096 tokens, 8.1
// behind a wider one, which is split over the GPU.
//
// Rounding: scores, maxima, sums and outputs are float32.  P enters the second
// product as a pair of bf16 (value and remainder, 2^-17 together), because one
// bf16 alone would add an error as large as the final bf16 rounding.  For
// groups of up to 8 heads the remainder rides in the rows 8..15 that the heads
// leave empty, at no further instruction.
#include <cooperative_groups.h>

#include "common.cuh"
#include "decode.h"

namespace gbf {
namespace {

namespace cg = cooperative_groups;

constexpr int kTile = 16;              // tokens per tile
// An item is one warp's alone (joining the warps costs about as much as four tiles) when it has at most 4 tiles, 8
// where a CTA has two items on average, and up to 16 as long as that is a 16th of the CTA's units.  192 requests up to
// 2048, 8 KV heads of 64: 80.1 us, 84.8 with 4 throughout; 48 on one KV head of 256, window 4096: 36.0, 45.7 with 16
// throughout; 64 requests up to 1024, 12 KV heads of 64: 28.9, 33.3 with none.
constexpr int kSoloOne = 4, kSoloTwo = 8, kSoloMost = 16;
// Units an item counts beside its tiles, for its queries, its start and its join: 24 requests of 32 KV heads take 48.8 us
// with 8 or 4, 60.8 with 0; window 4096 on one KV head 35.8 with 8, 37.2 with 4, 35.3 with 12, and 256 requests up to 512
// 52.3, 51.8 and 54.3.
constexpr int kOwn = 8;
constexpr int kSms = 152;
constexpr int kTogether = 8;           // most CTAs of a cluster that share an item
// What each of them takes at least where a smaller cluster would do, and at most (in tokens).  One request, 8 KV heads, 256
// tokens: 5.0 us with four CTAs of 64, 5.4 with eight, 6.9 split over the GPU; 4096 tokens 10.3 with eight of 512, 13.5 over
// the GPU, 8192 tokens 14.8 and 15.0; 8 requests of 2048 11.6 with four of 512 and 13.0, of 4096 21.7 and 20.5; 24 of 256
// 7.7 with one CTA each and 10.6, of 1024 18.8 and 15.6.
constexpr int kTogetherLeast = 64, kTogetherMost = 512;
// One warp takes an item alone, with no join at all, where it has at most four tiles (896 items of up to 64 tokens: 6.3
// us, 12.1 over the GPU; 160 items: 5.3, 5.5 with a CTA each, 10.1 over the GPU), or 16 where the items are too many for a
// CTA each (896 of 256 tokens: 16.8 us, 21.0 over the GPU, 23.1 with a CTA each; of 512 tokens 29.8, 29.9 and 32.4).
constexpr int kWarpTokens = 64, kWarpTokensMany = 256;
constexpr float kLn2 = 0.693147180559945f;

// Layout per padded head width: warps per CTA, ring depth, CTAs per SM.  Two stages ahead of the one in use keep 130 to
// 210 KB of an SM on their way, more than the bandwidth needs: at 64 three stages take 27.2 us on 64 requests of 12 heads
// and six 29.0 (a longer start), three CTAs per SM 95 us where two take 79; at 128 one CTA with six stages 58 us where two
// with three take 48.5, and two stages 48.8; at 256 two stages 57 us, three 54.5.
template <int DP>
struct Plan;
template <>
struct Plan<64> {
  static constexpr int kWarps = 4, kStages = 3, kPerSm = 2;
};
template <>
struct Plan<128> {
  static constexpr int kWarps = 4, kStages = 3, kPerSm = 2;
};
template <>
struct Plan<256> {
  static constexpr int kWarps = 4, kStages = 3, kPerSm = 1;
};

template <int DP>
constexpr int stage_bytes() { return 2 * kTile * DP * 2; }
// The join goes through shared memory half the columns at a time; floats per row, rows 8 banks apart.
template <int DP>
constexpr int join_stride() { return DP / 2 + 8; }
template <int DP>
constexpr int smem_bytes() {
  return Plan<DP>::kWarps * (Plan<DP>::kStages * stage_bytes<DP>() + 8 * join_stride<DP>() * 4);
}
// floats of one partial: 16 maxima, 16 sums, then the rows
template <int DP, bool WIDE>
constexpr int partial_floats() { return 32 + (WIDE ? 16 : 8) * DP; }

GBF_DEVICE float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

GBF_DEVICE void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
GBF_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
GBF_DEVICE void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

GBF_DEVICE void ldmatrix4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
GBF_DEVICE void ldmatrix4_trans(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
GBF_DEVICE void mma_bf16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------- the work split

struct Request {
  int len, lo, tiles;     // cached tokens [lo, len) and their tiles; an item is kOwn + tiles units, the tiles last
};

// EARLY: from L2, for a kernel that reads lengths before its pdl_wait() (see the join).
template <bool EARLY = false>
GBF_DEVICE int length_of(const PagedAttnArgs& a, int b) {
  if (!EARLY) return a.lens[b];
  int len;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(len) : "l"(a.lens + b) : "memory");
  return len;
}

template <bool EARLY = false>
GBF_DEVICE Request request_of(const PagedAttnArgs& a, int b) {
  Request r;
  r.len = length_of<EARLY>(a, b);
  if (r.len < 0) r.len = 0;
  if (r.len > a.room) r.len = a.room;
  r.lo = a.window > 0 && r.len > a.window ? r.len - a.window : 0;
  r.tiles = (r.len - r.lo + kTile - 1) / kTile;
  return r;
}

// a / b of values >= 0, b > 0, as a 32-bit division where they fit
GBF_DEVICE int64_t quotient(int64_t a, int64_t b) {
  if ((a | b) >> 31) return a / b;
  return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Where unit c * share lies: request, and units into that request.
struct Place {
  int64_t units;          // of the whole batch
  int64_t share;          // per CTA
  int64_t rest;           // units into request b
  int b;                  // -1: past the end
};

// Every thread of the block calls this; the result is the same in all.
template <int NT, bool EARLY = false>
GBF_DEVICE Place locate(const PagedAttnArgs& a, int64_t c, bool report) {
  __shared__ int64_t warp_sum[NT / 32];
  __shared__ Place place;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.hkv * a.chunks;
  const int per = (a.batch + NT - 1) / NT;       // (up to 2^30 requests: in 32 bits)
  const int b0 = tid * per < a.batch ? tid * per : a.batch;
  const int b1 = b0 + per < a.batch ? b0 + per : a.batch;
  int64_t mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    mine += request_of<EARLY>(a, b).tiles + kOwn;
    const int len = length_of<EARLY>(a, b);
    bad |= report && (len < 0 || len > a.room);
  }
  if (bad) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
  mine *= items;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) place.b = -1;
  __syncthreads();
  int64_t base = 0, units = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += warp_sum[w];
    units += warp_sum[w];
  }
  base += incl - mine;
  int64_t share = quotient(units + a.ctas - 1, a.ctas);
  if (share < a.min_units) share = a.min_units;
  const int64_t u = c * share;
  if (u >= base && u < base + mine) {       // exactly one thread, unless u is past the end
    int64_t rest = u - base;
    int b = b0;
    for (;;) {
      const int64_t n = static_cast<int64_t>(request_of<EARLY>(a, b).tiles + kOwn) * items;
      if (rest < n) break;
      rest -= n;
      ++b;
    }
    place.b = b;
    place.rest = rest;
  }
  __syncthreads();
  Place p;
  p.b = place.b;
  p.rest = place.rest;
  p.units = units;
  p.share = share;
  return p;
}

// A walk over the tiles of a CTA's range that belong to one warp.
template <int NW>
struct Cursor {
  int64_t left;           // units of the range behind the current segment
  Request r;
  int b, item;            // request; (KV head, row tile) within it
  int t0, t1;             // the segment: tiles of the item that lie in the range
  int t, step;            // this warp's tile, and to its next one
  int turn, solo_turn;    // warps' turns: at the segment's first tile; at the next short item
  int most_solo;
  bool whole, solo;       // the segment is the whole item; and one warp's
  bool mine;              // this warp takes part in it
  bool done;

  GBF_DEVICE void start(const PagedAttnArgs& a, const Place& p, int64_t units, int warp) {
    b = p.b;
    r = request_of(a, b);
    const int64_t n = r.tiles + kOwn;
    item = static_cast<int>(quotient(p.rest, n));
    left = units;
    turn = solo_turn = 0;
    most_solo = p.share * a.batch * a.hkv * a.chunks >= 2 * p.units ? kSoloTwo : kSoloOne;
    if (p.share >> 4 > most_solo) most_solo = p.share >> 4 < kSoloMost ? static_cast<int>(p.share >> 4) : kSoloMost;
    done = false;
    enter(static_cast<int>(p.rest - item * n), warp);
  }
  // TOGETHER: an equal share of one item's tiles, or a whole item, and nothing else; false: there is none
  GBF_DEVICE bool share_of_item(const PagedAttnArgs& a, int cta, int warp) {
    solo = a.log_ranks < 0;
    const int items = a.hkv * a.chunks, index = solo ? cta * NW + warp : cta >> a.log_ranks;
    if (index >= a.batch * items) return false;
    b = index / items;
    item = index - b * items;
    r = request_of(a, b);
    left = 0;
    turn = solo_turn = most_solo = 0;
    whole = done = false;
    mine = true;
    if (solo) {
      t = t0 = 0;
      t1 = r.tiles;
      step = 1;
    } else {
      const int64_t rank = cta - (index << a.log_ranks);
      t0 = static_cast<int>(r.tiles * rank >> a.log_ranks);
      t1 = static_cast<int>(r.tiles * (rank + 1) >> a.log_ranks);
      t = t0 + warp;
      step = NW;
    }
    return true;
  }
  // the segment that begins at unit u of the item
  GBF_DEVICE void enter(int u, int warp) {
    const int64_t rest = r.tiles + kOwn - u, n = rest < left ? rest : left;
    const int end = u + static_cast<int>(n);
    left -= n;
    t0 = u > kOwn ? u - kOwn : 0;
    t1 = end > kOwn ? end - kOwn : 0;
    whole = t0 == 0 && t1 == r.tiles && (t1 > 0 || u == 0);
    solo = whole && t1 <= most_solo;
    if (solo) {
      mine = solo_turn == warp;
      solo_turn = (solo_turn + 1) % NW;
      t = mine ? t0 : t1;
      step = 1;
    } else {
      mine = t1 > t0;     // (a range may begin or end in an item's own units)
      t = t0 + ((warp - turn) & (NW - 1));
      turn = (turn + t1 - t0) & (NW - 1);
      step = NW;
    }
  }
  // the next segment of the range; false behind the last one
  GBF_DEVICE bool next_segment(const PagedAttnArgs& a, int warp) {
    if (left <= 0) {
      done = true;
      return false;
    }
    if (++item == a.hkv * a.chunks) {
      item = 0;
      r = request_of(a, ++b);
    }
    enter(0, warp);
    return true;
  }
  // skip segments that hold no tile of this warp
  GBF_DEVICE void settle(const PagedAttnArgs& a, int warp) {
    while (!done && t >= t1) next_segment(a, warp);
  }
  GBF_DEVICE void advance(const PagedAttnArgs& a, int warp) {
    t += step;
    settle(a, warp);
  }
};

// ------------------------------------------------------------------ the kernel

// Writes four consecutive outputs.
GBF_DEVICE void store_out4(const PagedAttnArgs& a, int64_t at, float4 o) {
  if (a.out_fp8) {
    const float s = a.inv_out_scale;
    const uint32_t lo = f32x2_to_e4m3x2(o.x * s, o.y * s), hi = f32x2_to_e4m3x2(o.z * s, o.w * s);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + at) = lo | (hi << 16);
  } else {
    uint2 w;
    w.x = f32x2_to_bf16x2(o.x, o.y);
    w.y = f32x2_to_bf16x2(o.z, o.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) = w;
  }
}

GBF_DEVICE void store_out2(const PagedAttnArgs& a, int64_t at, float2 o) {
  if (a.out_fp8)
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.out) + at) =
        f32x2_to_e4m3x2(o.x * a.inv_out_scale, o.y * a.inv_out_scale);
  else
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at) = f32x2_to_bf16x2(o.x, o.y);
}

// DP: head width padded to 64, 128 or 256.  WIDE: 9..16 heads per row tile
// (else up to 8, with the remainders of P in rows 8..15).
// TOGETHER: the split into clusters (an equal share of an item's tiles is each
// CTA's, and each joins a part of the columns) or warps.
template <int DP, bool WIDE, bool TOGETHER>
__global__ void __launch_bounds__(Plan<DP>::kWarps * 32, Plan<DP>::kPerSm)
    paged_attention_kernel(const PagedAttnArgs a) {
  constexpr int NW = Plan<DP>::kWarps, NS = Plan<DP>::kStages, NT = NW * 32;
  constexpr int KS = DP / 16;                    // k steps of the score product
  constexpr int CPR = DP / 8;                    // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;                  // rows per warp-wide copy
  constexpr int HALVES = WIDE ? 2 : 1;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[2][NW][16], sm_l[2][NW][16];
  __shared__ uint32_t sm_valid[NW][NS];
  __shared__ float cta_m[16], cta_l[16];         // TOGETHER: this CTA's maxima and sums

  // In this order, and before any return: the join reads the lengths as soon as it starts, and what makes them complete by
  // then is that every CTA here has passed its wait before it lets the join begin.
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Cursor<NW> load, work;
  if (TOGETHER) {
    if (!work.share_of_item(a, blockIdx.x, warp)) return;  // (a warp without an item: nobody waits for it)
    const int len = a.lens[work.b];
    if (lane == 0 && (len < 0 || len > a.room)) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
  } else {
    const Place place = locate<NT>(a, blockIdx.x, blockIdx.x == 0);
    if (place.b < 0) return;
    const int64_t first_unit = static_cast<int64_t>(blockIdx.x) * place.share;
    const int64_t units = place.units - first_unit < place.share ? place.units - first_unit : place.share;
    work.start(a, place, units, warp);
  }

  unsigned char* stages = smem + warp * (NS * stage_bytes<DP>());
  const uint32_t stages_u = static_cast<uint32_t>(__cvta_generic_to_shared(stages));
  float* joined = reinterpret_cast<float*>(smem + NW * NS * stage_bytes<DP>());   // [NW][8][join_stride]
  if (a.d < DP) {                                // the padding columns stay zero
    for (int i = lane; i < NS * stage_bytes<DP>() / 16; i += 32)
      reinterpret_cast<uint4*>(stages)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }

  const uint32_t row_bytes = static_cast<uint32_t>(a.hkv) * a.d * 2;
  const int chunk_col = lane % CPR;              // this lane's 16-byte column, and row within a copy
  const int chunk_row = lane / CPR;
  const bool col_on = chunk_col * 8 < a.d;

  load = work;
  load.settle(a, warp);

  // Block-table entry of lane's token (lanes 0..15) of the load cursor's tile, requested one tile before its rows are,
  // and the cursor's step to the next tile.
  struct Fetch {
    int entry, offset, head;
    bool inside, on;
  };
  auto fetch_entry = [&]() {
    Fetch f{-1, 0, 0, false, !load.done};
    if (load.done) return f;
    f.head = load.item / a.chunks;
    const int tok = load.r.lo + load.t * kTile + (lane & 15);
    if (tok < load.r.len) {
      int blk;
      if (a.block_shift >= 0) {
        blk = tok >> a.block_shift;
        f.offset = tok & (a.block_size - 1);
      } else {
        blk = tok / a.block_size;
        f.offset = tok - blk * a.block_size;
      }
      f.inside = true;
      f.entry = a.table[static_cast<int64_t>(load.b) * a.table_stride + blk];
    }
    load.advance(a, warp);
    return f;
  };
  auto issue = [&](int stage, const Fetch& f) {
    if (f.on) {
      const bool ok = f.inside && f.entry >= 0 && f.entry < a.num_blocks;
      if (f.inside && !ok) raise_error(a.err, DEV_ERR_BLOCK_RANGE);
      const uint32_t row = ok ? static_cast<uint32_t>(f.entry * a.block_size + f.offset) : 0u;
      const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      if (lane == 0) sm_valid[warp][stage] = valid;
      const int64_t col = static_cast<int64_t>(f.head) * a.d * 2 + chunk_col * 16;
      const char* kp = static_cast<const char*>(a.k) + col;
      const char* vp = static_cast<const char*>(a.v) + col;
      const uint32_t dst = stages_u + stage * stage_bytes<DP>() + chunk_row * (DP * 2);
#pragma unroll
      for (int i = 0; i < kTile / RPI; ++i) {
        const int tr = i * RPI + chunk_row;
        const uint64_t off = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, tr)) * row_bytes;
        const uint32_t n = (valid >> tr) & 1u ? 16u : 0u;     // what is masked arrives as zeros
        const uint32_t at = dst + i * RPI * (DP * 2) + ((chunk_col ^ (tr & 7)) << 4);
        if (col_on) {
          cp_async16(at, kp + off, n);
          cp_async16(at + kTile * DP * 2, vp + off, n);
        }
      }
    }
    cp_async_commit();
  };

  Fetch next;
  {
    Fetch first[NS - 1];                         // their entries are on their way together
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) first[s] = fetch_entry();
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s, first[s]);
    next = fetch_entry();
  }

  // ldmatrix rows of this lane: K (tokens 0..7 | 0..7 | 8..15 | 8..15, columns 0 | 8 | 0 | 8 of the k step),
  // V transposed (tokens 0..7 | 8..15 | 0..7 | 8..15, columns 0 | 0 | 8 | 8 of a pair of column tiles)
  const int k_tok = (lane & 7) + ((lane >> 4) << 3), k_chunk = (lane >> 3) & 1;
  const int v_tok = (lane & 7) + (((lane >> 3) & 1) << 3), v_chunk = lane >> 4;
  const int g = lane >> 2, t4 = lane & 3;        // accumulator row, column pair
  // the swizzle moves a chunk within its 128-byte line only: four offsets each, the lines are constants apart
  uint32_t k_at[4], v_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k_at[i] = stages_u + k_tok * (DP * 2) + (((i * 2 + k_chunk) ^ (k_tok & 7)) << 4);
    v_at[i] = stages_u + kTile * DP * 2 + v_tok * (DP * 2) + (((i * 2 + v_chunk) ^ (v_tok & 7)) << 4);
  }

  int stage = 0, parity = 0;
  for (;;) {                                     // segments
    if (!work.mine) {
      if (!work.next_segment(a, warp)) break;
      continue;
    }
    const int head = work.item / a.chunks, row0 = (work.item - head * a.chunks) * 16;
    const int rows = a.group - row0 < 16 ? a.group - row0 : 16;
    const int64_t q_row0 = static_cast<int64_t>(work.b) * a.hq + static_cast<int64_t>(head) * a.group + row0;

    uint32_t qf[KS][WIDE ? 4 : 2];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int r = g + 8 * h;
        const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + (q_row0 + r) * a.d;
        const int c0 = ks * 16 + t4 * 2;
        qf[ks][h] = r < rows && c0 < a.d ? *reinterpret_cast<const uint32_t*>(qp + c0) : 0u;
        qf[ks][HALVES + h] = r < rows && c0 + 8 < a.d ? *reinterpret_cast<const uint32_t*>(qp + c0 + 8) : 0u;
      }
    }

    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m[HALVES], l[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.0f;
    }

    for (; work.t < work.t1; work.t += work.step) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      const uint32_t valid = sm_valid[warp][stage];
      const uint32_t base = stage * stage_bytes<DP>();
      issue(stage == 0 ? NS - 1 : stage - 1, next);    // into the stage the previous tile has left
      next = fetch_entry();

      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t kf[4];
        ldmatrix4(kf, base + k_at[ks & 3] + (ks >> 2) * 128);
        const uint32_t a1 = WIDE ? qf[ks][1] : 0u, a3 = WIDE ? qf[ks][3] : 0u;
        mma_bf16(s[0], qf[ks][0], a1, qf[ks][HALVES], a3, kf[0], kf[1]);
        mma_bf16(s[1], qf[ks][0], a1, qf[ks][HALVES], a3, kf[2], kf[3]);
      }

      uint32_t p_hi[HALVES][2], p_lo[HALVES][2];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        float x[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool on = (valid >> (n * 8 + t4 * 2 + e)) & 1u;
            x[n * 2 + e] = on ? s[n][h * 2 + e] * a.scale_log2 : -INFINITY;
          }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the reference follows the maximum only when that is more than 2^8 ahead: weights up to 2^8 are as good as
        // weights up to 1, and rescaling the accumulators is left out for most tiles
        if (__any_sync(0xffffffffu, top > m[h] + 8.0f)) {
          const float next = top > m[h] + 8.0f ? top : m[h];
          const float shrink = next == -INFINITY ? 1.0f : exp2_approx(m[h] - next);
          m[h] = next;
          l[h] *= shrink;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            o[n][h * 2] *= shrink;
            o[n][h * 2 + 1] *= shrink;
            if (!WIDE) {                         // rows 8..15 belong to the same heads
              o[n][2] *= shrink;
              o[n][3] *= shrink;
            }
          }
        }
        const float ref = m[h] == -INFINITY ? 0.0f : m[h];     // nothing seen yet: every weight is zero
        float p[4], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = exp2_approx(x[i] - ref);
          sum += p[i];
        }
        l[h] += sum;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t hi = f32x2_to_bf16x2(p[2 * n], p[2 * n + 1]);
          p_hi[h][n] = hi;
          p_lo[h][n] = f32x2_to_bf16x2(p[2 * n] - __uint_as_float(hi << 16),
                                       p[2 * n + 1] - __uint_as_float(hi & 0xffff0000u));
        }
      }

#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t vf[4];
        ldmatrix4_trans(vf, base + v_at[n & 3] + (n >> 2) * 128);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (WIDE) {
            mma_bf16(o[2 * n + e], p_hi[0][0], p_hi[HALVES - 1][0], p_hi[0][1], p_hi[HALVES - 1][1], vf[2 * e],
                     vf[2 * e + 1]);
            mma_bf16(o[2 * n + e], p_lo[0][0], p_lo[HALVES - 1][0], p_lo[0][1], p_lo[HALVES - 1][1], vf[2 * e],
                     vf[2 * e + 1]);
          } else {
            mma_bf16(o[2 * n + e], p_hi[0][0], p_lo[0][0], p_hi[0][1], p_lo[0][1], vf[2 * e], vf[2 * e + 1]);
          }
        }
      }
      stage = stage + 1 == NS ? 0 : stage + 1;
    }

#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if (work.solo) {                             // nothing to join: from the registers to the output
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int row = g + 8 * h;
        const float inv = l[h] == 0.0f ? 0.0f : 1.0f / l[h];
        if (row < rows) {
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            float2 v = WIDE ? make_float2(o[n][h * 2], o[n][h * 2 + 1])
                            : make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
            v.x *= inv;
            v.y *= inv;
            const int c = n * 8 + t4 * 2;
            if (c < a.d) store_out2(a, (q_row0 + row) * a.d + c, v);
          }
          if (t4 == 0 && a.lse) a.lse[q_row0 + row] = l[h] == 0.0f ? -INFINITY : (m[h] + log2f(l[h])) * kLn2;
        }
      }
      if (!work.next_segment(a, warp)) break;
      continue;
    }

    // ---- the warps' results of this segment, joined through shared memory
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
      if (t4 == 0) {
        sm_m[parity][warp][g + 8 * h] = m[h];
        sm_l[parity][warp][g + 8 * h] = l[h];
      }
    const bool whole = work.whole;
    float* part = a.ws + (2 * static_cast<int64_t>(blockIdx.x) + (work.t0 == 0 ? 1 : 0)) * partial_floats<DP, WIDE>();
    float* cta_o = reinterpret_cast<float*>(smem);         // TOGETHER: [rows][DP], where the stages were
#pragma unroll
    for (int pass = 0; pass < 2 * HALVES; ++pass) {
      const int h = pass >> 1, half = pass & 1;
      __syncthreads();                           // maxima are there; the join area is free again
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, sm_m[parity][w][g + 8 * h]);
      // (a NaN score is in the sums but not in the maximum, so that with no other score that is -inf still)
      const float f = exp2_approx(m[h] - (top == -INFINITY ? 0.0f : top));
      float* dst = joined + (warp * 8 + g) * join_stride<DP>() + t4 * 2;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        const int n = half * (DP / 16) + i;
        float2 v = WIDE ? make_float2(o[n][h * 2], o[n][h * 2 + 1])
                        : make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
        v.x *= f;
        v.y *= f;
        *reinterpret_cast<float2*>(dst + i * 8) = v;
      }
      __syncthreads();
      for (int i = tid; i < DP; i += NT) {       // 8 rows of DP / 8 float4s
        const int r = i / (DP / 8), ch = (i - r * (DP / 8)) * 4, c = half * (DP / 2) + ch, row = r + 8 * h;
        if (row >= rows || c >= a.d) continue;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float big = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) big = fmaxf(big, sm_m[parity][w][row]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(joined + (w * 8 + r) * join_stride<DP>() + ch);
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
          total += sm_l[parity][w][row] * exp2_approx(sm_m[parity][w][row] - (big == -INFINITY ? 0.0f : big));
        }
        if (TOGETHER) {
          *reinterpret_cast<float4*>(cta_o + row * DP + c) = acc;
          if (c == 0) {
            cta_m[row] = big;
            cta_l[row] = total;
          }
        } else if (whole) {
          const float inv = total == 0.0f ? 0.0f : 1.0f / total;
          acc.x *= inv;
          acc.y *= inv;
          acc.z *= inv;
          acc.w *= inv;
          store_out4(a, (q_row0 + row) * a.d + c, acc);
          if (c == 0 && a.lse) a.lse[q_row0 + row] = total == 0.0f ? -INFINITY : (big + log2f(total)) * kLn2;
        } else {
          *reinterpret_cast<float4*>(part + 32 + row * DP + c) = acc;
          if (c == 0) {
            part[row] = big;
            part[16 + row] = total;
          }
        }
      }
    }
    if (TOGETHER) {
      cg::cluster_group cluster = cg::this_cluster();
      const int ranks = 1 << a.log_ranks;
      cluster.sync();
      for (int i = static_cast<int>(cluster.block_rank()) * NT + tid; i < rows * (DP / 4); i += ranks * NT) {
        const int row = i / (DP / 4), c = (i - row * (DP / 4)) * 4;
        if (c >= a.d) continue;
        float m_of[kTogether], l_of[kTogether], top = -INFINITY, total = 0.0f;
        float4 o_of[kTogether], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          m_of[k] = -INFINITY;
          l_of[k] = 0.0f;
          o_of[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k < ranks) {
            m_of[k] = *cluster.map_shared_rank(cta_m + row, k);
            l_of[k] = *cluster.map_shared_rank(cta_l + row, k);
            o_of[k] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(cta_o + row * DP + c, k));
          }
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k) top = fmaxf(top, m_of[k]);
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const float f = m_of[k] == -INFINITY ? 0.0f : exp2_approx(m_of[k] - top);
          total += l_of[k] * f;
          acc.x += o_of[k].x * f;
          acc.y += o_of[k].y * f;
          acc.z += o_of[k].z * f;
          acc.w += o_of[k].w * f;
        }
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        store_out4(a, (q_row0 + row) * a.d + c, acc);
        if (c == 0 && a.lse) a.lse[q_row0 + row] = total == 0.0f ? -INFINITY : (top + log2f(total)) * kLn2;
      }
      cluster.sync();                            // the others have read this CTA's results
      break;
    }
    parity ^= 1;
    if (!work.next_segment(a, warp)) break;
  }
  cp_async_wait<0>();
}

// Joins the partials of the items that range borders cut.  Block x looks after
// border x + 1 (between CTAs x and x + 1), for the first border inside its
// item only; block y takes the head row y of the item's row tile.
template <int DP, bool WIDE>
__global__ void __launch_bounds__(128) paged_attention_join_kernel(const PagedAttnArgs a) {
  constexpr int LANES = DP / 4, PARTS = 128 / LANES;      // threads of a row; partials read side by side
  __shared__ float4 acc_s[PARTS][LANES];
  __shared__ float l_s[PARTS];
  __shared__ float m_s[PARTS];
  pdl_launch_dependents();
  const int c = blockIdx.x + 1;
  // Before pdl_wait(), beside the kernel this one follows (behind the wait: 3.5 us more of 49 on the decode batch, 2.5 of 37 at
  // width 256).  That kernel's CTAs have all passed their own wait by now, so whatever wrote the lengths is done and its
  // writes are in L2; they are read from there, because only a wait of this grid's own would vouch for what an SM's L1
  // still holds.  Nothing else may be read here: the partials are not there yet.
  const Place p = locate<128, true>(a, c, false);
  bool on = p.b >= 0;
  int item = 0, c0 = 0, c1 = 0;
  if (on) {
    const Request r = request_of<true>(a, p.b);
    item = static_cast<int>(quotient(p.rest, r.tiles + kOwn));
    const int64_t u = p.rest - static_cast<int64_t>(item) * (r.tiles + kOwn), begin = c * p.share - u;
    c0 = static_cast<int>(quotient(begin + kOwn, p.share));        // CTAs of the item's first and last tile
    c1 = static_cast<int>(quotient(begin + kOwn + r.tiles - 1, p.share));
    on = u > kOwn && c == c0 + 1;
  }
  const int head = item / a.chunks, row0 = (item - head * a.chunks) * 16, row = blockIdx.y;
  on = on && row0 + row < a.group;
  pdl_wait();
  if (!on) return;
  const int tid = threadIdx.x, part = tid / LANES, col = tid % LANES;
  // slot of CTA c0 is its last segment's, of the others their first one's
  auto slot = [&](int cta) {
    return a.ws + (2 * static_cast<int64_t>(cta) + (cta == c0 ? 1 : 0)) * partial_floats<DP, WIDE>();
  };
  float m = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const bool col_on = col * 4 < a.d;
#pragma unroll 4
  for (int cta = c0 + part; cta <= c1; cta += PARTS) {
    const float* s = slot(cta);
    const float sm = s[row], sl = s[16 + row];
    const float4 v = col_on ? *reinterpret_cast<const float4*>(s + 32 + row * DP + col * 4)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float top = fmaxf(m, sm), ref = top == -INFINITY ? 0.0f : top;
    const float fo = exp2_approx(m - ref), fn = exp2_approx(sm - ref);
    m = top;
    l = l * fo + sl * fn;
    acc.x = acc.x * fo + v.x * fn;
    acc.y = acc.y * fo + v.y * fn;
    acc.z = acc.z * fo + v.z * fn;
    acc.w = acc.w * fo + v.w * fn;
  }
  acc_s[part][col] = acc;
  if (col == 0) {
    m_s[part] = m;
    l_s[part] = l;
  }
  __syncthreads();
  if (part != 0 || !col_on) return;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) top = fmaxf(top, m_s[i]);
  float4 out = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const float f = exp2_approx(m_s[i] - (top == -INFINITY ? 0.0f : top));
    const float4 v = acc_s[i][col];
    total += l_s[i] * f;
    out.x += v.x * f;
    out.y += v.y * f;
    out.z += v.z * f;
    out.w += v.w * f;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  out.x *= inv;
  out.y *= inv;
  out.z *= inv;
  out.w *= inv;
  const int64_t q_row = static_cast<int64_t>(p.b) * a.hq + static_cast<int64_t>(head) * a.group + row0 + row;
  store_out4(a, q_row * a.d + col * 4, out);
  if (col == 0 && a.lse) a.lse[q_row] = total == 0.0f ? -INFINITY : (top + log2f(total)) * kLn2;
}

template <int DP, bool WIDE>
cudaError_t launch_together(const PagedAttnArgs& a, int items, cudaStream_t stream) {
  const cudaError_t e = allow_smem<paged_attention_kernel<DP, WIDE, true>>(smem_bytes<DP>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.log_ranks < 0 ? (items + Plan<DP>::kWarps - 1) / Plan<DP>::kWarps : items << a.log_ranks);
  cfg.blockDim = dim3(Plan<DP>::kWarps * 32);
  cfg.dynamicSmemBytes = smem_bytes<DP>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.log_ranks < 0 ? 1 : 1 << a.log_ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_attention_kernel<DP, WIDE, true>, a);
}

template <int DP, bool WIDE>
cudaError_t launch(PagedAttnArgs a, cudaStream_t stream) {
  constexpr int NW = Plan<DP>::kWarps;
  a.min_units = NW;
  const int64_t seen = a.window > 0 && a.window < a.room ? a.window : a.room;
  const int64_t items = static_cast<int64_t>(a.batch) * a.hkv * a.chunks;
  cudaError_t e = cudaSuccess;
  a.log_ranks = -1;                              // a warp per item
  bool together = seen <= kWarpTokens;
  if (!together && seen <= kTogether * kTogetherMost) {
    int i = 0, n = 0;
    while (1 << i < kTogether && seen > kTogetherLeast << i) ++i;
    auto fit = [&] { return resident_clusters<paged_attention_kernel<DP, WIDE, true>>(i, NW * 32, smem_bytes<DP>(), &n); };
    e = fit();
    while (e == cudaSuccess && i > 0 && items > n) {
      --i;
      e = fit();
    }
    if (e != cudaSuccess) return e;
    if (items <= n) {
      together = seen <= kTogetherMost << i;
      a.log_ranks = i;
    } else {
      together = seen <= kWarpTokensMany;
    }
  }
  if (together && items <= 1 << 28) return launch_together<DP, WIDE>(a, static_cast<int>(items), stream);
  e = allow_smem<paged_attention_kernel<DP, WIDE, false>>(smem_bytes<DP>());
  if (e != cudaSuccess) return e;
  const int64_t tiles = (seen + kTile - 1) / kTile;
  const int64_t units = (tiles + kOwn) * items;
  int64_t ctas = (units + NW - 1) / NW;
  if (ctas > kSms * Plan<DP>::kPerSm) ctas = kSms * Plan<DP>::kPerSm;
  a.ctas = static_cast<int>(ctas);
  e = launch_pdl(paged_attention_kernel<DP, WIDE, false>, dim3(a.ctas), dim3(NW * 32), smem_bytes<DP>(), stream, a);
  if (e != cudaSuccess || a.ctas == 1) return e;
  const int rows = a.group < 16 ? a.group : 16;
  return launch_pdl(paged_attention_join_kernel<DP, WIDE>, dim3(a.ctas - 1, rows), dim3(128), 0, stream, a);
}

}  // namespace

int64_t paged_attention_workspace(int hq, int hkv, int d) {
  const int rows = hq / hkv > 8 ? 16 : 8;
  const int dp = d <= 64 ? 64 : d <= 128 ? 128 : 256;
  const int per_sm = d <= 64 ? Plan<64>::kPerSm : d <= 128 ? Plan<128>::kPerSm : Plan<256>::kPerSm;
  return static_cast<int64_t>(kSms) * per_sm * 2 * (32 + rows * dp) * 4;
}

cudaError_t launch_paged_attention(PagedAttnArgs a, cudaStream_t stream) {
  a.group = a.hq / a.hkv;
  a.chunks = (a.group + 15) / 16;
  const int64_t room = static_cast<int64_t>(a.max_blocks) * a.block_size, most = 0x7fffffff - kTile;
  a.room = static_cast<int>(room < most ? room : most);
  a.block_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (a.block_size == 1 << s) a.block_shift = s;
  const bool wide = a.group > 8;
  if (a.d <= 64) return wide ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  if (a.d <= 128) return wide ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
  return wide ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
}

}  // namespace gbf
