// sample_tokens: the next token of each request from its logits, one given
// uniform number and its sampling parameters.
//
//   w_i = exp((l_i - max l) / T)
//   order: larger logit first, lower index first among equals
//   top-k: the first k;  top-p: of those, each one before which less than
//   top_p of their mass lies;  min-p: of those, w_i >= min_p
//   token: in index order, the first one at which the kept mass passes u times
//   its total.  T = 0: the lowest index of the maximum.
//
// Exactness.  The answer is an integer that jumps where a running sum passes a
// bound, and with 10^5 candidates of 10^-5 each a float32 sum would put one
// row in a hundred on the wrong side.  Weights are therefore 43-bit fixed-point
// integers (2^43 for the largest), computed to 2^-37 or better in pairs of
// float32, and every sum is a 64-bit integer sum: exact, so equal in any order
// and on any number of CTAs.  Float64 would do the same at about a fiftieth of
// the rate on this part.
//
// Work split: a row is one cluster of 1, 2, 4 or 8 CTAs, each with a
// contiguous slice.  The logits are read from HBM once; a slice that fits is
// kept in shared memory for the later passes, a larger one is read again from
// L2.  Top-k and top-p look for the border element of the sorted order without
// sorting: a histogram over 2048 bins of (max - l) / T (counts and masses)
// gives the bin it lies in, the bin's few elements are gathered and ranked by
// comparison, and a bin with too many of them (equal or almost equal logits)
// is cut further by (logit, index) until they are few.  Rows that ask for
// neither skip this.
#include <cooperative_groups.h>

#include "common.cuh"
#include "decode.h"

namespace gbf {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr float kBinsPerOctave = 64.0f;     // 32 octaves; what is smaller shares the last bin
constexpr int kList = 512;                  // candidates ranked by comparison
constexpr int kFix = 43;                    // 2^43: the weight of the largest logit
constexpr int kStageBytes = 72 * 1024;      // largest slice kept in shared memory

typedef unsigned long long u64;

// 2^43 * 2^(j / 64)
__device__ const u64 kPow[64] = {
    0x80000000000ull, 0x8164d1f3bc0ull, 0x82cd8698ac3ull, 0x843a28c3aceull, 0x85aac367cc5ull, 0x871f61969e9ull,
    0x88980e8092eull, 0x8a14d575497ull, 0x8b95c1e3ea9ull, 0x8d1adf5b7e6ull, 0x8ea4398b45dull, 0x9031dc43146ull,
    0x91c3d373ab1ull, 0x935a2b2f13eull, 0x94f4efa8fefull, 0x96942d37202ull, 0x9837f0518dcull, 0x99e0459320bull,
    0x9b8d39b9d55ull, 0x9d3ed9a72d0ull, 0x9ef5326091aull, 0xa0b0510fb97ull, 0xa27043030c5ull, 0xa43515ae09eull,
    0xa5fed6a9b15ull, 0xa7cd93b4e96ull, 0xa9a15ab4ea8ull, 0xab7a39b5a94ull, 0xad583eea42aull, 0xaf3b78ad691ull,
    0xb123f581d2bull, 0xb311c412a91ull, 0xb504f333f9eull, 0xb6fd91e328dull, 0xb8fbaf47630ull, 0xbaff5ab2134ull,
    0xbd08a39f581ull, 0xbf1799b67a7ull, 0xc12c4cca667ull, 0xc346ccda249ull, 0xc5672a11550ull, 0xc78d74c8abcull,
    0xc9b9bd866e3ull, 0xcbec14fef27ull, 0xce248c151f8ull, 0xd06333daef3ull, 0xd2a81d91f13ull, 0xd4f35aabcffull,
    0xd744fccad6aull, 0xd99d15c278bull, 0xdbfbb797dafull, 0xde60f4825e1ull, 0xe0ccdeec2a9ull, 0xe33f8972be9ull,
    0xe5b906e77c8ull, 0xe8396a503c5ull, 0xeac0c6e7dd2ull, 0xed4f301ed99ull, 0xefe4b99bdceull, 0xf281773c5a0ull,
    0xf5257d15248ull, 0xf7d0df730adull, 0xfa83b2db723ull, 0xfd3e0c0cf48ull,
};

// What a row's threads share.  One per CTA; ranks read and write each other's.
struct Shared {
  u64 pow[64];
  unsigned cnt[kBins], lo[kBins], hi[kBins];   // a histogram: counts, masses as low and high words
  unsigned list_key[kList], list_idx[kList];
  u64 list_w[kList];
  u64 warp_mass[kWarps], warp_rank[kWarps];
  unsigned warp_cnt[kWarps];
  u64 best;                                    // this rank's largest (key, ~index)
  u64 range_lo, range_hi;                      // of the searched bin's elements, this rank's
  u64 tot_mass;                                // of this rank's bins, or of its slice
  unsigned tot_cnt;
  unsigned list_n;                             // rank 0's: candidates gathered
  // found by one rank, written to all
  unsigned found_bin, found_cnt, before_cnt;
  u64 before_mass;
  u64 border;                                  // (key, ~index) of the last element kept
  u64 kept_mass;                               // of the elements up to the border
};

// Monotone 32-bit key of a float (larger float, larger key).
GBF_DEVICE unsigned key_of(float x) {
  const unsigned u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
GBF_DEVICE float of_key(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
GBF_DEVICE u64 rank_of(unsigned key, unsigned idx) { return (static_cast<u64>(key) << 32) | (0xffffffffu - idx); }

struct RowScale {
  float top;               // largest logit
  float c_hi, c_lo;        // log2(e) / T
};

// round(2^43 exp((l - top) / T)); relative error below 2^-37 + 2^-43 / w.
// (l - top) / T * log2(e) = ji / 64 + x + xl with |x| < 2^-6.99: 2^(ji / 64) from
// the table, 2^(x + xl) - 1 by its series with the linear term in two parts.
GBF_DEVICE u64 weight(const u64* pow, const RowScale& s, float l) {
  if (l == s.top) return 1ull << kFix;
  const float d = __fsub_rn(l, s.top);
  const float t = __fmul_rn(d, s.c_hi);
  if (!(t > -44.5f)) return 0;                          // below half a unit; also -inf
  const float e = __fsub_rn(d, l);                      // d + d_lo = l - top exactly
  const float d_lo = __fsub_rn(__fsub_rn(l, __fsub_rn(d, e)), __fadd_rn(s.top, e));
  const float t_lo = __fmaf_rn(d_lo, s.c_hi, __fmaf_rn(d, s.c_lo, __fmaf_rn(d, s.c_hi, -t)));
  const float q = __fadd_rn(__fmul_rn(t, 64.0f), 12582912.0f);       // 1.5 * 2^23: rounds to an integer
  const int ji = __float_as_int(q) - 0x4b400000;
  const float g = __fmaf_rn(__fsub_rn(q, 12582912.0f), -1.0f / 64.0f, t);
  const float x = __fadd_rn(g, t_lo), xl = __fsub_rn(t_lo, __fsub_rn(x, g));
  constexpr float kL = 0.693147180559945309f;           // ln 2 = kL + kLl
  constexpr float kLl = static_cast<float>(0.693147180559945309417 - static_cast<double>(kL));
  const float a = __fmul_rn(x, kL);
  float b = __fmaf_rn(xl, kL, __fmaf_rn(x, kLl, __fmaf_rn(x, kL, -a)));
  const float series = __fmaf_rn(x, __fmaf_rn(x, 0.00961812910763f, 0.0555041086648f), 0.240226506959f);
  b = __fmaf_rn(__fmul_rn(x, x), series, b);
  // a + b in units of 2^-38, read off the mantissas after adding 1.5 * 2^23 units (which holds up to 2^22 of
  // them): a (below 2^-7) to 2^-29, then the rest (below 0.97 * 2^-16) to 2^-38
  constexpr float kUa = 12582912.0f / 536870912.0f, kUb = 12582912.0f / 274877906944.0f;
  const float qa = __fadd_rn(a, kUa);
  const float rest = __fadd_rn(__fsub_rn(a, __fsub_rn(qa, kUa)), b);
  const float qb = __fadd_rn(rest, kUb);
  const int ia = __float_as_int(qa) - __float_as_int(kUa);
  const int ib = __float_as_int(qb) - __float_as_int(kUb);
  const long long i = static_cast<long long>(ia * 512 + ib);
  const u64 p = pow[ji & 63];
  const u64 w = p + static_cast<u64>((i * static_cast<long long>(p >> 12)) >> 26);
  const int shift = -(ji >> 6);
  return (w + ((1ull << shift) >> 1)) >> shift;
}

// Bin of a candidate: smaller logits never have a lower bin.
GBF_DEVICE int bin_of(const RowScale& s, float l) {
  if (l == s.top) return 0;
  const float t = __fmul_rn(__fmul_rn(__fsub_rn(s.top, l), s.c_hi), kBinsPerOctave);
  return t < static_cast<float>(kBins - 1) ? static_cast<int>(t) : kBins - 1;
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr unsigned kMinusInf = 0xff80u;
  static GBF_DEVICE void widen(uint4 v, float f[8]) { bf16x8_to_f32(v, f); }
  static GBF_DEVICE unsigned bits(const void* p, int64_t i) { return static_cast<const uint16_t*>(p)[i]; }
};
template <>
struct Elem<float> {
  static constexpr int N = 4;
  static constexpr unsigned kMinusInf = 0xff800000u;
  static GBF_DEVICE void widen(uint4 v, float f[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static GBF_DEVICE unsigned bits(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
};

// A row as aligned 16-byte vectors.  Vector v holds elements v * N - shift ...;
// what lies outside the row reads as -inf, and so does NaN.
template <typename T>
struct Row {
  static constexpr int N = Elem<T>::N;
  const char* base;        // 16-byte aligned
  int shift, vocab, vectors;
  const uint4* staged;     // vectors [v0, ...) in shared memory, or null
  int v0;

  GBF_DEVICE uint4 load(int v) const {
    const int e0 = v * N - shift;
    if (e0 >= 0 && e0 + N <= vocab) return ld_stream(base + static_cast<int64_t>(v) * 16);
    unsigned w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + i;
      const unsigned x = e >= 0 && e < vocab ? Elem<T>::bits(base, static_cast<int64_t>(v) * N + i) : Elem<T>::kMinusInf;
      if (N == 8) w[i >> 1] |= x << (16 * (i & 1));
      else w[i] = x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  GBF_DEVICE void get(int v, float f[N]) const {
    Elem<T>::widen(staged ? staged[v - v0] : load(v), f);
    tidy(f);
  }
  // NaN reads as -inf, -0 as +0 (equal logits have equal keys)
  static GBF_DEVICE void tidy(float f[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f[i] == f[i] ? f[i] + 0.0f : -INFINITY;
  }
};

// shared 64-bit add as two 32-bit ones: the carry shows in the old low word
GBF_DEVICE void add_mass(unsigned* lo, unsigned* hi, u64 w) {
  const unsigned wl = static_cast<unsigned>(w), wh = static_cast<unsigned>(w >> 32);
  const unsigned old = atomicAdd(lo, wl);
  const unsigned up = wh + (old + wl < old ? 1u : 0u);
  if (up) atomicAdd(hi, up);
}

GBF_DEVICE u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
GBF_DEVICE u64 warp_max64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// One row's cluster.
template <typename T>
struct Sampler {
  Shared* sh;
  cg::cluster_group cluster;
  unsigned rank, ranks;
  Row<T> row;
  RowScale scale;
  int v0, v1;              // this rank's vectors
  int tid, lane, warp;

  GBF_DEVICE Shared* of(unsigned r) { return cluster.map_shared_rank(sh, r); }

  GBF_DEVICE void clear_hist() {
    for (int i = tid; i < kBins; i += kThreads) sh->cnt[i] = sh->lo[i] = sh->hi[i] = 0;
  }

  // Sums this rank's share of the bins over all ranks, in order, and finds the
  // bin in which the running count (by_mass false) or mass passes `target`.
  // The total mass comes back in *all.  Three cluster barriers.
  GBF_DEVICE void find_bin(bool by_mass, u64 base_cnt, u64 base_mass, u64 target, double share, u64* all) {
    constexpr int kPer = kBins / kThreads;               // most bins per thread (one rank)
    cluster.sync();                                      // histograms complete
    const int mine = kBins / ranks, first = rank * mine;
    const int per = (mine + kThreads - 1) / kThreads;
    unsigned c = 0, bc[kPer];
    u64 m = 0, bm[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid * per + i;
      bc[i] = 0;
      bm[i] = 0;
      if (i >= per || j >= mine) continue;
      for (unsigned r = 0; r < ranks; ++r) {
        const Shared* o = of(r);
        bc[i] += o->cnt[first + j];
        bm[i] += (static_cast<u64>(o->hi[first + j]) << 32) + o->lo[first + j];
      }
      c += bc[i];
      m += bm[i];
    }
    unsigned ci = c;
    u64 mi = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned cu = __shfl_up_sync(0xffffffffu, ci, o);
      const u64 mu = __shfl_up_sync(0xffffffffu, mi, o);
      if (lane >= o) {
        ci += cu;
        mi += mu;
      }
    }
    if (lane == 31) {
      sh->warp_cnt[warp] = ci;
      sh->warp_mass[warp] = mi;
    }
    __syncthreads();
    unsigned cb = ci - c, tc = 0;
    u64 mb = mi - m, tm = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        cb += sh->warp_cnt[w];
        mb += sh->warp_mass[w];
      }
      tc += sh->warp_cnt[w];
      tm += sh->warp_mass[w];
    }
    if (tid == 0) {
      sh->tot_cnt = tc;
      sh->tot_mass = tm;
    }
    cluster.sync();                                      // totals of all ranks
    u64 total = 0;
    u64 cnt0 = base_cnt + cb, mass0 = base_mass + mb;
    for (unsigned r = 0; r < ranks; ++r) {
      const Shared* o = of(r);
      if (r < rank) {
        cnt0 += o->tot_cnt;
        mass0 += o->tot_mass;
      }
      total += o->tot_mass;
    }
    *all = total;
    if (share >= 0.0) {                                  // the target is a share of the total
      const double x = ceil(share * static_cast<double>(total));
      target = x < 1.0 ? 1ull : static_cast<u64>(x);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const u64 at = by_mass ? mass0 : cnt0;
      const u64 by = by_mass ? bm[i] : static_cast<u64>(bc[i]);
      if (by > 0 && at < target && at + by >= target) {  // one thread of the cluster, if any
        for (unsigned r = 0; r < ranks; ++r) {
          Shared* o = of(r);
          o->found_bin = first + tid * per + i;
          o->found_cnt = bc[i];
          o->before_cnt = static_cast<unsigned>(cnt0);
          o->before_mass = mass0;
        }
      }
      cnt0 += bc[i];
      mass0 += bm[i];
    }
    cluster.sync();                                      // the finding
  }

  // Border of the order's shortest prefix that holds `target` elements (or
  // that mass, or that share of the mass): sh->border and sh->kept_mass of all
  // ranks.  The first histogram is in place; true when it was overwritten.
  GBF_DEVICE bool select(bool by_mass, bool masses, u64 target, double share) {
    u64 total;
    if (tid == 0) sh->found_cnt = 0;
    find_bin(by_mass, 0, 0, target, share, &total);
    if (share >= 0.0) {
      const double x = ceil(share * static_cast<double>(total));
      target = x < 1.0 ? 1ull : static_cast<u64>(x);
    }
    unsigned n = sh->found_cnt;
    if (n == 0) {                                        // fewer than `target`: nothing is cut off
      if (tid == 0) {
        sh->border = 0;
        sh->kept_mass = total;
      }
      __syncthreads();
      return false;
    }
    const int bin = static_cast<int>(sh->found_bin);
    u64 lo = 0, hi = ~0ull;                              // ranks searched, once known
    bool by_range = false;
    if (n > kList) {
      // the bin's range of ranks
      u64 mn = ~0ull, mx = 0;
      for (int v = v0 + tid; v < v1; v += kThreads) {
        float f[Row<T>::N];
        row.get(v, f);
#pragma unroll
        for (int i = 0; i < Row<T>::N; ++i)
          if (f[i] != -INFINITY && bin_of(scale, f[i]) == bin) {
            const u64 k = rank_of(key_of(f[i]), v * Row<T>::N - row.shift + i);
            mn = k < mn ? k : mn;
            mx = k > mx ? k : mx;
          }
      }
      mn = ~warp_max64(~mn);
      mx = warp_max64(mx);
      if (lane == 0) {
        sh->warp_mass[warp] = mx;
        sh->warp_rank[warp] = mn;
      }
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) {
          mx = sh->warp_mass[w] > mx ? sh->warp_mass[w] : mx;
          mn = sh->warp_rank[w] < mn ? sh->warp_rank[w] : mn;
        }
        sh->range_lo = mn;
        sh->range_hi = mx;
      }
      cluster.sync();
      lo = ~0ull;
      hi = 0;
      for (unsigned r = 0; r < ranks; ++r) {
        const Shared* o = of(r);
        lo = o->range_lo < lo ? o->range_lo : lo;
        hi = o->range_hi > hi ? o->range_hi : hi;
      }
      by_range = true;
      for (int level = 0; n > kList && level < 8; ++level) {   // 11 of 64 bits each
        int s = 0;
        while (((hi - lo) >> s) >= kBins) ++s;
        const u64 before_cnt = sh->before_cnt, before_mass = sh->before_mass;
        cluster.sync();                                  // every rank is done with the last histogram and finding
        clear_hist();
        __syncthreads();
        for (int v = v0 + tid; v < v1; v += kThreads) {
          float f[Row<T>::N];
          row.get(v, f);
#pragma unroll
          for (int i = 0; i < Row<T>::N; ++i) {
            const u64 k = rank_of(key_of(f[i]), v * Row<T>::N - row.shift + i);
            if (f[i] == -INFINITY || k < lo || k > hi) continue;
            const int j = static_cast<int>((hi - k) >> s);
            atomicAdd(&sh->cnt[j], 1u);
            if (masses) add_mass(&sh->lo[j], &sh->hi[j], weight(sh->pow, scale, f[i]));
          }
        }
        u64 unused;
        find_bin(by_mass, before_cnt, before_mass, target, -1.0, &unused);
        n = sh->found_cnt;
        const u64 j = sh->found_bin;
        const u64 new_hi = hi - (j << s), span = (1ull << s) - 1;
        lo = new_hi - lo > span ? new_hi - span : lo;
        hi = new_hi;
      }
    }
    // gather the candidates on rank 0 and rank them by comparison
    const u64 before_cnt = sh->before_cnt, before_mass = sh->before_mass;
    Shared* head = of(0);
    if (rank == 0 && tid == 0) sh->list_n = 0;
    cluster.sync();
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float f[Row<T>::N];
      row.get(v, f);
#pragma unroll
      for (int i = 0; i < Row<T>::N; ++i) {
        if (f[i] == -INFINITY) continue;
        const unsigned key = key_of(f[i]), idx = v * Row<T>::N - row.shift + i;
        const u64 k = rank_of(key, idx);
        if (by_range ? (k < lo || k > hi) : bin_of(scale, f[i]) != bin) continue;
        const unsigned at = atomicAdd(&head->list_n, 1u);
        if (at < kList) {
          head->list_key[at] = key;
          head->list_idx[at] = idx;
          head->list_w[at] = weight(sh->pow, scale, f[i]);
        }
      }
    }
    cluster.sync();
    if (rank == 0) {
      const int found = static_cast<int>(sh->list_n < kList ? sh->list_n : kList);
      u64 last = ~0ull, mass = 0;
      for (int i = tid; i < found; i += kThreads) {
        const u64 k = rank_of(sh->list_key[i], sh->list_idx[i]);
        u64 cnt = before_cnt, w = before_mass;
        for (int j = 0; j < found; ++j)
          if (rank_of(sh->list_key[j], sh->list_idx[j]) > k) {
            ++cnt;
            w += sh->list_w[j];
          }
        if ((by_mass ? w : cnt) < target) {              // kept
          last = k < last ? k : last;
          mass += sh->list_w[i];
        }
      }
      last = ~warp_max64(~last);
      mass = warp_sum64(mass);
      __syncthreads();
      if (lane == 0) {
        sh->warp_mass[warp] = mass;
        sh->warp_rank[warp] = last;
      }
      __syncthreads();
      if (tid == 0) {
        mass = before_mass;
        last = ~0ull;
        for (int w = 0; w < kWarps; ++w) {
          mass += sh->warp_mass[w];
          last = sh->warp_rank[w] < last ? sh->warp_rank[w] : last;
        }
        for (unsigned r = 0; r < ranks; ++r) {
          of(r)->border = last;
          of(r)->kept_mass = mass;
        }
      }
    }
    cluster.sync();
    return by_range;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int staged) {
  constexpr int N = Elem<T>::N;
  extern __shared__ __align__(16) unsigned char dyn[];
  Sampler<T> s{reinterpret_cast<Shared*>(dyn), cg::this_cluster()};
  Shared* sh = s.sh;
  s.rank = s.cluster.block_rank();
  s.ranks = s.cluster.num_blocks();
  const int tid = s.tid = threadIdx.x, lane = s.lane = tid & 31, warp = s.warp = tid >> 5;
  for (int i = tid; i < 64; i += kThreads) sh->pow[i] = kPow[i];
  s.clear_hist();
  pdl_wait();
  pdl_launch_dependents();

  const int64_t b = blockIdx.x / s.ranks;
  const char* at = static_cast<const char*>(a.logits) + b * a.stride * static_cast<int64_t>(sizeof(T));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
  s.row.base = at - off;
  s.row.shift = off / static_cast<int>(sizeof(T));
  s.row.vocab = a.vocab;
  s.row.vectors = (s.row.shift + a.vocab + N - 1) / N;
  s.row.staged = nullptr;
  const int per = (s.row.vectors + s.ranks - 1) / s.ranks;
  const int v0 = s.v0 = min(static_cast<int>(s.rank) * per, s.row.vectors);
  const int v1 = s.v1 = min(v0 + per, s.row.vectors);
  s.row.v0 = v0;

  // pass 1: the only read of HBM; the largest logit and its lowest index
  uint4* stage = reinterpret_cast<uint4*>(dyn + sizeof(Shared));
  float best = -INFINITY;
  unsigned best_i = 0;
  auto look = [&](int v, uint4 raw) {
    if (staged) stage[v - v0] = raw;
    float f[N];
    Elem<T>::widen(raw, f);
    Row<T>::tidy(f);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (f[i] > best) {
        best = f[i];
        best_i = v * N - s.row.shift + i;
      }
  };
  int v = v0 + tid;
  for (; v + 3 * kThreads < v1; v += 4 * kThreads) {
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = s.row.load(v + u * kThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u) look(v + u * kThreads, raw[u]);
  }
  for (; v < v1; v += kThreads) look(v, s.row.load(v));
  u64 top = best == -INFINITY ? 0 : rank_of(key_of(best), best_i);
  top = warp_max64(top);
  if (lane == 0) sh->warp_mass[warp] = top;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) top = sh->warp_mass[w] > top ? sh->warp_mass[w] : top;
    sh->best = top;
  }
  s.cluster.sync();
  if (staged) s.row.staged = stage;
  top = 0;
  for (unsigned r = 0; r < s.ranks; ++r) {
    const u64 o = s.of(r)->best;
    top = o > top ? o : top;
  }

  const float temp = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.0f;
  const float mp = a.min_p ? a.min_p[b] : 0.0f;
  const float u = a.uniform[b];
  const bool bad = !(temp >= 0.0f && temp < INFINITY) || !(p == p) || !(mp <= 1.0f) || !(u >= 0.0f && u < 1.0f);
  if (bad || top == 0 || temp == 0.0f) {
    if (s.rank == 0 && tid == 0) {
      const bool none = bad || top == 0;
      if (none) raise_error(a.err, DEV_ERR_SAMPLING);
      a.tokens[b] = none ? -1 : static_cast<int32_t>(0xffffffffu - static_cast<unsigned>(top));
      if (a.logprob) a.logprob[b] = none ? __uint_as_float(0x7fc00000u) : 0.0f;
    }
    s.cluster.sync();                                    // no rank leaves while others read its memory
    return;
  }
  s.scale.top = of_key(static_cast<unsigned>(top >> 32));
  {
    const double c = 1.4426950408889634 / static_cast<double>(temp);
    s.scale.c_hi = c < 3.0e38 ? static_cast<float>(c) : 3.0e38f;
    s.scale.c_lo = c < 3.0e38 ? static_cast<float>(c - static_cast<double>(s.scale.c_hi)) : 0.0f;
  }

  // top-k and top-p: the border of the kept prefix
  const bool by_k = k > 0 && k < a.vocab, by_p = p < 1.0f;
  u64 border = 0;
  if (by_k || by_p) {
    auto histogram = [&]() {
      for (int i = v0 + tid; i < v1; i += kThreads) {
        float f[N];
        s.row.get(i, f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (f[e] == -INFINITY) continue;
          const int j = bin_of(s.scale, f[e]);
          atomicAdd(&sh->cnt[j], 1u);
          if (by_p)
            add_mass(&sh->lo[j], &sh->hi[j], weight(sh->pow, s.scale, f[e]));
        }
      }
    };
    histogram();
    bool again = false;
    if (by_k) {
      again = s.select(false, by_p, static_cast<u64>(k), -1.0);
      border = sh->border;
    }
    if (by_p) {
      double share = p > 0.0f ? static_cast<double>(p) : 0.0;
      u64 target = 0;
      if (by_k) {                                        // a share of what top-k kept
        const double x = ceil(share * static_cast<double>(sh->kept_mass));
        target = x < 1.0 ? 1ull : static_cast<u64>(x);
        share = -1.0;
        s.cluster.sync();                                // every rank has read its kept mass
        if (again) {
          s.clear_hist();
          __syncthreads();
          histogram();
        }
      }
      s.select(true, true, target, share);
      border = sh->border > border ? sh->border : border;
    }
  }
  const u64 least = mp > 0.0f ? static_cast<u64>(ceil(static_cast<double>(mp) * static_cast<double>(1ull << kFix))) : 0;

  // the kept mass in index order: a contiguous run of vectors per warp
  auto kept = [&](float f, unsigned idx) -> u64 {
    if (f == -INFINITY || rank_of(key_of(f), idx) < border) return 0;
    const u64 w = weight(sh->pow, s.scale, f);
    return w >= least ? w : 0;
  };
  const int run = (v1 - v0 + kWarps - 1) / kWarps;
  const int w0 = min(v0 + warp * run, v1), w1 = min(w0 + run, v1);
  auto lane_mass = [&](int i) {
    u64 m = 0;
    if (i < w1) {
      float f[N];
      s.row.get(i, f);
#pragma unroll
      for (int e = 0; e < N; ++e) m += kept(f[e], i * N - s.row.shift + e);
    }
    return m;
  };
  u64 mass = 0;
  for (int i = w0 + lane; i < w1; i += 32) mass += lane_mass(i);
  mass = warp_sum64(mass);
  __syncthreads();
  if (lane == 0) sh->warp_mass[warp] = mass;
  __syncthreads();
  u64 before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh->warp_mass[w];
    total += sh->warp_mass[w];
  }
  if (tid == 0) sh->tot_mass = total;
  s.cluster.sync();
  total = 0;
  for (unsigned r = 0; r < s.ranks; ++r) {
    const u64 o = s.of(r)->tot_mass;
    if (r < s.rank) before += o;
    total += o;
  }
  u64 target = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
  if (target >= total) target = total - 1;
  if (before <= target && target < before + mass) {      // one warp of the cluster
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const u64 mine = lane_mass(i0 + lane);
      u64 incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          u64 run_mass = before + incl - mine;
          float f[N];
          s.row.get(i0 + lane, f);
          bool done = false;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const unsigned idx = (i0 + lane) * N - s.row.shift + e;
            run_mass += kept(f[e], idx);
            if (!done && run_mass > target) {
              done = true;
              a.tokens[b] = static_cast<int32_t>(idx);
              if (a.logprob) {
                // ln(w / total) = (l - top) / T - ln(total / 2^43), both terms of one sign
                const float d = f[e] == s.scale.top ? 0.0f : (f[e] - s.scale.top) / temp;
                const u64 more = total - (1ull << kFix);
                a.logprob[b] = d - log1pf(static_cast<float>(more) * (1.0f / static_cast<float>(1ull << kFix)));
              }
            }
          }
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  s.cluster.sync();                                      // no rank leaves while others read its memory
}

template <typename T>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  constexpr int N = Elem<T>::N;
  const int64_t vectors = (static_cast<int64_t>(a.vocab) + N - 1) / N + 1;
  int ranks = 8;
  const int64_t slice = (vectors + ranks - 1) / ranks * 16;
  const int staged = slice <= kStageBytes ? 1 : 0;
  const size_t smem = sizeof(Shared) + (staged ? static_cast<size_t>(slice) : 0);
  const cudaError_t e = allow_smem<sample_kernel<T>>(static_cast<int>(sizeof(Shared)) + kStageBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, staged);
}

}  // namespace

cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t stream) {
  return a.f32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace gbf
