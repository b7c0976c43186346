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
// integers (2^43 for the largest), computed to 2^-36 or better in pairs of
// float32, and every sum is a 64-bit integer sum: exact, so equal in any order
// and on any number of CTAs.  Float64 would do the same at about a fiftieth of
// the rate on this part.
//
// Work split: a row is one cluster of 1, 2, 4 or 8 CTAs, each with a
// contiguous slice, and within it each warp with a contiguous run.  The logits
// are read from HBM once; a slice that fits is kept in shared memory for the
// later passes, a larger one is read again from L2.
//
// The border of top-k and top-p in the sorted order is found without sorting:
//   1. a histogram of counts over 4096 bins of (max - l) / T, 1/128 octave of
//      weight each (one shared atomic per element);
//   2. top-k: the bin the k-th element lies in.  Top-p: the histogram also sums
//      the elements' places in their bins, which gives each bin's mass to 50
//      ppm and so the few bins the border can lie in; one pass over the weights
//      then gives the total, the mass above those bins, and the masses within
//      them;
//   3. the few elements around the border (of a bin, or of 64ths of bins) are
//      gathered on every CTA of the cluster and sorted there; where they are too
//      many (thousands of equal or almost equal logits) they are first cut by
//      (logit, index).
// The pass of step 2 also sums each warp's run of the kept elements above the
// border's bins, so the draw only adds the few within them.  A row that asks for
// neither top-k nor top-p takes that pass alone.
//
// A row whose top-k border lies among its first 1024 elements is simpler: they
// are gathered on one CTA and sorted, and all the rest is done on that list.
// For a short top-k there is no histogram either: pass 1 gives the largest
// logits of as many disjoint groups of lanes as top-k keeps elements or more, and
// the smallest of those is a lower bound of the k-th largest logit.  With n
// groups it leaves about n ln n elements, in whatever order the logits come.
//
// The exact weight is the dear part (some 45 integer instructions, which run at
// half rate), so a row is first done in float32 with an error bound: the weight
// to 2^-32 in two float32 parts, summed as integers, and every decision checked
// against twice that bound.  A row in which all decisions clear it is done; the
// others (one in 500 of 128000 candidates with top_p up to 0.99, one in 4000 of
// 50257 without) are done again exactly.
//
// What bounds it: instructions and barriers, not HBM.  A nucleus row issues 107
// instructions per 32 elements (9 for pass 1, some 12 for the histogram, 55 for the
// weights, the rest for the border and the draw) at 2.5 a cycle and SM, and a
// cluster passes five barriers with an exchange behind each, 1 to 2 us apiece.
// Measured (device time, back to back): one row of 32000 bf16, nucleus, 17.7 us (temperature alone 8.0);
// 32 rows of 151936, mixed requests, 36.6 us (10 MB: 0.26 TB/s); 61 rows of 50257,
// temperature alone, 15.1 us; 256 rows of 128000 float32, nucleus, 177 us (131 MB:
// 0.74 TB/s).
//
// Ranks hand each other totals by remote stores into boxes (read locally behind
// the next barrier).
#include <cfloat>

#include <cooperative_groups.h>

#include "common.cuh"
#include "decode.h"
#include "tma.cuh"

namespace gbf {
namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 4096;
constexpr float kBinsPerOctave = 128.0f;    // 32 octaves; what is smaller shares the last bin
constexpr int kCells = kBins / 2;           // mass histogram in the same memory: low words, then high words
// With top-p alone an element adds 2^20 and its place in the bin, so that a bin's mass is known to 50 ppm: 42.3 for half a
// place (2^(1/16384)), 3.7 for the weight taken as linear within the bin, 4 for the places' own rounding (3 2^-24 of up to
// 2^18).  Behind that come the exponential (0.24 ppm), the products (0.24), 26 float32 additions on the way to a running
// sum (1.6) and the target's products (0.2): 52.3 in all, taken as 60.  It holds as long as no more than 4095 elements of
// a CTA fall in a bin (otherwise the border turns out to lie outside the bins searched, and all are).  Those of the last bin (weights below 2^-31.9) add vocab 2^-31.9 of the total at most.
constexpr float kBinError = 60e-6f, kLastBinError = 2.6e-10f;
constexpr int kList = 1024;                 // candidates that are sorted, an equal share of each rank's
constexpr int kGroup = 64;                  // bins per group (and groups): the two steps of a search over the bins
constexpr int kFew = 128;                   // up to this many are compared with each other
constexpr int kNear = 2048;                 // this rank's elements in the bins that may hold top-p's border
constexpr int kSpans = 32;                  // parts that the bins that may hold top-p's border are cut into
constexpr int kFix = 43;                    // 2^43: the weight of the largest logit
constexpr int kStageBytes = 66 * 1024;      // largest slice kept in shared memory
constexpr float kLeastTemperature = 1e-30f;

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
struct __align__(16) Shared {
  unsigned hist[kBins];
  u64 pow[64];
  float2 sixteenth[16];        // 2^(j / 16) in float32, and the rest of it relative to that
  u64 list[kList];             // candidates of every rank, as (key, ~index)
  union {
    struct {
      float group[8][kGroup];  // every rank's sums of the groups of bins,
      float bin[2][8][kGroup]; // and of the bins of a group, for two targets
    } search;
    u64 near[kNear];           // this rank's elements in the bins that may hold top-p's border
  };
  u64 span[8][kSpans];         // every rank's masses of the spans
  unsigned span_lo[kSpans], span_hi[kSpans];     // this rank's, being summed
  unsigned run_lo[kWarps], run_hi[kWarps];       // kept mass of each warp's run
  u64 warp_a[kWarps], warp_b[kWarps];
  u64 box[2][2][8];            // totals of the ranks: two boxes in turn, two values each
  unsigned list_n[8];          // how many every rank has
  unsigned mine_n, near_n;     // this rank's candidates, and elements near the border
  unsigned doubt;              // a float32 decision of this rank that did not clear its bound
  // found by one thread of the cluster, written to all ranks
  int found;
  u64 before;
};

// The CTA's shared memory: what its threads share, then its slice of the row.
// (Taken from the array at each use, so that accesses stay shared-memory ones;
// through a pointer kept in an object they would become generic.)
extern __shared__ __align__(16) unsigned char sample_smem[];
GBF_DEVICE Shared* mem() { return reinterpret_cast<Shared*>(sample_smem); }
GBF_DEVICE uint4* stage() { return reinterpret_cast<uint4*>(sample_smem + sizeof(Shared)); }

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
  float c_place;           // places (64ths of a bin) per unit of logit, and about its inverse
  float c_inverse;
  float cut;               // 60 octaves below the top
  unsigned n_top;          // exponent field of 2^N, see quick_weight
};

GBF_DEVICE float2 two(float x) { return make_float2(x, x); }
// b - a
GBF_DEVICE float2 sub2(float2 b, float2 a) { return __ffma2_rn(a, two(-1.0f), b); }

// From the table index ji, and the fraction's parts in the mantissas of qa and qb: the weight.
constexpr float kWa = 12582912.0f / 536870912.0f, kWb = 12582912.0f / 274877906944.0f;   // 1.5 * 2^23 units
GBF_DEVICE u64 assemble(const u64* pow, float nt, float q, float qa, float qb) {
  const int ji = __float_as_int(q) - 0x4b400000;
  const int i = (__float_as_int(qa) - __float_as_int(kWa)) * 512 + (__float_as_int(qb) - __float_as_int(kWb));
  const u64 p = pow[ji & 63];
  const long long part = static_cast<long long>(i) * static_cast<int>(p >> 13);
  const u64 w = p * 2 + static_cast<u64>(part >> 24);               // twice the weight, before the octave
  const u64 scaled = ((w >> (-(ji >> 6) & 63)) + 1) >> 1;
  return nt < 44.5f ? scaled : 0;                                   // below half a unit (and -inf): zero
}

// round(2^43 exp((l - top) / T)) of two logits; relative error below 2^-36, and half a unit.
// (l - top) / T * log2(e) = ji / 64 + x + xl with |x| < 2^-6.99: 2^(ji / 64) from
// the table, 2^(x + xl) - 1 by its series with the linear term in two parts.
GBF_DEVICE void weights(const u64* pow, const RowScale& s, float2 l, u64* w0, u64* w1) {
  const float2 one = two(1.0f);
  const float2 d = __fadd2_rn(l, two(-s.top));
  const float2 e = sub2(d, l);                                      // d + d_lo = l - top exactly
  const float2 d_lo = sub2(sub2(l, sub2(d, e)), __fadd2_rn(e, two(s.top)));
  const float2 nt = __fmul2_rn(d, two(-s.c_hi));                    // -t, t = d c_hi rounded
  float2 lo = __ffma2_rn(d, two(s.c_hi), nt);                       // what t lacks
  lo = __ffma2_rn(d, two(s.c_lo), lo);
  lo = __ffma2_rn(d_lo, two(s.c_hi), lo);
  const float2 q = __ffma2_rn(nt, two(-64.0f), two(12582912.0f));   // 1.5 * 2^23: rounds to an integer
  const float2 ng = __ffma2_rn(__fadd2_rn(q, two(-12582912.0f)), two(1.0f / 64.0f), nt);    // ji / 64 - t
  const float2 x = sub2(lo, ng);
  const float2 xl = sub2(lo, __fadd2_rn(x, ng));
  constexpr float kL = 0.693147180559945309f;                       // ln 2 = kL + kLl
  constexpr float kLl = static_cast<float>(0.693147180559945309417 - static_cast<double>(kL));
  const float2 na = __fmul2_rn(x, two(-kL));                        // -a, a = x kL rounded
  float2 b = __ffma2_rn(x, two(kL), na);
  b = __ffma2_rn(x, two(kLl), b);
  b = __ffma2_rn(xl, two(kL), b);
  float2 series = __ffma2_rn(x, two(0.00961812910763f), two(0.0555041086648f));
  series = __ffma2_rn(x, series, two(0.240226506959f));
  b = __ffma2_rn(__fmul2_rn(x, x), series, b);
  // a + b in units of 2^-38, read off the mantissas after adding 1.5 * 2^23 units (which holds up to 2^22 of
  // them): a (below 2^-7) to 2^-29, then the rest (below 0.97 * 2^-16) to 2^-38
  const float2 qa = sub2(two(kWa), na);
  const float2 rest = sub2(b, __fadd2_rn(na, __ffma2_rn(two(-kWa), one, qa)));
  const float2 qb = __fadd2_rn(rest, two(kWb));
  *w0 = assemble(pow, nt.x, q.x, qa.x, qb.x);
  *w1 = assemble(pow, nt.y, q.y, qa.y, qb.y);
}

// The float32 pass's weight: exp(l / T) over 2^N, in float32 hi + lo within 2^-32 (2^-33 seen over 10^7 logits), N as for
// the largest logit (scale.n_top), whose weight lies in [1/2, 1.03).  The argument l / T log2(e) = m + x + xl with m a
// multiple of 1/16, which a rounding addition leaves in the low bits of q; |x| <= 2^-5, exactly; 2^m from the table and an
// exponent, 2^(x + xl) - 1 = y + yl by a polynomial (minimax, 2^-36).  Logits more than 60 octaves below the top, -inf and
// NaN are taken as those there: 2^-60 each is lost in any sum.  For rows with |top| / T log2(e) < 2^14 (xl's own rounding:
// 2^-34).  Scalar instructions, whose constants and signs cost nothing: in pairs, half of what was issued were moves.
constexpr float kMagic = 786432.0f;         // 1.5 * 2^19: a float of 1/16 ulp
constexpr float kQuickRange = 16384.0f, kQuickHeat = 1e30f;
struct Quick {
  float w, lo;
};
GBF_DEVICE Quick quick_weight(unsigned table, const RowScale& s, float l) {
  l = fmaxf(l, s.cut);
  const float p = __fmul_rn(l, s.c_hi), q = __fadd_rn(p, kMagic);
  const float x0 = __fsub_rn(p, __fsub_rn(q, kMagic));              // exact
  float xl = __fmaf_rn(l, s.c_lo, __fmaf_rn(l, s.c_hi, -p));
  const float x = __fadd_rn(x0, xl);
  xl = __fsub_rn(xl, __fsub_rn(x, x0));
  constexpr float kL = 0.693147180559945309f;                       // ln 2 to 2^-28, times x: 2^-33
  const float r = __fmaf_rn(x, __fmaf_rn(x, 0.00961828f, 0.05550509f), 0.2402265f);
  const float b = __fmaf_rn(__fmul_rn(x, x), r, __fmul_rn(xl, kL));
  const float y = __fmaf_rn(x, kL, b);
  float yl = __fadd_rn(__fmaf_rn(x, kL, -y), b);
  float hi, rel;                                                    // 2^(j / 16), and what that lacks of itself
  asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(hi), "=f"(rel) : "r"(table + ((__float_as_uint(q) & 15u) << 3)));
  hi = __uint_as_float(__float_as_uint(hi) + ((__float_as_uint(q) << 19) & 0xff800000u) - s.n_top);
  yl = __fmaf_rn(rel, y, __fadd_rn(yl, rel));
  const float w = __fmaf_rn(hi, y, hi);
  return {w, __fmaf_rn(hi, yl, __fmaf_rn(hi, y, __fsub_rn(hi, w)))};
}

// Sums of such weights in integers: what 2 + w holds of w, in units of 2^-22, and the rest with lo to 2^-44.6, in units
// of 2^-44 (at most 2^21.9 of them a weight, and 520 weights a thread: a slice has at most 2^18 elements).
constexpr float kUa = 2.0f, kUb = 12582912.0f / 17592186044416.0f;  // 1.5 * 2^23 units
struct Sum {
  unsigned a;
  int b;
  GBF_DEVICE void add(const Sum& o) {
    a += o.a;
    b += o.b;
  }
  GBF_DEVICE u64 fixed() const {                                    // in units of 2^-kFix
    static_assert(kFix == 43, "");
    return (static_cast<u64>(a) << 21) + static_cast<u64>(static_cast<long long>(b >> 1));
  }
};
GBF_DEVICE Sum parts_of(const Quick& q) {
  const float a = __fadd_rn(q.w, kUa);
  const float b = __fadd_rn(__fadd_rn(__fsub_rn(q.w, __fsub_rn(a, kUa)), q.lo), kUb);
  return {__float_as_uint(a) - __float_as_uint(kUa), __float_as_int(b) - __float_as_int(kUb)};
}

// What a float32 sum of masses and a share of another may be apart by: twice 2^-32 of them; the weights' last places
// (2^-45 and a quarter of it each, which is 0.32 units of 2^-43, in both); one unit for each thread's two sums and each
// element near the border.
GBF_DEVICE u64 slack_of(u64 total, int vocab, unsigned ranks) {
  return (total >> 31) + (vocab - (vocab >> 3)) + ranks * (2 * kThreads + kNear);
}

// ln(w / total) = (l - top) / T - ln(total / the top's weight), both terms of one sign.
GBF_DEVICE float log_share(const RowScale& s, float l, float heat, u64 total, u64 of_top) {
  const float d = l == s.top ? 0.0f : (l - s.top) / heat;
  const u64 more = total > of_top ? total - of_top : 0;
  return d - log1pf(static_cast<float>(more) / static_cast<float>(of_top));
}

// Place of a candidate in 64ths of a bin, half a bin ahead: its bin, and 0..63 within it.  Smaller logits never have a
// lower place.
GBF_DEVICE int place_of(const RowScale& s, float l) {
  const float t = fminf(__fmul_rn(__fsub_rn(s.top, l), s.c_place), 64.0f * (kBins - 1) + 31.0f);
  return __float_as_int(__fadd_rn(t, 12582912.0f)) - (0x4b400000 - 32);
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr unsigned kMinusInf = 0xff80u;
  static GBF_DEVICE void widen(uint4 v, float f[8]) { bf16x8_to_f32(v, f); }
  static GBF_DEVICE uint4 pack(const float f[8]) { return f32x8_to_bf16x8(f); }
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
  static GBF_DEVICE uint4 pack(const float f[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static GBF_DEVICE unsigned bits(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
};

// NaN reads as -inf, -0 as +0 (equal logits have equal keys).
template <int N>
GBF_DEVICE void tidy(float f[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = fmaxf(f[i] + 0.0f, -INFINITY);
}

// A row as aligned 16-byte vectors of N elements, the first `shift` elements of
// which lie before it; what lies outside the row reads as -inf.  Passes behind
// the first one read pairs: pair j holds elements 2 j - shift and the next.
// STAGED: this rank's vectors v0 ... are in shared memory, tidied.
template <typename T, bool STAGED>
struct Row {
  static constexpr int N = Elem<T>::N;
  const char* base;        // 16-byte aligned
  int shift, vocab;
  int v0;
  int full0, full;         // the vectors that lie within the row: the first, and how many

  GBF_DEVICE uint4 load(int v) const {
    const int e0 = v * N - shift;
    if (static_cast<unsigned>(v - full0) < static_cast<unsigned>(full)) return ld_stream(base + static_cast<unsigned>(v) * 16u);
    unsigned w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned x = element(e0 + i);
      if (N == 8) w[i >> 1] |= x << (16 * (i & 1));
      else w[i] = x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  GBF_DEVICE unsigned element(int e) const {
    return e >= 0 && e < vocab ? Elem<T>::bits(base, static_cast<int64_t>(e) + shift) : Elem<T>::kMinusInf;
  }
  GBF_DEVICE float2 pair(int j) const {
    const int e = 2 * j - shift;
    float f[2];
    if (N == 8) {
      const unsigned w = STAGED ? reinterpret_cast<const unsigned*>(stage())[j - v0 * 4]
                                : e >= 0 && e + 1 < vocab ? reinterpret_cast<const unsigned*>(base)[j]
                                                          : element(e) | element(e + 1) << 16;
      f[0] = __uint_as_float(w << 16);
      f[1] = __uint_as_float(w & 0xffff0000u);
    } else {
      const uint2 w = STAGED ? reinterpret_cast<const uint2*>(stage())[j - v0 * 2]
                             : e >= 0 && e + 1 < vocab ? reinterpret_cast<const uint2*>(base)[j]
                                                       : make_uint2(element(e), element(e + 1));
      f[0] = __uint_as_float(w.x);
      f[1] = __uint_as_float(w.y);
    }
    if (!STAGED) tidy<2>(f);
    return make_float2(f[0], f[1]);
  }
  GBF_DEVICE uint4 raw(int v) const { return STAGED ? stage()[v - v0] : load(v); }
  GBF_DEVICE void get(int v, float f[N]) const {
    Elem<T>::widen(raw(v), f);
    if (!STAGED) tidy<N>(f);
  }
  // f(v, elements) for v = from, from + step, ... below end; each vector is loaded a turn ahead.  The elements as they
  // are (NaN, -0).
  template <typename F>
  GBF_DEVICE void each(int from, int end, int step, F f) const {
    if (from >= end) return;
    uint4 next = raw(from);
#pragma unroll 1
    for (int v = from; v < end; v += step) {
      float x[N];
      Elem<T>::widen(next, x);
      if (v + step < end) next = raw(v + step);
      f(v, x);
    }
  }
};

GBF_DEVICE float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// shared 64-bit add as two 32-bit ones: the carry shows in the old low word
GBF_DEVICE void add_mass(unsigned* lo, unsigned* hi, u64 w) {
  const unsigned wl = static_cast<unsigned>(w), wh = static_cast<unsigned>(w >> 32);
  const unsigned old = atomicAdd(lo, wl);
  const unsigned up = wh + (old + wl < old ? 1u : 0u);
  if (up) atomicAdd(hi, up);
}
GBF_DEVICE u64 mass_of(unsigned lo, unsigned hi) { return (static_cast<u64>(hi) << 32) + lo; }

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
GBF_DEVICE u64 warp_scan64(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// floor(x 2^64) for 0 <= x < 1: a 64-bit fraction, exact from 2^-40 on.  (Products of masses and float32 shares are
// taken in integers; a float64 instruction would cost a block of 512 threads some 250 cycles.)
GBF_DEVICE u64 fraction_of(float x) { return __float2ull_rz(x * 18446744073709551616.0f); }
// ceil(share * total), at least 1
GBF_DEVICE u64 share_of(float share, u64 total) {
  if (!(share > 0.0f)) return 1;
  if (share >= 1.0f) return ~0ull;
  const u64 f = fraction_of(share), hi = __umul64hi(f, total) + (f * total != 0 ? 1 : 0);
  return hi > 0 ? hi : 1;
}

// One row's cluster.
template <typename T, bool STAGED>
struct Sampler {
  cg::cluster_group cluster;
  unsigned rank, ranks;
  Row<T, STAGED> row;
  RowScale scale;
  int v0, v1, j0, j1;      // this rank's vectors, and pairs
  int tid, lane, warp;
  int turn;                // box of the next exchange

  GBF_DEVICE Shared* of(unsigned r) { return cluster.map_shared_rank(mem(), r); }

  GBF_DEVICE void clear() {
    for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(mem()->hist)[i] = make_uint4(0, 0, 0, 0);
  }
  GBF_DEVICE void weigh(float2 l, u64* w0, u64* w1) {
    weights(mem()->pow, scale, l, w0, w1);
    if (scale.top == INFINITY) {                         // the infinite logits share all of the mass
      *w0 = l.x == INFINITY ? 1ull << kFix : 0;
      *w1 = l.y == INFINITY ? 1ull << kFix : 0;
    }
  }
  // a logit below those of all places up to place - 64
  GBF_DEVICE float logit_of(int place) {
    return scale.top == INFINITY ? -FLT_MAX : fmaxf(scale.top - place * scale.c_inverse, -FLT_MAX);
  }
  GBF_DEVICE int place(float l) {
    return scale.top == INFINITY ? (l == INFINITY ? 32 : 64 * kBins - 1) : place_of(scale, l);
  }

  // Sums over the block of every thread's a and b, the same in all threads.
  GBF_DEVICE void block_sum(u64* a, u64* b) {
    const u64 wa = warp_sum64(*a), wb = warp_sum64(*b);
    __syncthreads();
    if (lane == 0) {
      mem()->warp_a[warp] = wa;
      mem()->warp_b[warp] = wb;
    }
    __syncthreads();
    *a = warp_sum64(lane < kWarps ? mem()->warp_a[lane] : 0);
    *b = warp_sum64(lane < kWarps ? mem()->warp_b[lane] : 0);
  }
  // Every rank's (a, b), the same in all threads of a rank, to all ranks'
  // boxes; a cluster barrier.
  GBF_DEVICE const u64 (*exchange(u64 a, u64 b))[8] {
    if (tid < ranks) {
      Shared* o = of(tid);
      o->box[turn][0][rank] = a;
      o->box[turn][1][rank] = b;
    }
    cluster.sync();
    const u64(*got)[8] = mem()->box[turn];
    turn ^= 1;
    return got;
  }

  // A warp's running sum over 64 values, each summed over the ranks' rows (lane
  // l: values 2 l and 2 l + 1).
  struct Scan {
    float y, xy, incl, total;
  };
  struct Hit {
    int at;                    // value at which the sum reaches a target; -1: it stays below
    float before, upto;        // the sum before it, and with it
  };
  GBF_DEVICE Scan scan64(const float (*rows)[kGroup], float base) {
    float x = 0.0f, y = 0.0f;
    for (unsigned r = 0; r < ranks; ++r) {
      const float2 v = reinterpret_cast<const float2*>(rows[r])[lane];
      x += v.x;
      y += v.y;
    }
    Scan s{y, x + y, x + y, 0.0f};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float up = __shfl_up_sync(0xffffffffu, s.incl, o);
      if (lane >= o) s.incl += up;
    }
    s.incl += base;
    s.total = __shfl_sync(0xffffffffu, s.incl, 31);
    return s;
  }
  GBF_DEVICE Hit hit64(const Scan& s, float t) {
    const unsigned m = __ballot_sync(0xffffffffu, s.incl >= t);
    const int src = m ? __ffs(m) - 1 : 0;
    const bool second = s.incl - s.y < t;                // (in the lane that reaches t)
    const int at = 2 * lane + (second ? 1 : 0);
    const float before = s.incl - (second ? s.y : s.xy), upto = second ? s.incl : s.incl - s.y;
    Hit h{__shfl_sync(0xffffffffu, at, src), __shfl_sync(0xffffffffu, before, src), __shfl_sync(0xffffffffu, upto, src)};
    if (!m) h.at = -1;
    return h;
  }
  // The bins in which the running sum over bins 0, 1, ... and all ranks reaches
  // two targets: by groups of 64 bins, then the bins of the groups they lie
  // in, read from every rank's histogram.  value(h, j): of bin j that holds h.
  // Float32 sums: exact for counts (at most 2^20), and good to 2^-19 for masses
  // (a part of kBinError).  One cluster barrier, and another has to pass before a rank
  // writes to its histogram again or ends.
  template <typename Value, typename Targets>
  GBF_DEVICE void find_bins(Value value, Targets targets, Hit out[2]) {
    static_assert(kBins == 8 * kThreads && kGroup * kGroup == kBins && kThreads == 8 * kGroup, "");
    __syncthreads();                                     // this rank's histogram is complete
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += value(mem()->hist[tid * 8 + i], tid * 8 + i);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 7) < ranks) of(tid & 7)->search.group[rank][tid >> 3] = sum;
    cluster.sync();
    const Scan groups = scan64(mem()->search.group, 0.0f);
    float t[2];
    targets(groups.total, t);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      out[k] = hit64(groups, t[k]);
      const unsigned r = tid >> 6;
      const int j = out[k].at * kGroup + (tid & 63);
      if (out[k].at >= 0 && r < ranks) mem()->search.bin[k][r][tid & 63] = value(of(r)->hist[j], j);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (out[k].at >= 0) {
        const Hit h = hit64(scan64(mem()->search.bin[k], out[k].before), t[k]);
        out[k].before = h.before;
        out[k].upto = h.upto;
        out[k].at = out[k].at * kGroup + (h.at < 0 ? kGroup - 1 : h.at);
      }
  }

  // The same over kCells cells of masses in the histogram's memory, one target:
  // mem()->found and mem()->before of all ranks.  Three barriers.
  GBF_DEVICE void find_cell(u64 base, u64 target) {
    constexpr int kMost = kCells / kThreads;
    if (tid == 0) mem()->found = -1;
    cluster.sync();
    const int mine = kCells / ranks, first = rank * mine;
    const int per = (mine + kThreads - 1) / kThreads;
    u64 val[kMost], part = 0;
#pragma unroll 1
    for (int i = 0; i < kMost; ++i) {
      u64 lo = 0, hi = 0;
      if (i < per && tid * per + i < mine)
        for (unsigned r = 0; r < ranks; ++r) {
          lo += of(r)->hist[first + tid * per + i];
          hi += of(r)->hist[kCells + first + tid * per + i];
        }
      val[i] = (hi << 32) + lo;
      part += val[i];
    }
    const u64 incl = warp_scan64(part, lane);
    if (lane == 31) mem()->warp_a[warp] = incl;
    __syncthreads();
    u64 at = base + incl - part, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += mem()->warp_a[w];
      all += mem()->warp_a[w];
    }
    const u64(*box)[8] = exchange(all, 0);
    for (unsigned r = 0; r < rank; ++r) at += box[0][r];
#pragma unroll 1
    for (int i = 0; i < kMost; ++i) {
      if (at < target && at + val[i] >= target)          // one thread of the cluster, if any
        for (unsigned r = 0; r < ranks; ++r) {
          of(r)->found = first + tid * per + i;
          of(r)->before = at;
        }
      at += val[i];
    }
    cluster.sync();
  }

  // A candidate of this rank to the list of every rank, or of the first `heads`.
  GBF_DEVICE void offer(u64 k, unsigned heads) {
    const unsigned share = kList / ranks, at = atomicAdd(&mem()->mine_n, 1u);
    if (at < share)
      for (unsigned r = 0; r < heads; ++r) of(r)->list[rank * share + at] = k;
  }
  // Closes the lists (the threads' offers are behind a barrier of the block): a
  // cluster barrier; false when one of them is too short.
  GBF_DEVICE bool close_lists() {
    if (tid < ranks) of(tid)->list_n[rank] = mem()->mine_n;
    cluster.sync();
    bool fits = true;
    for (unsigned r = 0; r < ranks; ++r) fits = fits && mem()->list_n[r] <= kList / ranks;
    return fits;
  }
  struct Border {
    u64 rank;                  // (key, ~index) of the last element kept
    bool sure;                 // it clears the target by the slack (or slack is 0)
  };
  // The lists of all ranks in one row; how many there are.
  GBF_DEVICE unsigned pack(u64* order) {
    unsigned n = 0;
    for (unsigned r = 0; r < ranks; ++r) {
      const unsigned c = min(mem()->list_n[r], kList / ranks);
      for (unsigned i = tid; i < c; i += kThreads) order[n + i] = mem()->list[r * (kList / ranks) + i];
      n += c;
    }
    return n;
  }
  // Those of the lists' candidates that keep(c) is true for, in any order (mine_n is 0 before); how many.
  template <typename Keep>
  GBF_DEVICE unsigned pack_some(u64* order, Keep keep) {
    const unsigned share = kList / ranks;
#pragma unroll
    for (unsigned j = tid; j < kList; j += kThreads)
      if (j % share < mem()->list_n[j / share]) {
        const u64 c = mem()->list[j];
        if (keep(c)) order[atomicAdd(&mem()->mine_n, 1u)] = c;
      }
    __syncthreads();
    return mem()->mine_n;
  }
  // Sorts n <= kList values, larger first: bitonic, a warp's 64 values in its lanes
  // as long as the steps stay within them.  Zeros go behind, up to a power of two.
  // They stand `from` values into the histogram's memory.
  __device__ __noinline__ static void sort_down(unsigned from, unsigned n) {
    static_assert(kList == 2 * kThreads, "");
    u64* order = reinterpret_cast<u64*>(mem()->hist) + from;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned size = 64;
    while (size < n) size *= 2;
    for (unsigned i = n + tid; i < size; i += kThreads) order[i] = 0;
    __syncthreads();
    const unsigned i0 = warp * 64 + lane, i1 = i0 + 32;
    const bool on = static_cast<unsigned>(warp) * 64 < size;
    u64 x = on ? order[i0] : 0, y = on ? order[i1] : 0;
    auto keep = [](u64 mine, u64 other, bool larger) { return (mine > other) == larger ? mine : other; };
#pragma unroll 1
    for (unsigned width = 2; width <= size; width *= 2) {
      if (width > 64) {                                  // steps across warps: through shared memory
        if (on) {
          order[i0] = x;
          order[i1] = y;
        }
#pragma unroll 1
        for (unsigned step = width / 2; step >= 64; step /= 2) {
          __syncthreads();
          if (static_cast<unsigned>(tid) < size / 2) {
            const unsigned i = 2 * tid - (tid & (step - 1)), j = i + step;
            const u64 p = order[i], q = order[j];
            if ((p < q) == ((i & width) == 0)) {
              order[i] = q;
              order[j] = p;
            }
          }
        }
        __syncthreads();
        if (on) {
          x = order[i0];
          y = order[i1];
        }
      }
      if (width >= 64) {                                 // the lane's own two
        const bool down = (i0 & width) == 0;
        const u64 larger = x > y ? x : y, smaller = x > y ? y : x;
        x = down ? larger : smaller;
        y = down ? smaller : larger;
      }
#pragma unroll 1
      for (unsigned step = width / 2 < 16 ? width / 2 : 16; step > 0; step /= 2) {
        const u64 ox = __shfl_xor_sync(0xffffffffu, x, step), oy = __shfl_xor_sync(0xffffffffu, y, step);
        const bool low = (lane & step) == 0;
        x = keep(x, ox, low == ((i0 & width) == 0));
        y = keep(y, oy, low == ((i1 & width) == 0));
      }
    }
    if (on) {
      order[i0] = x;
      order[i1] = y;
    }
    __syncthreads();
  }

  // Ranks n candidates, the same in every rank, packed in the histogram's memory
  // (a few by comparison with each other, more by a bitonic sort, larger first):
  // the last of them before which less than `target` lies, `before` lying before
  // all.  value(l): what a candidate counts for.
  template <typename Value>
  GBF_DEVICE Border border_of(unsigned n, u64 before, u64 target, u64 slack, Value value) {
    static_assert(2 * kList * sizeof(u64) <= sizeof(unsigned) * kBins && kFew <= kThreads, "");
    u64* order = reinterpret_cast<u64*>(mem()->hist);
    u64 last = ~0ull;
    bool sure = false;
    auto decide = [&](u64 k, u64 at, u64 w) {
      if (at >= target) return;
      last = k;
      sure = at + w >= target + slack && (at == 0 || at + slack < target);
    };
    if (n <= kFew) {
      u64* weight = order + kList;
      __syncthreads();
      u64 k = 0, w = 0, at = before;
      if (tid < n) {
        k = order[tid];
        weight[tid] = w = value(of_key(static_cast<unsigned>(k >> 32)));
      }
      __syncthreads();
      if (tid < n) {
#pragma unroll 4
        for (unsigned j = 0; j < n; ++j)
          if (order[j] > k) at += weight[j];
        decide(k, at, w);
      }
      return conclude(last, sure);
    }
    sort_down(0, n);
    // the border: two candidates per thread
    constexpr int kPer = kList / kThreads;
    u64 w[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const unsigned j = tid * kPer + i;
      w[i] = j < n ? value(of_key(static_cast<unsigned>(order[j] >> 32))) : 0;
      sum += w[i];
    }
    const u64 incl = warp_scan64(sum, lane);
    if (lane == 31) mem()->warp_a[warp] = incl;
    __syncthreads();
    const u64 warps = warp_scan64(lane < kWarps ? mem()->warp_a[lane] : 0, lane);
    u64 at = before + incl - sum + (warp ? __shfl_sync(0xffffffffu, warps, warp - 1) : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const unsigned j = tid * kPer + i;
      if (j < n) decide(order[j], at, w[i]);
      at += w[i];
    }
    return conclude(last, sure);
  }
  // the smallest of the threads' borders
  GBF_DEVICE Border conclude(u64 last, bool sure) {
    last = ~warp_max64(~last);
    __syncthreads();
    if (lane == 0) mem()->warp_a[warp] = last;
    Border out;
    out.sure = __syncthreads_or(sure);
    out.rank = ~warp_max64(lane < kWarps ? ~mem()->warp_a[lane] : 0);
    return out;
  }

  // An exclusive sum over the block of each thread's value, and the total.
  GBF_DEVICE u64 block_before(u64 v, u64* total) {
    const u64 incl = warp_scan64(v, lane);
    __syncthreads();
    if (lane == 31) mem()->warp_a[warp] = incl;
    __syncthreads();
    const u64 warps = warp_scan64(lane < kWarps ? mem()->warp_a[lane] : 0, lane);
    *total = __shfl_sync(0xffffffffu, warps, 31);
    return incl - v + (warp ? __shfl_sync(0xffffffffu, warps, warp - 1) : 0);
  }

  // The row's draw when the lists hold its first elements, top-k's border among
  // them: on one CTA, without the others.  In the thread that returns true.
  GBF_DEVICE bool draw_of_lists(unsigned k, bool by_p, float p, u64 least, float u, unsigned* token, float* l, u64* mass) {
    u64* order = reinterpret_cast<u64*>(mem()->hist);
    u64* by_index = order + kList;
    u64* weight = mem()->near;
    const unsigned n = pack(order), kept = min(n, k);
    sort_down(0, n);
    constexpr int kPer = kList / kThreads;
    u64 w[kPer], sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const unsigned j = tid * kPer + i;
      const float l0 = j < kept ? of_key(static_cast<unsigned>(order[j] >> 32)) : -INFINITY;
      const float l1 = j + 1 < kept ? of_key(static_cast<unsigned>(order[j + 1] >> 32)) : -INFINITY;
      weigh(make_float2(l0, l1), &w[i], &w[i + 1]);
      sum += w[i] + w[i + 1];
    }
    u64 at = block_before(sum, &total);
    const u64 target = by_p ? share_of(p, total) : ~0ull;
    unsigned most = 0;                                     // kept by all criteria: the first so many
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const unsigned j = tid * kPer + i;
      const bool on = j < kept && at < target && w[i] >= least;
      at += w[i];
      weight[j] = w[i];
      by_index[j] = (order[j] << 32) | j;                  // ~index above: lower indexes first
      most += __syncthreads_count(on);
    }
    sort_down(kList, most);
    sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const unsigned j = tid * kPer + i;
      w[i] = j < most ? weight[static_cast<unsigned>(by_index[j])] : 0;
      sum += w[i];
    }
    at = block_before(sum, &total);
    *mass = total;
    const u64 aim = __umul64hi(fraction_of(u), total);
    bool here = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (at <= aim && aim < at + w[i]) {
        const u64 x = by_index[tid * kPer + i];
        *token = 0xffffffffu - static_cast<unsigned>(x >> 32);
        *l = of_key(static_cast<unsigned>(order[static_cast<unsigned>(x)] >> 32));
        here = true;
      }
      at += w[i];
    }
    return here;
  }

  // The rank (key, ~index) of the last element before which less than `target`
  // (elements, or mass) lies.  It is one of the elements with places p0..p1 and
  // ranks >= lo, before which `before` lies.
  GBF_DEVICE u64 border_within(bool by_mass, int p0, int p1, u64 lo, u64 before, u64 target) {
    u64 hi = ~0ull;
    int s = 0;
    // these places' logits lie between these two, with room for the roundings
    float l_hi = INFINITY, l_lo = -FLT_MAX;
    if (scale.top != INFINITY) {
      if (p0 >= 64) l_hi = scale.top - (p0 - 64) * scale.c_inverse;
      if (p1 < 64 * (kBins - 1)) l_lo = fmaxf(scale.top - (p1 + 64) * scale.c_inverse, -FLT_MAX);
    }
    // rounds: gather the candidates; when there are too many, the range of their ranks, then (and again) that range
    // cut into cells, of which the target's one stays, and gather again
    enum { kGather, kRange, kCut };
    int level = 0;
    for (int todo = kGather;;) {
      u64 mn = ~0ull, mx = 0;
      if (todo == kGather && tid == 0) mem()->mine_n = 0;
      if (todo == kCut) clear();
      if (todo == kGather) __syncthreads();
      else cluster.sync();                               // every rank is done with the last histogram
#pragma unroll 1
      for (int v = v0 + tid; v < v1; v += kThreads) {
        float f[Row<T, STAGED>::N];
        row.get(v, f);
        bool any = false;
#pragma unroll
        for (int e = 0; e < Row<T, STAGED>::N; ++e) any = any || (f[e] >= l_lo && f[e] <= l_hi);
        if (!any) continue;
#pragma unroll 1
        for (int e = 0; e < Row<T, STAGED>::N; e += 2) {
          const int j = v * (Row<T, STAGED>::N / 2) + e / 2;
          const float2 q = row.pair(j);
          u64 w[2] = {1, 1};
          if (by_mass && todo == kCut) weigh(q, &w[0], &w[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float l = i ? q.y : q.x;
            const u64 k = rank_of(key_of(l), 2 * j + i - row.shift);
            const int n = place(l);
            if (l < l_lo || l > l_hi || k < lo || k > hi || n < p0 || n > p1) continue;
            if (todo == kGather) {
              offer(k, ranks);
            } else if (todo == kRange) {
              mn = k < mn ? k : mn;
              mx = k > mx ? k : mx;
            } else {
              const int cell = static_cast<int>((hi - k) >> s);
              add_mass(&mem()->hist[cell], &mem()->hist[kCells + cell], w[i]);
            }
          }
        }
      }
      if (todo == kGather) {
        __syncthreads();
        if (close_lists() || level == 8) break;
        todo = level == 0 ? kRange : kCut;
      } else if (todo == kRange) {
        mn = ~warp_max64(~mn);
        mx = warp_max64(mx);
        __syncthreads();
        if (lane == 0) {
          mem()->warp_a[warp] = mx;
          mem()->warp_b[warp] = mn;
        }
        __syncthreads();
        mx = warp_max64(lane < kWarps ? mem()->warp_a[lane] : 0);
        mn = ~warp_max64(lane < kWarps ? ~mem()->warp_b[lane] : 0);
        const u64(*box)[8] = exchange(mn, mx);
        lo = ~0ull;
        hi = 0;
        for (unsigned r = 0; r < ranks; ++r) {
          lo = box[0][r] < lo ? box[0][r] : lo;
          hi = box[1][r] > hi ? box[1][r] : hi;
        }
        todo = kCut;
      } else {
        find_cell(before, target);
        if (mem()->found >= 0) {                         // (always: the target lies within)
          before = mem()->before;
          hi -= static_cast<u64>(mem()->found) << s;
          const u64 span = (1ull << s) - 1;
          lo = hi - lo > span ? hi - span : lo;
        }
        ++level;
        todo = kGather;
      }
      if (todo == kCut) {
        s = 0;
        while (((hi - lo) >> s) >= kCells) ++s;
      }
    }
    return border_of(pack(reinterpret_cast<u64*>(mem()->hist)), before, target, 0, [&](float l) {
             u64 w0 = 1, w1;
             if (by_mass) weigh(two(l), &w0, &w1);
             return w0;
           }).rank;
  }
};

// border_within as a call (it is needed in two places and long), on a copy, so
// that the caller's object stays in registers.
struct BorderTurn {
  u64 border;
  int turn;
};
template <typename T, bool STAGED>
__device__ __noinline__ BorderTurn border_call(Sampler<T, STAGED> s, bool by_mass, int p0, int p1, u64 lo, u64 before,
                                               u64 target) {
  const u64 border = s.border_within(by_mass, p0, p1, lo, before, target);
  return {border, s.turn};
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  constexpr int N = Elem<T>::N;
  Sampler<T, STAGED> s{cg::this_cluster()};
  s.rank = s.cluster.block_rank();
  s.ranks = s.cluster.num_blocks();
  s.turn = 0;
  // Shared memory of another CTA may be touched only once that CTA runs: every rank says so here, and the first exchange
  // waits for all of them (behind the row's read, where that costs nothing).
  s.cluster.barrier_arrive();
  const int tid = s.tid = threadIdx.x, lane = s.lane = tid & 31, warp = s.warp = tid >> 5;
  if (tid < 64) mem()->pow[tid] = kPow[tid];
  if (tid < 16) {
    const u64 p = kPow[4 * tid];
    const float hi = __ull2float_rn(p);
    mem()->sixteenth[tid] =
        make_float2(hi * 0x1p-43f, __ll2float_rn(static_cast<long long>(p - __float2ull_rn(hi))) / hi);
  }
  s.clear();
  pdl_wait();
  pdl_launch_dependents();

  const int64_t b = blockIdx.x / s.ranks;
  const char* at = static_cast<const char*>(a.logits) + b * a.stride * static_cast<int64_t>(sizeof(T));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
  s.row.base = at - off;
  s.row.shift = off / static_cast<int>(sizeof(T));
  s.row.vocab = a.vocab;
  const int vectors = (s.row.shift + a.vocab + N - 1) / N;
  s.row.full0 = s.row.shift ? 1 : 0;
  s.row.full = max((s.row.shift + a.vocab) / N - s.row.full0, 0);
  const int per = (vectors + s.ranks - 1) / s.ranks;
  const int v0 = s.v0 = s.row.v0 = min(static_cast<int>(s.rank) * per, vectors);
  const int v1 = s.v1 = min(v0 + per, vectors);
  s.j0 = v0 * (N / 2);
  s.j1 = v1 * (N / 2);
  const float temp = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.0f;
  const float mp = a.min_p ? a.min_p[b] : 0.0f;
  const float u = a.uniform[b];

  const float heat = fmaxf(temp, kLeastTemperature);
  {
    // log2(e) / T in two parts: the quotient of the high part, and the quotient of what it leaves
    constexpr float kHi = 1.44269504088896341f;
    constexpr float kLo = static_cast<float>(1.4426950408889634074 - static_cast<double>(kHi));
    s.scale.c_hi = __fdiv_rn(kHi, heat);
    s.scale.c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-s.scale.c_hi, heat, kHi), kLo), heat);
    s.scale.c_place = s.scale.c_hi * (kBinsPerOctave * 64.0f);
    s.scale.c_inverse = heat * (0.693147180559945f / (kBinsPerOctave * 64.0f));
  }

  // top-k: lanes per group, with at least k groups in the cluster
  const bool by_k = k > 0 && k < a.vocab, by_p = p < 1.0f;
  const int lanes = kThreads * static_cast<int>(s.ranks);
  const int group = !by_k ? 0 : k <= lanes / 32 ? 32 : k <= lanes / 4 ? 4 : k <= lanes ? 1 : 0;

  // pass 1: the only read of HBM; the largest logit, and the smallest of the groups' largest ones
  float most = -INFINITY;
  auto look = [&](int v, uint4 raw) {
    float f[N];
    Elem<T>::widen(raw, f);
    tidy<N>(f);
    if (STAGED) stage()[v - v0] = Elem<T>::pack(f);
#pragma unroll
    for (int i = 0; i < N; ++i) most = fmaxf(most, f[i]);
  };
  int v = v0 + tid;
#pragma unroll 1
  for (; v + 3 * kThreads < v1; v += 4 * kThreads) {
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = s.row.load(v + u * kThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u) look(v + u * kThreads, raw[u]);
  }
#pragma unroll 1
  for (; v < v1; v += kThreads) look(v, s.row.load(v));
  // (as keys, over the lanes, the warps and the ranks; 0: no candidate)
  const unsigned mine = most == -INFINITY ? 0u : key_of(most);
  unsigned top = __reduce_max_sync(0xffffffffu, mine), low = mine;
  if (group == 4) {
    low = max(low, __shfl_xor_sync(0xffffffffu, low, 1));
    low = max(low, __shfl_xor_sync(0xffffffffu, low, 2));
  }
  low = group == 32 ? top : __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    mem()->warp_a[warp] = top;
    mem()->warp_b[warp] = low;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<unsigned>(mem()->warp_a[lane]) : 0u);
  low = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<unsigned>(mem()->warp_b[lane]) : 0xffffffffu);
  s.cluster.barrier_wait();                              // all ranks have started
  {
    const u64(*box)[8] = s.exchange(top, low);
    for (unsigned r = 0; r < s.ranks; ++r) {
      top = max(top, static_cast<unsigned>(box[0][r]));
      low = min(low, static_cast<unsigned>(box[1][r]));
    }
  }
  const float floor_k = group > 0 && low > 0 ? of_key(low) : -FLT_MAX;
  s.scale.top = of_key(top);
  const float quick_top = __fmul_rn(s.scale.top, s.scale.c_hi);
  s.scale.cut = s.scale.top - 41.5f * heat;
  s.scale.n_top = ((__float_as_uint(__fadd_rn(quick_top, kMagic)) << 19) & 0xff800000u) + 0x800000u;

  const bool bad = !(temp >= 0.0f && temp < INFINITY) || !(p == p) || !(mp <= 1.0f) || !(u >= 0.0f && u < 1.0f);
  if (bad || top == 0) {
    if (s.rank == 0 && tid == 0) {
      raise_error(a.err, DEV_ERR_SAMPLING);
      a.tokens[b] = -1;
      if (a.logprob) a.logprob[b] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  if (temp == 0.0f) {                                    // the lowest index of the largest logit
    unsigned first = 0xffffffffu;
    if (most == s.scale.top)
#pragma unroll 1
      for (int j = s.j0 + tid * (N / 2); j < s.j1; j += kThreads * (N / 2)) {
#pragma unroll 1
        for (int e = 0; e < N / 2; ++e) {
          const float2 f = s.row.pair(j + e);
          const unsigned i = 2 * (j + e) - s.row.shift;
          if (f.y == s.scale.top) first = min(first, i + 1);
          if (f.x == s.scale.top) first = min(first, i);
        }
      }
    first = __reduce_min_sync(0xffffffffu, first);
    __syncthreads();
    if (lane == 0) mem()->warp_a[warp] = first;
    __syncthreads();
    first = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<unsigned>(mem()->warp_a[lane]) : 0xffffffffu);
    const u64(*box)[8] = s.exchange(first, 0);
    for (unsigned r = 0; r < s.ranks; ++r) first = min(first, static_cast<unsigned>(box[0][r]));
    if (s.rank == 0 && tid == 0) {
      a.tokens[b] = static_cast<int32_t>(first);
      if (a.logprob) a.logprob[b] = 0.0f;
    }
    return;
  }
  const u64 least = mp > 0.0f ? __float2ull_ru(mp * static_cast<float>(1ull << kFix)) : 0;

  // The row's draw from the elements with logits >= from and places <= p1, top-k's border among them: gathered on rank 0.
  // False when a rank has more than its share of them.
  auto draw_first = [&](float from, int p1) {
    if (tid == 0) mem()->mine_n = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = v0 + tid; i < v1; i += kThreads) {
      float f[N];
      s.row.get(i, f);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (f[e] >= from && s.place(f[e]) <= p1)
          s.offer(rank_of(key_of(f[e]), static_cast<unsigned>(i * N + e - s.row.shift)), 1);
    }
    __syncthreads();
    if (!s.close_lists()) {
      s.cluster.sync();                                    // every rank has read the lists' sizes
      return false;
    }
    unsigned token;
    float l;
    u64 mass;
    if (s.rank == 0 && s.draw_of_lists(k, by_p, p, least, u, &token, &l, &mass)) {
      a.tokens[b] = static_cast<int32_t>(token);
      if (a.logprob) a.logprob[b] = log_share(s.scale, l, heat, mass, 1ull << kFix);
    }
    return true;
  };
  // (shared addresses that stay in registers: the compiler would derive them again at each use)
  unsigned hist_at, sixteenth;
  asm volatile("mov.u32 %0, %1;" : "=r"(hist_at) : "r"(smem_u32(mem()->hist)));
  asm volatile("mov.u32 %0, %1;" : "=r"(sixteenth) : "r"(smem_u32(mem()->sixteenth)));
  u64 border = 0;                                        // ranks below it are cut off
  int b0 = 0, b1 = kBins - 1;                            // bins the border of top-p lies in
  typename Sampler<T, STAGED>::Hit hit[2];
  hit[0].at = -1;
  // first without a histogram, where the groups leave few elements; then with one
  bool counted = !(group > 0 && lanes / group <= kFew && (low > 0 || a.vocab <= kList));
  for (;; counted = true) {
    float from = floor_k;
    int p1 = 64 * kBins;
    bool listed = !counted;
    if (counted && (by_k || by_p)) {
      const unsigned one = by_k ? 1u : 1u << 20, offset = by_k ? 0u : 63u;
      auto count = [&](float l, int at) {                  // (without a branch for each element)
        asm volatile("{ .reg .pred p; setp.ge.f32 p, %0, %1; @p red.shared.add.u32 [%2], %3; }" ::"f"(l), "f"(floor_k),
                     "r"(hist_at + ((static_cast<unsigned>(at) >> 6) << 2)), "r"(one + (at & offset))
                     : "memory");
      };
      if (s.scale.top == INFINITY)
        s.row.each(v0 + tid, v1, kThreads, [&](int, const float(&f)[N]) {
#pragma unroll
          for (int e = 0; e < N; ++e) count(f[e], s.place(f[e]));
        });
      else
        s.row.each(v0 + tid, v1, kThreads, [&](int, const float(&f)[N]) {
#pragma unroll
          for (int e = 0; e < N; ++e) count(f[e], place_of(s.scale, f[e]));
        });
      // counts, or with top-p alone the bins' masses: middle weight times (count - ln 2 / 128 * sum of offsets)
      s.find_bins(
          [&](unsigned h, int j) {
            if (by_k) return static_cast<float>(h);
            const float c = static_cast<float>(h >> 20), places = static_cast<float>(h & 0xfffffu);
            return (c - 0.00541521235f / 64.0f * (places - 32.0f * c)) * exp2_approx(-j / kBinsPerOctave);
          },
          [&](float total, float* t) {
            const float error = kBinError + kLastBinError * static_cast<float>(a.vocab);
            const float r = (1.0f - error) / (1.0f + error);
            t[0] = by_k ? static_cast<float>(k) : p * r * total;
            t[1] = by_k ? INFINITY : p / r * total;
          },
          hit);
      if (by_k) {
        listed = hit[0].at >= 0 && hit[0].upto <= kList;
        if (hit[0].at < kBins - 1) from = fmaxf(s.logit_of(64 * hit[0].at + 128), floor_k);    // (the last bin has no end)
        p1 = 64 * hit[0].at + 63;
      } else {
        b0 = hit[0].at < 0 ? kBins - 1 : hit[0].at;
        b1 = hit[1].at < 0 ? kBins - 1 : hit[1].at;
      }
    }
    if (listed && draw_first(from, p1)) return;
    if (counted) break;
  }
  if (by_k && hit[0].at >= 0) {                          // (else fewer than k candidates)
    const BorderTurn found = border_call<T, STAGED>(s, false, 64 * hit[0].at, 64 * hit[0].at + 63, 0,
                                                    static_cast<u64>(hit[0].before), static_cast<u64>(k));
    border = found.border;
    s.turn = found.turn;
    b1 = hit[0].at;
  }

  // A contiguous run of vectors per warp.
  const int run_v = (v1 - v0 + kWarps - 1) / kWarps, run = run_v * (N / 2);
  const int u0 = min(v0 + warp * run_v, v1), u1 = min(u0 + run_v, v1);
  // a finite logit below this one has a weight below min_p by more than any rounding
  float floor_l = -FLT_MAX;
  if (mp > 0.0f && s.scale.top != INFINITY)
    floor_l = fmaxf(__fadd_rd(s.scale.top, (log2f(mp) - 0.01f) * heat * 0.69322f), -FLT_MAX);
  const u64 k_border = border;
  const float border_l = border ? of_key(static_cast<unsigned>(border >> 32)) : -FLT_MAX;
  const float from_l = by_p ? border_l : fmaxf(border_l, floor_l);
  // float32 first, unless two criteria meet in one sum or top-k leaves little (even on the shortest slices: one row of
  // 1000 bf16 8.0 us, 8.6 exactly; 256 rows of 4000 21.8 and 22.6)
  bool exact = by_k || (by_p && mp > 0.0f) || !(fabsf(quick_top) < kQuickRange) ||
               heat > kQuickHeat;

  // min-p's bound in the float32 pass's weights
  const Quick w_top = quick_weight(sixteenth, s.scale, s.scale.top);
  const float mp_w = mp > 0.0f ? mp * w_top.w : 0.0f;

  // With top-p alone the lists are free at first: the candidates near the border go to all ranks with the totals.
  bool direct = by_p && !by_k;

  for (;; exact = true, direct = false) {
    // The kept mass of each run.  With top-p, also the mass in all and above the border's bins; what lies in them
    // goes to a list, and its mass to the span of bins.
    // (a logit above above_l lies in a bin before b0, one below below_l behind b1)
    float above_l = INFINITY, below_l = -FLT_MAX;
    // (by two places, which are rounded by half of one and are as far from (top - l) c_place by 2^-4 at most)
    if (by_p && s.scale.top != INFINITY) {
      if (b0 > 0) above_l = __fadd_ru(s.scale.top, -(64 * b0 - 34) * s.scale.c_inverse);
      if (b1 < kBins - 1) below_l = fmaxf(__fadd_rd(s.scale.top, -(64 * b1 + 33) * s.scale.c_inverse), -FLT_MAX);
    }
    const int p0 = 64 * b0, p1 = 64 * b1 + 63;           // the bins' places, in spans of 2^coarse
    const int coarse = max(0, 32 - __clz(p1 - p0) - 5);
    if (tid < kSpans) mem()->span_lo[tid] = mem()->span_hi[tid] = 0;
    if (tid == 0) mem()->near_n = mem()->mine_n = mem()->doubt = 0;
    __syncthreads();
    u64 kept = 0, above = 0, all = 0;
    auto weight_of = [&](float l) {                      // the weight that this turn's sums are made of
      u64 w0, w1;
      if (exact) {
        s.weigh(two(l), &w0, &w1);
      } else {
        w0 = parts_of(quick_weight(sixteenth, s.scale, l)).fixed();
      }
      return w0;
    };
    // an element that may lie in the border's bins: true when it does
    auto near = [&](float l, unsigned i, u64 w) {
      const int n = s.place(l);
      if (n < p0) return false;
      if (n <= p1) {
        const int span = (n - p0) >> coarse;
        add_mass(&mem()->span_lo[span], &mem()->span_hi[span], w);
        const unsigned at = atomicAdd(&mem()->near_n, 1u);
        if (at < kNear) mem()->near[at] = rank_of(key_of(l), i);
      }
      return true;
    };
    if (!exact) {
      Sum sum{};
      if (by_p) {
        Sum sum_above{};
        s.row.each(u0 + lane, u1, 32, [&](int i, const float(&f)[N]) {
          bool any = false;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const Sum w = parts_of(quick_weight(sixteenth, s.scale, f[e]));
            sum.add(w);
            asm("{ .reg .pred p; setp.gt.f32 p, %2, %3; @p add.u32 %0, %0, %4; @p add.s32 %1, %1, %5; }"
                : "+r"(sum_above.a), "+r"(sum_above.b) : "f"(f[e]), "f"(above_l), "r"(w.a), "r"(w.b));
            any = any | (f[e] <= above_l & f[e] >= below_l);
          }
          if (any)
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float l = f[e] + 0.0f;                 // (-0 as 0)
              if (l > above_l || !(l >= below_l)) continue;
              const u64 w = weight_of(l);
              if (!near(l, static_cast<unsigned>(i * N + e - s.row.shift), w)) above += w;
            }
        });
        all = sum.fixed();
        kept = above += sum_above.fixed();
      } else if (mp > 0.0f) {
        // (weights as float32 numbers: 2^-23 of each other)
        const float mp_lo = mp_w * (1.0f - 0x1p-21f), mp_hi = mp_w * (1.0f + 0x1p-21f);
        s.row.each(u0 + lane, u1, 32, [&](int, const float(&f)[N]) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const Quick w = quick_weight(sixteenth, s.scale, f[e]);
            if (w.w > mp_lo && w.w < mp_hi && f[e] != s.scale.top) mem()->doubt = 1;
            if (!(w.w < mp_w)) sum.add(parts_of(w));
          }
        });
        kept = sum.fixed();
      } else {
        s.row.each(u0 + lane, u1, 32, [&](int, const float(&f)[N]) {
#pragma unroll
          for (int e = 0; e < N; ++e) sum.add(parts_of(quick_weight(sixteenth, s.scale, f[e])));
        });
        kept = sum.fixed();
      }
    } else {
#pragma unroll 1
      for (int i = u0 + lane; i < u1; i += 32) {
        float f[N];
        s.row.get(i, f);
        bool any = false;
#pragma unroll
        for (int e = 0; e < N; ++e) any = any || f[e] >= from_l;
        if (!any) continue;
#pragma unroll
        for (int q = 0; q < N; q += 4) {                 // two pairs at once: a weight is a long chain
          u64 w[4];
          s.weigh(make_float2(f[q], f[q + 1]), &w[0], &w[1]);
          s.weigh(make_float2(f[q + 2], f[q + 3]), &w[2], &w[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float l = f[q + e];
            const unsigned at = static_cast<unsigned>(i * N + q + e - s.row.shift);
            if (l < from_l || (l == border_l && rank_of(key_of(l), at) < k_border)) continue;
            all += w[e];
            if (by_p && l <= above_l && near(l, at, w[e])) continue;
            above += w[e];
            if (w[e] >= least) kept += w[e];
          }
        }
      }
    }
    kept = warp_sum64(kept);
    if (lane == 0) {
      mem()->run_lo[warp] = static_cast<unsigned>(kept);
      mem()->run_hi[warp] = static_cast<unsigned>(kept >> 32);
    }
    if (by_p) {
      s.block_sum(&above, &all);
      const unsigned share = kList / s.ranks;
      if (direct) {
        const unsigned n = mem()->near_n;
        if (n <= share)
          for (unsigned i = tid; i < n * s.ranks; i += kThreads)
            s.of(i % s.ranks)->list[s.rank * share + i / s.ranks] = mem()->near[i / s.ranks];
        if (tid < s.ranks) s.of(tid)->list_n[s.rank] = n;
      }
      // spans and whether the list holds them all to all ranks with the totals
      if (tid < kSpans * 8 && (tid >> 5) < s.ranks)
        s.of(tid >> 5)->span[s.rank][lane] = mass_of(mem()->span_lo[lane], mem()->span_hi[lane]);
      const u64(*box)[8] = s.exchange(above, all | (mem()->near_n > kNear ? 1ull << 63 : 0));
      above = all = 0;
      bool many = false;
      for (unsigned r = 0; r < s.ranks; ++r) {
        above += box[0][r];
        all += box[1][r] & ~(1ull << 63);
        many |= (box[1][r] >> 63) != 0;
      }
      const u64 target = share_of(p, all);
      u64 mass = 0;
      for (unsigned r = 0; r < s.ranks; ++r) mass += mem()->span[r][lane];
      const u64 incl = above + warp_scan64(mass, lane);
      const unsigned reached = __ballot_sync(0xffffffffu, incl >= target);
      if ((above >= target || reached == 0) && (b0 > 0 || b1 < kBins - 1)) {      // not in these bins: search them all
        b0 = 0;
        b1 = kBins - 1;
        s.cluster.sync();                                // every rank has read its spans
        continue;
      }
      const int hit = max(__ffs(reached) - 1, 0);
      const u64 before = __shfl_sync(0xffffffffu, incl - mass, hit);
      u64* order = reinterpret_cast<u64*>(mem()->hist);
      auto in_span = [&](u64 c) { return ((s.place(of_key(static_cast<unsigned>(c >> 32))) - p0) >> coarse) == hit; };
      unsigned n = 0;                                    // the span's elements
      if (direct) {
        for (unsigned r = 0; r < s.ranks; ++r) direct = direct && mem()->list_n[r] <= share;
        if (direct) n = s.pack_some(order, in_span);
        else s.cluster.sync();                           // every rank has read the lists' sizes
      }
      if (!direct && !many) {                            // from this rank's list to all
        for (unsigned i = tid; i < mem()->near_n; i += kThreads)
          if (in_span(mem()->near[i])) s.offer(mem()->near[i], s.ranks);
        __syncthreads();
        many = !s.close_lists();
        if (!many) n = s.pack(order);
      }
      if (!many) {
        const auto found = s.border_of(n, before, target, exact ? 0 : slack_of(target, a.vocab, s.ranks), weight_of);
        if (!exact && !found.sure) {
          if (direct) s.cluster.sync();                  // every rank has read its spans and lists
          continue;
        }
        border = found.rank;
      } else {
        s.cluster.sync();                                // every rank has read the lists' sizes
        if (!exact) continue;
        const BorderTurn found = border_call<T, STAGED>(
            s, true, p0 + (hit << coarse), min(p0 + ((hit + 1) << coarse) - 1, p1), k_border, before, target);
        border = found.border;
        s.turn = found.turn;
      }
      // what is kept of the elements in the border's bins
      auto keep = [&](u64 rank) {
        if (rank < border) return;
        const u64 w = weight_of(of_key(static_cast<unsigned>(rank >> 32)));
        if (w < least) return;
        const int of_run = (static_cast<int>((0xffffffffu - static_cast<unsigned>(rank) + s.row.shift) >> 1) - s.j0) / run;
        add_mass(&mem()->run_lo[of_run], &mem()->run_hi[of_run], w);
      };
      if (mem()->near_n <= kNear) {
#pragma unroll 1
        for (unsigned i = tid; i < mem()->near_n; i += kThreads) keep(mem()->near[i]);
      } else {
#pragma unroll 1
        for (int i = 2 * s.j0 + tid; i < 2 * s.j1; i += kThreads) {
          const float2 f = s.row.pair(i / 2);
          const float l = i & 1 ? f.y : f.x;
          const int n = s.place(l);
          if (l != -INFINITY && n >= p0 && n <= p1) keep(rank_of(key_of(l), i - s.row.shift));
        }
      }
    }
    __syncthreads();

    // the draw: the rank, and in it the run, that the target lies in
    const u64 mine = lane < kWarps ? mass_of(mem()->run_lo[lane], mem()->run_hi[lane]) : 0;
    const u64 incl_runs = warp_scan64(mine, lane);
    const u64 my_total = __shfl_sync(0xffffffffu, incl_runs, 31);
    u64 before = 0, total = 0;
    bool doubt = false;
    {
      const u64(*box)[8] = s.exchange(my_total, mem()->doubt);
      for (unsigned r = 0; r < s.ranks; ++r) {
        if (r < s.rank) before += box[0][r];
        total += box[0][r];
        doubt |= box[1][r] != 0;
      }
    }
    if (doubt) continue;
    const u64 target = __umul64hi(fraction_of(u), total);  // below total
    const bool here = target >= before && target < before + my_total;
    if (exact && !here) return;
    int token = -1;
    float token_l = 0.0f;
    if (here) {
      const int of_run = __ffs(__ballot_sync(0xffffffffu, before + incl_runs > target)) - 1;
      before += __shfl_sync(0xffffffffu, incl_runs - mine, of_run);
      const int r0 = s.j0 + of_run * run, r1 = min(r0 + run, s.j1);
      const u64 slack = exact ? 0 : slack_of(total, a.vocab, s.ranks);
#pragma unroll 1
      for (int i0 = r0; i0 < r1; i0 += kThreads) {       // the whole CTA walks that run
        const int j = i0 + tid;
        u64 w[2] = {0, 0};
        float2 f = make_float2(-INFINITY, -INFINITY);
        if (j < r1) {
          f = s.row.pair(j);
          if (exact) {
            s.weigh(f, &w[0], &w[1]);
          } else {
            const Quick q0 = quick_weight(sixteenth, s.scale, f.x), q1 = quick_weight(sixteenth, s.scale, f.y);
            w[0] = q0.w < mp_w ? 0 : parts_of(q0).fixed();
            w[1] = q1.w < mp_w ? 0 : parts_of(q1).fixed();
          }
          const unsigned i = 2 * j - s.row.shift;
          if (f.x == -INFINITY || rank_of(key_of(f.x), i) < border || (exact && w[0] < least)) w[0] = 0;
          if (f.y == -INFINITY || rank_of(key_of(f.y), i + 1) < border || (exact && w[1] < least)) w[1] = 0;
        }
        u64 incl = warp_scan64(w[0] + w[1], lane);
        __syncthreads();
        if (lane == 31) mem()->warp_a[warp] = incl;
        __syncthreads();
        const u64 sums = warp_scan64(lane < kWarps ? mem()->warp_a[lane] : 0, lane);
        incl += before + (warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
        u64 at = incl - w[0] - w[1];
        if (at <= target && target < incl) {             // one thread
          const bool second = at + w[0] <= target;
          if (second) at += w[0];
          else incl = at + w[0];
          if ((at == 0 || at + slack <= target) && target + slack < incl) {
            token = 2 * j + (second ? 1 : 0) - s.row.shift;
            token_l = second ? f.y : f.x;
          }
        }
        before += __shfl_sync(0xffffffffu, sums, 31);
        if (target < before) break;
      }
    }
    if (!exact) {                                        // done unless the token lies too near its neighbours
      const bool found = __syncthreads_or(token >= 0);
      const u64(*box)[8] = s.exchange(found, 0);
      for (unsigned r = 0; r < s.ranks; ++r) doubt |= box[0][r] != 0;
      if (!doubt) continue;                              // (no rank has found it)
    }
    if (token >= 0) {
      a.tokens[b] = token;
      if (a.logprob)
        a.logprob[b] = log_share(s.scale, token_l, heat, total, exact ? 1ull << kFix : parts_of(w_top).fixed());
    }
    return;
  }
}

// Clusters of 1, 2, 4 and 8 CTAs that are there at once with two CTAs on an SM (a bound for a choice, not for correctness).
constexpr int kShared[4] = {304, 152, 74, 36};
// Dynamic shared memory of a CTA that is to have an SM for itself.
constexpr int kAloneBytes = 120 * 1024;
static_assert(sizeof(Shared) + kStageBytes < kAloneBytes && 2 * kAloneBytes > 228 * 1024, "");

template <typename T, bool STAGED>
cudaError_t launch(const SampleArgs& a, int ranks, size_t smem, cudaStream_t stream) {
  const cudaError_t e = allow_smem<sample_kernel<T, STAGED>>(kAloneBytes);
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, STAGED>, a);
}

template <typename T>
cudaError_t plan(const SampleArgs& a, cudaStream_t stream) {
  constexpr int N = Elem<T>::N;
  const int64_t vectors = (static_cast<int64_t>(a.vocab) + N - 1) / N + 1;
  auto slice = [&](int ranks) { return (vectors + ranks - 1) / ranks * 16; };
  // (of the kernel with an SM for each CTA)
  auto alone_at = [](int i, int* n) { return resident_clusters<sample_kernel<T, true>>(i, kThreads, kAloneBytes, n); };
  // CTAs per row: as many as leave an SM to each CTA, because two on one SM cost each other more than half a slice is
  // worth (64 rows of 32000, nucleus: 27 us with two, 28 with four; 16 rows: 21.6 with four, 23.5 with eight) ...
  int i = 3, n = 0;
  cudaError_t e = alone_at(i, &n);
  while (e == cudaSuccess && i > 0 && a.batch > n) e = alone_at(--i, &n);
  if (e != cudaSuccess) return e;
  bool alone = a.batch <= n;
  // ... and twice that, two on one SM, where a slice would not fit in shared memory (32 rows of 151936, nucleus: 51 us
  // with eight, 60 with four; 200 rows of 50257: 73 with two, 82 with one; 256 of 32000, which fit: 62 with one, 69 with
  // two) and they are all there at once (76 rows of 128000: 66 with two, 74 with four)
  if (i < 3 && slice(1 << i) > kStageBytes && (i == 0 || a.batch <= kShared[i + 1])) {
    ++i;
    alone = false;
  }
  // very long rows: so that a bin's count and a thread's sums hold
  if (a.vocab > 256 * 1024 && i < 2) {
    i = 2;
    alone = false;
  }
  // Where they fit, CTAs are kept from sharing an SM (by the shared memory they ask for): in a run of calls, the second
  // call's would otherwise settle in pairs beside the first one's (61 rows of 50257: 14.9 us, or 21.8 in half of the
  // processes; 152 rows of 30000: 16.5 and 24).
  const size_t bytes = static_cast<size_t>(slice(1 << i));
  if (bytes <= kStageBytes) return launch<T, true>(a, 1 << i, alone ? kAloneBytes : sizeof(Shared) + bytes, stream);
  return launch<T, false>(a, 1 << i, alone ? kAloneBytes : sizeof(Shared), stream);
}

}  // namespace

cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t stream) {
  return a.f32 ? plan<float>(a, stream) : plan<__nv_bfloat16>(a, stream);
}

}  // namespace gbf
