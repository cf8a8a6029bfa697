// Tokens drawn from rows of logits with temperature, top-k, top-p and min-p.
//
// The candidates of a row stand in one order: larger logits first, equal ones by index.  Each filter
// keeps a first part of that order (top-k the first k, top-p the shortest part whose weight reaches p of what
// top-k left, min-p those within ln(min_p) T of the largest), so all of them together keep the
// candidates up to one (key, index): the row's cut.  The draw is by index: the first kept token where
// the running sum of weights passes u times their total.
//
// Sums are exact.  A weight, e^((l - max) / T), is a whole number of 2^-43 of the largest (weight()
// below: an error of at most 2^-28 of itself before that rounding), and sums of whole numbers depend on no
// order: a row gives the same token however it is split, and products with u and p are compared in whole
// numbers too.  In 32-bit floats a sum over a vocabulary is off by more than a single token weighs.
//
// A row is a cluster's (of one CTA, where there are many rows): each warp takes a stretch of it.  The
// first pass over the logits only takes maxima, of four groups a thread.  Where top-k is asked for,
// a CTA's ceil(k / C)-th largest group maximum (C CTAs) has as many logits at or above it, so the least of these
// over the cluster has k: the candidates are at or above it, and there are few more than k, found in
// the groups whose maximum is.  Without top-k, top-p needs every weight: a second pass sums them into
// 1024 intervals of logits below the largest, 1/64 T wide each, the last one without an end (by keys, which had 64 of them an octave,
// a cut at a T of 1.5 and a p of 0.99 came to lie in the last one and took three passes: 393 rows of 151936 logits 800 us, not
// 501).  That gives the total and the interval that the cut lies in.
// Up to 2048 candidates are gathered in one CTA, which finishes the row: cuts and the draw are each a search
// for the place where a running count or weight reaches a goal, by a histogram of the candidates and
// a last step over the few of one interval.  Where there are more, that CTA is given the interval's candidates
// alone and finds the cut, and a last pass of the cluster draws.  An interval of too many (flat rows) is cut up
// again until it is one key, whose ties go by index.
//
// What bounds it, at 151936 logits: one row (12 us with top-k 50, 31 with top-p alone, call after call in a graph), latency: three
// to seven meetings of the cluster, the passes' loads, of L2 after the first, and code that is fetched once and run once.  Many
// rows: 393 float ones with top-k 50 take 75 us, 3.2 TB/s: a row's first pass is followed by some 8 us of short steps, which the
// other resident CTAs' passes cover in part.  393 with top-p alone take 355 us, without any filter 183 to 187: the weights' pass is
// 41 instructions a logit, 70 with the intervals; the candidates' pass behind it (6000 of a row of such logits) takes half as long.
// Two CTAs an SM leave 64 registers a thread; with all paths in one function some 500 bytes of a thread's values are kept in
// local memory.  Rows that are not whole 16 bytes are read an element at a time: 64 float rows of 151937 logits with top-k 50
// take 21.8 us, of 151936 14.9; bf16 ones with filtered logits 54.0 and 27.2.
#include <cooperative_groups.h>

#include "tree_step.h"
#include "vg_common.cuh"
#include "vg_internal.h"

namespace cg = cooperative_groups;

namespace vg {
namespace {

constexpr int NT = 512;     // threads of a CTA
constexpr int W = NT / 32;
constexpr int NB = 1024;    // intervals of a histogram
constexpr int CAP = 2048;   // candidates that one CTA finishes
constexpr int kSmall = 256; // of these, so many by comparing each with each
constexpr int kMaxC = 16;   // CTAs of a cluster
constexpr int NG = 4;       // groups of a thread
constexpr uint32_t kNone = 0;  // key of what is no candidate: -inf and NaN
constexpr uint32_t kLowest = 0x00800000u;  // of the most negative float

// ---------------------------------------------------------------- weights
// 2^(-j / 32) in two floats, from the series of e^x (terms to x^24 / 24!: below 2^-53 for x < 1).
struct PowerTable {
  float hi[32], lo[32];
  PowerTable() = default;
  constexpr explicit PowerTable(int) : hi(), lo() {
    for (int j = 0; j < 32; ++j) {
      const double x = j * (0.693147180559945309417232121458 / 32);
      double term = 1, sum = 1;
      for (int i = 1; i <= 24; ++i) {
        term *= x / i;
        sum += term;
      }
      hi[j] = static_cast<float>(1 / sum);
      lo[j] = static_cast<float>(1 / sum - static_cast<double>(hi[j]));
    }
  }
};
__device__ const PowerTable g_powers = PowerTable(0);

// For the weights of a row: l stands for l - off, hi + lo is log2(e) / T, and ah + al that times top - off; least is the l - off
// of a weight of 2^-100.
struct Scale {
  float off, hi, lo, ah, al, least;
};
__device__ __forceinline__ Scale make_scale(float top, double c) {
  const double a = top * c;
  // ah is a whole number of 2^-16: less a whole number of 2^-5, and as long as |a| + 100 is below 2^8, it is a float again.
  // A larger |a| is taken off first, which is exact for all logits that weigh anything: they are within a factor of two
  const bool large = !(fabs(a) < 128.0);
  Scale s;
  s.off = large ? top : 0.f;
  s.hi = static_cast<float>(c);
  s.lo = static_cast<float>(c - static_cast<double>(s.hi));
  const double b = large ? 0.0 : a, h = rint(b * 0x1p16) * 0x1p-16;
  s.ah = static_cast<float>(h);
  s.al = static_cast<float>(b - h);
  s.least = (s.ah - 100.f) / s.hi;
  return s;
}

// e^((l - top) / T), for l <= top (of NaN and -inf 0), as a sum of whole numbers of 2^-14, 2^-29 and 2^-43, each with kRound*
// on it.  With x = l - off, the exponent ah + al - x (hi + lo) is n + j / 32 + r, |r| <= 2^-6: n + j / 32 comes from its float,
// and (ah - n - j / 32) - x hi in one rounding is r but for the small parts.  2^-r - 1 is its series to r^4 (the next term is
// below 2^-39).  What errs is the float arithmetic on r and on that sum, below 2^-6: 2^-28.5 of the weight at most, 2^-31 as a
// rule, and what the three parts leave out, 2^-40.  In floats, two logits to an instruction: in whole numbers of 64 bits the
// weights of 393 rows of 151936 logits took 150 us.
constexpr float kRoundA = 768.f, kRoundB = 1.5f * 0x1p-6f, kRoundC = 1.5f * 0x1p-20f;  // 1.5 2^23 units

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }

// The parts of two weights, without and with what was added to round them.
struct Parts2 {
  float2 a, b, c, ra, rb, rc;
};
__device__ __forceinline__ Parts2 parts2(float2 l, const Scale& s, const PowerTable& powers) {
  float2 x = sub2(both(s.off), l);  // (off - l)
  x = make_float2(fminf(x.x, -s.least), fminf(x.y, -s.least));
  const float2 hi = both(s.hi), ah = both(s.ah);
  const float2 big = fma2(fma2(x, hi, ah), both(32.f), both(12582912.f));  // 1.5 2^23: its last bits are round(32 p)
  const uint32_t b0 = __float_as_uint(big.x), b1 = __float_as_uint(big.y);
  const float2 r = add2(fma2(x, hi, fma2(add2(big, both(-12582912.f)), both(-0x1p-5f), ah)), fma2(x, both(s.lo), both(s.al)));
  constexpr double k = 0.693147180559945309417232121458;
  constexpr float c1 = -k, c2 = k * k / 2, c3 = -k * k * k / 6, c4 = k * k * k * k / 24;
  const float2 e = mul2(r, fma2(r, fma2(r, fma2(r, both(c4), both(c3)), both(c2)), both(c1)));  // 2^-r - 1
  const float2 t = make_float2(powers.hi[b0 & 31u], powers.hi[b1 & 31u]);
  const float2 u = make_float2(powers.lo[b0 & 31u], powers.lo[b1 & 31u]);
  const float2 n = make_float2(__uint_as_float((127u << 23) - ((b0 & 0xfe0u) << 18)),
                               __uint_as_float((127u << 23) - ((b1 & 0xfe0u) << 18)));  // 2^-n
  const float2 v = mul2(t, n), y = mul2(fma2(t, e, u), n);
  const float2 h = add2(v, y), rest = sub2(y, sub2(h, v));
  Parts2 w;
  w.ra = add2(h, both(kRoundA));
  w.a = add2(w.ra, both(-kRoundA));
  const float2 q = add2(sub2(h, w.a), rest);
  w.rb = add2(q, both(kRoundB));
  w.b = add2(w.rb, both(-kRoundB));
  w.rc = add2(sub2(q, w.b), both(kRoundC));
  w.c = add2(w.rc, both(-kRoundC));
  return w;
}
// The units of a part, from its rounded form; a weight in whole numbers of 2^-43.
__device__ __forceinline__ int units(float part, float round) { return __float_as_int(part) - __float_as_int(round); }
__device__ __forceinline__ uint64_t whole(float ra, float rb, float rc) {
  return static_cast<uint64_t>((static_cast<int64_t>(units(ra, kRoundA)) << 29) +
                               (static_cast<int64_t>(units(rb, kRoundB)) << 14) + units(rc, kRoundC));
}
__device__ __noinline__ uint64_t weight(float l, const Scale& s, const PowerTable& powers) {  // (for the few: less code)
  const Parts2 w = parts2(both(l), s, powers);
  return whole(w.ra.x, w.rb.x, w.rc.x);
}
// The sum of at most 1000 weights (a part is 2^14 + 2^5 units at most, and floats add whole numbers below 2^24 exactly), by
// even and odd ones.
constexpr int kSumMost = 1000;
struct Sum {
  float2 a = {0.f, 0.f}, b = {0.f, 0.f}, c = {0.f, 0.f};
  __device__ __forceinline__ void add(const Parts2& w, bool x, bool y) {
    const float2 is = make_float2(x ? 1.f : 0.f, y ? 1.f : 0.f);
    a = fma2(w.a, is, a);
    b = fma2(w.b, is, b);
    c = fma2(w.c, is, c);
  }
  __device__ __forceinline__ uint64_t value() const {
    const auto one = [](float x, float y, float unit) { return static_cast<int64_t>(x * unit) + static_cast<int64_t>(y * unit); };
    return static_cast<uint64_t>((one(a.x, a.y, 0x1p14f) << 29) + (one(b.x, b.y, 0x1p29f) << 14) + one(c.x, c.y, 0x1p43f));
  }
};

// Order-preserving keys of finite logits: larger ones have larger keys, -0 and +0 the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > neg_inf())) return kNone;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// The first search's intervals are even in logits: NB of 1 / steps below the largest, the last one without an end.  (Each
// operation rounds monotonically: an interval is a range of keys.)
__device__ __forceinline__ int interval_of(float l, float top, float steps) {
  return __float_as_int(__fmaf_rn(__fsub_rn(top, l), steps, 8388608.f)) - 0x4b000000;  // (2^23: the last bit is a whole)
}
// The least and the largest key of an interval, found by a warp: either half splits its range in sixteen.
__device__ __forceinline__ void keys_of_interval(int b, float top, float steps, uint32_t& lo, uint32_t& hi) {
  const int lane = threadIdx.x & 31, half = lane >> 4;
  // the least key in interval b or before it, and before b
  uint32_t a = kLowest, z = key_of(top);
  const int most = b - half;
#pragma unroll 1
  for (int round = 0; round < 8; ++round) {  // (16^8 keys)
    const uint32_t step = (z - a) / 16 + 1;
    const uint64_t from = static_cast<uint64_t>(step) * (lane & 15);
    const uint32_t last = a + static_cast<uint32_t>(min(from + step - 1, static_cast<uint64_t>(z - a)));
    const uint32_t in = __ballot_sync(0xffffffffu, min(interval_of(logit_of(last), top, steps), NB - 1) <= most) >> (half * 16);
    const int first = max(__ffs(in & 0xffffu) - 1, 0);  // (none: before the first interval, where no key is)
    const uint32_t base = a;
    a = base + step * first;
    z = base + static_cast<uint32_t>(min(static_cast<uint64_t>(step) * (first + 1) - 1, static_cast<uint64_t>(z - base)));
  }
  lo = b < NB - 1 ? __shfl_sync(0xffffffffu, a, 0) : kLowest;
  const uint32_t next = __shfl_sync(0xffffffffu, a, 16);
  hi = b > 0 ? next - 1 : key_of(top);
}

// A temperature above 0 as it is used, for the weights and for the filtered logits.
__device__ __forceinline__ float within(float temperature) { return fminf(fmaxf(temperature, 0x1p-70f), 0x1p70f); }

// The place in the order of a logit (its bits) and an index.
__device__ __forceinline__ uint64_t place_of(uint64_t x) {
  return (static_cast<uint64_t>(~key_of(__uint_as_float(static_cast<uint32_t>(x >> 32)))) << 32) | static_cast<uint32_t>(x);
}

// A token's probability, rounded once (the two whole numbers lose no more than 2^-53 in a double; a quotient of floats was off by
// up to three roundings).  One row of 151936 logits takes 11.95 us so, 11.75 with that.
__device__ __forceinline__ float share(uint64_t weight, uint64_t total) {
  return __double2float_rn(static_cast<double>(weight) / static_cast<double>(total));
}

// floor(f s) (up: ceil) for a float 0 <= f < 1.
__device__ __forceinline__ uint64_t times(float f, uint64_t s, bool up) {
  const uint32_t b = __float_as_uint(f);
  const int ex = static_cast<int>(b >> 23);
  const uint64_t m = ex ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (ex ? ex : 1);  // f = m 2^-sh, sh >= 24
  const uint64_t lo = m * s, hi = __umul64hi(m, s);
  uint64_t v, rest;
  if (sh < 64) {
    v = (hi << (64 - sh)) | (lo >> sh);
    rest = lo << (64 - sh);
  } else if (sh < 128) {
    v = sh == 64 ? hi : hi >> (sh - 64);
    rest = lo | (sh == 64 ? 0 : hi << (128 - sh));
  } else {
    v = 0;
    rest = lo | hi;
  }
  return v + (up && rest != 0 ? 1 : 0);
}

// ---------------------------------------------------------------- shared memory of a CTA
struct Found {
  int bin, count;         // the interval, candidates in it
  int above, pad;         // candidates above it
  uint64_t mass_above;    // their weight
};
struct __align__(16) Shared {
  union {
    uint32_t hist[4 * NB];  // counts, three parts of weights
    unsigned long long order[CAP];  // (the first CTA's) the candidates: inverted key, index
  };
  unsigned long long mine[CAP];  // this CTA's candidates
  unsigned long long warps[2][W];
  unsigned long long xch[2][2][kMaxC];  // two values of every CTA, in two buffers by turns
  unsigned long long mass[kSmall];  // kept candidates' weights
  unsigned long long few[2][32];  // an interval's last candidates and their weights
  PowerTable powers;
  Found found;
  uint32_t cut_key, cut_idx;
  uint32_t lo, hi;  // an interval's keys
  uint32_t bound;  // an interval's lower end
  int n_mine, n_groups, n_few;
  unsigned long long place;
  float steps;  // intervals of the first search by a logit
  double log_min_p, per_octave;  // T ln(min_p), log2(e) / T
  Scale scale;

  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < 4 * NB; i += NT) hist[i] = 0;
  }
};

// A candidate and the three parts of its weight to an interval b of a histogram: words of 32 bits, which shared memory adds
// without an answer to wait for (a wider word it would compare and try again).  Their sums fit for 2^17 - 2^8 candidates: the
// second part of a rounded weight is between -(2^14 + 2^5) and 2^14 + 2^5.
__device__ __forceinline__ void add_one(uint32_t* hist, int b, uint32_t a, uint32_t mid, uint32_t c) {
  atomicAdd(hist + b, 1u);
  atomicAdd(hist + NB + b, a);
  atomicAdd(hist + 2 * NB + b, mid);
  atomicAdd(hist + 3 * NB + b, c);
}
__device__ __forceinline__ void add_one(uint32_t* hist, int b, uint64_t w) {
  add_one(hist, b, static_cast<uint32_t>(w >> 29), static_cast<uint32_t>(w >> 14) & 0x7fffu, static_cast<uint32_t>(w) & 0x3fffu);
}
// The same for the interval at an address, where `yes`, with the parts as rounded floats: what a float's bits are more than its
// units is taken off by the count (get_mass).
__device__ __forceinline__ void add_one_if(bool yes, uint32_t at) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(at),
               "r"(static_cast<uint32_t>(yes))
               : "memory");
}
__device__ __forceinline__ void add_one_if(bool yes, uint32_t at, float a, float mid, float c) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t"
      "@p red.shared.add.u32 [%0 + %5], %2;\n\t@p red.shared.add.u32 [%0 + %6], %3;\n\t"
      "@p red.shared.add.u32 [%0 + %7], %4;\n\t}" ::"r"(at),
      "r"(static_cast<uint32_t>(yes)), "r"(__float_as_uint(a)), "r"(__float_as_uint(mid)), "r"(__float_as_uint(c)), "n"(4 * NB), "n"(8 * NB), "n"(12 * NB)
      : "memory");
}
// Two neighbouring intervals' weights are added to m (floats: they were added as such).
__device__ __forceinline__ void get_mass(const uint32_t* hist, int b, uint64_t (&m)[2], bool floats = false) {
  uint2 a = *reinterpret_cast<const uint2*>(hist + NB + b), mid = *reinterpret_cast<const uint2*>(hist + 2 * NB + b),
        c = *reinterpret_cast<const uint2*>(hist + 3 * NB + b);
  if (floats) {
    const uint2 n = *reinterpret_cast<const uint2*>(hist + b);
    a.x -= n.x * __float_as_uint(kRoundA), a.y -= n.y * __float_as_uint(kRoundA);
    mid.x -= n.x * __float_as_uint(kRoundB), mid.y -= n.y * __float_as_uint(kRoundB);
    c.x -= n.x * __float_as_uint(kRoundC), c.y -= n.y * __float_as_uint(kRoundC);
  }
  const auto whole = [](uint32_t a, uint32_t mid, uint32_t c) {
    return (static_cast<uint64_t>(a) << 29) +
           static_cast<uint64_t>((static_cast<int64_t>(static_cast<int>(mid)) << 14) + static_cast<int>(c));
  };
  m[0] += whole(a.x, mid.x, c.x);
  m[1] += whole(a.y, mid.y, c.y);
}

// 16 bytes of logits as floats.
__device__ __forceinline__ void unpack(const uint4& x, float (&v)[4]) {
  v[0] = __uint_as_float(x.x);
  v[1] = __uint_as_float(x.y);
  v[2] = __uint_as_float(x.z);
  v[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void unpack(const uint4& x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// The largest finite number of a type; the smaller of two floats, NaN if one is.
__device__ __forceinline__ float largest(float) { return 3.402823466e38f; }
__device__ __forceinline__ float largest(__nv_bfloat16) { return __uint_as_float(0x7f7f0000u); }
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The largest of a word and a vector (of a type, as loaded), NaN passed over; no logit; the logit of such a word.
__device__ __forceinline__ uint32_t none_of(float) { return 0xff800000u; }
__device__ __forceinline__ uint32_t none_of(__nv_bfloat16) { return 0xff80ff80u; }
__device__ __forceinline__ uint32_t most_of(float, uint32_t m, const uint4& x) {
  return __float_as_uint(fmaxf(fmaxf(fmaxf(__uint_as_float(m), __uint_as_float(x.x)), __uint_as_float(x.y)),
                               fmaxf(__uint_as_float(x.z), __uint_as_float(x.w))));
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t most_of(__nv_bfloat16, uint32_t m, const uint4& x) {
  return max2(max2(max2(m, x.x), max2(m, x.y)), max2(max2(m, x.z), max2(m, x.w)));  // (m first: no NaN stays)
}
__device__ __forceinline__ float most_of(float, uint32_t m) { return __uint_as_float(m); }
__device__ __forceinline__ float most_of(__nv_bfloat16, uint32_t m) {
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
struct Row {
  static constexpr int L = 16 / sizeof(T);  // logits of a vector
  Shared& s;
  const T* src;    // the row
  bool vec;        // it is read 16 bytes at a time
  int C, rank;     // CTAs of the cluster, this one
  int begin, end;  // this warp's stretch
  int turn;        // of the exchange buffers
  float cut;        // candidates above it, and of those like it up to index cut_idx, are in
  uint32_t cut_idx;

  __device__ __forceinline__ bool in(float l, int idx) const {
    return l > cut || (l == cut && static_cast<uint32_t>(idx) <= cut_idx);
  }
  __device__ __forceinline__ void take_cut() {
    cut = logit_of(s.cut_key);
    cut_idx = s.cut_idx;
  }
  __device__ __forceinline__ void meet() {
    if (C > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  template <typename P>
  __device__ __forceinline__ P* theirs(P* p, int r) {
    return C > 1 ? cg::this_cluster().map_shared_rank(p, r) : p;
  }
  // Two values of every CTA (its first thread's), seen by all.
  __device__ __forceinline__ const unsigned long long (*exchange(uint64_t a, uint64_t b))[kMaxC] {
    turn ^= 1;
    if (static_cast<int>(threadIdx.x) < C) {
      *theirs(&s.xch[turn][0][rank], threadIdx.x) = a;
      *theirs(&s.xch[turn][1][rank], threadIdx.x) = b;
    }
    meet();
    return s.xch[turn];
  }
  // Sums of a (and b) before this thread, in thread order, and over the CTA.
  template <int N>
  __device__ __forceinline__ void sums(const uint64_t (&a)[N], uint64_t (&before)[N], uint64_t (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = a[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, x[k], o);
        if (lane >= o) x[k] += u;
      }
    }
    __syncthreads();
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < N; ++k) s.warps[k][warp] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t mine = s.warps[k][lane % W];
      uint64_t t = mine;
#pragma unroll
      for (int o = 1; o < W; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, t, o, W);
        if (lane % W >= o) t += u;
      }
      total[k] = __shfl_sync(0xffffffffu, t, W - 1);
      before[k] = __shfl_sync(0xffffffffu, t - mine, warp) + x[k] - a[k];
    }
  }
  __device__ __forceinline__ void scan(uint64_t a, uint64_t& before, uint64_t& total) {
    const uint64_t v[1] = {a};
    uint64_t b[1], t[1];
    sums(v, b, t);
    before = b[0];
    total = t[0];
  }
  __device__ __forceinline__ void scan2(uint64_t a, uint64_t b, uint64_t& before_a, uint64_t& before_b, uint64_t& total_a,
                                        uint64_t& total_b) {
    const uint64_t v[2] = {a, b};
    uint64_t u[2], t[2];
    sums(v, u, t);
    before_a = u[0];
    before_b = u[1];
    total_a = t[0];
    total_b = t[1];
  }
  // The vector of logits at i (-inf past the stretch, which ends at `end`).
  __device__ __forceinline__ void at(int i, float (&v)[L]) const { at(i, end, v); }
  __device__ __forceinline__ void at(int i, int end, float (&v)[L]) const {
    if (vec && i + L <= end) {
      unpack(*reinterpret_cast<const uint4*>(src + i), v);
    } else {
#pragma unroll
      for (int e = 0; e < L; ++e) v[e] = i + e < end ? as_float(src[i + e]) : neg_inf();
    }
#pragma unroll
    for (int e = 0; e < L; ++e) v[e] = min_nan(v[e], largest(T()));
  }
  // f(logits, index of the first) for this thread's vectors, AHEAD more on the way (1: enough where f is long, and fewer words
  // to move: the weights of 393 rows of 151936 logits take 117 us so, 135 with 4).  (Not unrolled: where a pass is a few
  // turns a warp, fetching more code takes longer than running it.)
  template <int AHEAD = 4, typename F>
  __device__ __forceinline__ void each(F f) const {
    int i = begin + (threadIdx.x & 31) * L;
    uint4 q[AHEAD];
    auto fetch = [&](uint4& x, int j) {
      if (vec && j + L <= end) x = *reinterpret_cast<const uint4*>(src + j);
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(q[d], i + d * 32 * L);
#pragma unroll 1
    for (; i < end; i += 32 * L) {
      float v[L];
      if (vec && i + L <= end) {
        unpack(q[0], v);
#pragma unroll
        for (int e = 0; e < L; ++e) v[e] = min_nan(v[e], largest(T()));
      } else {
        at(i, v);
      }
#pragma unroll
      for (int d = 0; d + 1 < AHEAD; ++d) q[d] = q[d + 1];
      fetch(q[AHEAD - 1], i + AHEAD * 32 * L);
      f(v, i);
    }
  }
};

// Of the values c[] in [lo, hi] that the threads of a CTA hold (n of them, no two alike), in ascending order, the
// first where the running count (sum of w[]: mass) reaches goal, which their total does.
template <typename T, int E>
__device__ uint64_t find(Row<T>& x, bool mass, uint64_t goal, uint64_t lo, uint64_t hi, int n, const uint64_t (&c)[E],
                         const uint64_t (&w)[E]) {
  Shared& s = x.s;
  const int tid = threadIdx.x, lane = tid & 31;
  uint64_t base = 0;
  while (n > 32) {
    const int shift = max(0, 54 - __clzll(static_cast<long long>(hi - lo)));  // (at most 1024 intervals)
    __syncthreads();
    s.clear();
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (c[e] < lo || c[e] > hi) continue;
      const int b = static_cast<int>((c[e] - lo) >> shift);
      if (mass) add_one(s.hist, b, w[e]);
      else atomicAdd(&s.hist[b], 1u);
    }
    __syncthreads();
    const uint2 k = *reinterpret_cast<const uint2*>(s.hist + 2 * tid);
    uint64_t m[2] = {k.x, k.y}, before, total;
    if (mass) {
      m[0] = m[1] = 0;
      get_mass(s.hist, 2 * tid, m);
    }
    x.scan(m[0] + m[1], before, total);
    before += base;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < goal && before + m[e] >= goal)
        s.found = Found{2 * tid + e, static_cast<int>(e ? k.y : k.x), 0, 0, before};
      before += m[e];
    }
    __syncthreads();
    const Found f = s.found;
    base = f.mass_above;
    lo += static_cast<uint64_t>(f.bin) << shift;
    hi = min(hi, lo + ((uint64_t{1} << shift) - 1));
    n = f.count;
  }
  __syncthreads();
  if (tid == 0) s.n_few = 0;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (c[e] < lo || c[e] > hi) continue;
    const int i = atomicAdd(&s.n_few, 1);
    s.few[0][i] = c[e];
    s.few[1][i] = mass ? w[e] : 1;
  }
  __syncthreads();
  if (tid < 32) {
    const uint64_t mine = lane < n ? s.few[0][lane] : 0, y = lane < n ? s.few[1][lane] : 0;
    uint64_t run = base;
    for (int j = 0; j < n; ++j)
      if (s.few[0][j] <= mine) run += s.few[1][j];
    if (lane < n && run >= goal && run - y < goal) s.place = mine;
  }
  __syncthreads();
  return s.place;
}

// One row, by the CTAs of a cluster.
// Rows of a call: all in one launch, or the ones that need their weights summed in a first, the ones with few candidates in a
// second one.
enum Rows { kAllRows, kHeavyRows, kLightRows };

template <typename T>
__device__ __forceinline__ void sample_row(const SampleParams& p, int rows) {
  // keys of a 16-bit float lie 2^16 apart or further: an interval of that many holds one at most.  (Groups' maxima are
  // counted by intervals of 2^14 keys of 32 bits, 0.016 wide for logits of 8 to 16: a thousand reach some ten below the largest)
  constexpr int kKeyBits = sizeof(T) == 2 ? 16 : 0, kFirstShift = sizeof(T) == 2 ? 16 : 14;
  constexpr int L = Row<T>::L;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = rows == kLightRows ? p.few : p.ctas;
  const int rank = static_cast<int>(blockIdx.x) % C, row = static_cast<int>(blockIdx.x) / C;
  const int set = row / p.rows_per_set;
  if (p.set_rows) {
    const int used = p.set_rows[set];
    if (used < 0 || used > p.rows_per_set) {
      if (tid == 0 && rows != kLightRows) report(p.status, VG_ERR_DEVICE_BOUNDS);
      return;
    }
    if (row - set * p.rows_per_set >= used) return;
  }
  const float temp = p.temperature ? p.temperature[set] : 1.f;
  const float top_p = p.top_p ? p.top_p[set] : 1.f;
  const float min_p = p.min_p ? p.min_p[set] : 0.f;
  int top_k = p.top_k ? p.top_k[set] : 0;
  const bool greedy = temp == 0.f;
  if (!(temp >= 0.f && temp < INFINITY) || !(top_p == top_p) || !(min_p <= 1.f)) {  // (NaN too)
    if (rank == 0 && tid == 0 && rows != kLightRows) {
      report(p.status, VG_ERR_DEVICE_BOUNDS);
      p.token[row] = -1;
      if (p.prob) p.prob[row] = 0.f;
    }
    return;
  }
  const bool light = greedy || (top_k > 0 ? top_k <= CAP : min_p > 0.f && !(top_p < 1.f));
  if (rows != kAllRows && light != (rows == kLightRows)) return;
  // Every CTA of the cluster must be running before the first write into its shared memory.
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (greedy) top_k = 1;
  if (top_k >= p.V) top_k = 0;
  const bool use_k = top_k > 0, use_p = !greedy && top_p < 1.f, use_m = !greedy && min_p > 0.f;
  const int per = ((p.V + C * W - 1) / (C * W) + 7) & ~7;  // logits of a warp
  const int first = min(p.V, (rank * W + warp) * per);
  Row<T> x{sh, reinterpret_cast<const T*>(p.logits) + row * p.logit_stride, p.vec != 0, C, rank, first,
           min(p.V, first + per), 0, -3.402823466e38f, 0xffffffffu};
  if (tid < 32) {
    sh.powers.hi[tid] = g_powers.hi[tid];
    sh.powers.lo[tid] = g_powers.lo[tid];
  }
  if (tid == 0) {
    const double t = greedy ? 1.0 : static_cast<double>(within(temp));
    sh.per_octave = 1.4426950408889634074 / t;
    sh.steps = static_cast<float>(64 / t);
    if (use_m) sh.log_min_p = t * log(static_cast<double>(min_p));
    sh.n_mine = sh.n_groups = 0;
    sh.bound = kLowest;
  }
  // the groups' maxima
  float gmax[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) gmax[g] = neg_inf();
  if (x.vec) {
    constexpr int ON = 2 * NG;  // vectors on the way
    uint4 q[ON];
    uint32_t most[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) most[g] = none_of(T());
    for (int i = x.begin + lane * L; i < x.end; i += ON * 32 * L) {
#pragma unroll
      for (int g = 0; g < ON; ++g) {
        q[g] = make_uint4(none_of(T()), none_of(T()), none_of(T()), none_of(T()));
        const int j = i + g * 32 * L;
        if (j + L <= x.end) q[g] = *reinterpret_cast<const uint4*>(x.src + j);
      }
#pragma unroll
      for (int g = 0; g < ON; ++g) most[g % NG] = most_of(T(), most[g % NG], q[g]);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) gmax[g] = most_of(T(), most[g]);
  }
  if (!x.vec || (x.end - x.begin) % L) {  // (vectors that the loop above left out)
    for (int i = x.begin + lane * L; i < x.end; i += NG * 32 * L) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int j = i + g * 32 * L;
        if (x.vec && j + L <= x.end) continue;
#pragma unroll 1
        for (int e = j; e < min(j + L, x.end); ++e) gmax[g] = fmaxf(gmax[g], as_float(x.src[e]));
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) gmax[g] = fminf(gmax[g], largest(T()));
  uint32_t gkey[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) gkey[g] = key_of(gmax[g]);
  uint32_t kmax = kNone;
#pragma unroll
  for (int g = 0; g < NG; ++g) kmax = max(kmax, gkey[g]);
  auto cta_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) sh.warps[0][warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(sh.warps[0][lane % W]));
  };
  kmax = cta_max(kmax);
  // top-k: a bound that k logits of the row reach
  uint32_t bound = kLowest;
  const bool few_k = use_k && top_k <= CAP;
  if (few_k) {
    sh.clear();
    __syncthreads();
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t d = (kmax - gkey[g]) >> kFirstShift;
      if (gkey[g] != kNone && d < NB) atomicAdd(&sh.hist[d], 1u);
    }
    __syncthreads();
    const int want = (top_k + C - 1) / C;
    const uint32_t c0 = sh.hist[2 * tid], c1 = sh.hist[2 * tid + 1];
    uint64_t before, total;
    x.scan(c0 + c1, before, total);
    const int b0 = static_cast<int>(before);
    if (b0 < want && b0 + static_cast<int>(c0 + c1) >= want) {
      const uint32_t bin = 2 * tid + (b0 + static_cast<int>(c0) >= want ? 0 : 1);
      const uint32_t down = ((bin + 1) << kFirstShift) - 1;
      sh.bound = kmax > down + kLowest ? kmax - down : kLowest;
    }
    __syncthreads();
    bound = sh.bound;
  }
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (C > 1) {
    const auto v = x.exchange(kmax, bound);
    for (int r = 0; r < C; ++r) {
      kmax = max(kmax, static_cast<uint32_t>(v[0][r]));
      bound = min(bound, static_cast<uint32_t>(v[1][r]));
    }
  }
  const bool empty = kmax == kNone;  // nothing to draw from
  const float top = logit_of(kmax);
  if (tid == 0) sh.scale = make_scale(top, sh.per_octave);
  __syncthreads();
  const Scale scale = sh.scale;
  // min-p: the smallest key it keeps
  uint32_t key_min = kLowest;
  if (use_m && !empty) {
    const float least = __double2float_ru(static_cast<double>(top) + sh.log_min_p);
    key_min = min(kmax, max(key_min, key_of(least)));
  }

  // Searches the key where the running count (weight: mass) from the largest key down reaches `goal` (of the
  // weight: p of the total, found on the way), among the candidates of the cut.  It lies in [lo, hi], above which lie
  // `above` candidates of weight mass_above.
  enum Cut { kNoCut, kFew, kFewHere, kOneKey };  // no cut; at most CAP down to lo; in [lo, hi]; one key in [lo, hi]
  uint32_t lo = kLowest, hi = kmax;
  int above = 0, here = 0;
  uint64_t goal = 0, mass_above = 0;
  auto search = [&](bool mass) -> Cut {
    lo = kLowest;
    hi = kmax;
    above = 0;
    mass_above = 0;
    int shift = 0;
    for (bool start = true;; start = false) {
      sh.clear();
      __syncthreads();
      if (start) {
        uint32_t rest = 0;
        Sum rest_sum;
        const float steps = mass ? sh.steps : 64.f;
        const bool cutting = x.cut > -3.402823466e38f;
        const uint32_t hist = smem_u32(sh.hist);
        // (without branches: of 32 logits one nearly always is in an interval)
        auto places = [&](const float (&v)[L], int i, bool (&hit)[L], bool (&low)[L], uint32_t (&at)[L]) {
#pragma unroll
          for (int e = 0; e < L; ++e) hit[e] = v[e] >= -3.402823466e38f;
          if (cutting) {
#pragma unroll
            for (int e = 0; e < L; ++e) hit[e] = x.in(v[e], i + e);
          }
#pragma unroll
          for (int e = 0; e < L; ++e) {
            const int b = interval_of(v[e], top, steps);
            low[e] = hit[e] & (b >= NB - 1);
            hit[e] = hit[e] & (b < NB - 1);
            at[e] = hist + 4 * static_cast<uint32_t>(b);
            rest += low[e];  // (much of the row: added up by thread)
          }
        };
        if (mass) {
          x.template each<1>([&](const float (&v)[L], int i) {
            bool hit[L], low[L];
            uint32_t at[L];
            places(v, i, hit, low, at);
#pragma unroll
            for (int e = 0; e < L; e += 2) {
              const Parts2 w = parts2(make_float2(v[e], v[e + 1]), scale, sh.powers);
              add_one_if(hit[e], at[e], w.ra.x, w.rb.x, w.rc.x);
              add_one_if(hit[e + 1], at[e + 1], w.ra.y, w.rb.y, w.rc.y);
              rest_sum.add(w, low[e], low[e + 1]);
            }
          });
        } else {
          x.template each<1>([&](const float (&v)[L], int i) {
            bool hit[L], low[L];
            uint32_t at[L];
            places(v, i, hit, low, at);
#pragma unroll
            for (int e = 0; e < L; ++e) add_one_if(hit[e], at[e]);
          });
        }
        rest = __reduce_add_sync(0xffffffffu, rest);
        const uint64_t rest_mass = mass ? warp_sum(rest_sum.value()) : 0;
        if (lane == 0 && rest) {
          atomicAdd(&sh.hist[NB - 1], rest);
          if (mass) {  // (the sum of the parts is whole, whatever they are)
            atomicAdd(&sh.hist[2 * NB - 1], static_cast<uint32_t>(rest_mass >> 29) + rest * __float_as_uint(kRoundA));
            atomicAdd(&sh.hist[3 * NB - 1], (static_cast<uint32_t>(rest_mass >> 14) & 0x7fffu) + rest * __float_as_uint(kRoundB));
            atomicAdd(&sh.hist[4 * NB - 1], (static_cast<uint32_t>(rest_mass) & 0x3fffu) + rest * __float_as_uint(kRoundC));
          }
        }
      } else {  // (few of the row)
        const float flo = logit_of(lo), fhi = logit_of(hi);
        x.each([&](const float (&v)[L], int i) {
#pragma unroll
          for (int e = 0; e < L; ++e) {
            if (!(v[e] >= flo && v[e] <= fhi) || !x.in(v[e], i + e)) continue;
            const uint32_t b = (hi - key_of(v[e])) >> shift;
            if (mass) add_one(sh.hist, b, weight(v[e], scale, sh.powers));
            else atomicAdd(&sh.hist[b], 1u);
          }
        });
      }
      x.meet();
      // this CTA's share of the intervals, summed over the cluster: a thread takes two of one CTA's, C neighbouring
      // threads the same two
      const int b = (rank * (NT / C) + tid / C) * 2;
      uint64_t n[2], m[2] = {0, 0};
      {
        const uint32_t* theirs = x.theirs(sh.hist, tid % C);
        const uint2 c = *reinterpret_cast<const uint2*>(theirs + b);
        n[0] = c.x;
        n[1] = c.y;
        if (mass) get_mass(theirs, b, m, start);
      }
      for (int o = 1; o < C; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          n[k] += __shfl_xor_sync(0xffffffffu, n[k], o);
          m[k] += __shfl_xor_sync(0xffffffffu, m[k], o);
        }
      }
      const bool one = tid % C == 0;
      uint64_t bn, bm, tn, tm;
      x.scan2(one ? n[0] + n[1] : 0, one ? m[0] + m[1] : 0, bn, bm, tn, tm);
      const auto v = x.exchange(tn, tm);
      uint64_t sum_n = 0, sum_m = 0;
      for (int r = 0; r < C; ++r) {
        if (r == rank) {
          bn += sum_n;
          bm += sum_m;
        }
        sum_n += v[0][r];
        sum_m += v[1][r];
      }
      if (start && mass) goal = max(times(fmaxf(top_p, 0.f), sum_m, true), uint64_t{1});
      if (start && !mass && sum_n <= goal) return kNoCut;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint64_t have = mass ? mass_above + bm : above + bn, add = mass ? m[k] : n[k];
        if (one && have < goal && have + add >= goal) {
          const Found f{b + k, static_cast<int>(n[k]), above + static_cast<int>(bn), 0, mass_above + bm};
          for (int r = 0; r < C; ++r) *x.theirs(&sh.found, r) = f;
        }
        bn += n[k];
        bm += m[k];
      }
      x.meet();
      const Found f = sh.found;
      above = f.above;
      here = f.count;
      mass_above = f.mass_above;
      if (start) {
        if (warp == 0) {
          keys_of_interval(f.bin, top, mass ? sh.steps : 64.f, lo, hi);
          if (lane == 0) {
            sh.lo = lo;
            sh.hi = hi;
          }
        }
        __syncthreads();
        lo = sh.lo;
        hi = sh.hi;
      } else {
        hi -= static_cast<uint32_t>(f.bin) << shift;
        const uint32_t width = (1u << shift) - 1;
        if (hi - lo > width) lo = hi - width;
      }
      if (above + here <= CAP) return kFew;
      if (here <= CAP) return kFewHere;
      if (hi - lo <= (1u << kKeyBits) - 1) return kOneKey;
      shift = kKeyBits;
      while ((hi - lo) >> shift >= NB) ++shift;
    }
  };
  // The sum of every thread's n in the warps before this one, by index, and over the cluster.
  auto sum_before = [&](uint64_t n, uint64_t& total) {
    n = warp_sum(n);
    uint64_t before, t;
    x.scan(lane == 0 ? n : 0, before, t);
    before = __shfl_sync(0xffffffffu, before, 0);
    const auto v = x.exchange(t, 0);
    total = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before += total;
      total += v[0][r];
    }
    return before;
  };
  // The first of this warp's logits, by index, where the running sum of f exceeds q; `run` before them.
  auto first_past = [&](uint64_t run, uint64_t q, auto f, auto found) {
    for (int i0 = x.begin; i0 < x.end; i0 += 32 * L) {
      float v[L];
      x.at(i0 + lane * L, v);
      uint64_t y[L], sum = 0;
#pragma unroll
      for (int e = 0; e < L; ++e) sum += y[e] = f(v[e], i0 + lane * L + e);
      uint64_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const uint64_t here = run + incl - sum, all = run + __shfl_sync(0xffffffffu, incl, 31);
      if (q < all) {
        if (here <= q && q < here + sum) {
          uint64_t r = here;
#pragma unroll
          for (int e = 0; e < L; ++e) {
            if (r <= q && q < r + y[e]) found(v[e], i0 + lane * L + e, y[e]);
            r += y[e];
          }
        }
        return;
      }
      run = all;
    }
  };
  // The cut at the q-th (1 ..) candidate, by index, of those with keys in [lo, hi] (all the same key).
  auto cut_ties = [&](uint64_t q) {
    const float flo = logit_of(lo), fhi = logit_of(hi);
    auto tie = [&](float l, int idx) { return static_cast<uint64_t>(l >= flo && l <= fhi && x.in(l, idx)); };
    uint64_t n = 0, total;
    x.each([&](const float (&v)[L], int i) {
#pragma unroll
      for (int e = 0; e < L; ++e) n += tie(v[e], i + e);
    });
    const uint64_t before = sum_before(n, total);
    n = warp_sum(n);
    if (before < q && before + n >= q) {
      first_past(before, q - 1, tie, [&](float l, int idx, uint64_t) {
        for (int r = 0; r < C; ++r) {
          *x.theirs(&sh.cut_key, r) = key_of(l);
          *x.theirs(&sh.cut_idx, r) = static_cast<uint32_t>(idx);
        }
      });
    }
    x.meet();
    x.take_cut();
  };
  // This CTA's candidates of [from, to] (logit, index), unsorted, in its mine[]; how many (more than CAP: the rest are not there):
  // from the groups whose maximum is among them, which are listed and then read by all threads.
  auto collect = [&](uint32_t from, uint32_t to) {
    const float flo = logit_of(from), fhi = logit_of(to);
    const bool cutting = x.cut > -3.402823466e38f;
    uint16_t* groups = reinterpret_cast<uint16_t*>(sh.hist);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const bool is = gkey[g] >= from && gkey[g] != kNone;
      const uint32_t who = __ballot_sync(0xffffffffu, is);
      int at = 0;
      if (lane == 0 && who) at = atomicAdd(&sh.n_groups, __popc(who));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
      if (is) groups[at] = static_cast<uint16_t>(g * NT + tid);
    }
    __syncthreads();
    const int vectors = (per + NG * 32 * L - 1) / (NG * 32 * L), n_vectors = sh.n_groups * vectors;  // (of a group, of all)
    const uint32_t inverse = 0xffffffffu / vectors + 1;  // (e / vectors for e < 2^16)
    static_assert(NT * NG * (1 + (1 << 17) / (NT * NG * L)) < 1 << 16, "a CTA has at most 2^17 logits, in NT NG groups");
    for (int e = tid; e - lane < n_vectors; e += NT) {
      const int which = vectors == 1 ? e : __umulhi(e, inverse), group = e < n_vectors ? groups[which] : 0, whose = group % NT;
      const int begin = min(p.V, (rank * W + whose / 32) * per), end = min(p.V, begin + per);
      const int i = e < n_vectors ? begin + ((e - which * vectors) * NG * 32 + group / NT * 32 + whose % 32) * L : end;
      float v[L];
      x.at(i, end, v);
      uint32_t mine = 0;
#pragma unroll
      for (int k = 0; k < L; ++k) mine |= static_cast<uint32_t>((v[k] >= flo) & (v[k] <= fhi)) << k;
      if (cutting) {
#pragma unroll
        for (int k = 0; k < L; ++k) mine &= ~(static_cast<uint32_t>(!x.in(v[k], i + k)) << k);
      }
      if (!__any_sync(0xffffffffu, mine)) continue;
      int at = __popc(mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
      }
      int base = 0;
      if (lane == 31) base = atomicAdd(&sh.n_mine, at);
      at += __shfl_sync(0xffffffffu, base, 31) - __popc(mine);
#pragma unroll
      for (int k = 0; k < L; ++k) {
        if ((mine >> k & 1) && at < CAP)
          sh.mine[at] = (static_cast<uint64_t>(__float_as_uint(v[k])) << 32) | static_cast<uint32_t>(i + k);
        at += mine >> k & 1;
      }
    }
    __syncthreads();
    const int n = sh.n_mine;
    __syncthreads();
    if (tid == 0) sh.n_mine = sh.n_groups = 0;
    return n;
  };
  // Every candidate from `from` up in the first CTA's order[]; how many, or -1: more than CAP.
  uint32_t least = 0;
  auto gather = [&](uint32_t from) {
    least = from;
    const int n = collect(from, kmax);
    const auto v = x.exchange(n, 0);
    int all = 0, before = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = all;
      all += static_cast<int>(v[0][r]);
    }
    if (all > CAP) return -1;
    unsigned long long* dst = x.theirs(sh.order, 0);
    for (int i = tid; i < n; i += NT) dst[before + i] = place_of(sh.mine[i]);
    x.meet();
    return all;
  };
  // This thread's of `all` candidates and their weights.
  constexpr int E = CAP / NT;
  uint64_t c[E], w[E];
  auto load = [&](const unsigned long long* from, int all, bool logits) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = tid + e * NT;
      c[e] = i < all ? logits ? place_of(from[i]) : from[i] : ~uint64_t{0};
      w[e] = i < all ? weight(logit_of(~static_cast<uint32_t>(c[e] >> 32)), scale, sh.powers) : 0;
    }
  };
  auto first_of = [](uint32_t key) { return static_cast<uint64_t>(~key) << 32; };  // a key's first and last place
  auto last_of = [](uint32_t key) { return (static_cast<uint64_t>(~key) << 32) | 0xffffffffu; };
  auto send_cut = [&](uint64_t place) {
    if (tid < C) {
      *x.theirs(&sh.cut_key, tid) = ~static_cast<uint32_t>(place >> 32);
      *x.theirs(&sh.cut_idx, tid) = static_cast<uint32_t>(place);
    }
  };
  // Whether every CTA's candidates from lo up fit its list: then they are in c and w, else the ones of [lo, hi] are.
  auto hold = [&] {
    int n = 0;
    bool fit = above + here <= CAP * C;
    if (fit) {
      n = collect(lo, kmax);
      const auto v = x.exchange(n, 0);
      for (int r = 0; r < C; ++r) fit = fit && v[0][r] <= CAP;
    }
    if (!fit) n = collect(lo, hi);
    load(sh.mine, n, true);
    return fit;
  };
  // The cut among the `here` candidates of [lo, hi] where count or weight reaches q: the first CTA gets them all.
  auto cut_here = [&](bool mass, uint64_t q) {
    const bool fit = hold();
    uint64_t k = 0, before, total;
#pragma unroll
    for (int e = 0; e < E; ++e) k += c[e] >= first_of(hi) && c[e] <= last_of(lo);
    x.scan(k, before, total);
    const auto v = x.exchange(total, 0);
    for (int r = 0; r < rank; ++r) before += v[0][r];
    unsigned long long* dst = x.theirs(sh.order, 0);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c[e] >= first_of(hi) && c[e] <= last_of(lo)) dst[before++] = c[e];
    x.meet();
    if (rank == 0) {
      uint64_t c2[E], w2[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = tid + e * NT;
        c2[e] = i < here ? sh.order[i] : ~uint64_t{0};
        w2[e] = mass && i < here ? weight(logit_of(~static_cast<uint32_t>(c2[e] >> 32)), scale, sh.powers) : 0;
      }
      send_cut(find<T, E>(x, mass, q, first_of(hi), last_of(lo), here, c2, w2));
    }
    x.meet();
    x.take_cut();
    return fit;
  };
  const float u = p.u[row];
  auto mark_of = [&](uint64_t sum) { return u >= 1.f ? sum - 1 : times(u > 0.f ? u : 0.f, sum, false); };
  int all = -1;       // candidates gathered in the first CTA: all that may be kept
  bool held = false;  // or each CTA has its own
  if (!empty) {
    if (few_k) all = gather(use_p ? bound : max(bound, key_min));
    else if (use_m && !use_k && !use_p) all = gather(key_min);
    if (all < 0 && use_k) {
      goal = top_k;
      const Cut cut = search(false);
      if (cut == kFew) {
        all = gather(lo);
      } else if (cut != kNoCut) {
        if (cut == kOneKey) cut_ties(goal - above);
        else held = cut_here(false, goal - above);
      }
      goal = 0;
    }
    if (all < 0 && use_p) {
      const Cut cut = search(true);
      if (cut == kFew || key_min > lo) all = gather(max(lo, key_min));
      if (all < 0) {
        // ties of one weight: as many as reach the goal
        const float l = logit_of(!kKeyBits ? lo : hi >> 31 ? hi & 0xffff0000u : lo | 0xffffu);
        const uint64_t y = weight(l, scale, sh.powers), q = goal - mass_above;
        if (cut == kOneKey) cut_ties(y ? (q + y - 1) / y : 1);
        else held = cut_here(true, q);
      }
    }
  }
  if (all >= 0 && all <= kSmall) {
    if (rank == 0) {
      // a thread a candidate: its rank is how many stand before it
      const uint64_t mine = tid < all ? sh.order[tid] : ~uint64_t{0};
      int r = 0;
      if (tid < all) {
#pragma unroll 4
        for (int j = 0; j < all; ++j) r += sh.order[j] < mine;
        sh.mine[r] = mine;
      }
      __syncthreads();
      // from here on thread t has the one of rank t
      const uint64_t place = tid < all ? sh.mine[tid] : ~uint64_t{0};
      const bool ranked = tid < all && (!use_k || tid < top_k);
      const uint64_t y = ranked ? weight(logit_of(~static_cast<uint32_t>(place >> 32)), scale, sh.powers) : 0;
      uint64_t before, sum;
      x.scan(y, before, sum);
      if (use_p && goal == 0) goal = max(times(fmaxf(top_p, 0.f), sum, true), uint64_t{1});
      const bool keep = ranked && (!use_p || before < goal) && (tid == 0 || place <= last_of(key_min));
      const int kept = __syncthreads_count(keep);  // (a first part)
      if (tid == kept - 1) sh.place = before + y;
      if (p.filtered) send_cut(sh.mine[kept - 1]);  // (without, the other CTAs are gone)
      if (tid < kept) {
        sh.order[tid] = place & 0xffffffffu;
        sh.mass[tid] = y;
      }
      __syncthreads();
      const uint64_t total = sh.place, mark = mark_of(total);
      if (tid < kept) {
        const uint64_t idx = place & 0xffffffffu;
        uint64_t run = 0;
#pragma unroll 4
        for (int j = 0; j < kept; ++j) run += sh.order[j] < idx ? sh.mass[j] : 0;
        if (run <= mark && mark < run + y) {
          p.token[row] = static_cast<int32_t>(idx);
          if (p.prob) p.prob[row] = share(y, total);
        }
      }
    }
    if (!p.filtered) return;  // (nobody touches another CTA's memory any more)
    x.meet();
    x.take_cut();
  } else if (all >= 0) {
    if (rank == 0) {
      load(sh.order, all, false);
      const uint64_t lowest = first_of(kmax), highest = last_of(least);
      uint64_t cut = highest;
      if (use_k && all > top_k) cut = find<T, E>(x, false, top_k, lowest, highest, all, c, w);
      auto inside = [&](uint64_t& sum) {  // candidates up to the cut and their weight; the others' become 0
        uint64_t n = 0, z0, z1, k = 0;
        sum = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (c[e] > cut) w[e] = 0;
          else n += c[e] != ~uint64_t{0};
          sum += w[e];
        }
        x.scan2(n, sum, z0, z1, k, sum);
        return static_cast<int>(k);
      };
      uint64_t sum;
      int n = inside(sum);
      if (use_p) {
        if (goal == 0) goal = max(times(fmaxf(top_p, 0.f), sum, true), uint64_t{1});
        // (what lies below min-p's bound may not have been gathered: then top-p cuts nothing more)
        if (goal <= sum) cut = find<T, E>(x, true, goal, lowest, min(highest, cut), n, c, w);
      }
      cut = min(cut, last_of(key_min));
      if (p.filtered) send_cut(cut);  // (without, the other CTAs are gone)
      n = inside(sum);
      // the draw, by index
      uint64_t index[E];
#pragma unroll
      for (int e = 0; e < E; ++e) index[e] = c[e] <= cut ? c[e] & 0xffffffffu : ~uint64_t{0};
      const uint64_t token = find<T, E>(x, true, mark_of(sum) + 1, 0, p.V - 1, n, index, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (index[e] == token) {
          p.token[row] = static_cast<int32_t>(token);
          if (p.prob) p.prob[row] = share(w[e], sum);
        }
      }
    }
    if (!p.filtered) return;  // (nobody touches another CTA's memory any more)
    x.meet();
    x.take_cut();
  } else if (!empty) {
    if (logit_of(key_min) > x.cut) {
      x.cut = logit_of(key_min);
      x.cut_idx = 0xffffffffu;
    }
    if (held) {
      // each CTA has its candidates; the draw is the CTA's where the running sum passes the mark
      const uint64_t cut = first_of(key_of(x.cut)) | x.cut_idx;
      uint64_t index[E], n = 0, sum = 0, z0, z1, mine, count;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool is = c[e] <= cut;
        index[e] = is ? c[e] & 0xffffffffu : ~uint64_t{0};
        w[e] = is ? w[e] : 0;
        n += is;
        sum += w[e];
      }
      x.scan2(n, sum, z0, z1, count, mine);
      const auto v = x.exchange(mine, 0);
      uint64_t before = 0, total = 0;
      for (int r = 0; r < C; ++r) {
        if (r == rank) before = total;
        total += v[0][r];
      }
      const uint64_t mark = mark_of(total);
      if (before <= mark && mark < before + mine) {
        const uint64_t token = find<T, E>(x, true, mark - before + 1, 0, p.V - 1, static_cast<int>(count), index, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (index[e] == token) {
            p.token[row] = static_cast<int32_t>(token);
            if (p.prob) p.prob[row] = share(w[e], total);
          }
        }
      }
    } else {
      auto mass = [&](float l, int idx) { return x.in(l, idx) ? weight(l, scale, sh.powers) : uint64_t{0}; };
      Sum part;
      uint64_t total;
      x.template each<1>([&](const float (&v)[L], int i) {
#pragma unroll
        for (int e = 0; e < L; e += 2)
          part.add(parts2(make_float2(v[e], v[e + 1]), scale, sh.powers), x.in(v[e], i + e), x.in(v[e + 1], i + e + 1));
      });
      uint64_t sum = part.value();
      const uint64_t before = sum_before(sum, total), mark = mark_of(total);
      sum = warp_sum(sum);
      if (before <= mark && mark < before + sum) {
        first_past(before, mark, mass, [&](float, int idx, uint64_t y) {
          p.token[row] = idx;
          if (p.prob) p.prob[row] = share(y, total);
        });
      }
    }
  } else if (rank == 0 && tid == 0) {
    report(p.status, VG_ERR_DEVICE_BOUNDS);
    p.token[row] = -1;
    if (p.prob) p.prob[row] = 0.f;
  }
  if (!p.filtered) return;
  // (a kept logit stays finite: what takes -inf for a token that was cut, and +inf for no distribution, reads these rows)
  constexpr float kMost = 3.402823466e38f;
  const float t = within(temp);
  float* dst = p.filtered + row * p.filtered_stride;
  x.each([&](const float (&v)[L], int i) {
    float f[L];
#pragma unroll
    for (int e = 0; e < L; ++e)
      f[e] = empty || !x.in(v[e], i + e) ? neg_inf() : greedy ? 0.f : fminf(fmaxf(__fdiv_rn(v[e], t), -kMost), kMost);
    if (p.vec_out && i + L <= x.end) {
#pragma unroll
      for (int e = 0; e < L; e += 4)
        *reinterpret_cast<float4*>(dst + i + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < L; ++e)
        if (i + e < x.end) dst[i + e] = f[e];
    }
  });
}

template <typename T>
__global__ void __launch_bounds__(NT, 2) sample_kernel(const SampleParams p, int rows) {
  // (the second launch starts when all CTAs of the first one have had everything before them; it needs nothing of the
  // first one's, but must not end before it)
  if (rows != kLightRows) pdl_wait();
  pdl_launch_dependents();
  sample_row<T>(p, rows);
  if (rows == kLightRows) pdl_wait();
}

template <typename T>
cudaError_t launch_rows(const SampleParams& p, int rows, cudaStream_t stream) {
  const int ctas = rows == kLightRows ? p.few : p.ctas;
  cudaError_t e;
  if (ctas > 8) {
    static std::atomic<int> nonportable[64] = {};  // (set once per device; any thread)
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!nonportable[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      nonportable[dev].store(1, std::memory_order_release);
    }
  }
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_rows) * ctas);
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p, rows);
}

template <typename T>
cudaError_t launch_sample_t(const SampleParams& p, cudaStream_t stream) {
  if (p.few == p.ctas) return launch_rows<T>(p, kAllRows, stream);
  const cudaError_t e = launch_rows<T>(p, kHeavyRows, stream);
  return e != cudaSuccess ? e : launch_rows<T>(p, kLightRows, stream);
}

}  // namespace

// One or two CTAs a row for many rows, whose passes then overlap; four as long as all rows' are resident at once, and up to 16
// while they fill half of the SMs: 8 rows of 151936 logits take 11.7 us on 8 CTAs each and 14.3 on 16, 16 rows 12.3 on 4 and
// 13.4 on 8, 120 rows 26.3 on 2 and 32.2 on 4.  Rows that need every weight take several times as long as ones with few
// candidates: they are given four CTAs (120 rows: 144 us, on two 175) in a launch of their own, before the others', which
// fill up what they leave.
void sample_ctas(int V, int n_rows, int sms, int* ctas, int* few) {
  constexpr int kMostOfACta = (1 << 17) - (1 << 9);  // (see add_one; a warp's share is rounded up to 8)
  static_assert(kMostOfACta <= NT * (kSumMost - 16), "and a thread's weights are few enough for a Sum");
  int least = 1;
  while (V > least * kMostOfACta) least *= 2;
  int most = least;
  while (most < kMaxC && V > most * 4096) most *= 2;
  int c = max(least, min(most, n_rows <= 8 * sms ? 2 : 1));
  while (c < most && 2 * c * n_rows <= (c < 4 ? 2 * sms : sms / 2)) c *= 2;
  *few = c;
  *ctas = max(c, min(most, 4));
}

cudaError_t launch_sample(const SampleParams& p, cudaStream_t stream) {
  return p.bf16 ? launch_sample_t<__nv_bfloat16>(p, stream) : launch_sample_t<float>(p, stream);
}

}  // namespace vg
