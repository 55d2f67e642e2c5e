// Verification of drafted tokens against the target's probabilities, from
// given random numbers, with the log-probabilities of the tokens that stand.
//
//   p = softmax(x / T), q = softmax(y / T) (without draft logits: 1 at the draft)
//   draft d of a row stands if u q(d) < p(d); at the first that does not the
//   sequence gets a token from w = max(p - q, 0) instead (without draft
//   logits: p without d), after the last draft one from w = p:
//   the first index whose cumulated w exceeds u' times the whole of w.
//   T = 0: a draft stands if it is the largest logit's first index, and that is the token.
//
// All rows are read once, which is what the call cannot do without: 2 or 4
// bytes a logit and one exponential each.  Three launches, four for large calls:
//   rows     a CTA per (row, slice of the vocabulary): the slice's maximum and
//            the sum relative to it
//   stop     a CTA per entry: tests its drafts (in small calls the next launch
//            does, every part alike, which costs less)
//   weights  a CTA per (entry, part of the vocabulary): sums what the part weighs
//            in the row where the entry stopped, run by run; the row, or pair of
//            rows, is read again, in part from L2
//   draw     a CTA per entry: the run that holds the place drawn, and the token
//            in it (the whole row where p and q nearly agree)
//
// Measured (GB300): 128 entries of 0 to 4 drafts over 201088 bf16 logits 95 us
// (255 MB, 38 us at the copy rate): rows 42, tests 6, weights 39 (300
// instructions per 32 vectors of both rows, and entries that have nothing to draw
// beside others that have), draw 8.  48 entries of up to 7 looked-up drafts over 100003 fp16 34 us,
// one entry with 3 drafts over 50257 fp32 17.5 us: the chains of loads of the
// launches, which wait for one another on the device.
//
// Arithmetic.  Where the tests are concerned fp32 sums do: a test is decided
// wrongly only where u q and p agree to some 2^-22.  The draw is another
// matter: among 200 k cumulated masses one border or another lies within 2^-24
// of every place, so the masses are 64-bit fixed point in units of 2^-40 of
// the whole (one rounding a vector of 16 bytes), and
//   - the exponent is kept in two parts (x - max times log2 e / T loses 2^-24
//     of up to 20 otherwise), which leaves the hardware exponential's error,
//     some 2^-23 of the mass;
//   - masses from 2^-12 of the whole on, of which there are few, are listed and
//     take an exponential of two fp32 parts (off by 2^-40 of itself);
//   - max(p - q, 0) needs the ratio of the two sums as exactly: they are
//     summed again in the same way from the two rows; weights are taken with the
//     fp32 sums' ratio and corrected by what that is off, and where little is
//     left of them the draw takes them again with the exact one.
// Integer sums are the same in every order.  FP64 is not used: its rate on this
// GPU would cost more than all the rest.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace {

typedef unsigned long long u64;

constexpr float kLowest = -3.402823466e38f;  // fp32's lowest finite value

template <int kType>
struct Elem;
template <>
struct Elem<0> {
  typedef float T;
  static constexpr int kVec = 4;
  static SA_DEV void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static SA_DEV float largest(uint4 v) {
    return fmaxf(fmax3(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)), __uint_as_float(v.w));
  }
  static SA_DEV float one(T v) { return v; }
  static SA_DEV T lowest() { return -INFINITY; }
};
template <>
struct Elem<1> {
  typedef uint16_t T;
  static constexpr int kVec = 8;
  static SA_DEV void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static SA_DEV float largest(uint4 v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static SA_DEV uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static SA_DEV float one(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static SA_DEV T lowest() { return 0xff80u; }
};
template <>
struct Elem<2> {
  typedef uint16_t T;
  static constexpr int kVec = 8;
  static SA_DEV void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static SA_DEV float largest(uint4 v) {
    const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmaxf(f.x, f.y);
  }
  static SA_DEV uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static SA_DEV float one(T v) { return __half2float(*reinterpret_cast<const __half*>(&v)); }
  static SA_DEV T lowest() { return 0xfc00u; }
};

SA_DEV float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
SA_DEV int warp_min(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <class T>
SA_DEV T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The softmax's scale log2 e / T in two parts.  Valid temperatures: 0 (greedy,
// with the probabilities of temperature 1) up to 1e36.
struct Scale {
  float hi, lo, temperature;
  bool valid, greedy;
  SA_DEV explicit Scale(float t) {
    valid = t >= 0.f && t <= 1e36f;
    greedy = t == 0.f;
    temperature = greedy || !valid ? 1.f : t;
    constexpr float kLog2eLo = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
    const float q = __fdiv_rn(kLog2e, temperature);
    hi = fminf(q, 1e38f);
    lo = q < 1e38f ? __fdiv_rn(fmaf(-q, temperature, kLog2e) + kLog2eLo, temperature) : 0.f;
  }
};

// ---------------------------------------------------------------- all rows
constexpr int kStatThreads = 256;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kStatVecs = 4;       // 16-byte vectors that a thread works on, and as many that are on their way
constexpr int kStatPerSm = 4;      // CTAs that an SM holds
constexpr int kStatMostVecs = 32;  // vectors of a thread, at most about (more slices where rows are few)

// A thread's running sum of 2^((x - top) scale).
struct Running {
  float top, sum;
};

// Adds the vectors a thread holds.
template <int kType>
SA_DEV void add_powers(Running& r, const uint4 (&w)[kStatVecs], float scale) {
  typedef Elem<kType> E;
  float top = r.top;
#pragma unroll
  for (int i = 0; i < kStatVecs; ++i) top = fmaxf(top, E::largest(w[i]));
  const float by = (r.top - top) * scale;
  r.sum *= ex2(by);
  r.top = top;
  float2 sum = make_float2(0.f, 0.f);
  const float2 s2 = make_float2(scale, scale);
  const float ref = top * scale;
  if (fabsf(ref) < 1048576.f) {
    // one fused x scale - ref, put right at the end for what ref was rounded by
    const float2 minus = make_float2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < kStatVecs; ++i) {
      float f[E::kVec];
      E::unpack(w[i], f);
#pragma unroll
      for (int e = 0; e < E::kVec; e += 2) {
        const float2 t = ffma2(make_float2(f[e], f[e + 1]), s2, minus);
        sum = fadd2(sum, make_float2(ex2(t.x), ex2(t.y)));
      }
    }
    r.sum += (sum.x + sum.y) * ex2(-fmaf(top, scale, -ref));
    return;
  }
  // where ref's rounding would swamp the exponent the difference comes first
  const float2 minus = make_float2(-top, -top);
#pragma unroll
  for (int i = 0; i < kStatVecs; ++i) {
    float f[E::kVec];
    E::unpack(w[i], f);
#pragma unroll
    for (int e = 0; e < E::kVec; e += 2) {
      const float2 t = fmul2(fadd2(make_float2(f[e], f[e + 1]), minus), s2);
      sum = fadd2(sum, make_float2(ex2(t.x), ex2(t.y)));
    }
  }
  r.sum += sum.x + sum.y;
}

// CTA: slice `slice` (`turns` x kStatThreads vectors) of target row or draft
// `index`.  The row is on its way while the first warp finds the sequence that
// it belongs to.
template <int kType>
__global__ void __launch_bounds__(kStatThreads, kStatPerSm) verify_rows_kernel(const VerifyArgs a, int slices, int turns) {
  typedef Elem<kType> E;
  typedef typename E::T T;
  __shared__ float4 red[kStatWarps];
  __shared__ int seq_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / slices, slice = blockIdx.x - item * slices;
  const bool draft = item >= a.rows;
  const int index = draft ? item - a.rows : item;
  const T* x = draft ? static_cast<const T*>(a.draft_logits) + static_cast<int64_t>(index) * a.draft_stride
                     : static_cast<const T*>(a.logits) + static_cast<int64_t>(index) * a.stride;

  // 16-byte vectors as they are aligned in memory, what is outside the row -inf
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % E::kVec);
  const T* base = x - shift;
  const int end = shift + a.vocab, whole0 = shift > 0, whole1 = end / E::kVec;  // vectors that are whole
  const int v0 = slice * turns * kStatThreads, v1 = min(v0 + turns * kStatThreads, (end + E::kVec - 1) / E::kVec);
  const auto load = [&](int v) {
    union {
      uint4 q;
      T t[E::kVec];
    } part;
    if (v >= whole0 && v < min(whole1, v1)) return __ldg(reinterpret_cast<const uint4*>(base) + v);
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) {
      const int at = v * E::kVec + e;
      part.t[e] = v < v1 && at >= shift && at < end ? base[at] : E::lowest();
    }
    return part.q;
  };
  const auto load_some = [&](int v, uint4 (&w)[kStatVecs]) {
    if (v - tid >= whole0 && v - tid + kStatVecs * kStatThreads <= min(whole1, v1)) {
      const uint4* from = reinterpret_cast<const uint4*>(base) + v;
#pragma unroll
      for (int i = 0; i < kStatVecs; ++i) w[i] = __ldg(from + i * kStatThreads);
    } else {
#pragma unroll
      for (int i = 0; i < kStatVecs; ++i) w[i] = load(v + i * kStatThreads);
    }
  };
  uint4 w[kStatVecs];
  load_some(v0 + tid, w);
  if (warp == 0) {
    // the sequences that end at or before the row, or (one draft fewer than rows each) before the draft
    const int first = a.cu[0];
    int seqs = 0, behind = 0;
    for (int j0 = 0; j0 < a.num_seqs; j0 += 32) {
      const int j = j0 + lane;
      int rows = 0, upto = 0x7fffffff;
      if (j < a.num_seqs) {
        upto = a.cu[j + 1];
        rows = upto - a.cu[j];
      }
      if (draft) {
        const uint32_t full = __ballot_sync(0xffffffffu, rows > 0);
        if (j < a.num_seqs) upto -= first + behind + __popc(full & (2u << lane) - 1u);
        behind += __popc(full);
      }
      const uint32_t done = __ballot_sync(0xffffffffu, j < a.num_seqs && upto <= index);
      seqs += __popc(done);
      if (done != 0xffffffffu) break;
    }
    if (!draft && index < first) seqs = a.num_seqs;
    if (lane == 0) seq_sh = seqs;
  }
  __syncthreads();
  const int b = seq_sh;
  if (b >= a.num_seqs || (a.live != nullptr && a.live[b] < 0)) return;  // a row of no entry, or of one that was not served
  const Scale sc(a.temperature[b]);
  if (!sc.valid || (draft && sc.greedy)) return;
  Running r{kLowest, 0.f};
  int arg = 0x7fffffff;
  for (int v = v0 + tid;; v += kStatVecs * kStatThreads) {
    const bool more = v - tid + kStatVecs * kStatThreads < v1;
    uint4 next[kStatVecs];
    if (more) load_some(v + kStatVecs * kStatThreads, next);  // on their way meanwhile
    const float before = r.top;
    add_powers<kType>(r, w, sc.hi);
    if (sc.greedy && (r.top > before || arg == 0x7fffffff)) {  // the first of the largest so far
      arg = 0x7fffffff;
#pragma unroll
      for (int i = kStatVecs - 1; i >= 0; --i) {
        float f[E::kVec];
        E::unpack(w[i], f);
#pragma unroll
        for (int e = E::kVec - 1; e >= 0; --e)
          if (f[e] == r.top) arg = (v + i * kStatThreads) * E::kVec + e - shift;
      }
    }
    if (!more) break;
#pragma unroll
    for (int i = 0; i < kStatVecs; ++i) w[i] = next[i];
  }
  const float top = warp_max(r.top);
  const float sum = warp_sum(r.sum * ex2((r.top - top) * sc.hi));
  if (sc.greedy) arg = warp_min(r.top == top ? arg : 0x7fffffff);
  if (lane == 0) red[warp] = make_float4(top, sum, __int_as_float(arg), 0.f);
  __syncthreads();
  if (tid != 0) return;
  float4 all = red[0];
#pragma unroll
  for (int i = 1; i < kStatWarps; ++i) all.x = fmaxf(all.x, red[i].x);
  all.y = 0.f;
  arg = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < kStatWarps; ++i) {
    const float4 f = red[i];
    all.y += f.y * ex2((f.x - all.x) * sc.hi);
    if (f.x == all.x) arg = min(arg, __float_as_int(f.z));
  }
  all.z = __int_as_float(arg);
  a.parts[static_cast<int64_t>(item) * slices + slice] = all;
}

// ---------------------------------------------------------------- exponentials
// 2^(k / 16) in two parts, from repeated square roots.
constexpr double root2(double x) {  // Newton's iteration, x in [1, 2]
  double r = x;
  for (int i = 0; i < 40; ++i) r = 0.5 * (r + x / r);
  return r;
}
struct Powers {
  float hi[16], lo[16];
  constexpr Powers() : hi(), lo() {
    const double step = root2(root2(root2(root2(2.0))));
    double v = 1.0;
    for (int k = 0; k < 16; ++k) {
      hi[k] = static_cast<float>(v);
      lo[k] = static_cast<float>(v - static_cast<double>(hi[k]));
      v *= step;
    }
  }
};
__constant__ Powers kPowers{};

struct Pair {
  float hi, lo;
};

// a - b, and what it was rounded by.
SA_DEV Pair minus(float a, float b) {
  const float d = __fadd_rn(a, -b), c = __fadd_rn(d, -a);
  return {d, __fadd_rn(__fadd_rn(a, -__fadd_rn(d, -c)), -__fadd_rn(b, c))};
}
// t = (x - top) scale in two parts.
SA_DEV Pair exponent(float x, float top, const Scale& s) {
  const Pair d = minus(x, top);
  const float hi = __fmul_rn(d.hi, s.hi);
  return {hi, __fmaf_rn(d.hi, s.hi, -hi) + __fmaf_rn(d.hi, s.lo, d.lo * s.hi)};
}
// An exponent at which nothing is left (fp64's least): a token masked in both
// rows, by whatever value, does not stand.
constexpr float kNothing = -1074.f;

// Whether u a < 2^t b, for sums a and b (1 to 2^18), u of 0 or from 2^-126 on, and any t that is not nothing: small
// powers are brought up, large ones cut off (2^64 b is more than any u a), so that neither leaves fp32's range where it
// decides.
SA_DEV bool less(float u, float a, Pair t, float b) {
  const bool small = t.hi < -64.f;
  const float e = ex2(small ? t.hi + 64.f : fminf(t.hi, 64.f));
  return u == 0.f || u * (small ? 18446744073709551616.f : 1.f) * a < fmaf(e, t.lo * kLn2, e) * b;
}
// 2^t, t <= 0, off by 2^-40.4 of itself at most and 2^-43 on average where a mass is heavy (t > -12; the same steps against
// exact values): 2^(n + k/16) (1 + g + g^2/2 + ...), g = ln 2 times the rest of t, |g| <= ln 2 / 32.
// 0 from t = -60 down, where no unit of 2^-40 is left (a ratio of two sums brings back 2^18 at most), and where t is -inf
// or, behind it, a NaN: a token that is heavy in one row may be anything in the other, and the scale holds for t > -127
// alone.
__device__ __noinline__ Pair power_pair(Pair t) {
  if (!(t.hi > -60.f)) return {0.f, 0.f};
  const float m = rintf(t.hi * 16.f), rest = fmaf(m, -0.0625f, t.hi) + t.lo;  // the first difference is exact
  const float rest_lo = t.lo - (rest - fmaf(m, -0.0625f, t.hi));
  const int i = static_cast<int>(m), k = i & 15;
  constexpr float kLn2Lo = static_cast<float>(0.693147180559945309 - static_cast<double>(kLn2));
  const float g = __fmul_rn(rest, kLn2), g_lo = fmaf(rest, kLn2, -g) + fmaf(rest, kLn2Lo, rest_lo * kLn2);
  // e^g - 1 in two parts: g and its square, whose parts matter (one fp32 for all but g would be off by 2^-34), then
  // g^3 (1/6 + g/24 + g^2/120)
  const float half = 0.5f * g, b = __fmul_rn(half, g), b_lo = fmaf(half, g, -b);
  const float cube = fmaf(g * b, fmaf(g, fmaf(g, 1.f / 60, 1.f / 12), 1.f / 3), b_lo + fmaf(g_lo, g, g_lo));
  const float e = __fadd_rn(g, b), e_lo = (b - (e - g)) + cube;  // |g| > |b|
  const float hi = kPowers.hi[k], lo = kPowers.lo[k];
  const float a = __fmul_rn(hi, e), a_lo = fmaf(hi, e, -a);
  const float sum = __fadd_rn(hi, a), sum_lo = a - (sum - hi);  // |hi| > |a|
  const float rest2 = sum_lo + (a_lo + fmaf(hi, e_lo, fmaf(lo, e, lo)));
  const float scale = __int_as_float((127 + (i >> 4)) << 23);
  return {sum * scale, rest2 * scale};
}
SA_DEV Pair to_pair(u64 m) {
  const float hi = __ull2float_rn(m);
  return {hi, __ll2float_rn(static_cast<long long>(m - static_cast<u64>(hi)))};
}
// Of a mass below 2^20 of its row's largest: the product stays below 2^61.
__device__ __noinline__ long long to_units(Pair e, float unit) { return __float2ll_rn(e.hi * unit) + __float2ll_rn(e.lo * unit); }

// ---------------------------------------------------------------- an entry
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 16;
constexpr int kWeightsPerSm = 4;  // CTAs of the weights' launch that an SM holds, one fewer where it tests the drafts too
constexpr int kHeavyLog2 = 12;  // masses from 2^-12 of the whole on are heavy
constexpr int kUnitLog2 = 40;   // masses in units of 2^-40 of (about) the whole
// Units of max(p - q, 0) up to which the draw weighs the row's tokens again.  With the near ratio, off by 2^-23, the tokens
// on which p and q agree to that get or lose their sign: 2^-23 of the whole at most, which is nothing beside most of w, but
// all of it where w comes to no more (of 20 million entries, a third with u next to 1 so that rows alike are refused at all,
// 304 got a token whose border lay up to 2.3 x 2^-24 of the whole away, or one of p where nothing was left; all had less
// than 2^-20 of the whole in w, and with this limit none is off by more than 0.12 x 2^-24).  From 2^-16 on it is 2^-7 of w.
constexpr u64 kEnough = 1ull << (kUnitLog2 - 16);
constexpr int kList = 1024;     // vectors with heavy masses that a CTA keeps a list of

struct RowStat {
  float top, sum;
  int arg;
  SA_DEV bool none() const { return sum == 0.f; }
  SA_DEV bool bad() const { return !(sum >= 0.f) || sum > 3e38f; }
};

// Of a run of tokens: what they weigh with the near ratio, and what that loses
// for each unit that the ratio is more; the sums of both rows' masses.
struct alignas(16) Sums {
  u64 weight, slope, p, q;
};

// Where an entry stopped and what its last token is drawn from; in the
// workspace between the second launch and the third.
struct alignas(16) Stop {
  RowStat p, q;
  int row, draft;  // row: -1 for an entry without rows; draft: the one that did not stand, or -1
  int drawn;       // 0: the token is written already, or there is none
  int pad[3];
};

SA_DEV float unit_of(float u) { return fminf(fmaxf(u, 0.f), 0.99999994f); }
// A power of two that brings the whole, `sum`, to 2^kUnitLog2 or just below.
SA_DEV float unit_for(float sum) {
  const int e = (__float_as_int(sum) >> 23) - 127 + 1;  // sum < 2^e, and at least 2^-1 (the largest counts 1)
  return __int_as_float((127 + kUnitLog2 - e) << 23);
}
SA_DEV float log_share(float x, const RowStat& s, const Scale& sc) {
  return __fdiv_rn(x - s.top, sc.temperature) - logf(s.sum);
}

template <class T>
SA_DEV const T* row_of(const VerifyArgs& a, int row) {
  return static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride;
}
template <class T>
SA_DEV const T* draft_of(const VerifyArgs& a, int draft) {
  return static_cast<const T*>(a.draft_logits) + static_cast<int64_t>(draft) * a.draft_stride;
}
SA_DEV bool has_rows(const VerifyArgs& a, int b) { return min(a.cu[b + 1], a.rows) > max(a.cu[b], 0); }

// The rows of an entry, and where it stops.
template <int kType>
class Entry {
 public:
  typedef Elem<kType> E;
  typedef typename E::T T;
  struct Shared {
    int count[kWarps];
    int first;
  };

  SA_DEV Entry(Shared& sh, const VerifyArgs& a, int slices) : sh_(sh), a_(a), slices_(slices) {}

  // Tests the drafts of entry b; `writes`: and writes what is decided by that.  The same in all threads.
  SA_DEV Stop stop(int b, bool writes) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Stop s;
    s.drawn = 0;
    s.draft = -1;
    int full = 0;
    for (int j = tid; j < b; j += kThreads) full += a_.cu[j + 1] > a_.cu[j];
    full = warp_sum(full);
    const int row0 = max(a_.cu[b], 0), n = min(a_.cu[b + 1], a_.rows) - row0;
    if (lane == 0) sh_.count[warp] = full;
    if (tid == 0) sh_.first = max(n - 1, 0);
    __syncthreads();
    s.row = -1;
    if (n <= 0) {
      if (writes && tid == 0) a_.accepted[b] = a_.rejected[b] = 0;
      return s;
    }
    if (a_.live != nullptr && a_.live[b] < 0) {  // its logits are of nothing: none of its drafts stands, and none is refused
      s.row = row0;
      if (writes) {
        for (int i = tid; i < n; i += kThreads) {
          a_.tokens[row0 + i] = -1;
          a_.logp[row0 + i] = 0.f;
        }
        if (tid == 0) a_.accepted[b] = a_.rejected[b] = 0;
      }
      return s;
    }
    int draft0 = row0 - a_.cu[0];  // one draft fewer than rows in every entry before that has rows
    for (int w = 0; w < kWarps; ++w) draft0 -= sh_.count[w];
    const Scale sc(a_.temperature[b]);
    // the drafts, a warp each; what an earlier stop makes void is overwritten below
    for (int i = warp; i < n - 1; i += kWarps) {
      bool stands = false;
      if (sc.valid && has_draft(draft0 + i)) {
        const int token = a_.drafts[draft0 + i];
        const bool inside = token >= 0 && token < a_.vocab;
        const float x = inside ? E::one(row_of<T>(a_, row0 + i)[token]) : -INFINITY;
        const float y = inside && a_.draft_logits != nullptr ? E::one(draft_of<T>(a_, draft0 + i)[token]) : 0.f;
        const float u = unit_of(a_.u[row0 + i]);
        const RowStat p = stat(row0 + i, sc);
        if (!p.bad() && !p.none() && inside) {
          const Pair tp = exponent(x, p.top, sc);
          if (sc.greedy) {
            stands = token == p.arg;
          } else if (a_.draft_logits == nullptr) {
            stands = tp.hi > kNothing && less(u, p.sum, tp, 1.f);
          } else {
            // u q < p by their ratio, if either is anything
            const RowStat q = stat(a_.rows + draft0 + i, sc);
            const Pair tq = exponent(y, q.top, sc);
            Pair t = minus(tp.hi, tq.hi);
            t.lo += tp.lo - tq.lo;
            stands = !q.bad() && !q.none() && tp.hi > kNothing && (!(tq.hi > kNothing) || less(u, p.sum, t, q.sum));
          }
          if (stands && writes && lane == 0) {
            a_.tokens[row0 + i] = token;
            a_.logp[row0 + i] = log_share(x, p, sc);
          }
        }
      }
      if (!stands && lane == 0) atomicMin(&sh_.first, i);
    }
    __syncthreads();
    const int j = sh_.first;
    s.row = row0 + j;
    if (writes) {
      for (int i = j + 1 + tid; i < n; i += kThreads) {
        a_.tokens[row0 + i] = -1;
        a_.logp[row0 + i] = 0.f;
      }
      if (tid == 0) {
        a_.accepted[b] = j;
        a_.rejected[b] = n - 1 - j;
      }
    }
    const auto put = [&](int token, float logp) {
      if (writes && tid == 0) {
        a_.tokens[s.row] = token;
        a_.logp[s.row] = logp;
      }
      return s;
    };
    const bool refused = j < n - 1;
    if (!sc.valid || (refused && !has_draft(draft0 + j))) return put(-1, NAN);
    if (refused) s.draft = draft0 + j;
    s.p = stat(s.row, sc);
    const bool minus_q = refused && a_.draft_logits != nullptr && !sc.greedy;
    if (minus_q) s.q = stat(a_.rows + s.draft, sc);
    if (s.p.bad()) return put(-1, NAN);
    if (s.p.none()) return put(-1, -INFINITY);
    if (sc.greedy) return put(s.p.arg, log_share(s.p.top, s.p, sc));
    if (minus_q && (s.q.bad() || s.q.none())) return put(-1, NAN);
    s.drawn = 1;
    return s;
  }
 private:
  SA_DEV bool has_draft(int i) const { return i >= 0 && i < a_.num_drafts; }
  // Of target row `item`, or of draft item - rows; by a whole warp.
  SA_DEV RowStat stat(int item, const Scale& sc) const {
    const float4* parts = a_.parts + static_cast<int64_t>(item) * slices_;
    const int lane = threadIdx.x & 31;
    RowStat r{kLowest, 0.f, 0x7fffffff};
    if (slices_ <= 32) {
      const float4 f = lane < slices_ ? parts[lane] : make_float4(kLowest, 0.f, __int_as_float(0x7fffffff), 0.f);
      r.top = warp_max(f.x);
      r.sum = warp_sum(f.y * ex2((f.x - r.top) * sc.hi));
      if (sc.greedy) r.arg = warp_min(f.x == r.top ? __float_as_int(f.z) : 0x7fffffff);
      return r;
    }
    for (int i = lane; i < slices_; i += 32) r.top = fmaxf(r.top, parts[i].x);
    r.top = warp_max(r.top);
    for (int i = lane; i < slices_; i += 32) {
      const float4 f = parts[i];
      r.sum += f.y * ex2((f.x - r.top) * sc.hi);
      if (f.x == r.top) r.arg = min(r.arg, __float_as_int(f.z));
    }
    r.sum = warp_sum(r.sum);
    r.arg = warp_min(r.arg);
    return r;
  }

  Shared& sh_;
  const VerifyArgs& a_;
  int slices_;
};

// What the tokens of a row (x_), less those of a draft row (y_), weigh.
template <int kType>
class Weights {
 public:
  typedef Elem<kType> E;
  typedef typename E::T T;
  static constexpr int kVec = E::kVec;

  // A vector's logits that are heavy in neither row (-inf in the others' place), and which those are, a bit each.
  struct Vector {
    float x[kVec], y[kVec];
    uint32_t heavy;
  };

  SA_DEV Weights(const VerifyArgs& a, const Stop& s, const Scale& sc)
      : vocab_(a.vocab), vectors_((a.vocab + kVec - 1) / kVec), sc_(sc), p_(s.p), q_(s.q) {
    x_ = row_of<T>(a, s.row);
    y_ = nullptr;
    unit_ = unit_for(s.p.sum);
    heavy_ = heavy_from(s.p);
    d_least_ = fmaxf(__fdiv_rn(-150.f, sc.hi), -3e38f);
    if (s.draft >= 0 && a.draft_logits != nullptr) {
      y_ = draft_of<T>(a, s.draft);
      near_ = __fdiv_rn(s.p.sum, s.q.sum);
      // (equal rows' sums can fall on either side of a power of two; in one unit what they leave is 0)
      unit_q_ = fabsf(near_ - 1.f) < 0.001f ? unit_ : unit_for(s.q.sum);
      heavy_q_ = heavy_from(s.q);
    } else if (s.draft >= 0) {
      without_ = a.drafts[s.draft];
    }
  }
  SA_DEV bool minus_q() const { return y_ != nullptr; }
  SA_DEV void make_plain() {
    y_ = nullptr;
    without_ = -1;
  }
  SA_DEV int vectors() const { return vectors_; }
  SA_DEV float x_at(int index) const { return E::one(x_[index]); }

  // The vectors of one warp's run among `runs`.
  SA_DEV int run_length(int runs) const { return (vectors_ + runs - 1) / runs; }

  // A vector as it comes from memory.
  struct Raw {
    uint4 x, y;
  };
  SA_DEV Raw fetch(int v) const {
    Raw w;
    w.x = raw(x_, v);
    if (y_ != nullptr) w.y = raw(y_, v);
    return w;
  }
  SA_DEV void unpack(const Raw& w, Vector& t) const {
    bool any = E::largest(w.x) >= heavy_;
    E::unpack(w.x, t.x);
    if (y_ != nullptr) {
      any |= E::largest(w.y) >= heavy_q_;
      E::unpack(w.y, t.y);
    }
    t.heavy = 0;
    if (any) {  // they leave the light path
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (t.x[e] >= heavy_ || (y_ != nullptr && t.y[e] >= heavy_q_)) {
          t.heavy |= 1u << e;
          t.x[e] = t.y[e] = -INFINITY;
        }
      }
    }
  }

  // What the logits of vector v weigh that are not heavy, before the unit, with
  // the near ratio (kSums: adding to the rows' masses and the slope) or with
  // the exact one.
  template <bool kSums>
  SA_DEV void light_weights(int v, const Vector& t, float2 (&r)[kVec / 2], float2& p, float2& q, float2& slope) const {
#pragma unroll
    for (int e = 0; e < kVec; e += 2) {
      float2 m = light(t.x[e], t.x[e + 1], p_.top);
      if (y_ != nullptr) {
        float2 n = light(t.y[e], t.y[e + 1], q_.top);
        if constexpr (kSums) p = fadd2(p, m), q = fadd2(q, n);
        m = ffma2(n, make_float2(-near_, -near_), m);
        if constexpr (!kSums) m = ffma2(n, make_float2(-more_, -more_), m);
        if constexpr (kSums) slope = fadd2(slope, make_float2(m.x > 0.f ? n.x : 0.f, m.y > 0.f ? n.y : 0.f));
        m = make_float2(fmaxf(m.x, 0.f), fmaxf(m.y, 0.f));
      }
      r[e / 2] = m;
    }
    if (without_ >= v * kVec && without_ < (v + 1) * kVec) {
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        if (v * kVec + e == without_) r[e / 2].x = 0.f;
        if (v * kVec + e + 1 == without_) r[e / 2].y = 0.f;
      }
    }
  }
  static SA_DEV float sum_of(const float2 (&r)[kVec / 2]) {
    float2 s = r[0];
#pragma unroll
    for (int e = 1; e < kVec / 2; ++e) s = fadd2(s, r[e]);
    return s.x + s.y;
  }
  SA_DEV u64 units(float f) const { return __float2uint_rn(f * unit_); }
  SA_DEV u64 units_q(float f) const { return __float2uint_rn(f * unit_q_); }

  // Adds a heavy token with the near ratio.
  SA_DEV void add_heavy(Sums& to, int index) const {
    const Pair p = power_pair(exponent(E::one(x_[index]), p_.top, sc_));
    if (y_ == nullptr) {
      if (index != without_) to.weight += to_units(p, unit_);
      return;
    }
    const Pair q = power_pair(exponent(E::one(y_[index]), q_.top, sc_));
    const long long m = difference(p, q, near_, 0.f);
    to.weight += m;
    to.p += to_units(p, unit_);
    to.q += to_units(q, unit_q_);
    if (m > 0) to.slope += to_units(q, unit_q_);
  }
  // What a heavy token weighs with the exact ratio.
  SA_DEV u64 heavy_weight(int index) const {
    if (index == without_) return 0;
    const Pair p = power_pair(exponent(E::one(x_[index]), p_.top, sc_));
    if (y_ == nullptr) return to_units(p, unit_);
    return difference(p, power_pair(exponent(E::one(y_[index]), q_.top, sc_)), ratio_.hi, ratio_.lo);
  }

  // The ratio of the two rows' sums, from their masses.
  SA_DEV void set_ratio(u64 all_p, u64 all_q) {
    if (y_ == nullptr) return;
    const Pair a = to_pair(all_p), b = to_pair(all_q);
    const float hi = __fdiv_rn(a.hi, b.hi);
    const float lo = __fdiv_rn(fmaf(-hi, b.hi, a.hi) + fmaf(-hi, b.lo, a.lo), b.hi);
    const float scale = __fdiv_rn(unit_q_, unit_);  // a power of two
    ratio_ = {hi * scale, lo * scale};
    more_ = (ratio_.hi - near_) + ratio_.lo;
    fall_ = more_ * __fdiv_rn(unit_, unit_q_);
  }
  // What a run weighs with the exact ratio, but for tokens that get or lose their sign between near and exact ratio: each
  // weighs less than the ratios' difference times itself.
  SA_DEV u64 exact(const Sums& v) const {
    return max(static_cast<long long>(v.weight) - __float2ll_rn(__ull2float_rn(v.slope) * fall_), 0LL);
  }
  // What vector v weighs with the exact ratio; r: its light logits'.
  SA_DEV u64 vector_weight(int v, Vector& t, float2 (&r)[kVec / 2]) const {
    float2 none = make_float2(0.f, 0.f);
    unpack(fetch(v), t);
    light_weights<false>(v, t, r, none, none, none);
    u64 m = units(sum_of(r));
#pragma unroll 1
    for (uint32_t bits = t.heavy; bits != 0; bits &= bits - 1) m += heavy_weight(v * kVec + __ffs(bits) - 1);
    return m;
  }

 private:
  SA_DEV float heavy_from(const RowStat& s) const {  // the logit from which a mass is heavy
    float l;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(l) : "f"(s.sum));
    return s.top + __fdiv_rn(l - kHeavyLog2, sc_.hi);
  }
  // Vector v of a row, counted from its first logit; -inf behind its end.
  SA_DEV uint4 raw(const T* row, int v) const {
    const int at = v * kVec;
    if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0 && at + kVec <= vocab_) return __ldg(reinterpret_cast<const uint4*>(row) + v);
    union {
      uint4 q;
      T t[kVec];
    } w;
#pragma unroll
    for (int e = 0; e < kVec; ++e) w.t[e] = at + e < vocab_ ? row[at + e] : E::lowest();
    return w.q;
  }
  // 2^((x - top) scale) of two logits to some 2^-23 of itself, 0 far below.
  SA_DEV float2 light(float x, float y, float top) const {
    float2 d = fadd2(make_float2(x, y), make_float2(-top, -top));
    float2 d_lo = make_float2(0.f, 0.f);
    if constexpr (kType == 0) {
      // what d was rounded by; the difference of two 16-bit logits is exact where it matters (neither below 2^-13 of
      // the other)
      const float2 b = fadd2(d, make_float2(-x, -y));
      const float2 c = fadd2(d, make_float2(-b.x, -b.y));
      d_lo = fadd2(fadd2(make_float2(x, y), make_float2(-c.x, -c.y)), fadd2(make_float2(-top, -top), make_float2(-b.x, -b.y)));
      d_lo = make_float2(d.x > d_least_ ? d_lo.x : 0.f, d.y > d_least_ ? d_lo.y : 0.f);
    }
    d = make_float2(fmaxf(d.x, d_least_), fmaxf(d.y, d_least_));
    const float2 hi = fmul2(d, make_float2(sc_.hi, sc_.hi));
    // minus what hi was rounded by, and minus what the scale was
    float2 lo = ffma2(d, make_float2(-sc_.lo, -sc_.lo), ffma2(d, make_float2(-sc_.hi, -sc_.hi), hi));
    if constexpr (kType == 0) lo = ffma2(d_lo, make_float2(-sc_.hi, -sc_.hi), lo);
    const float2 e = make_float2(ex2(hi.x), ex2(hi.y));
    return ffma2(e, fmul2(lo, make_float2(-kLn2, -kLn2)), e);
  }
  // e_p - ratio e_q in units, 0 at least.
  SA_DEV long long difference(Pair p, Pair q, float ratio, float ratio_lo) const {
    const float c = __fmul_rn(q.hi, ratio), c_lo = fmaf(q.hi, ratio, -c) + fmaf(q.hi, ratio_lo, q.lo * ratio);
    return max(to_units(p, unit_) - to_units({c, c_lo}, unit_), 0LL);
  }

  const T* x_;
  const T* y_;
  int vocab_, vectors_, without_ = -1;  // without: the draft that is taken out
  Scale sc_;
  RowStat p_, q_;
  float unit_, unit_q_ = 0.f;       // masses are e times unit
  float heavy_, heavy_q_ = 0.f;     // logits from which a mass is heavy
  float d_least_;                   // a difference at which nothing is left
  float near_ = 0.f;                // about the ratio of the sums: p - q is e_p - ratio e_q, but for a factor
  float more_ = 0.f, fall_ = 0.f;   // what the exact ratio is more; units of weight that a unit of slope costs
  Pair ratio_ = {0.f, 0.f};         // the exact ratio
};

// The parts of the workspace behind the slices' sums.
struct Places {
  int slices, parts;
  bool by_row;  // an entry's place goes by its first row, not by its number: there are more entries than rows
  Stop* stops;  // [min(rows, most entries)]
  Sums* sums;   // [the same][parts][kWarps]
  SA_DEV int of(const VerifyArgs& a, int b) const { return by_row ? max(a.cu[b], 0) : b; }  // (of an entry that has rows)
};

// CTA: tests entry b's drafts.
template <int kType>
__global__ void __launch_bounds__(kThreads) verify_stop_kernel(const __grid_constant__ VerifyArgs a, const Places w) {
  __shared__ typename Entry<kType>::Shared sh;
  const int b = blockIdx.x;
  cudaGridDependencySynchronize();
  const Stop s = Entry<kType>(sh, a, w.slices).stop(b, true);
  if (threadIdx.x == 0 && s.row >= 0) w.stops[w.of(a, b)] = s;
}

// CTA: a part of entry b's vocabulary, cut into a run for each warp.  kTests:
// tests the entry's drafts itself, all parts alike.
template <int kType, bool kTests>
__global__ void __launch_bounds__(kThreads, kTests ? kWeightsPerSm - 1 : kWeightsPerSm) verify_weights_kernel(const __grid_constant__ VerifyArgs a, const Places w) {
  constexpr int kVec = Elem<kType>::kVec;
  __shared__ Sums sums[kWarps];
  __shared__ uint32_t list[kList];  // vector in the CTA's run << 8 | its heavy logits, a bit each
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / w.parts, part = blockIdx.x - b * w.parts;
  if (tid == 0) listed = 0;
  __syncthreads();
  cudaGridDependencySynchronize();  // by all: this launch is not over before the others are
  const int place = w.of(a, b);
  Stop s;
  if constexpr (kTests) {
    __shared__ typename Entry<kType>::Shared entry_sh;
    s = Entry<kType>(entry_sh, a, w.slices).stop(b, part == 0);
    if (part == 0 && tid == 0 && s.row >= 0) w.stops[place] = s;
  } else {
    if (!has_rows(a, b)) return;
    s = w.stops[place];
  }
  if (!s.drawn) return;
  const Weights<kType> weights(a, s, Scale(a.temperature[b]));
  const int run = weights.run_length(w.parts * kWarps), v_cta = part * kWarps * run;
  const int v0 = min(v_cta + warp * run, weights.vectors()), v1 = min(v0 + run, weights.vectors());
  Sums own{0, 0, 0, 0};
  typename Weights<kType>::Raw next;
  if (v0 + lane < v1) next = weights.fetch(v0 + lane);
#pragma unroll 1
  for (int v = v0 + lane; v < v1; v += 32) {
    typename Weights<kType>::Vector t;
    float2 r[kVec / 2], p = make_float2(0.f, 0.f), q = p, slope = p;
    weights.unpack(next, t);
    if (v + 32 < v1) next = weights.fetch(v + 32);
    weights.template light_weights<true>(v, t, r, p, q, slope);
    own.weight += weights.units(Weights<kType>::sum_of(r));
    if (weights.minus_q()) {
      own.p += weights.units(p.x + p.y);
      own.q += weights.units_q(q.x + q.y);
      own.slope += weights.units_q(slope.x + slope.y);
    }
    if (t.heavy != 0) {
      const int at = atomicAdd(&listed, 1);
      if (at < kList) {
        list[at] = static_cast<uint32_t>(v - v_cta) << 8 | t.heavy;
      } else {
#pragma unroll 1
        for (uint32_t bits = t.heavy; bits != 0; bits &= bits - 1) weights.add_heavy(own, v * kVec + __ffs(bits) - 1);
      }
    }
  }
  own.weight = warp_sum(own.weight);
  if (weights.minus_q()) {
    own.p = warp_sum(own.p);
    own.q = warp_sum(own.q);
    own.slope = warp_sum(own.slope);
  }
  if (lane == 0) sums[warp] = own;
  __syncthreads();
  // the heavy tokens, evenly over the threads; integer sums do not depend on the order
  for (int i = tid; i < min(listed, kList); i += kThreads) {
    const int in_cta = static_cast<int>(list[i] >> 8);
    Sums some{0, 0, 0, 0};
#pragma unroll 1
    for (uint32_t bits = list[i] & 0xffu; bits != 0; bits &= bits - 1)
      weights.add_heavy(some, (v_cta + in_cta) * kVec + __ffs(bits) - 1);
    Sums& to = sums[in_cta / run];
    atomicAdd(&to.weight, some.weight);
    if (weights.minus_q()) {
      atomicAdd(&to.slope, some.slope);
      atomicAdd(&to.p, some.p);
      atomicAdd(&to.q, some.q);
    }
  }
  __syncthreads();
  if (tid < kWarps) w.sums[(static_cast<int64_t>(place) * w.parts + part) * kWarps + tid] = sums[tid];
}

struct DrawShared {
  u64 scan[2][kWarps];
  int found, spare;
};

// Inclusive sum over the CTA's threads, and its total; the buffers alternate.
SA_DEV u64 block_scan(DrawShared& sh, int turn, u64 x, u64& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 other = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += other;
  }
  u64* sums = sh.scan[turn & 1];
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) x += sums[w];
    total += sums[w];
  }
  return x;
}

// CTA: draws entry b's last token.
template <int kType>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const __grid_constant__ VerifyArgs a, const Places w) {
  constexpr int kVec = Elem<kType>::kVec;
  __shared__ DrawShared sh;
  __shared__ int holder_sh;
  __shared__ u64 before_sh;
  const int tid = threadIdx.x, b = blockIdx.x;
  cudaGridDependencySynchronize();  // by all: this launch is not over before the others are
  if (!has_rows(a, b)) return;
  const int place = w.of(a, b);
  const Stop s = w.stops[place];
  if (!s.drawn) return;
  const Scale sc(a.temperature[b]);
  Weights<kType> weights(a, s, sc);
  const float u = unit_of(a.u[min(a.cu[b + 1], a.rows) - 1]);
  const auto target_of = [&](u64 total) {  // floor(total u), below total
    return __umul64hi(total << 4, static_cast<u64>(u * 4294967296.f) << 28);
  };
  int turn = 0;
  const int runs = w.parts * kWarps;  // <= kThreads
  static_assert(kMaxParts * kWarps <= kThreads, "a run to each thread");
  Sums mine{0, 0, 0, 0};
  if (tid < runs) mine = w.sums[static_cast<int64_t>(place) * runs + tid];
  if (weights.minus_q()) {
    u64 p, q;
    block_scan(sh, turn++, mine.p, p);
    block_scan(sh, turn++, mine.q, q);
    weights.set_ratio(p, q);
  }
  u64 total, target, before = 0;
  int first = 0, last = weights.vectors();  // the vectors among which the token is
  const u64 run_weight = weights.exact(mine), upto = block_scan(sh, turn++, run_weight, total);
  if (tid == 0) sh.found = 0, sh.spare = -1;
  if (total >= (weights.minus_q() ? kEnough : 1)) {
    // the run that holds the place drawn
    target = target_of(total);
    if (target >= upto - run_weight && target < upto) holder_sh = tid, before_sh = upto - run_weight;
    __syncthreads();
    const int run = weights.run_length(runs);
    first = min(holder_sh * run, last);
    last = min(first + run, last);
    before = before_sh;
  } else {
    // Little is left of w, next to what the runs' weights are off by: the whole row again, with the exact ratio.  Where
    // that leaves nothing, the target's own probabilities.
#pragma unroll 1
    for (int again = 0; again < 2; ++again) {
      if (again == 1 || !weights.minus_q()) weights.make_plain();
      u64 sum = 0;
      for (int v = tid; v < last; v += kThreads) {
        typename Weights<kType>::Vector t;
        float2 r[kVec / 2];
        sum += weights.vector_weight(v, t, r);
      }
      block_scan(sh, turn++, sum, total);
      if (total > 0) break;
    }
    target = target_of(total);
  }
  // A vector to each thread.  With the exact ratio they may come to a few units
  // less than the run did: then (pass 1) the last token that weighs something
  // is taken, or that p allows.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int v0 = first; v0 < last; v0 += kThreads) {
      const int v = v0 + tid;
      typename Weights<kType>::Vector t;
      float2 r[kVec / 2];
      t.heavy = 0;
      const u64 weight = v < last ? weights.vector_weight(v, t, r) : 0;
      u64 all, at = 0;
      if (pass == 0) {
        at = before + block_scan(sh, turn++, weight, all) - weight;
        before += all;
      }
      if (v < last && (pass == 1 || (target >= at && target < at + weight))) {
        int token = -1, any = -1, allowed = -1;
        float f[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = e & 1 ? r[e / 2].y : r[e / 2].x;
#pragma unroll 1
        for (int e = 0; e < kVec && v * kVec + e < a.vocab; ++e) {
          const int index = v * kVec + e;
          const u64 m = t.heavy >> e & 1u ? weights.heavy_weight(index) : weights.units(f[0]);
          if (token < 0 && target < at + m) token = index;
          if (m > 0 || f[0] > 0.f) any = index;
          if (weights.x_at(index) > -INFINITY) allowed = index;
          at += m;
#pragma unroll
          for (int k = 0; k + 1 < kVec; ++k) f[k] = f[k + 1];
        }
        if (pass == 0) {
          sh.spare = token < 0 ? any : token;
          sh.found = 1;
        } else {
          atomicMax(&sh.spare, any >= 0 ? 1 << 18 | any : allowed);
        }
      }
      if (pass == 0 && target < before) break;
    }
    __syncthreads();
    if (sh.found) break;
  }
  if (tid == 0 && sh.spare >= 0) {
    const int token = sh.spare & ((1 << 18) - 1);
    a.tokens[s.row] = token;
    a.logp[s.row] = log_share(weights.x_at(token), s.p, sc);
  }
}

// Vectors of a row however it is aligned, in turns of a CTA.
int turns_for(int dtype, int vocab) {
  const int vec = dtype == 0 ? Elem<0>::kVec : Elem<1>::kVec;
  return ceil_div(ceil_div(static_cast<long long>(vocab) + vec - 1, vec), kStatThreads);
}
int most_slices(int dtype, int vocab) { return ceil_div(turns_for(dtype, vocab), kStatVecs); }

template <int kType>
cudaError_t launch_type(const VerifyArgs& a, cudaStream_t s) {
  const long long items = a.rows + (a.draft_logits != nullptr ? a.num_drafts : 0);
  // A row in as few slices as keep the GPU busy (what it holds at once, a few times), each a whole number of turns that
  // a thread has in flight, so that none is nearly empty.
  const int all = turns_for(kType, a.vocab);
  int slices = std::max(ceil_div(all, kStatMostVecs), 1);
  if (items > 0)
    slices = std::max(slices, static_cast<int>(std::min<long long>(most_slices(kType, a.vocab), 3LL * kStatPerSm * device_sms() / items)));
  const int turns = ceil_div(ceil_div(all, slices), kStatVecs) * kStatVecs;
  slices = ceil_div(all, turns);
  if (items > 0)
    verify_rows_kernel<kType><<<static_cast<unsigned>(items * slices), kStatThreads, 0, s>>>(a, slices, turns);
  // An entry in parts of eight vectors a thread at least, four where there are few entries, and in no more than five
  // times what the GPU holds at once (not all entries have anything to draw; 128 x 201088 bf16 with 16 parts 94 us, with 8
  // 103).  Parts that come in one turn test the drafts themselves (one entry 18.3 us, with a launch of its own for that
  // 19.5), else all but the first turn would wait for the same tests again (128 x 201088: 105 us with 8 parts each).
  const int wave = kWeightsPerSm * device_sms();
  int parts = 1;
  while (parts < kMaxParts && 2LL * parts * a.num_seqs <= 5LL * wave &&
         parts * kThreads * (4LL * parts * a.num_seqs <= wave ? 4 : 8) * Elem<kType>::kVec < a.vocab)
    parts *= 2;
  const bool tests_apart = static_cast<long long>(parts) * a.num_seqs > (kWeightsPerSm - 1) * device_sms();
  Places w;
  w.slices = slices;
  w.parts = parts;
  uint8_t* behind = reinterpret_cast<uint8_t*>(a.parts) +
                    static_cast<size_t>(a.rows) * 2 * most_slices(kType, a.vocab) * sizeof(float4);
  w.by_row = a.num_seqs > a.rows;
  w.stops = reinterpret_cast<Stop*>(behind);
  w.sums = reinterpret_cast<Sums*>(behind + static_cast<size_t>(std::min(a.rows, kKv4MaxRequests)) * sizeof(Stop));
  // Each waits for the one before on the device, so that its launch does not come on top.
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs));
  cudaError_t e = tests_apart ? cudaLaunchKernelEx(&cfg, verify_stop_kernel<kType>, a, w) : cudaSuccess;
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * parts);
  e = cudaLaunchKernelEx(&cfg, tests_apart ? verify_weights_kernel<kType, false> : verify_weights_kernel<kType, true>, a, w);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs));
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<kType>, a, w);
}

}  // namespace

size_t verify_workspace_bytes(int dtype, int rows, int vocab) {
  return static_cast<size_t>(rows) * 2 * most_slices(dtype, vocab) * sizeof(float4) +
         static_cast<size_t>(std::min(rows, kKv4MaxRequests)) * (sizeof(Stop) + kMaxParts * kWarps * sizeof(Sums));
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_type<0>(a, s);
  if (a.dtype == 1) return launch_type<1>(a, s);
  return launch_type<2>(a, s);
}

}  // namespace sa
