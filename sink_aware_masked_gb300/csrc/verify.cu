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
// bytes a logit and one exponential each.  A first launch does that, a CTA per
// (row, slice of the vocabulary): the slice's maximum and the sum relative to
// it, from registers.  A second launch gives each sequence to a cluster: it
// tests the drafts and draws the last token from the one row (or pair of
// rows) in which it stopped, read again, mostly from L2.
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
//     take an exponential of two fp32 parts (off by some 2^-40);
//   - max(p - q, 0) needs the ratio of the two sums as exactly: they are
//     summed again in the same way from the two rows.
// Integer sums are the same in every order.  FP64 is not used: its rate on this
// GPU would cost more than all the rest.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace {

namespace cg = cooperative_groups;

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

// A sequence's rows [row0, row0 + n) and drafts [draft0, ...): the drafts of
// all sequences stand one after another, n - 1 of a sequence that has rows.
struct Rows {
  int row0, n, draft0;
};

// ---------------------------------------------------------------- all rows
constexpr int kStatThreads = 256;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kStatVecs = 8;       // 16-byte vectors that a thread has in flight
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
__global__ void __launch_bounds__(kStatThreads, 3) verify_rows_kernel(const VerifyArgs a, int slices, int turns) {
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
  if (b >= a.num_seqs) return;  // a row of no entry
  const Scale sc(a.temperature[b]);
  if (!sc.valid || (draft && sc.greedy)) return;
  Running r{kLowest, 0.f};
  int arg = 0x7fffffff;
  for (int v = v0 + tid;;) {
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
    v += kStatVecs * kStatThreads;
    if (v - tid >= v1) break;
    load_some(v, w);
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

// t = (x - top) scale in two parts.
SA_DEV Pair exponent(float x, float top, const Scale& s) {
  const float d = __fadd_rn(x, -top), b = __fadd_rn(d, -x);
  const float d_lo = __fadd_rn(__fadd_rn(x, -__fadd_rn(d, -b)), -__fadd_rn(top, b));  // what d was rounded by
  const float hi = __fmul_rn(d, s.hi);
  return {hi, __fmaf_rn(d, s.hi, -hi) + __fmaf_rn(d, s.lo, d_lo * s.hi)};
}
// 2^t to some 2^-23 of itself; 0 below fp32's normal numbers.
SA_DEV float power(Pair t) {
  const float e = ex2(t.hi);
  return t.hi > -126.f ? fmaf(e, t.lo * kLn2, e) : 0.f;
}
// 2^t to some 2^-40 of itself, t in (-60, 0]: 2^(n + k/16) (1 + g + g^2/2 + ...), g = ln 2 times the rest of t,
// |g| <= ln 2 / 32.
SA_DEV Pair power_pair(Pair t) {
  const float m = rintf(t.hi * 16.f), rest = fmaf(m, -0.0625f, t.hi) + t.lo;  // the first difference is exact
  const float rest_lo = t.lo - (rest - fmaf(m, -0.0625f, t.hi));
  const int i = static_cast<int>(m), k = i & 15;
  constexpr float kLn2Lo = static_cast<float>(0.693147180559945309 - static_cast<double>(kLn2));
  const float g = __fmul_rn(rest, kLn2), g_lo = fmaf(rest, kLn2, -g) + fmaf(rest, kLn2Lo, rest_lo * kLn2);
  const float more = fmaf(g * g, fmaf(g, fmaf(g, fmaf(g, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f), g_lo);  // e^g - 1 - g
  const float hi = kPowers.hi[k], lo = kPowers.lo[k];
  const float a = __fmul_rn(hi, g), a_lo = fmaf(hi, g, -a);
  const float sum = __fadd_rn(hi, a), sum_lo = a - (sum - hi);  // |hi| > |a|
  const float rest2 = sum_lo + (a_lo + fmaf(hi, more, fmaf(lo, g, lo)));
  const float scale = __int_as_float((127 + (i >> 4)) << 23);
  return {sum * scale, rest2 * scale};
}
SA_DEV Pair to_pair(u64 m) {
  const float hi = __ull2float_rn(m);
  return {hi, __ll2float_rn(static_cast<long long>(m - static_cast<u64>(hi)))};
}
SA_DEV long long to_units(Pair e, float unit) { return __float2ll_rn(e.hi * unit) + __float2ll_rn(e.lo * unit); }

// ---------------------------------------------------------------- a sequence
constexpr int kThreads = 512;
constexpr int kPerSm = 2;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kHeavyLog2 = 12;  // masses from 2^-12 of the whole on are heavy
constexpr int kUnitLog2 = 40;   // masses in units of 2^-40 of (about) the whole
constexpr int kList = 2048;     // vectors with heavy masses that a CTA keeps a list of

struct RowStat {
  float top, sum;
  int arg;
  SA_DEV bool none() const { return sum == 0.f; }
  SA_DEV bool bad() const { return !(sum >= 0.f) || sum > 3e38f; }
};

// Of a run of tokens: what they weigh with the near ratio, and what that loses
// for each unit that the ratio is more; the sums of both rows' masses.
struct Sums {
  u64 weight, p, q, slope;
};

struct Shared {
  Sums exchange[2][kMaxCluster];
  Sums warp[kWarps];
  u64 weight[kWarps];  // the warps' runs' weights
  int count[kWarps];
  u64 scan[kWarps];
  int first, listed, found, spare;
  uint32_t list[kList];  // vector in the CTA's run << 8 | its heavy logits, a bit each
};

template <int kType>
class Sequence {
 public:
  typedef Elem<kType> E;
  typedef typename E::T T;

  SA_DEV Sequence(Shared& sh, const VerifyArgs& a, int slices)
      : sh_(sh), a_(a), cluster_(cg::this_cluster()), slices_(slices), rank_(cluster_.block_rank()),
        ctas_(cluster_.num_blocks()) {}

  SA_DEV void run(int b) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (ctas_ > 1) cluster_.barrier_arrive();
    int full = 0;
    for (int j = tid; j < b; j += kThreads) full += a_.cu[j + 1] > a_.cu[j];
    full = warp_sum(full);
    if (lane == 0) sh_.count[warp] = full;
    const int row0 = max(a_.cu[b], 0), n = min(a_.cu[b + 1], a_.rows) - row0;
    if (tid == 0) sh_.first = max(n - 1, 0), sh_.listed = 0;
    my_run();
    if (ctas_ > 1) cluster_.barrier_wait();  // every CTA of the cluster runs: its shared memory may be written
    __syncthreads();
    int draft0 = row0 - a_.cu[0];  // one draft fewer than rows in every sequence before that has rows
    for (int w = 0; w < kWarps; ++w) draft0 -= sh_.count[w];
    if (n <= 0) {
      if (rank_ == 0 && tid == 0) a_.accepted[b] = a_.rejected[b] = 0;
      return;
    }
    const Scale sc(a_.temperature[b]);
    // the drafts, a warp each; what an earlier stop makes void is overwritten below
    for (int i = warp; i < n - 1; i += kWarps) {
      bool stands = false;
      if (sc.valid && draft0 + i < a_.num_drafts) {
        const int token = a_.drafts[draft0 + i];
        const RowStat p = stat(row0 + i, sc);
        if (!p.bad() && !p.none() && token >= 0 && token < a_.vocab) {
          const float x = logit(row0 + i, token);
          if (sc.greedy) {
            stands = token == p.arg;
          } else {
            const float u = unit_of(a_.u[row0 + i]);
            const Pair tp = exponent(x, p.top, sc);
            if (a_.draft_logits == nullptr) {
              stands = u * p.sum < power(tp);
            } else {
              // u q < p by their ratio, which stays in range where both are small
              const RowStat s = stat(a_.rows + draft0 + i, sc);
              const float y = draft_logit(draft0 + i, token);
              const Pair tq = exponent(y, s.top, sc);
              const float ratio = y == -INFINITY ? INFINITY : ex2((tp.hi - tq.hi) + (tp.lo - tq.lo)) * __fdiv_rn(s.sum, p.sum);
              stands = !s.bad() && !s.none() && x > -INFINITY && u < ratio;
            }
          }
          if (stands && rank_ == 0 && lane == 0) {
            a_.tokens[row0 + i] = token;
            a_.logp[row0 + i] = log_share(x, p, sc);
          }
        }
      }
      if (!stands && lane == 0) atomicMin(&sh_.first, i);
    }
    __syncthreads();
    const int j = sh_.first, row = row0 + j;
    if (rank_ == 0) {
      for (int i = j + 1 + tid; i < n; i += kThreads) {
        a_.tokens[row0 + i] = -1;
        a_.logp[row0 + i] = 0.f;
      }
      if (tid == 0) {
        a_.accepted[b] = j;
        a_.rejected[b] = n - 1 - j;
      }
    }
    const bool refused = j < n - 1;
    if (!sc.valid || (refused && draft0 + j >= a_.num_drafts)) return put(row, -1, NAN);
    const RowStat p = stat(row, sc);
    if (p.bad()) return put(row, -1, NAN);
    if (p.none()) return put(row, -1, -INFINITY);
    if (sc.greedy) return put(row, p.arg, log_share(p.top, p, sc));
    Weights w;
    w.p = p;
    w.unit = unit_for(p.sum);
    w.heavy = heavy_from(p, sc);
    w.without = -1;
    w.minus_q = false;
    x_ = static_cast<const T*>(a_.logits) + static_cast<int64_t>(row) * a_.stride;
    y_ = nullptr;
    if (refused && a_.draft_logits == nullptr) w.without = a_.drafts[draft0 + j];
    if (refused && a_.draft_logits != nullptr) {
      const RowStat q = stat(a_.rows + draft0 + j, sc);
      if (q.bad() || q.none()) return put(row, -1, NAN);
      w.q = q;
      w.minus_q = true;
      w.heavy_q = heavy_from(q, sc);
      w.near = __fdiv_rn(p.sum, q.sum);
      w.ratio = {w.near, 0.f};
      y_ = static_cast<const T*>(a_.draft_logits) + static_cast<int64_t>(draft0 + j) * a_.draft_stride;
    }
    if (!draw(w, sc, row, unit_of(a_.u[row0 + n - 1]))) {
      // nothing is left of w: the target's own probabilities
      w.minus_q = false;
      w.without = -1;
      __syncthreads();
      if (tid == 0) sh_.listed = 0;
      __syncthreads();
      draw(w, sc, row, unit_of(a_.u[row0 + n - 1]));
    }
  }

 private:
  struct Weights {
    RowStat p, q;
    float unit;            // masses are e times unit
    float heavy, heavy_q;  // logits from which a mass is heavy
    float near;            // about the ratio of the sums: p - q is e_p - ratio e_q, but for a factor
    Pair ratio;            // the same as exactly as the sums are known
    int without;           // the draft that is taken out, or -1
    bool minus_q;
  };

  static SA_DEV float heavy_from(const RowStat& s, const Scale& sc) {
    float l;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(l) : "f"(s.sum));
    return s.top + __fdiv_rn(l - kHeavyLog2, sc.hi);
  }
  static SA_DEV float unit_of(float u) { return fminf(fmaxf(u, 0.f), 0.99999994f); }
  // A power of two that brings the whole, `sum`, to 2^kUnitLog2 or just below.
  static SA_DEV float unit_for(float sum) {
    const int e = (__float_as_int(sum) >> 23) - 127 + 1;  // sum < 2^e, and at least 2^-1 (the largest counts 1)
    return __int_as_float((127 + kUnitLog2 - e) << 23);
  }

  // Of target row `item`, or of draft item - rows; by a whole warp.
  SA_DEV RowStat stat(int item, const Scale& sc) const {
    const float4* parts = a_.parts + static_cast<int64_t>(item) * slices_;
    RowStat r{kLowest, 0.f, 0x7fffffff};
    for (int i = threadIdx.x & 31; i < slices_; i += 32) r.top = fmaxf(r.top, parts[i].x);
    r.top = warp_max(r.top);
    for (int i = threadIdx.x & 31; i < slices_; i += 32) {
      const float4 f = parts[i];
      r.sum += f.y * ex2((f.x - r.top) * sc.hi);
      if (f.x == r.top) r.arg = min(r.arg, __float_as_int(f.z));
    }
    r.sum = warp_sum(r.sum);
    r.arg = warp_min(r.arg);
    return r;
  }
  SA_DEV float logit(int row, int token) const {
    return E::one(static_cast<const T*>(a_.logits)[static_cast<int64_t>(row) * a_.stride + token]);
  }
  SA_DEV float draft_logit(int draft, int token) const {
    return E::one(static_cast<const T*>(a_.draft_logits)[static_cast<int64_t>(draft) * a_.draft_stride + token]);
  }
  static SA_DEV float log_share(float x, const RowStat& s, const Scale& sc) {
    return __fdiv_rn(x - s.top, sc.temperature) - logf(s.sum);
  }
  SA_DEV void put(int row, int token, float logp) const {
    if (rank_ != 0 || threadIdx.x != 0) return;
    a_.tokens[row] = token;
    a_.logp[row] = logp;
  }

  // Every CTA of the cluster gives its sums and takes all of them in rank order.
  template <class F>
  SA_DEV void exchange(const Sums& own, F take) {
    if (ctas_ == 1) {
      take(own);
      return;
    }
    Sums* buf = sh_.exchange[parity_];
    parity_ ^= 1;  // the other half may still be read by a slower CTA
    if (threadIdx.x < ctas_) cluster_.map_shared_rank(buf, threadIdx.x)[rank_] = own;
    cluster_.sync();
    for (unsigned r = 0; r < ctas_; ++r) take(buf[r]);
  }

  // The vectors of a row (counted from its first logit) that the warp has, one run of them.
  SA_DEV void my_run() {
    const int vectors = (a_.vocab + E::kVec - 1) / E::kVec, parts = ctas_ * kWarps;
    run_ = (vectors + parts - 1) / parts;
    v0_ = min((static_cast<int>(rank_) * kWarps + static_cast<int>(threadIdx.x >> 5)) * run_, vectors);
    v1_ = min(v0_ + run_, vectors);
  }
  // Logits of vector v; -inf behind the row's end.
  SA_DEV void load(const T* row, int v, float* f) const {
    const int at = v * E::kVec;
    if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0 && at + E::kVec <= a_.vocab) {
      E::unpack(__ldg(reinterpret_cast<const uint4*>(row) + v), f);
    } else {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) f[e] = at + e < a_.vocab ? E::one(row[at + e]) : -INFINITY;
    }
  }

  // 2^((x - top) scale) of two logits to some 2^-23 of itself, 0 far below; d_least is where that is.
  static SA_DEV float2 light(float x, float y, float top, float d_least, const Scale& sc) {
    float2 d = fadd2(make_float2(x, y), make_float2(-top, -top));
    float2 d_lo = make_float2(0.f, 0.f);
    if constexpr (kType == 0) {
      // what d was rounded by; the difference of two 16-bit logits is exact where it matters (neither below 2^-13 of
      // the other)
      const float2 b = fadd2(d, make_float2(-x, -y));
      const float2 c = fadd2(d, make_float2(-b.x, -b.y));
      d_lo = fadd2(fadd2(make_float2(x, y), make_float2(-c.x, -c.y)), fadd2(make_float2(-top, -top), make_float2(-b.x, -b.y)));
      d_lo = make_float2(x > -INFINITY ? d_lo.x : 0.f, y > -INFINITY ? d_lo.y : 0.f);
    }
    d = make_float2(fmaxf(d.x, d_least), fmaxf(d.y, d_least));
    const float2 s2 = make_float2(sc.hi, sc.hi);
    const float2 hi = fmul2(d, s2);
    float2 lo = ffma2(d, make_float2(sc.lo, sc.lo), ffma2(d, s2, make_float2(-hi.x, -hi.y)));
    if constexpr (kType == 0) lo = ffma2(d_lo, s2, lo);
    const float2 e = make_float2(ex2(hi.x), ex2(hi.y));
    return ffma2(e, fmul2(lo, make_float2(kLn2, kLn2)), e);
  }
  static SA_DEV float least_difference(const Scale& sc) { return fmaxf(__fdiv_rn(-150.f, sc.hi), -3e38f); }

  // e_p - ratio e_q in units, 0 at least.
  static SA_DEV long long difference(Pair p, Pair q, Pair ratio, float unit) {
    const float c = __fmul_rn(q.hi, ratio.hi), c_lo = fmaf(q.hi, ratio.hi, -c) + fmaf(q.hi, ratio.lo, q.lo * ratio.hi);
    return max(to_units(p, unit) - to_units({c, c_lo}, unit), 0LL);
  }
  // What a token weighs, in units, where its mass is heavy.
  SA_DEV long long heavy_weight(float x, float y, int index, const Weights& w, const Scale& sc) const {
    if (index == w.without) return 0;
    const Pair p = power_pair(exponent(x, w.p.top, sc));
    return w.minus_q ? difference(p, power_pair(exponent(y, w.q.top, sc)), w.ratio, w.unit) : to_units(p, w.unit);
  }
  // A vector's logits, and which of them are heavy, a bit each.
  SA_DEV uint32_t load_both(int v, const Weights& w, float (&x)[E::kVec], float (&y)[E::kVec]) const {
    load(x_, v, x);
    bool any = largest(x) >= w.heavy;
    if (w.minus_q) {
      load(y_, v, y);
      any |= largest(y) >= w.heavy_q;
    }
    uint32_t bits = 0;
    if (any) {
#pragma unroll
      for (int e = 0; e < E::kVec; ++e)
        bits |= static_cast<uint32_t>(x[e] >= w.heavy || (w.minus_q && y[e] >= w.heavy_q)) << e;
    }
    return bits;
  }
  static SA_DEV float largest(const float (&x)[E::kVec]) {
    float m = fmaxf(x[0], x[1]);
#pragma unroll
    for (int e = 2; e < E::kVec; e += 2) m = fmax3(m, x[e], x[e + 1]);
    return m;
  }
  // What the logits of a vector weigh that are not heavy, before the unit, with
  // the ratio w.near + more.  kSums: also adds to the rows' masses and the slope.
  template <bool kSums>
  SA_DEV void light_weights(int v, uint32_t heavy, const float (&x)[E::kVec], const float (&y)[E::kVec], const Weights& w,
                            float more, float d_least, const Scale& sc, float2 (&r)[E::kVec / 2], float2& p, float2& q,
                            float2& slope) const {
    const float2 near = make_float2(-w.near, -w.near), rest = make_float2(-more, -more);
#pragma unroll
    for (int e = 0; e < E::kVec; e += 2) {
      float2 m = light(x[e], x[e + 1], w.p.top, d_least, sc);
      if (w.minus_q) {
        float2 n = light(y[e], y[e + 1], w.q.top, d_least, sc);
        if (heavy >> e & 3u) {
          if (heavy >> e & 1u) m.x = n.x = 0.f;
          if (heavy >> e & 2u) m.y = n.y = 0.f;
        }
        if constexpr (kSums) p = fadd2(p, m), q = fadd2(q, n);
        m = ffma2(n, near, m);
        if constexpr (!kSums) m = ffma2(n, rest, m);
        if constexpr (kSums) slope = fadd2(slope, make_float2(m.x > 0.f ? n.x : 0.f, m.y > 0.f ? n.y : 0.f));
        m = make_float2(fmaxf(m.x, 0.f), fmaxf(m.y, 0.f));
      } else if (heavy >> e & 3u) {
        if (heavy >> e & 1u) m.x = 0.f;
        if (heavy >> e & 2u) m.y = 0.f;
      }
      r[e / 2] = m;
    }
    if (w.without >= v * E::kVec && w.without < (v + 1) * E::kVec) {
#pragma unroll
      for (int e = 0; e < E::kVec; e += 2) {
        if (v * E::kVec + e == w.without) r[e / 2].x = 0.f;
        if (v * E::kVec + e + 1 == w.without) r[e / 2].y = 0.f;
      }
    }
  }
  static SA_DEV float sum_of(const float2 (&r)[E::kVec / 2]) {
    float2 s = r[0];
#pragma unroll
    for (int e = 1; e < E::kVec / 2; ++e) s = fadd2(s, r[e]);
    return s.x + s.y;
  }
  // f(x, y, index) for the heavy logits of the CTA's listed vectors, evenly over its threads.
  template <class F>
  SA_DEV void each_listed(const Weights& w, F f) const {
    const int v_cta = static_cast<int>(rank_) * kWarps * run_;
    for (int i = threadIdx.x; i < min(sh_.listed, kList); i += kThreads) {
      const int v = v_cta + static_cast<int>(sh_.list[i] >> 8);
      for (uint32_t bits = sh_.list[i] & 0xffu; bits != 0; bits &= bits - 1) {
        const int index = v * E::kVec + __ffs(bits) - 1;
        f(E::one(x_[index]), w.minus_q ? E::one(y_[index]) : 0.f, index, v);
      }
    }
  }
  // Enters a vector in the list of those with heavy logits; false if it is full.
  SA_DEV bool enter(int v, uint32_t bits) {
    const int at = atomicAdd(&sh_.listed, 1);
    if (at >= kList) return false;
    sh_.list[at] = static_cast<uint32_t>(v - static_cast<int>(rank_) * kWarps * run_) << 8 | bits;
    return true;
  }

  // Draws the token of `row`; false (for all CTAs alike) if nothing has weight.
  // One pass over the run: weights with the ratio that the first launch's sums
  // give, which is off by some 2^-22, and the rows' masses, which give the ratio
  // as exactly as the draw needs it.  The weights change by the slope then (the
  // few that get or lose their sign between are below the square of that).
  SA_DEV bool draw(Weights& w, const Scale& sc, int row, float u) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float d_least = least_difference(sc), unit_q = w.minus_q ? unit_for(w.q.sum) : 0.f;
    Sums own{0, 0, 0, 0};
    const auto add_heavy = [&](Sums& to, float x, float y, int index) {
      if (!w.minus_q) {
        to.weight += heavy_weight(x, y, index, w, sc);
        return;
      }
      const Pair p = power_pair(exponent(x, w.p.top, sc)), q = power_pair(exponent(y, w.q.top, sc));
      const long long m = difference(p, q, {w.near, 0.f}, w.unit);
      to.weight += m;
      to.p += to_units(p, w.unit);
      to.q += to_units(q, unit_q);
      if (m > 0) to.slope += to_units(q, unit_q);
    };
#pragma unroll 2
    for (int v = v0_ + lane; v < v1_; v += 32) {
      float x[E::kVec], y[E::kVec];
      float2 r[E::kVec / 2], p = make_float2(0.f, 0.f), q = p, slope = p;
      const uint32_t heavy = load_both(v, w, x, y);
      light_weights<true>(v, heavy, x, y, w, 0.f, d_least, sc, r, p, q, slope);
      own.weight += __float2uint_rn(sum_of(r) * w.unit);
      if (w.minus_q) {
        own.p += __float2uint_rn((p.x + p.y) * w.unit);
        own.q += __float2uint_rn((q.x + q.y) * unit_q);
        own.slope += __float2uint_rn((slope.x + slope.y) * unit_q);
      }
      if (heavy != 0 && !enter(v, heavy)) {
#pragma unroll
        for (int e = 0; e < E::kVec; ++e)
          if (heavy >> e & 1u) add_heavy(own, x[e], w.minus_q ? y[e] : 0.f, v * E::kVec + e);
      }
    }
    own.weight = warp_sum(own.weight);
    if (w.minus_q) {
      own.p = warp_sum(own.p);
      own.q = warp_sum(own.q);
      own.slope = warp_sum(own.slope);
    }
    if (lane == 0) sh_.warp[warp] = own;
    __syncthreads();
    each_listed(w, [&](float x, float y, int index, int v) {
      Sums one{0, 0, 0, 0};
      add_heavy(one, x, y, index);
      Sums& to = sh_.warp[(v - static_cast<int>(rank_) * kWarps * run_) / run_];
      atomicAdd(&to.weight, one.weight);
      if (w.minus_q) {
        atomicAdd(&to.p, one.p);
        atomicAdd(&to.q, one.q);
        atomicAdd(&to.slope, one.slope);
      }
    });
    __syncthreads();
    Sums all{0, 0, 0, 0}, every{0, 0, 0, 0};
    for (int i = 0; i < kWarps; ++i) add(all, sh_.warp[i]);
    exchange(all, [&](const Sums& v) { add(every, v); });
    float fall = 0.f;  // units of weight that a unit of slope costs
    if (w.minus_q) {
      const Pair a = to_pair(every.p), b = to_pair(every.q);
      const float hi = __fdiv_rn(a.hi, b.hi);
      const float lo = __fdiv_rn(fmaf(-hi, b.hi, a.hi) + fmaf(-hi, b.lo, a.lo), b.hi);
      const float scale = __fdiv_rn(unit_q, w.unit);  // a power of two
      w.ratio = {hi * scale, lo * scale};
      fall = ((w.ratio.hi - w.near) + w.ratio.lo) * __fdiv_rn(w.unit, unit_q);
    }
    const auto weight_of = [&](const Sums& v) {
      return static_cast<u64>(max(static_cast<long long>(v.weight) - __float2ll_rn(__ull2float_rn(v.slope) * fall), 0LL));
    };
    u64 total = 0, before = 0, mine_all = weight_of(all);
    if (ctas_ == 1) {
      total = mine_all;
    } else {
      const Sums* buf = sh_.exchange[parity_ ^ 1];
      for (unsigned r = 0; r < ctas_; ++r) {
        if (r < rank_) before += weight_of(buf[r]);
        total += weight_of(buf[r]);
      }
    }
    if (total == 0) return false;
    // floor(total u), below total
    const u64 target = __umul64hi(total << 4, static_cast<u64>(u * 4294967296.f) << 28);
    if (target < before || target >= before + mine_all) return true;  // another CTA has it
    // the warp's run that holds it (or, the parts rounded one by one, the last with any)
    int holder = 0;
    u64 start = before;
    for (int i = 0; i < kWarps; ++i) {
      const u64 m = weight_of(sh_.warp[i]);
      if (m > 0) {
        holder = i;
        start = before;
        if (target < before + m) break;
      }
      before += m;
    }
    before = start;
    const float more = (w.ratio.hi - w.near) + w.ratio.lo;
    const int first = (static_cast<int>(rank_) * kWarps + holder) * run_;
    const int last = min(first + run_, (a_.vocab + E::kVec - 1) / E::kVec);
    float x[E::kVec], y[E::kVec];
    float2 r[E::kVec / 2], none = make_float2(0.f, 0.f);
    uint32_t heavy = 0;
    const auto vector_weight = [&](int v) {
      heavy = load_both(v, w, x, y);
      light_weights<false>(v, heavy, x, y, w, more, d_least, sc, r, none, none, none);
      u64 m = __float2uint_rn(sum_of(r) * w.unit);
#pragma unroll 1
      for (uint32_t bits = heavy; bits != 0; bits &= bits - 1) {
        const int index = v * E::kVec + __ffs(bits) - 1;
        m += heavy_weight(E::one(x_[index]), w.minus_q ? E::one(y_[index]) : 0.f, index, w, sc);
      }
      return m;
    };
    const auto put_token = [&](int token) {
      a_.tokens[row] = token;
      a_.logp[row] = log_share(E::one(x_[token]), w.p, sc);
    };
    if (threadIdx.x == 0) sh_.found = 0, sh_.spare = -1;
    for (int v0 = first; v0 < last && target >= before; v0 += kThreads) {  // a vector to each thread
      const int v = v0 + static_cast<int>(threadIdx.x);
      const u64 mine = v < last ? vector_weight(v) : 0;
      u64 upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 other = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += other;
      }
      __syncthreads();  // the sums have been read
      if (lane == 31) sh_.scan[warp] = upto;
      __syncthreads();
      u64 at = before + upto - mine;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) at += sh_.scan[i];
        before += sh_.scan[i];
      }
      if (target >= at && target < at + mine) {
        // the first whose own rounded weight passes it, or (rounding) the last with any
        int token = -1, any = -1;
#pragma unroll
        for (int e = 0; e < E::kVec; ++e) {
          const int index = v * E::kVec + e;
          const float f = e & 1 ? r[e / 2].y : r[e / 2].x;
          const u64 m = heavy >> e & 1u ? static_cast<u64>(heavy_weight(x[e], w.minus_q ? y[e] : 0.f, index, w, sc))
                                        : __float2uint_rn(f * w.unit);
          if (token < 0 && target < at + m) token = index;
          if (m > 0 || f > 0.f) any = index;
          at += m;
        }
        put_token(token < 0 ? any : token);
        sh_.found = 1;
      }
    }
    __syncthreads();
    if (sh_.found) return true;
    // The run's vectors come to a few units less than the run did with the near
    // ratio: the last token of it that weighs something, or that p allows.
    for (int v = first + static_cast<int>(threadIdx.x); v < last; v += kThreads) {
      const u64 m = vector_weight(v);
      int best = -1;
#pragma unroll
      for (int e = 0; e < E::kVec; ++e) {
        const float f = e & 1 ? r[e / 2].y : r[e / 2].x;
        const bool weighs = f > 0.f || (heavy >> e & 1u && m > 0);
        if (x[e] > -INFINITY && v * E::kVec + e < a_.vocab && v * E::kVec + e != w.without)
          best = max(best, (weighs ? 1 << 18 : 0) + v * E::kVec + e);
      }
      if (best >= 0) atomicMax(&sh_.spare, best);
    }
    __syncthreads();
    if (threadIdx.x == 0 && sh_.spare >= 0) put_token(sh_.spare & ((1 << 18) - 1));
    return true;
  }
  static SA_DEV void add(Sums& to, const Sums& v) {
    to.weight += v.weight;
    to.p += v.p;
    to.q += v.q;
    to.slope += v.slope;
  }

  Shared& sh_;
  const VerifyArgs& a_;
  cg::cluster_group cluster_;
  int slices_;
  unsigned rank_, ctas_;
  int parity_ = 0;
  int run_ = 0, v0_ = 0, v1_ = 0;  // vectors of a warp, and the warp's
  const T* x_ = nullptr;
  const T* y_ = nullptr;
};

template <int kType>
__global__ void __launch_bounds__(kThreads, kPerSm) verify_draw_kernel(const __grid_constant__ VerifyArgs a, int slices) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks();
  {
    Sequence<kType> s(sh, a, slices);
    s.run(blockIdx.x / ctas);
  }
  if (ctas > 1) cluster.sync();  // no CTA leaves while another may still write to its shared memory
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
  // A row in as few slices as keep the GPU busy (3 CTAs an SM, a few turns of them), each a whole number of turns that
  // a thread has in flight, so that none is nearly empty.
  const int all = turns_for(kType, a.vocab);
  int slices = std::max(ceil_div(all, kStatMostVecs), 1);
  if (items > 0)
    slices = std::max(slices, static_cast<int>(std::min<long long>(most_slices(kType, a.vocab), 9LL * device_sms() / items)));
  const int turns = ceil_div(ceil_div(all, slices), kStatVecs) * kStatVecs;
  slices = ceil_div(all, turns);
  if (items > 0)
    verify_rows_kernel<kType><<<static_cast<unsigned>(items * slices), kStatThreads, 0, s>>>(a, slices, turns);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Enough CTAs for a sequence to be quick, not so many that the batch comes in several turns.
  int ctas = 1;
  while (ctas < kMaxCluster && ctas * 8192 < a.vocab && 2LL * ctas * a.num_seqs <= 2 * device_sms() * kPerSm) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<kType>, a, slices);
}

}  // namespace

size_t verify_workspace_bytes(int dtype, int rows, int vocab) {
  return static_cast<size_t>(rows) * 2 * most_slices(dtype, vocab) * sizeof(float4);
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_type<0>(a, s);
  if (a.dtype == 1) return launch_type<1>(a, s);
  return launch_type<2>(a, s);
}

}  // namespace sa
