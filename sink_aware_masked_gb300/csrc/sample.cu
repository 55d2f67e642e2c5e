// Token sampling with temperature, top-k, top-p and min-p from given random
// numbers, with the token's log-probability (what the GRPO loss takes as
// logp_old).
//
//   e_i = exp((x_i - max x) / T),  Z = sum e
//   order: larger x first, of equal ones the lower index
//   top-k keeps the first k; top-p of those the shortest run whose mass is at
//   least p times theirs; min-p of those the ones with e_i >= min_p
//   token = the first index, in index order, whose kept mass up to and
//   including it exceeds u times the kept mass
//
// A row belongs to a CTA, or, where the vocabulary is longer than one CTA's
// slice, to a cluster of two or four.  Pass 1 reads it from HBM and leaves the
// maximum, Z and every thread's own maximum; later passes find it in L2.
//
//   Nothing to select: the token lies in the chunk whose mass, known from
//   pass 1, holds u Z; that chunk alone is read again.
//   top-k or min-p: the threads' maxima (or min-p itself) bound the kept
//   logits from below.  Pass 2 collects the few that reach the bound, and one
//   CTA sorts them; what is kept is a run at their front.
//   Otherwise (top-p alone, top-k in the thousands, long lists): a histogram
//   (count and mass) over equal steps of x finds the step in which a cut
//   lies; its members, if few, are ranked by one CTA, else they are split
//   again by their exact key (x's bits and the index, so all keys differ)
//   until they are few.  A last pass sums what is kept.
//
// Measured (GB300): 1 x 50257 fp32 with top-k and top-p 13.7 us; 256 x 201088
// bf16 at T = 0.9 (103 MB, 15 us at the copy rate; three batches in turn, so that
// none is found in L2): no selection 61 us, greedy 47, top-k 200 81, min-p 0.02
// 64, top-p 0.95 215, top-k 5000 180, all of these mixed 119.  The first rows' pass 1
// runs at HBM speed, later ones' is bound by issue and latency (with the next
// rows brought into L2 ahead the time is the same); what a row waits for is
// the latency of its phases, with two CTAs on an SM.
//
// Arithmetic.  e is fp32 (the difference before the scale: a large logit must
// not lose what tells it from its neighbours).  Partial sums of a thread are
// fp32, and so is Z, in a fixed order; masses that decide are 64-bit fixed
// point: those of chunks in units of 2^-40, inside the chunk that holds the
// token as fine as its mass allows, those of logits under selection in units
// of Z 2^-43.  Integer sums are the
// same in every order, so histogram atomics leave the result reproducible,
// and 2^18 roundings lose at most 2^-22 (chunks) or 2^-25 of the whole.  FP64 is
// not used: its rate on this GPU would cost more than all the rest.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 4;
constexpr int kSliceLogits = 16384;       // a slice this long is not shared out further
constexpr int kIndexBits = 18;            // vocabularies up to 2^18
constexpr int kBins = 1024;
constexpr int kGather = kThreads;         // members that the last step of a search ranks, one per thread
constexpr int kList = 2048;               // candidates that are sorted at once
constexpr int kSlice = 8192;              // candidates of a slice that are kept for a search's passes
constexpr int kRuns = 512;                // runs of indices; 512 of 512 are the largest vocabulary
constexpr int kQueue = kSlice / kWarps;    // candidates a warp can hold back: 31 and a vector of each lane
constexpr int kChunks = 16;               // runs of a slice whose masses are kept apart
constexpr int kUnroll = 4;                // vectors a thread has in flight
constexpr float kMassOne = 8796093022208.f;   // 2^43
constexpr float kSumOne = 1099511627776.f;    // 2^40
constexpr int kLowBits = 13;
constexpr float kLowest = -3.402823466e38f;   // fp32's lowest finite value

typedef unsigned long long u64;

struct Pick {  // what a histogram step found
  int bin;
  u64 members;     // candidates in the bin
  u64 count, mass; // of all bins before it
  u64 target;
};

struct Histogram {
  uint32_t count[kBins], mass_hi[kBins], mass_lo[kBins];  // this CTA's
  uint32_t all_count[kBins];                              // CTA 0: the row's
  u64 all_mass[kBins];
  u64 key[kGather], key_mass[kGather], sorted[kGather], sorted_mass[kGather];
};

struct alignas(16) Sorted {
  u64 key[kList];
  u64 bin[kRuns];  // masses by index
};

struct Shared {
  u64 exchange[2][kMaxCluster][2];
  u64 warp_u[kWarps], warp_v[kWarps];
  float chunk_max[kChunks][kWarps], chunk_sum[kChunks][kWarps];
  u64 chunk_mass[kChunks][kWarps];
  u64 cut, cut_mass;
  Pick pick;
  int gathered, found, last;
  int slice_n;
  union {
    Histogram h;
    Sorted s;
  };
  float slice_x[kSlice];
  uint16_t slice_at[kSlice];  // index in the slice
};

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
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
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

// Larger x, larger key; -0 and +0 are one value.
SA_DEV uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
SA_DEV float key_value(uint32_t key) {
  return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}
SA_DEV u64 full_key(float x, int index) {
  return static_cast<u64>(order_key(x)) << kIndexBits | ((1u << kIndexBits) - 1 - index);
}

SA_DEV float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <class T>
SA_DEV T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <class T>
SA_DEV T warp_scan(T x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

template <int kType>
class Row {
 public:
  typedef Elem<kType> E;
  typedef typename E::T T;

  SA_DEV Row(Shared& sh) : sh_(sh), cluster_(cg::this_cluster()) {
    rank_ = cluster_.block_rank();
    ctas_ = cluster_.num_blocks();
  }

  SA_DEV void run(const SampleArgs& a, int row, int slice) {
    const int tid = threadIdx.x;
    cluster_.barrier_arrive();
    vocab_ = a.vocab;
    first_ = min(static_cast<int>(rank_) * slice, a.vocab);
    const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride + first_;
    shift_ = static_cast<int>((reinterpret_cast<uintptr_t>(x) / sizeof(T)) % E::kVec);
    base_ = x - shift_;
    end_ = shift_ + min(slice, a.vocab - first_);
    vectors_ = end_ > shift_ ? (end_ + E::kVec - 1) / E::kVec : 0;
    const int turns = (vectors_ + kThreads - 1) / kThreads;
    chunk_turns_ = max((turns + kChunks - 1) / kChunks, 1);
    chunk_turns_ = (chunk_turns_ + kUnroll - 1) / kUnroll * kUnroll;

    const float temperature = a.temperature[row], top_p = a.top_p[row], min_p = a.min_p[row], u = a.u[row];
    int k = a.top_k[row];
    // up to 1e36, so that 1 / T stays a normal number and a difference that overflows has no mass either way
    const bool valid = temperature >= 0.f && temperature <= 1e36f && top_p == top_p && min_p == min_p && u == u;
    const bool greedy = temperature == 0.f;
    temperature_ = greedy || !valid ? 1.f : temperature;
    scale_ = fminf(__fdiv_rn(kLog2e, temperature_), 1e38f);
    if (greedy || top_p <= 0.f) k = 1;
    const bool by_count = k > 0 && k < vocab_, by_mass = top_p < 1.f, by_floor = min_p > 0.f;
    const bool chunks = !by_count && !by_mass && !by_floor;

    if (!valid) {
      cluster_.barrier_wait();
      if (rank_ == 0 && tid == 0) put(a, row, -1, NAN, NAN);
      return;
    }
    const float thread_max = pass1(chunks);
    cluster_.barrier_wait();  // every CTA of the cluster runs: its shared memory may be written
    reduce(thread_max, by_count && k > 1 ? k : 0);
    if (z_ == 0.f || max_ == INFINITY || z_ != z_) {
      const float v = z_ == 0.f ? -INFINITY : NAN;  // nothing is allowed, or something is not a number
      if (rank_ == 0 && tid == 0) put(a, row, -1, v, v);
      return;
    }
    to_fixed_ = __fdiv_rn(kMassOne, z_);

    if (k == 1) {  // the largest, of equal ones the lowest index
      int at = vocab_;
      each_from(max_, [&](float, int index) { at = min(at, index); });
      at = block_min(at);
      int best = vocab_;
      exchange(static_cast<u64>(at), [&](u64 v) { best = min(best, static_cast<int>(v)); });
      if (rank_ == 0 && tid == 0) put(a, row, best, -ln(z_), 0.f);
      return;
    }
    // below 1, so that the kept mass exceeds the target
    const float share = fminf(fmaxf(u, 0.f), 0.99999994f);
    cut_ = 0;
    min_mass_ = fminf(min_p, 1.f);
    if (chunks) {
      sample_chunks(a, row, share);
      return;
    }
    // what lies below floor is not kept, nor does its mass count for top-p
    float floor = -INFINITY;
    if (by_count) floor = count_floor();
    if (by_floor && !(by_count && by_mass)) floor = fmaxf(floor, mass_floor(min_mass_ * 0.999f));
    if (floor > -INFINITY && sample_list(a, row, floor, by_count ? k : vocab_, by_mass ? top_p : 1.f, by_count, share))
      return;
    // what lies below (1 - p) Z / vocab holds less than (1 - p) Z together; 1 % to spare for rounding
    if (!by_count && by_mass)
      floor = fmaxf(floor, mass_floor((1.f - top_p) * 0.99f * z_ / vocab_));
    floor_ = floor;
    if (by_floor && !by_count && !by_mass) make_slice_list();
    if (by_count || by_mass) {
      // steps for the first histogram: the candidates' range, or what holds all mass that counts
      const float range = floor > -INFINITY ? max_ - floor : 30.f * temperature_;
      per_step_ = range > 0.f ? fminf((kBins - 1) / range, 1e30f) : 0.f;
      u64 kept = 0;
      if (by_count) kept = search(true, k, 0.f, by_mass);
      if (by_mass) search(false, by_count ? part_of(kept, top_p) : 0, top_p, true);
    }
    const u64 least = min_p_cut();
    cut_ = cut_ > least ? cut_ : least;
    if (listed_) {
      __syncthreads();  // the histogram's place is used again
      pick(a, row, share, first_, end_ - shift_, ctas_ > 1, [&](auto f) {
        for (int i = tid; i < list_n_; i += kThreads) {
          const float x = sh_.slice_x[i];
          const int index = first_ + sh_.slice_at[i];
          const float e = kept_mass(x, index);
          if (e > 0.f) f(index, static_cast<u64>(e * to_fixed_), x);
        }
      });
      return;
    }
    chunk_masses();
    sample_chunks(a, row, share);
  }

 private:
  // Every CTA of the cluster gives a number and takes all of them in rank order.
  template <class F>
  SA_DEV void exchange(u64 v, F take) {
    if (ctas_ == 1) {
      take(v);
      return;
    }
    u64 (*buf)[2] = sh_.exchange[parity_];
    parity_ ^= 1;  // the other half may still be read by a slower CTA
    if (threadIdx.x < ctas_) cluster_.map_shared_rank(&buf[0][0], threadIdx.x)[2 * rank_] = v;
    cluster_.sync();
    for (unsigned r = 0; r < ctas_; ++r) take(buf[r][0]);
  }
  SA_DEV void sync_all() {
    if (ctas_ == 1)
      __syncthreads();
    else
      cluster_.sync();
  }

  // Vector v of the slice, aligned as in global memory, -inf outside the slice.
  SA_DEV uint4 load(int v) const {
    union {
      uint4 q;
      T t[E::kVec];
    } w;
    if (v * E::kVec >= shift_ && (v + 1) * E::kVec <= end_) return __ldg(reinterpret_cast<const uint4*>(base_) + v);
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) {
      const int i = v * E::kVec + e;
      w.t[e] = i >= shift_ && i < end_ ? base_[i] : E::lowest();
    }
    return w.q;
  }
  SA_DEV int index_of(int v) const { return first_ + v * E::kVec - shift_; }

  // f(vectors, number of the first) for the slice's vectors in [turn0, turn1) x threads, some of the thread's at
  // once, which are kThreads apart; padding is -inf.
  template <class F>
  SA_DEV void turns_of_groups(int turn0, int turn1, F f) {
    const int tid = threadIdx.x, whole = end_ / E::kVec / kThreads;  // turns of whole vectors, the first one aside
    const auto checked = [&](int t) {
      const int v = t * kThreads + tid;
      if (v < vectors_) {
        const uint4 w[1] = {load(v)};
        f(w, v);
      }
    };
    int t = turn0;
    if (t == 0 && shift_ > 0 && t < turn1) checked(t++);
    for (; t + kUnroll <= min(turn1, whole); t += kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(base_) + (t + i) * kThreads + tid);
      f(w, t * kThreads + tid);
    }
#pragma unroll 1
    for (; t < turn1; ++t) checked(t);
  }
  // f(vector, its number), one by one.
  template <class F>
  SA_DEV void turns_of_vectors(int turn0, int turn1, F f) {
    turns_of_groups(turn0, turn1, [&](const auto& w, int v) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(w) / sizeof(uint4)); ++i) f(w[i], v + i * kThreads);
    });
  }
  template <class F>
  SA_DEV void each_vector(F f) {
    turns_of_vectors(0, (vectors_ + kThreads - 1) / kThreads, f);
  }
  // f(x, index) for the slice's logits from floor on, above -inf.
  template <class F>
  SA_DEV void each_from(float floor, F f) {
    each_vector([&](uint4 w, int v) {
      if (!(E::largest(w) >= floor)) return;
      float x[E::kVec];
      E::unpack(w, x);
#pragma unroll
      for (int e = 0; e < E::kVec; ++e)
        if (x[e] >= floor && x[e] > -INFINITY) f(x[e], index_of(v) + e);
    });
  }
  SA_DEV int chunks() const {
    return ((vectors_ + kThreads - 1) / kThreads + chunk_turns_ - 1) / chunk_turns_;
  }

  // Maximum and sum of one pass, the sum relative to the running maximum; per
  // chunk and warp, or (by_chunk false) per warp as chunk 0.
  SA_DEV float pass1(bool by_chunk) {
    const int warp = threadIdx.x >> 5, turns = (vectors_ + kThreads - 1) / kThreads;
    const int step = by_chunk ? chunk_turns_ : max(turns, 1);
    float top = kLowest;  // so that a difference with -inf is -inf
    // In the ordinary range the exponent is one fused x * scale - ref, with
    // ref the rounded top * scale; what ref was rounded by is put right at
    // the end.  Beyond it (where ref's rounding would swamp the exponent) the
    // difference is taken first.
    float ref = 0.f;
    bool fused = false;
    for (int c = 0; c * step < max(turns, 1); ++c) {
      float2 sum = make_float2(0.f, 0.f);
      turns_of_groups(c * step, min((c + 1) * step, turns), [&](const auto& w, int) {
        constexpr int kGroup = sizeof(w) / sizeof(uint4);
        float m = E::largest(w[0]);
#pragma unroll
        for (int i = 1; i < kGroup; ++i) m = fmaxf(m, E::largest(w[i]));
        if (m > top) {
          const float next = m * scale_;
          const bool next_fused = fabsf(next) < 1048576.f;
          float by = ref - next;
          if (!fused || !next_fused) {  // from top's or ref's basis to m's or next's: ref and next are rounded
            by = (top - m) * scale_;
            if (fused) by -= fmaf(top, scale_, -ref);
            if (next_fused) by += fmaf(m, scale_, -next);
          }
          const float f = ex2(by);
          sum.x *= f;
          sum.y *= f;
          top = m;
          ref = next;
          fused = next_fused;
        }
        const float2 c2 = make_float2(scale_, scale_), r2 = make_float2(-ref, -ref);
        const bool by_fma = fused;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          float x[E::kVec];
          E::unpack(w[i], x);
          if (by_fma) {
#pragma unroll
            for (int e = 0; e < E::kVec; e += 2) {
              const float2 t = ffma2(make_float2(x[e], x[e + 1]), c2, r2);
              sum = fadd2(sum, make_float2(ex2(t.x), ex2(t.y)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) sum.x += ex2((x[e] - top) * scale_);
          }
        }
      });
      float total = sum.x + sum.y;
      if (fused) total *= ex2(-fmaf(top, scale_, -ref));
      const float warp_top = warp_max(top);
      const float warp_total = warp_sum(total * ex2((top - warp_top) * scale_));
      if ((threadIdx.x & 31) == 0) sh_.chunk_max[c][warp] = warp_top, sh_.chunk_sum[c][warp] = warp_total;
    }
    pass1_parts_ = (by_chunk ? chunks() : 1) * kWarps;
    return top;
  }

  // From pass 1, with one exchange: max_, z_ (0: no logit above -inf, NaN: a
  // NaN or +inf among them), the chunks' sums relative to max_ in fixed
  // point, and the bound of the k largest.  Every warp does it all.
  SA_DEV void reduce(float thread_max, int k) {
    const int lane = threadIdx.x & 31;
    uint32_t least = quota_key(thread_max, k);
    __syncthreads();
    const float* maxima = &sh_.chunk_max[0][0];
    const float* sums = &sh_.chunk_sum[0][0];
    float top = kLowest, sum = 0.f;
    for (int i = lane; i < pass1_parts_; i += 32) top = fmaxf(top, maxima[i]);
    top = warp_max(top);
    for (int i = lane; i < pass1_parts_; i += 32) sum += sums[i] * ex2((maxima[i] - top) * scale_);
    sum = warp_sum(sum);
    if (ctas_ == 1) {
      max_ = top;
      z_ = sum;
    } else {
      u64 (*buf)[2] = sh_.exchange[parity_];
      parity_ ^= 1;
      if (threadIdx.x < ctas_) {
        u64* to = cluster_.map_shared_rank(&buf[0][0], threadIdx.x) + 2 * rank_;
        to[0] = static_cast<u64>(__float_as_uint(top)) << 32 | __float_as_uint(sum);
        to[1] = least;
      }
      cluster_.sync();
      max_ = kLowest;
      for (unsigned r = 0; r < ctas_; ++r) {
        max_ = fmaxf(max_, __uint_as_float(static_cast<uint32_t>(buf[r][0] >> 32)));
        least = min(least, static_cast<uint32_t>(buf[r][1]));
      }
      z_ = 0.f;
      for (unsigned r = 0; r < ctas_; ++r)
        z_ += __uint_as_float(static_cast<uint32_t>(buf[r][0])) *
              ex2((__uint_as_float(static_cast<uint32_t>(buf[r][0] >> 32)) - max_) * scale_);
    }
    count_key_ = least;
    for (int i = threadIdx.x; i < pass1_parts_; i += kThreads)
      (&sh_.chunk_mass[0][0])[i] = static_cast<u64>(sums[i] * ex2((maxima[i] - max_) * scale_) * kSumOne);
    __syncthreads();
  }

  // ceil(mass * p)
  static SA_DEV u64 part_of(u64 mass, float p) {
    const u64 m = mass << 20, q = static_cast<u64>(fmaxf(p, 0.f) * 4294967296.f) << 12;  // mass < 2^44, p < 1
    return __umul64hi(m, q) + (m * q != 0);
  }
  // The mass of everything, given that of the candidates: theirs alone where
  // no more is left than rounding, so that equal masses are counted exactly.
  SA_DEV u64 whole_mass(u64 candidates) const {
    const u64 all = static_cast<u64>(z_ * to_fixed_);
    return all > candidates + (candidates >> 20) ? all : candidates;
  }

  // floor(mass * u), below mass.
  static SA_DEV u64 u_of(u64 mass, float u) {
    return __umul64hi(mass << 4, static_cast<u64>(u * 4294967296.f) << 28);  // mass < 2^60, u < 1
  }

  static SA_DEV float ln(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y * kLn2;
  }

  SA_DEV float mass(float x) const { return ex2((x - max_) * scale_); }
  // min-p of 1 keeps what equals the largest, by its key, since a smaller logit's e may round to 1 (a large temperature,
  // a near tie).
  SA_DEV u64 min_p_cut() const { return min_mass_ >= 1.f ? static_cast<u64>(order_key(max_)) << kIndexBits : 0; }
  SA_DEV u64 fixed(float x) const { return static_cast<u64>(mass(x) * to_fixed_); }

  SA_DEV int block_min(int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((threadIdx.x & 31) == 0) sh_.warp_u[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) x = min(x, static_cast<int>(sh_.warp_u[w]));
    return x;
  }

  // The logit at which e is `least`, rounded down.
  SA_DEV float mass_floor(float least) const {
    const float f = max_ + ln(least) * temperature_ * (least < 1.f ? 1.0001f : 1.f);
    return f - fabsf(f) * 2.4e-7f;
  }

  // A value that k / ctas of the threads' maxima reach (the largest such one,
  // to the upper 16 bits of its key), as a key: at least k logits of the row
  // reach the least of these over the row's CTAs.  0 where there is none.
  SA_DEV uint32_t quota_key(float thread_max, int k) const {
    const int quota = (k + ctas_ - 1) / ctas_;
    if (k <= 0 || quota > kThreads) return 0;
    const uint32_t key = thread_max > kLowest ? order_key(thread_max) : 0;
    uint32_t lo = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t mid = lo | 1u << bit;
      if (__syncthreads_count(key >= mid) >= quota) lo = mid;
    }
    return lo;
  }
  SA_DEV float count_floor() const {
    const float f = key_value(count_key_);
    return f > kLowest ? f : -INFINITY;  // key 0: some CTA has too few logits above -inf, or k is large
  }

  // Collects the logits from floor on, sorts them and samples from their
  // front.  False (for all CTAs alike) if they are too many.
  SA_DEV bool sample_list(const SampleArgs& a, int row, float floor, int k, float top_p, bool by_count, float share) {
    const int tid = threadIdx.x;
    if (tid == 0) sh_.gathered = 0;
    __syncthreads();
    each_from(floor, [&](float x, int index) {
      const int at = atomicAdd(&sh_.gathered, 1);
      if (at < kList) sh_.s.key[at] = full_key(x, index);
    });
    sync_all();
    // CTA 0 takes the others' lists behind its own
    int counts[kMaxCluster], n = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      counts[r] = r < static_cast<int>(ctas_) ? *cluster_.map_shared_rank(&sh_.gathered, r) : 0;
      n += counts[r];
    }
    if (n <= kList && rank_ == 0) {
      int at = counts[0];
#pragma unroll
      for (int r = 1; r < kMaxCluster; ++r) {
        const u64* from = cluster_.map_shared_rank(sh_.s.key, r < static_cast<int>(ctas_) ? r : 0);
        for (int i = tid; i < counts[r]; i += kThreads) sh_.s.key[at + i] = from[i];
        at += counts[r];
      }
    }
    sync_all();  // the lists have been read
    if (n > kList) return false;
    if (rank_ != 0) return true;

    sort_keys(n);
    // masses of the first k, in order: kPer entries per thread
    constexpr int kPer = kList / kThreads;
    u64 upto[kPer], own = 0;
    float e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      e[j] = i < min(n, k) ? mass(key_value(static_cast<uint32_t>(sh_.s.key[i] >> kIndexBits))) : 0.f;
      own += static_cast<u64>(e[j] * to_fixed_);
      upto[j] = own;
    }
    const u64 before = block_scan(own, sh_.warp_u) - own;
    u64 all = 0;
    for (int w = 0; w < kWarps; ++w) all += sh_.warp_u[w];
    // top-p counts against the first k, or, without top-k, against everything
    const u64 target = top_p < 1.f ? part_of(by_count ? all : whole_mass(all), top_p) : ~0ull;
    const u64 least = min_p_cut();
    int kept = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      const u64 excluded = before + (j > 0 ? upto[j > 0 ? j - 1 : 0] : 0);
      if (i < min(n, k) && e[j] >= min_mass_ && e[j] > 0.f && (i == 0 || excluded < target) && sh_.s.key[i] >= least)
        ++kept;
    }
    kept = block_sum_int(kept);  // they are the first ones
    pick(a, row, share, 0, vocab_, false, [&](auto f) {
      for (int i = tid; i < kept; i += kThreads) {
        const u64 key = sh_.s.key[i];
        const float x = key_value(static_cast<uint32_t>(key >> kIndexBits));
        f((1 << kIndexBits) - 1 - static_cast<int>(key & ((1u << kIndexBits) - 1)), static_cast<u64>(mass(x) * to_fixed_),
          x);
      }
    });
    return true;
  }

  // The token among kept entries, indices [lo, lo + span): first the run of
  // indices that holds the target, then the index in it.  each(f) calls
  // f(index, mass, x) for the thread's entries; across: every CTA has some,
  // in index order.
  template <class Each>
  SA_DEV void pick(const SampleArgs& a, int row, float share, int lo, int span, bool across, Each each) {
    const int tid = threadIdx.x, width = max((span + kRuns - 1) / kRuns, 1);
    constexpr int kRun = kRuns / kThreads;
    u64 target = 0, total = 0;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
      for (int i = tid; i < kRuns; i += kThreads) sh_.s.bin[i] = 0;
      __syncthreads();
      each([&](int index, u64 m, float) {
        if (level == 0)
          atomicAdd(&sh_.s.bin[(index - lo) / width], m);
        else if (index >= lo && index < lo + width)
          sh_.s.bin[index - lo] = m;
      });
      __syncthreads();
      u64 in = 0;
#pragma unroll
      for (int j = 0; j < kRun; ++j) in += sh_.s.bin[tid * kRun + j];
      u64* sums = level == 0 ? sh_.warp_u : sh_.warp_v;
      u64 run = block_scan(in, sums) - in;
      if (level == 0) {
        for (int w = 0; w < kWarps; ++w) total += sums[w];
        u64 before = 0;
        const u64 own = total;
        if (across) {
          unsigned r = 0;
          total = 0;
          exchange(own, [&](u64 v) {
            if (r++ < rank_) before += v;
            total += v;
          });
        }
        target = u_of(total, share);
        if (!(before <= target && before + own > target)) return;  // exactly one CTA holds it
        target -= before;
      }
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        const u64 next = run + sh_.s.bin[tid * kRun + j];
        if (next > target && run <= target) {
          sh_.found = tid * kRun + j;
          sh_.cut_mass = run;
        }
        run = next;
      }
      __syncthreads();
      if (level == 0) {
        lo += sh_.found * width;
        target -= sh_.cut_mass;
        __syncthreads();
      }
    }
    const int token = lo + sh_.found;
    each([&](int index, u64 m, float x) {  // logq of a token that is kept alone is 0 exactly
      if (index == token) put_token(a, row, token, x, m == total ? mass(x) : __fdiv_rn(static_cast<float>(total), to_fixed_));
    });
  }

  // The slice's candidates (floor_ and above) into shared memory, if those of
  // every slice fit.  A warp claims places for all its lanes at once.
  SA_DEV void make_slice_list() {
    const int lane = threadIdx.x & 31;
    listed_ = floor_ > -INFINITY || end_ - shift_ <= kSlice;
    if (threadIdx.x == 0) sh_.slice_n = 0;
    __syncthreads();
    if (listed_) {
      each_vector_of_warp([&](uint4 w, int v) {
        claim(w, v, [&](int total) {
          int at = 0;
          if (lane == 0) at = atomicAdd(&sh_.slice_n, total);
          return __shfl_sync(0xffffffffu, at, 0);
        }, sh_.slice_x, sh_.slice_at, kSlice);
      });
    }
    __syncthreads();
    list_n_ = sh_.slice_n;
    const bool mine = listed_ && list_n_ <= kSlice;
    listed_ = true;
    exchange(mine, [&](u64 v) { listed_ &= v != 0; });
  }

  // f(vector, number) for every vector with a logit from floor_ on among the
  // warp's 32; all lanes take part, those without a vector with padding.
  template <class F>
  SA_DEV void each_vector_of_warp(F f) {
    const int turns = (vectors_ + kThreads - 1) / kThreads;
    uint4 none;
    T* fill = reinterpret_cast<T*>(&none);
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) fill[e] = E::lowest();
    for (int t = 0; t < turns; t += kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int v = (t + i) * kThreads + threadIdx.x;
        w[i] = v < vectors_ ? load(v) : none;
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (__any_sync(0xffffffffu, E::largest(w[i]) >= floor_)) f(w[i], (t + i) * kThreads + threadIdx.x);
    }
  }

  // Sorts sh_.s.key[0 .. n), largest first; the keys differ.
  SA_DEV void sort_keys(int n) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (n <= kThreads) {  // a key's place is the number of larger ones
      const u64 mine = tid < n ? sh_.s.key[tid] : 0;
      if (tid == n) sh_.s.key[n] = 0;  // n + 1 <= kList
      __syncthreads();
      int place = 0;
      if ((tid & ~31) < n)
        for (int j = 0; j < n; j += 2) {
          const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sh_.s.key[j]);
          place += (two.x > mine) + (two.y > mine);
        }
      __syncthreads();
      if (tid < n) sh_.s.key[place] = mine;
      __syncthreads();
      return;
    }
    int size = 2 * kThreads;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kThreads) sh_.s.key[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = 2; k <= size; k *= 2)
#pragma unroll 1
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < size / 2; i += kThreads) {
          const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
          const u64 x = sh_.s.key[lo], y = sh_.s.key[hi];
          if ((x < y) == ((lo & k) == 0)) sh_.s.key[lo] = y, sh_.s.key[hi] = x;
        }
        // pairs at most 32 apart stay inside the 64 keys of one warp
        if (j > 32 || (j == 1 && k >= 64))
          __syncthreads();
        else
          __syncwarp();
      }
    __syncthreads();
  }

  SA_DEV int block_sum_int(int x) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh_.warp_u[threadIdx.x >> 5] = x;
    __syncthreads();
    int s = 0;
    for (int w = 0; w < kWarps; ++w) s += static_cast<int>(sh_.warp_u[w]);
    __syncthreads();
    return s;
  }

  // f(x, index) for the slice's candidates: from their list, or, while there
  // is none, from memory.  There a warp queues what it finds and calls f for
  // 32 at a time, since among neighbours few lanes have a candidate.
  template <class F>
  SA_DEV void each_candidate(F f) {
    if (listed_) {
      for (int i = threadIdx.x; i < list_n_; i += kThreads) f(sh_.slice_x[i], first_ + sh_.slice_at[i]);
      return;
    }
    if (floor_ == -INFINITY) {  // every logit is one (256 x 201088, top-k 5000: 180 us; by the queue 281)
      each_from(floor_, f);
      return;
    }
    const int lane = threadIdx.x & 31;
    float* queue_x = sh_.slice_x + (threadIdx.x >> 5) * kQueue;
    uint16_t* queue_at = sh_.slice_at + (threadIdx.x >> 5) * kQueue;
    int n = 0;
    const auto drain = [&](int least) {
      __syncwarp();
      while (n >= least && n > 0) {
        const int i = n - 32 + lane;
        if (i >= 0) f(queue_x[i], first_ + queue_at[i]);
        n = max(n - 32, 0);
      }
      __syncwarp();
    };
    each_vector_of_warp([&](uint4 w, int v) {
      claim(w, v, [&](int total) {
        const int at = n;
        n += total;
        return at;
      }, queue_x, queue_at, kQueue);
      if (n >= 32) drain(32);
    });
    drain(1);
  }

  // Writes a vector's candidates of all the warp's lanes to a list, from the
  // place that claim_places(their number) gives; those beyond cap are dropped.
  template <class F>
  SA_DEV void claim(uint4 w, int v, F claim_places, float* xs, uint16_t* ats, int cap) {
    float x[E::kVec];
    E::unpack(w, x);
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) mine |= static_cast<uint32_t>(x[e] >= floor_ && x[e] > -INFINITY) << e;
    const int count = __popc(mine), upto = warp_scan(count);
    int at = claim_places(__shfl_sync(0xffffffffu, upto, 31)) + upto - count;
    const int index = index_of(v) - first_;
#pragma unroll
    for (int e = 0; e < E::kVec; ++e)
      if (mine >> e & 1u) {
        if (at < cap) {
          xs[at] = x[e];
          ats[at] = static_cast<uint16_t>(index + e);
        }
        ++at;
      }
  }

  SA_DEV int step_of(float x) const { return static_cast<int>(fminf((max_ - x) * per_step_, kBins - 1.f)); }

  // Histogram of what bin_of gives a bin (>= 0), summed over the cluster; the
  // first bin at which count or mass reaches the target, starting from before.
  template <class F>
  SA_DEV Pick histogram(bool by_count, u64 target, float top_p, u64 count0, u64 mass0, bool masses, F bin_of) {
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += kThreads) sh_.h.count[i] = sh_.h.mass_hi[i] = sh_.h.mass_lo[i] = 0;
    __syncthreads();
    each_candidate([&](float x, int index) {
      const int bin = bin_of(x, index);
      if (bin < 0) return;
      atomicAdd(&sh_.h.count[bin], 1u);
      if (!masses) return;
      const u64 m = fixed(x);
      atomicAdd(&sh_.h.mass_hi[bin], static_cast<uint32_t>(m >> kLowBits));
      atomicAdd(&sh_.h.mass_lo[bin], static_cast<uint32_t>(m & ((1u << kLowBits) - 1)));
    });
    sync_all();
    const int share = kBins / ctas_;
    for (int i = rank_ * share + tid; i < static_cast<int>(rank_ + 1) * share; i += kThreads) {
      uint32_t n = 0;
      u64 m = 0;
      for (unsigned r = 0; r < ctas_; ++r) {
        n += cluster_.map_shared_rank(sh_.h.count, r)[i];
        m += (static_cast<u64>(cluster_.map_shared_rank(sh_.h.mass_hi, r)[i]) << kLowBits) +
             cluster_.map_shared_rank(sh_.h.mass_lo, r)[i];
      }
      cluster_.map_shared_rank(sh_.h.all_count, 0)[i] = n;
      cluster_.map_shared_rank(sh_.h.all_mass, 0)[i] = m;
    }
    sync_all();
    if (rank_ == 0) {
      constexpr int kPer = kBins / kThreads;
      u64 n = 0, m = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) n += sh_.h.all_count[tid * kPer + j], m += sh_.h.all_mass[tid * kPer + j];
      const u64 n_in = block_scan(n, sh_.warp_u), m_in = block_scan(m, sh_.warp_v);
      if (tid == 0) sh_.found = kBins;
      __syncthreads();
      u64 nb = count0 + n_in - n, mb = mass0 + m_in - m;
      if (target == 0) {
        u64 candidates = 0;
        for (int w = 0; w < kWarps; ++w) candidates += sh_.warp_v[w];
        target = part_of(whole_mass(candidates), top_p);
      }
      Pick p, lastp;
      p.target = lastp.target = target;
      p.bin = kBins;
      int last = -1;  // the thread's last bin with members
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int bin = tid * kPer + j;
        const u64 c = sh_.h.all_count[bin], ms = sh_.h.all_mass[bin];
        const bool reached = (by_count ? nb + c : mb + ms) >= target;
        if (c > 0) last = bin, lastp.bin = bin, lastp.members = c, lastp.count = nb, lastp.mass = mb;
        if (reached && c > 0 && p.bin == kBins) p.bin = bin, p.members = c, p.count = nb, p.mass = mb;
        nb += c;
        mb += ms;
      }
      if (p.bin < kBins) atomicMin(&sh_.found, p.bin);
      __syncthreads();
      const int hit = sh_.found;
      __syncthreads();
      if (hit == kBins) {  // rounding kept the sum below the target: the last bin that has members
        if (tid == 0) sh_.found = -1;
        __syncthreads();
        if (last >= 0) atomicMax(&sh_.found, last);
        __syncthreads();
        if (last >= 0 && sh_.found == last) sh_.pick = lastp;
        if (sh_.found < 0 && tid == 0) sh_.pick = Pick{-1, 0, count0, mass0, target};
      } else if (p.bin == hit) {
        sh_.pick = p;
      }
      __syncthreads();
      if (tid > 0 && tid < ctas_) *cluster_.map_shared_rank(&sh_.pick, tid) = sh_.pick;
    }
    sync_all();
    return sh_.pick;
  }

  SA_DEV u64 block_scan(u64 x, u64* sums) {
    x = warp_scan(x);
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 31) sums[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x += sums[i];
    return x;
  }

  // Moves cut_ to the key of the last candidate that is kept and returns the
  // mass of the kept ones.  Candidates below the present cut do not count.
  // Target 0: top_p of the mass of everything.  Without `masses` (a cut by
  // count alone) none are summed, and none is returned.
  SA_DEV u64 search(bool by_count, u64 target, float top_p, bool masses) {
    const int tid = threadIdx.x;
    const u64 cut = cut_;
    Pick p = histogram(by_count, target, top_p, 0, 0, masses, [&](float x, int index) {
      return cut == 0 || full_key(x, index) >= cut ? step_of(x) : -1;
    });
    const int step = p.bin;
    if (!listed_ && step >= 0 && step < kBins - 1 && per_step_ > 0.f) {
      // Nothing below this step counts any more (the last step holds all that lies beyond the range): what is left
      // is mostly few enough for a list.
      const float edge = max_ - (step + 1.01f) / per_step_;
      floor_ = fmaxf(floor_, edge - fabsf(edge) * 2.4e-7f);
      make_slice_list();
    }
    u64 lo = 0, hi = ~0ull;
    if (p.members > kGather) {  // the members' range of keys
      u64 least = ~0ull, most = 0;
      each_candidate([&](float x, int index) {
        const u64 key = full_key(x, index);
        if (key >= cut && step_of(x) == step) least = least < key ? least : key, most = most > key ? most : key;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const u64 a = __shfl_xor_sync(0xffffffffu, least, o), b = __shfl_xor_sync(0xffffffffu, most, o);
        least = least < a ? least : a;
        most = most > b ? most : b;
      }
      if ((tid & 31) == 0) sh_.warp_u[tid >> 5] = least, sh_.warp_v[tid >> 5] = most;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) {
        least = least < sh_.warp_u[w] ? least : sh_.warp_u[w];
        most = most > sh_.warp_v[w] ? most : sh_.warp_v[w];
      }
      exchange(least, [&](u64 v) { least = least < v ? least : v; });
      exchange(most, [&](u64 v) { most = most > v ? most : v; });
      lo = least;
      hi = most;
    }
    while (p.members > kGather) {  // keys differ, so each turn leaves fewer
      int shift = 0;
      while (((hi - lo) >> shift) >= kBins) ++shift;
      p = histogram(by_count, p.target, 0.f, p.count, p.mass, masses, [&](float x, int index) {
        const u64 key = full_key(x, index);
        return key >= cut && key >= lo && key <= hi && step_of(x) == step ? static_cast<int>((hi - key) >> shift) : -1;
      });
      const u64 top = hi - (static_cast<u64>(p.bin) << shift);
      const u64 width = (1ull << shift) - 1;
      lo = top - lo > width ? top - width : lo;
      hi = top;
    }
    // the members to CTA 0, which ranks them
    if (tid == 0) sh_.gathered = 0;
    sync_all();
    {
      int* n = cluster_.map_shared_rank(&sh_.gathered, 0);
      u64* keys = cluster_.map_shared_rank(sh_.h.key, 0);
      u64* masses = cluster_.map_shared_rank(sh_.h.key_mass, 0);
      each_candidate([&](float x, int index) {
        const u64 key = full_key(x, index);
        if (key >= cut && key >= lo && key <= hi && step_of(x) == step) {
          const int at = atomicAdd(n, 1);
          if (at < kGather) keys[at] = key, masses[at] = fixed(x);
        }
      });
    }
    sync_all();
    if (rank_ == 0) {
      const int n = min(sh_.gathered, kGather);
      u64 key = 0;
      if (tid < n) {
        key = sh_.h.key[tid];
        int r = 0;
        for (int j = 0; j < n; ++j) r += sh_.h.key[j] > key;
        sh_.h.sorted[r] = key;
        sh_.h.sorted_mass[r] = sh_.h.key_mass[tid];
      }
      if (tid == 0) sh_.found = n - 1;
      __syncthreads();
      const u64 m = p.mass + block_scan(tid < n ? sh_.h.sorted_mass[tid] : 0, sh_.warp_u);
      const bool reached = (by_count ? p.count + tid + 1 : m) >= p.target;
      if (tid < n && reached) atomicMin(&sh_.found, tid);
      __syncthreads();
      if (tid == max(sh_.found, 0)) {
        sh_.cut = n > 0 ? sh_.h.sorted[tid] : cut;
        sh_.cut_mass = m;
      }
      __syncthreads();
      if (tid > 0 && tid < ctas_) {
        *cluster_.map_shared_rank(&sh_.cut, tid) = sh_.cut;
        *cluster_.map_shared_rank(&sh_.cut_mass, tid) = sh_.cut_mass;
      }
    }
    sync_all();
    cut_ = sh_.cut;
    return sh_.cut_mass;
  }

  SA_DEV float kept_mass(float x, int index) const {
    if (cut_ != 0 && (static_cast<u64>(order_key(x)) < (cut_ >> kIndexBits) || full_key(x, index) < cut_)) return 0.f;
    const float e = mass(x);
    return e >= min_mass_ ? e : 0.f;
  }

  // The kept mass of every chunk, by warp.
  SA_DEV void chunk_masses() {
    __syncthreads();
    for (int c = 0; c < chunks(); ++c) {
      float sum = 0.f;
      turns_of_vectors(c * chunk_turns_, min((c + 1) * chunk_turns_, (vectors_ + kThreads - 1) / kThreads),
                       [&](uint4 w, int v) {
                         if (!(E::largest(w) >= floor_)) return;
                         float x[E::kVec];
                         E::unpack(w, x);
#pragma unroll
                         for (int e = 0; e < E::kVec; ++e)
                           if (x[e] >= floor_) sum += kept_mass(x[e], index_of(v) + e);
                       });
      sum = warp_sum(sum);
      if ((threadIdx.x & 31) == 0) sh_.chunk_mass[c][threadIdx.x >> 5] = static_cast<u64>(sum * kSumOne);
    }
    __syncthreads();
  }

  // Index order: the CTAs' slices, in them chunks, turns, threads and elements.
  SA_DEV void sample_chunks(const SampleArgs& a, int row, float share) {
    const int tid = threadIdx.x, lane = tid & 31;
    // a lane's chunk (kChunks <= 32), and the slice, in every warp alike
    u64 mine = 0;
    if (lane < chunks())
      for (int w = 0; w < kWarps; ++w) mine += sh_.chunk_mass[lane][w];
    const u64 chunk_upto = warp_scan(mine);
    const u64 slice = __shfl_sync(0xffffffffu, chunk_upto, 31);
    u64 total = 0, before = 0;
    unsigned r = 0;
    exchange(slice, [&](u64 v) {
      if (r++ < rank_) before += v;
      total += v;
    });
    const u64 target = u_of(total, share);
    if (!(before <= target && before + slice > target)) return;  // exactly one CTA holds the target
    const unsigned beyond = __ballot_sync(0xffffffffu, before + chunk_upto > target);
    const int chunk = __ffs(beyond) - 1;
    // From here on the masses before the chunk are left out, and the unit is as fine as 64 bits allow: the chunk's
    // mass, at least 1 in the old unit, becomes 2^57 to 2^58 in the new one.  So logits whose masses are 0 each in
    // the old unit, and more than 0 only together, are met by the walk one by one.  (The warps' sums lost less than
    // one old unit each, so that the walk's own sum stays below 17 * 2^58.)
    const u64 chunk_mass = __shfl_sync(0xffffffffu, mine, chunk);
    const int finer = __clzll(chunk_mass) - 6;  // the chunk's mass is below 2^58
    const u64 goal = (target - before - __shfl_sync(0xffffffffu, chunk_upto - mine, chunk)) << finer;
    const float one = kSumOne * __int_as_float((127 + finer) << 23);
    before = 0;
    if (tid == 0) sh_.found = -1, sh_.last = max(chunk * chunk_turns_ * kThreads * E::kVec, shift_);
    __syncthreads();
    const int turns = (vectors_ + kThreads - 1) / kThreads;
    for (int t = chunk * chunk_turns_; t < min((chunk + 1) * chunk_turns_, turns); ++t) {
      const int v = t * kThreads + tid;
      u64 e[E::kVec], own = 0;
      int last = -1;
      if (v < vectors_) {
        float x[E::kVec];
        E::unpack(load(v), x);
#pragma unroll
        for (int i = 0; i < E::kVec; ++i) {
          e[i] = x[i] >= floor_ ? static_cast<u64>(kept_mass(x[i], index_of(v) + i) * one) : 0;
          own += e[i];
          if (e[i] > 0) last = i;
        }
      }
      const u64 upto = before + block_scan(own, sh_.warp_u);
      if (last >= 0) {
        atomicMax(&sh_.last, v * E::kVec + last);
        if (upto > goal && upto - own <= goal) {
          u64 run = upto - own;
          bool hit = false;
#pragma unroll
          for (int i = 0; i < E::kVec; ++i) {
            run += e[i];
            if (!hit && run > goal) sh_.found = v * E::kVec + i, hit = true;
          }
        }
      }
      __syncthreads();
      if (sh_.found >= 0) break;
      for (int w = 0; w < kWarps; ++w) before += sh_.warp_u[w];
      __syncthreads();
    }
    // the chunk's sum was rounded elsewhere: where the walk falls short of the goal, the last kept one
    const int at = sh_.found >= 0 ? sh_.found : sh_.last;
    if (tid == 0)
      put_token(a, row, first_ + at - shift_, E::one(base_[at]), static_cast<float>(total) * (1.f / kSumOne));
  }

  SA_DEV void put_token(const SampleArgs& a, int row, int token, float x, float kept) const {
    const float d = __fdiv_rn(x - max_, temperature_);
    put(a, row, token, d - ln(z_), d - ln(kept));
  }
  static SA_DEV void put(const SampleArgs& a, int row, int token, float logp, float logq) {
    a.tokens[row] = token;
    a.logp[row] = logp;
    a.logq[row] = logq;
  }

  Shared& sh_;
  cg::cluster_group cluster_;
  const T* base_;
  unsigned rank_, ctas_;
  int parity_ = 0;
  int vocab_, first_, shift_, end_, vectors_, chunk_turns_, pass1_parts_;
  int list_n_ = 0;
  bool listed_ = false;
  uint32_t count_key_;
  float temperature_, scale_, max_, z_, to_fixed_, min_mass_, floor_ = -INFINITY, per_step_;
  u64 cut_;
};

template <int kType>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Row<kType> row(*reinterpret_cast<Shared*>(smem));
  row.run(a, blockIdx.x / cg::this_cluster().num_blocks(), slice);
}

template <int kType>
cudaError_t launch_type(const SampleArgs& a, cudaStream_t s) {
  // CTAs per row go by the vocabulary alone, so that a row's result does not
  // depend on the batch around it.
  int ctas = 1;
  while (ctas < kMaxCluster && ceil_div(a.vocab, ctas) > kSliceLogits) ctas *= 2;
  const int vec = Elem<kType>::kVec;
  const int slice = ceil_div(ceil_div(a.vocab, ctas), vec) * vec;
  const auto kernel = sample_kernel<kType>;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(kernel, sizeof(Shared));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  if (a.dtype == 0) return launch_type<0>(a, s);
  if (a.dtype == 1) return launch_type<1>(a, s);
  return launch_type<2>(a, s);
}

}  // namespace sa
