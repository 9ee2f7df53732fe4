// asv_sample.cu -- sample_tokens: tokens drawn from rows of logits by given random numbers.
//
// Of a row x, with T > 0:  w_i = exp((x_i - max x) / T).  The entries in order (value descending, index ascending at
// equal values): top-k keeps the first k; top-p of these the ones with less than p of their mass before them; min-p those
// with w_i >= min_p.  All three keep a beginning of the order, so the kept set is a cut, the pair (value, index) of its last
// entry.  The token is the first kept index whose cumulative mass (over kept entries, by index) passes u times the
// kept mass; the distribution is w over the kept mass.
//
// Whole numbers come out, so a border must fall where exact arithmetic has it.  Weights are worked out to 2^-29 of themselves
// and summed in units of 2^-44 in 64-bit integers, which makes their sums exact in any order.  That costs some 40
// instructions an entry, half of them at half the rate, so few are weighed so:
//   - The row streams once, for the maxima of groups of the threads' vectors and, where the whole row's mass counts, a
//     running sum of fp32 weights (two operations and ex2).  Its error is bounded; a border within the bound counts as
//     undecided.
//   - Where the n largest maxima of threads bound the kept set from below (top-k; a nucleus, by one of two trials; min-p's
//     border), the groups that reach the bound are read again, out of L2, and the few entries from it on are put in order:
//     rank and mass before each, then the draw.
//   - A draw from the whole row finds the warp's run that u falls into by the fp32 sums and weighs that run alone.
//   - What stays undecided, or has too many candidates, takes an estimate of the border by a histogram and one pass that
//     weighs the row exactly and collects what is near the border (search_near); where even that does not settle it, many
//     values apart by less than a bin, histograms of exact masses level by level (search).
//
// A cluster of CTAs has a row, each a run of its vectors, each warp a run of the CTA's.  All CTAs come to the same
// decisions from the same exchanged numbers.  Up to 76 rows one launch does all; above, a launch of small CTAs whose chains
// of exchanges overlap, and one that has the rows it left, a cluster of eight large CTAs each.
//
// What bounds it (one call among others; the row's bytes at 6.79 TB/s in brackets): one row of 32,000, top-k, 11.1 us: four
// exchanges of a cluster and code that runs once, 43 % of its waits for instructions; 64 bf16 rows of 151,936, top-p,
// 23.4 [2.9], of which a row's chain is 19; 64 flat fp32 rows 80 [5.7]: 48 million warp instructions, 54 % of the issue slots;
// 352 fp32 rows of 128,256 with distributions 170 [53]; 1024 mixed rows of 151,936 150 [46]: 86 for the first launch, 58 for
// the few rows of the second, each a chain of some 20 exchanges.
// What the bound of the candidates lives on is that large entries lie anywhere: where whole runs are masked, or logits fall with
// the index, it admits too many, and the row takes the general way (one row at top-p 0.9: 14 us, with its last third masked 79).
#include <algorithm>
#include <climits>

#include "asv_device.cuh"
#include "asv_sample.h"

namespace asv {

namespace {

#include "exp2_table.inc"

constexpr int kNucleus = 64;             // maxima of threads that a nucleus is first looked for above
constexpr int kGroups = 20;              // groups of a thread's vectors, at most
constexpr int kScan = 1024;              // groups that are read again, at most
constexpr int kFew = 128;                // candidates up to which each is compared with each
constexpr int kBins = 2048;
constexpr int kMaxCtas = 8;
constexpr int kAhead = 4;                // vectors a lane has in flight
constexpr int kMostAhead = 8;            // the same at most, when the row streams from HBM
constexpr uint64_t kOne = uint64_t(1) << kSampleUnitBits;  // the largest weight

template <class T>
constexpr int kVec = 16 / int(sizeof(T));  // entries of a 16-byte vector

struct Cut {
  uint32_t key;   // entries with larger keys are kept, and those of this key up to the index
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return (k > key) | ((k == key) & (i <= index)); }
};

// What a launch does with its rows: all of it; the first way alone, leaving what that does not settle marked in the
// tokens; or those rows in general.
enum Part { kAll, kFirst, kRest };
constexpr int kLeft = INT_MIN, kTaken = INT_MIN + 1;

template <int THREADS, Part PART>
struct __align__(16) Shared {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32;
  static constexpr int kBuckets = THREADS < 256 ? THREADS : 256;
  static constexpr int kList = THREADS < 256 ? 256 : 512;  // candidates that are put in order
  union {                                          // one after the other
    float group[PART != kRest ? (kGroups + 1) * THREADS : 1];  // maxima of groups of a thread's vectors; of the row's ends
    uint2 bins[PART != kFirst ? kBins : 1];        // a histogram's 64-bit sums
    struct {
      uint4 sorted[kList];                         // the candidates in order
      uint64_t place[kFew];                        // the candidates' places in the order, where there are few
      uint64_t bin_mass[kBuckets];
      uint32_t bin_start[kBuckets];
    };
  };
  uint4 list[kList];                               // candidates of the row: key, index, weight
  uint64_t before[kList];                          // mass before each, by value or by index
  uint2 own[kList];                                // this CTA's candidates: key, index
  float tops[THREADS];                             // the threads' maxima
  uint16_t scan[kScan];                            // groups whose vectors are read again
  uint32_t table[PART != kFirst ? 1024 : 1];       // kExp2Table, where the whole row is weighed
  uint64_t chunk[kWarps];                          // sums of the warps' runs
  uint64_t run_mass[PART != kFirst ? kWarps : 1], count[PART != kFirst ? kWarps : 1];  // the same of all, and counts
  uint64_t room[kWarps], room2[kWarps];
  uint64_t pick_before, pick_sum, total;
  float2 sums[kWarps];                             // the warps' maxima and fast sums next to them
  float4 ends;                                     // of the CTA: maximum, bound of the candidates, whether it is bad, sum
  float2 lead[2];                                  // a bound, and the sum of threads' maxima from it on; a lower one
  Cut cut;
  int n_scan, n_own, found, pick, first;
  int first_own;                                   // of the list's, this CTA's first
  uint32_t least_key, most_key, found_key;         // of what was collected; of the token
  long long row;                                   // the next one
  __device__ __forceinline__ uint32_t* bin_ends() { return reinterpret_cast<uint32_t*>(tops); }  // (read by then)
};

// ------------------------------------------------------------------ a row

template <class T>
struct Row {
  const T* base;     // the 16-byte vector with the first entry
  int off;           // entries of it before the first
  int V, vectors;
  int rank, ctas, per_cta, per_warp;
  int v0, v1;        // this warp's vectors
#ifdef ASV_CHECKED
  uint32_t* check_log;
#endif
  __device__ __forceinline__ bool holds(int v) const {  // a whole vector of the row
    return v >= 0 && (long long)v * kVec<T> >= off && (long long)(v + 1) * kVec<T> - off <= V;
  }
  __device__ __forceinline__ bool whole(int v) const {
    return (v > 0 || off == 0) && (long long)(v + 1) * kVec<T> - off <= V;
  }
  // the vectors of warp w of CTA c
  __device__ __forceinline__ int run_start(int c, int w) const { return min(c * per_cta + w * per_warp, vectors); }
  __device__ __forceinline__ int run_end(int c, int w) const {
    return max(min(min(c * per_cta + (w + 1) * per_warp, (c + 1) * per_cta), vectors), run_start(c, w));
  }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16_t x) { return bf16_lo(x.bits); }

__device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}

// Entry e of a vector.
template <class T>
__device__ __forceinline__ float entry_of(const uint4& w, int e) {
  const int i = sizeof(T) == 2 ? e / 2 : e;
  const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
  return sizeof(T) == 4 ? __uint_as_float(x) : e % 2 ? bf16_hi(x) : bf16_lo(x);
}

// f(entries e and e + 1 of a vector, e), two at a time: a loop, whose instructions are fetched once.
template <class T, class F>
__device__ __forceinline__ void pairs(uint4 w, F f) {
#pragma unroll kVec<T> == 4 ? 2 : 1
  for (int e = 0; e < kVec<T>; e += 2) {
    if constexpr (sizeof(T) == 2) {
      f(bf16_lo(w.x), bf16_hi(w.x), e);
      w = make_uint4(w.y, w.z, w.w, 0);
    } else {
      f(__uint_as_float(w.x), __uint_as_float(w.y), e);
      w = make_uint4(w.z, w.w, 0, 0);
    }
  }
}

template <class T>
__device__ __forceinline__ float entry(const Row<T>& r, int i) {
  if (!ASV_GUARD(r, i >= 0 && i < r.V)) return -INFINITY;
  return widen(r.base[r.off + i]);
}

// A vector; entries that are not the row's are -inf.
template <class T>
__device__ __forceinline__ uint4 edge_vector(const Row<T>& r, int v) {
  constexpr int kBits = 8 * int(sizeof(T));
  uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int e = kVec<T> - 1; e >= 0; --e) {  // the last entry first, moved up by those before it
    const int i = v * kVec<T> - r.off + e;
    uint32_t x = kBits == 16 ? 0xff80u : 0xff800000u;
    if (i >= 0 && i < r.V) memcpy(&x, r.base + r.off + i, sizeof(T));
    if constexpr (kBits == 16)
      w = make_uint4((w.x << 16) | x, __funnelshift_l(w.x, w.y, 16), __funnelshift_l(w.y, w.z, 16),
                     __funnelshift_l(w.z, w.w, 16));
    else
      w = make_uint4(x, w.x, w.y, w.z);
  }
  return w;
}

template <class T>
__device__ __forceinline__ uint4 load_vector(const Row<T>& r, int v) {
  return r.whole(v) ? __ldg(reinterpret_cast<const uint4*>(r.base) + v) : edge_vector(r, v);
}

// f(vector, number) for a warp's vectors [v0, v1), kAhead of them a lane in flight; one instance of f.  BACK: from the last
// on (what was read last is likeliest still in L2).
template <bool BACK = false, class T, class F>
__device__ __forceinline__ void stream(const Row<T>& r, int v0, int v1, F f) {
  const int w0 = r.off > 0 ? 1 : 0, w1 = (r.off + r.V) / kVec<T>;  // whole ones
  const uint4* p = reinterpret_cast<const uint4*>(r.base);
  int v = v0 + int(threadIdx.x % 32);
  auto number = [&](int v) { return BACK ? v0 + v1 - 1 - v : v; };
  auto whole = [&](int v) { return (number(v) >= w0) & (number(v) < w1); };
  uint4 w[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    const int at = v + 32 * i;
    if (((at < v1) & whole(at)) && ASV_GUARD(r, r.holds(number(at)))) w[i] = __ldg(p + number(at));
  }
#pragma unroll 1
  for (; v < v1; v += 32) {
    uint4 now = w[0];
    if (!whole(v)) now = edge_vector(r, number(v));
#pragma unroll
    for (int i = 1; i < kAhead; ++i) w[i - 1] = w[i];
    const int at = v + 32 * kAhead;
    if (((at < v1) & whole(at)) && ASV_GUARD(r, r.holds(number(at)))) w[kAhead - 1] = __ldg(p + number(at));
    f(now, number(v));
  }
}

// Keys in the order of the values (equal for -0 and 0); 0 is no value's.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// ------------------------------------------------------------------ weights

// How weights follow from values.  k_top / 1024 + rest is the maximum's x c, which the fine sums' whole references are
// next to, unless it is beyond +-4000 (`far`).
struct Scale {
  float M;         // the row's maximum
  float c, c_lo;   // log2(e) / T
  float rest;
  int k_top;
  bool far;
};

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number

struct Exponent {
  float hi, lo;
};

// (x - M) / T in log2 units, x - M as a sum of two floats (Knuth's TwoSum).
__device__ __forceinline__ Exponent exponent(float x, const Scale& sc) {
  const float s = x - sc.M, bb = s - x, err = (x - (s - bb)) + (-sc.M - bb);
  const float hi = s * sc.c;
  return {hi, fmaf(s, sc.c, -hi) + fmaf(s, sc.c_lo, err * sc.c)};
}

// Shifts whose amounts may be any: 32 and more, and below 0, leave nothing.
__device__ __forceinline__ uint32_t shift_right(uint32_t x, int by) {
  uint32_t y;
  asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
  return y;
}
__device__ __forceinline__ uint32_t shift_left(uint32_t x, int by) {
  uint32_t y;
  asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
  return y;
}

// exp((x - M) / T) in units of 2^-44, rounded down: 2^(hi + lo) by the table (k / 1024 next to hi, r the rest, |r| <= 2^-11)
// and Taylor's first terms of 2^r - 1 in fp32; the rest is whole numbers, to 2^-30 of the weight.  (As pairs of floats, to
// 2^-39, it took 50 instructions, and with 64-bit whole numbers, to 2^-34, as many cycles; 32-bit ones run at half the rate
// of fp32's, 64-bit ones at a quarter.)
__device__ __forceinline__ uint64_t units_of(float x, const Scale& sc, const uint32_t* table) {
  const Exponent t = exponent(x, sc);
  const float m = fmaf(fmaxf(t.hi, -4090.0f), 1024.0f, kMagic);
  const int k = __float_as_int(m) - __float_as_int(kMagic);
  const float z = (fmaf(m - kMagic, -1.0f / 1024.0f, t.hi) + t.lo) * kLn2Hi;
  const float more = fmaf(z * z, fmaf(z, 1.0f / 6.0f, 0.5f), z);                                             // 2^r - 1
  const int more32 = __float_as_int(fmaf(more, 4294967296.0f, kMagic)) - __float_as_int(kMagic);  // in units of 2^-32
  const int base = int(table[k & 1023]);
  const uint32_t w = uint32_t(base + __mulhi(base, more32));  // in units of 2^-30
  const int down = -(k >> 10) - (kSampleUnitBits - 30);
  const uint32_t low = shift_right(w, down) | shift_left(w, -down), high = shift_right(w, down + 32);
  return (uint64_t(high) << 32) | low;
}

__device__ __forceinline__ Scale scale_of(float M, float c, float c_lo) {
  Scale sc = {M, c, c_lo, 0.0f, 0, !(fabsf(M * c) < 4000.0f)};
  if (!sc.far) {
    const float hi = M * c, lo = fmaf(M, c_lo, fmaf(M, c, -hi)), m = fmaf(hi, 1024.0f, kMagic);
    sc.k_top = __float_as_int(m) - __float_as_int(kMagic);
    sc.rest = fmaf(m - kMagic, -1.0f / 1024.0f, hi) + lo;
  }
  return sc;
}

__device__ __noinline__ uint64_t weight(float x, const Scale sc, const uint32_t* table) { return units_of(x, sc, table); }

// Whether a vector whose largest entry is x has weights that count.
__device__ __forceinline__ bool weighs(float x, const Scale& sc) { return (x - sc.M) * sc.c > -float(kSampleUnitBits + 3); }

// ------------------------------------------------------------------ sums over the row

__device__ __forceinline__ void row_sync() {  // all threads of the row's CTAs
  __syncwarp();
  if (cluster_size() > 1) cluster_sync();
  else __syncthreads();
}

__device__ __forceinline__ uint64_t ld_peer_u64(const uint64_t* p, int rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(dsmem_map(smem_addr(p), uint32_t(rank))) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer_u32(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_map(smem_addr(p), uint32_t(rank))) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t shfl_up_u64(uint64_t x, int d) { return __shfl_up_sync(0xffffffffu, x, d); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Inclusive sums over the block's threads.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* room) {
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint64_t y = shfl_up_u64(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) room[w] = x;
  __syncthreads();
  for (int i = 0; i < w; ++i) x += room[i];
  return x;
}

// ------------------------------------------------------------------ fast sums

// The sums that stream with the row are of fp32 weights 2^t, t = fma(x, c, -ref).  With D = (max - x) c a term is off by
// the rounding of c (D 2^-24 in t), of t ((D + 8) 2^-24, a reference is at most 8 below what it met) and ex2 (2^-22), a
// thread's sum by its move to the row's maximum (ex2 again) and the additions (three within a vector; the running sum
// carries its own errors).  Averaged over the mass, D is at most the entropy, log2 V <= 19: in all
// (ln 2 (2 * 19 + 8) + 4 + 4 + 4 + 3) 2^-24 < 2^-18 of the sum.
// References are whole parts of what fp32 holds exactly next to a term only within +-2^20: what lies below is left out, and
// a row whose maximum is not well above that, or lies above the range, does without these sums.
constexpr int kFastBits = 18;
constexpr float kFastRange = 1048576.0f;

struct Partial {
  float ref = -INFINITY;  // log2 units
  float hi = 0.0f, lo = 0.0f;
  // the sum with `top` (log2 units, at least any term's) for reference
  __device__ __forceinline__ float next_to(float top) const {
    return ref > -INFINITY ? (hi + lo) * ex2_approx(ref - top) : 0.0f;
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float vector_max(const uint4& w, bf16_t*) {
  uint32_t m, n;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w.x), "r"(w.y));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(w.z), "r"(w.w));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
  return max_nan(bf16_lo(m), bf16_hi(m));
}
__device__ __forceinline__ float vector_max(const uint4& w, float*) {
  return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
}

// One vector's weights onto a running sum.
template <int N>
__device__ __forceinline__ void add_weights(Partial& s, const float (&x)[N], float top, float c) {
  const float t = top * c;
  if (!(t > -kFastRange)) return;
  if (t > s.ref + 8.0f) {
    const float keep = ex2_approx(s.ref - t);
    s.hi *= keep;
    s.lo *= keep;
    s.ref = t;
  }
  const float2 cc = make_float2(c, c), rr = make_float2(-s.ref, -s.ref);
  float2 w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    w[e] = ffma2(make_float2(x[2 * e], x[2 * e + 1]), cc, rr);
    w[e].x = ex2_approx(w[e].x);
    w[e].y = ex2_approx(w[e].y);
  }
#pragma unroll
  for (int n = N / 2; n > 1; n /= 2)
#pragma unroll
    for (int e = 0; e < n / 2; ++e) w[e] = fadd2(w[2 * e], w[2 * e + 1]);
  const float v = w[0].x + w[0].y;
  const float sum = s.hi + v, bb = sum - s.hi;
  s.lo += (s.hi - (sum - bb)) + (v - bb);
  s.hi = sum;
}

// ------------------------------------------------------------------ candidates

// The same where the whole row's mass is drawn from, and fp32's errors are what leaves a draw undecided: exponents as sums of
// two floats next to a whole reference.  What is left is ex2 (2^-22), a product, three additions within the vector, and the
// move to the maximum (ex2 and two products): 15 * 2^-24 < 2^-20.
constexpr int kFineBits = 20;

template <int N>
__device__ __forceinline__ void add_weights_fine(Partial& s, const float (&x)[N], float top, float c, float c_lo) {
  const float most = top * c;
  if (!(most > -kFastRange)) return;
  if (most > s.ref + 8.0f) {
    const float ref = rintf(most), keep = ex2_approx(s.ref - ref);  // (a power of two)
    s.hi *= keep;
    s.lo *= keep;
    s.ref = ref;
  }
  const float2 cc = make_float2(c, c), cl = make_float2(c_lo, c_lo), rr = make_float2(-s.ref, -s.ref);
  const float2 one = make_float2(1.0f, 1.0f), ln2 = make_float2(kLn2Hi, kLn2Hi), far = make_float2(-120.0f, -120.0f);
  float2 w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const float2 y = make_float2(x[2 * e], x[2 * e + 1]);
    const float2 p = fmul2(y, cc), low = ffma2(y, cl, ffma2(y, cc, make_float2(-p.x, -p.y)));
    const float2 t = fadd2(p, rr), bb = fsub2(t, p), err = fadd2(fsub2(p, fsub2(t, bb)), fsub2(rr, bb));
    // (what is too far below to count may be -inf, and its errors nothing)
    const bool a = t.x > far.x, b = t.y > far.y;
    const float2 v = make_float2(a ? ex2_approx(t.x) : 0.0f, b ? ex2_approx(t.y) : 0.0f);
    const float2 l = fadd2(low, err), more = fmul2(make_float2(a ? l.x : 0.0f, b ? l.y : 0.0f), ln2);
    w[e] = ffma2(v, more, v);
  }
#pragma unroll
  for (int n = N / 2; n > 1; n /= 2)
#pragma unroll
    for (int e = 0; e < n / 2; ++e) w[e] = fadd2(w[2 * e], w[2 * e + 1]);
  const float v = w[0].x + w[0].y;
  const float sum = s.hi + v, bb = sum - s.hi;
  s.lo += (s.hi - (sum - bb)) + (v - bb);
  s.hi = sum;
}

// A running sum in units, once the row's maximum is known.
__device__ __forceinline__ uint64_t units_of_sum(const Partial& s, const Scale& sc, bool fine) {
  if (!(s.ref > -INFINITY)) return 0;
  const float shift = fine ? ex2_approx(s.ref - float(sc.k_top) * (1.0f / 1024.0f)) : ex2_approx(fmaf(-sc.M, sc.c, s.ref));
  const float v = (s.hi + s.lo) * shift;
  return uint64_t((fine ? fmaf(v, -sc.rest * kLn2Hi, v) : v) * float(kOne));
}

// A bound of the n-th largest of sh.tops (1 <= n <= kThreads) from below, to sixteen bits, and the largest, by a warp: the
// longest beginning of a key that n of the keys reach, two bits a step.
template <class S>
__device__ __forceinline__ void nth_largest(const S& sh, int n, float& nth, float& top) {
  constexpr int kEach = S::kThreads / 32;
  const int lane = threadIdx.x % 32;
  uint32_t key[kEach], most = 0;
#pragma unroll
  for (int i = 0; i < kEach; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(sh.tops + lane * kEach + i);
    key[i] = key_of(x.x), key[i + 1] = key_of(x.y), key[i + 2] = key_of(x.z), key[i + 3] = key_of(x.w);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) most = max(most, key[i]);
  most = __reduce_max_sync(0xffffffffu, most);
  top = value_of(most);
  uint32_t at = n == 1 ? most : 0;
  for (int bit = n == 1 ? 0 : 30; bit >= 16; bit -= 2) {
    // how many reach each of the three next beginnings, 10 bits each
    const uint32_t one = at + (1u << bit), two = at + (2u << bit), three = at + (3u << bit);
    uint32_t count = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      count += (key[i] >= one ? 1u : 0u) + (key[i] >= two ? 1u << 10 : 0u) + (key[i] >= three ? 1u << 20 : 0u);
    count = __reduce_add_sync(0xffffffffu, count);
    at = int(count >> 20) >= n ? three : int((count >> 10) & 1023u) >= n ? two : int(count & 1023u) >= n ? one : at;
  }
  nth = at < key_of(-INFINITY) ? -INFINITY : value_of(at);
}

// Where the thread's groups of vectors lie: vector q of the thread is first + 32 q, and in group q / per_group.
template <class T>
struct Groups {
  int per_group;
  __device__ __forceinline__ explicit Groups(const Row<T>& r) {
    const int each = (r.per_warp + 31) / 32;
    per_group = ((each + kGroups - 1) / kGroups + kMostAhead - 1) / kMostAhead * kMostAhead;
  }
};

// The CTA's entries from tau on, out of the groups of vectors whose maximum reaches it, to sh.own (those that have
// room; sh.n_own counts them all).
template <int AHEAD, class S, class T>
__device__ __noinline__ void collect(S& sh, const Row<T> r, float tau) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.n_scan = sh.n_own = 0;
  __syncthreads();
#pragma unroll 4
  for (int g = 0; g < kGroups; ++g) {
    if (sh.group[g * S::kThreads + tid] >= tau) {
      const int at = atomicAdd(&sh.n_scan, 1);
      if (at < kScan) sh.scan[at] = uint16_t(g * S::kThreads + tid);
    }
  }
  __syncthreads();
  const int n = sh.n_scan, per_group = Groups<T>(r).per_group;
  if (n > kScan) {
    if (tid == 0) sh.n_own = S::kList + 1;
    return;
  }
  auto take = [&](const uint4& w, int v) {
    float x[kVec<T>];
    unpack(w, x);
    uint32_t some = 0;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) some |= (x[e] >= tau ? 1u : 0u) << e;
    for (; some != 0; some &= some - 1) {
      const int e = __ffs(some) - 1, index = v * kVec<T> - r.off + e;
      if (index < 0 || index >= r.V) continue;
      const int to = atomicAdd(&sh.n_own, 1);
      if (to < S::kList) sh.own[to] = make_uint2(key_of(entry_of<T>(w, e)), uint32_t(index));
    }
  };
  const int w0 = r.off > 0 ? 1 : 0, w1 = (r.off + r.V) / kVec<T>;
  // the (whole) vector that number x of all groups' is, < 0: none
  auto vector_at = [&](int x) {
    const int k = x / per_group, q = x - k * per_group;
    if (k >= n) return -1;
    if (!ASV_GUARD(r, k >= 0 && k < kScan)) return -1;
    const int g = sh.scan[k] / S::kThreads, t = sh.scan[k] % S::kThreads, warp = t / 32;
    const int v = max(r.run_start(r.rank, warp), w0) + t % 32 + 32 * (g * per_group + q);
    return v < min(r.run_end(r.rank, warp), w1) ? v : -1;
  };
  const uint4* p = reinterpret_cast<const uint4*>(r.base);
#pragma unroll 1
  for (int x = tid; x < n * per_group; x += AHEAD * S::kThreads) {
    int v[AHEAD];
    uint4 w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      v[i] = vector_at(x + i * S::kThreads);
      w[i] = v[i] >= 0 && ASV_GUARD(r, r.holds(v[i])) ? __ldg(p + v[i]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (v[i] >= 0) take(w[i], v[i]);
  }
  // the row's ends (as they were streamed)
  if (sh.group[kGroups * S::kThreads + tid] >= tau) {
    const int edge = tid % 32 == 0 ? 0 : w1;
    take(edge_vector(r, edge), edge);
  }
}

// The row's candidates of all CTAs, with their weights (kOne each without), to sh.list; their number, or -1 if there is no
// room.
template <class S>
__device__ __noinline__ int share_out(S& sh, const Scale sc, int ctas, bool weigh) {
  const int lane = threadIdx.x % 32;
  const int own = lane < ctas ? int(ld_peer_u32(&sh.n_own, lane)) : 0;
  int upto = own;
#pragma unroll
  for (int d = 1; d < kMaxCtas; d *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  if (__any_sync(0xffffffffu, lane < ctas && (own > S::kList || upto > S::kList))) return -1;
  const int n = __shfl_sync(0xffffffffu, upto, kMaxCtas - 1);
  if (threadIdx.x == int(cluster_rank())) sh.first_own = upto - own;
  for (int i0 = 0; i0 < n; i0 += S::kThreads) {
    const int i = i0 + threadIdx.x;
    int c = 0, start = 0;
#pragma unroll
    for (int k = 0; k < kMaxCtas - 1; ++k) {
      const int end = __shfl_sync(0xffffffffu, upto, k);
      if (i >= end) c = k + 1, start = end;
    }
    if (i < n) {
      const uint64_t e = ld_peer_u64(reinterpret_cast<const uint64_t*>(sh.own + (i - start)), c);
      const uint32_t key = uint32_t(e), index = uint32_t(e >> 32);
      const uint64_t w = weigh ? weight(value_of(key), sc, kExp2Table) : kOne;
      sh.list[i] = make_uint4(key, index, uint32_t(w), uint32_t(w >> 32));
    }
  }
  __syncthreads();
  return n;
}

__device__ __forceinline__ uint64_t weight_in(const uint4& e) { return (uint64_t(e.w) << 32) | e.z; }

// The warps' sums of all CTAs, added up by each warp.
template <class S>
__device__ __forceinline__ uint64_t all_chunks(const S& sh, int ctas) {
  uint64_t x = 0;
  for (int i = threadIdx.x % 32; i < ctas * S::kWarps; i += 32) x += ld_peer_u64(sh.chunk + i % S::kWarps, i / S::kWarps);
  return warp_sum(x);
}

// p of a mass, p as a fraction of 2^64, rounded up.
__device__ __forceinline__ uint64_t part_of(uint64_t part, uint64_t mass) {
  return __umul64hi(part, mass) + (part * mass != 0 ? 1 : 0);
}

// Whether p of a mass is a whole number of the largest weights.  The border is then right behind some of several equal largest
// entries, whose sums are exact, and what weighs less than a unit decides whether the next one is in.
__device__ __forceinline__ bool even_border(uint64_t part, uint64_t mass) {
  return part > 0 && part * mass == 0 && part_of(part, mass) % kOne == 0;
}

// A weight below 2^-44, in units of 2^-88, and whether a sum of them is more than 2^-53 of the mass, which 64 bits see.
__device__ __forceinline__ uint64_t light_units(float x, float M, float c) {
  const float t = (x - M) * c;
  return t < -float(kSampleUnitBits) ? uint64_t(ex2_approx(t + 88.0f)) : 0;
}
__device__ __forceinline__ bool light_counts(uint64_t sum, uint64_t mass) { return sum > mass >> 9; }

// Numbers 0 .. n - 1 (n <= kList) by bins: bin b has sh.scan[bin_start[b]] up to sh.scan[bin_ends()[b] - 1], in any order.
// (Each candidate against each takes 1 us at 75 of them, this 2.5; at 350 they take 12 and 4.)
template <class S, class F>
__device__ __forceinline__ void by_bins(S& sh, int n, F bin_of) {
  const int tid = threadIdx.x;
  uint32_t *count = sh.bin_ends(), *start = sh.bin_start;
  if (tid < S::kBuckets) count[tid] = 0;
  __syncthreads();
  for (int e = tid; e < n; e += S::kThreads) atomicAdd(count + bin_of(e), 1u);
  __syncthreads();
  const uint64_t own = tid < S::kBuckets ? count[tid] : 0;
  const uint32_t upto = uint32_t(block_scan(own, sh.room) - own);
  if (tid < S::kBuckets) start[tid] = count[tid] = upto;
  __syncthreads();
  for (int e = tid; e < n; e += S::kThreads) sh.scan[atomicAdd(count + bin_of(e), 1u)] = uint16_t(e);
  __syncthreads();
}

// Few candidates' ranks: a group of threads counts for one those before it.
template <class S>
__device__ __forceinline__ void sort_few(S& sh, int n) {
  const int tid = threadIdx.x;
  if (tid < n) sh.place[tid] = (uint64_t(sh.list[tid].x) << 32) | ~sh.list[tid].y;
  __syncthreads();
  int g = 1;
  while (g < 32 && 2 * g * n <= S::kThreads) g *= 2;
  const int e = tid / g;  // (n <= kFew <= kThreads)
  const uint64_t mine = sh.place[min(e, n - 1)];
  int rank = 0;
#pragma unroll 4
  for (int j = tid % g; j < n; j += g) rank += sh.place[j] > mine;
  for (int o = 1; o < g; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (tid % g == 0 && e < n) sh.sorted[rank] = sh.list[e];
}

// The candidates in order, to sh.sorted, and the mass before each, to sh.before.  Where they are many, by bins of their
// values, from `top` down to `low`, and within a bin by comparison.
template <class S>
__device__ __noinline__ void sort_list(S& sh, int n, float top, float low) {
  const int tid = threadIdx.x;
  if (n <= kFew) {
    sort_few(sh, n);
  } else {
    const float scale = top > low ? float(S::kBuckets) / (top - low) : 0.0f;
    auto bin_of = [&](int e) { return int(fminf((top - value_of(sh.list[e].x)) * scale, float(S::kBuckets - 1))); };
    by_bins(sh, n, bin_of);
    for (int e = tid; e < n; e += S::kThreads) {
      const uint4 mine = sh.list[e];
      const int bin = bin_of(e), end = int(sh.bin_ends()[bin]);
      int rank = int(sh.bin_start[bin]);
      for (int q = rank; q < end; ++q) {
        const uint4& other = sh.list[sh.scan[q]];
        rank += (other.x > mine.x) | ((other.x == mine.x) & (other.y < mine.y));
      }
      sh.sorted[rank] = mine;
    }
  }
  __syncthreads();
  constexpr int kEach = S::kList / S::kThreads;
  uint64_t w[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    w[i] = kEach * tid + i < n ? weight_in(sh.sorted[kEach * tid + i]) : 0;
    sum += w[i];
  }
  uint64_t upto = block_scan(sum, sh.room) - sum;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    sh.before[kEach * tid + i] = upto;
    upto += w[i];
  }
  __syncthreads();
}

// The mass of the first m candidates with lower indices than each, to sh.before.  Where they are many, by bins of the V
// indices.
template <class S>
__device__ __forceinline__ void masses_by_index(S& sh, int m, int V) {
  const int tid = threadIdx.x;
  if (m <= kFew) {
    int g = 1;
    while (g < 32 && 2 * g * m <= S::kThreads) g *= 2;
    const int e = tid / g;
    const uint32_t index = sh.sorted[min(e, m - 1)].y;
    uint64_t mass = 0;
#pragma unroll 4
    for (int j = tid % g; j < m; j += g) {
      const uint4 y = sh.sorted[j];
      if (y.y < index) mass += weight_in(y);
    }
    for (int o = 1; o < g; o *= 2) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    if (tid % g == 0 && e < m) sh.before[e] = mass;
    __syncthreads();
    return;
  }
  const uint32_t scale = uint32_t((uint64_t(S::kBuckets) << 32) / uint32_t(V + S::kBuckets));
  auto bin_of = [&](int e) { return int(__umulhi(sh.sorted[e].y, scale)); };
  by_bins(sh, m, bin_of);
  uint64_t* mass = sh.bin_mass;
  uint64_t own = 0;  // of the thread's bin
  if (tid < S::kBuckets)
    for (uint32_t q = sh.bin_start[tid]; q < sh.bin_ends()[tid]; ++q) own += weight_in(sh.sorted[sh.scan[q]]);
  const uint64_t upto = block_scan(own, sh.room) - own;
  if (tid < S::kBuckets) mass[tid] = upto;
  __syncthreads();
  for (int e = tid; e < m; e += S::kThreads) {
    const uint32_t index = sh.sorted[e].y;
    const int bin = bin_of(e);
    uint64_t before = mass[bin];
    for (uint32_t q = sh.bin_start[bin]; q < sh.bin_ends()[bin]; ++q) {
      const uint4& other = sh.sorted[sh.scan[q]];
      if (other.y < index) before += weight_in(other);
    }
    sh.before[e] = before;
  }
  __syncthreads();
}

struct Drawn {
  int token;
  float value;     // its logit
  uint64_t total;  // the mass of all that is kept
};

// Settles a row by its n candidates, which are all its entries from some value on: its first k where k > 0, else all that
// can be kept (`closed`: nothing else is, for its weight; if not, the list has to reach past the nucleus).  `mass`, off by
// `off` at most: of the row, where k = 0 and p < 1.  False: the list does not settle it (sh.cut and the result are then
// nothing).
template <class S>
__device__ __noinline__ bool settle(S& sh, int n, int k, float p, uint64_t least, bool closed, uint64_t mass,
                                    uint64_t off, uint64_t draw, float M, float tau, int V, Drawn& d) {
  const int tid = threadIdx.x;
  sort_list(sh, n, M, tau);
  const uint64_t sum = k > 0 && k < n ? sh.before[k] : sh.before[n - 1] + weight_in(sh.sorted[n - 1]);
  if (k > 0) {
    mass = sum;
    off = 0;
  }
  uint64_t low = ~uint64_t(0), high = ~uint64_t(0);
  if (p < 1.0f) {
    const uint64_t part = uint64_t(p * 18446744073709551616.0f);
    low = max(part_of(part, mass - min(off, mass)), uint64_t(1));
    high = max(part_of(part, mass + off), uint64_t(1)) + (off > 0 ? 1 : 0);  // (the border itself is undecided too)
    if (k > 0 && even_border(part, mass)) return false;
  }
  bool unsure = k == 0 && p < 1.0f && !closed && sum < high;
  // the kept ones are the first m
  int m = 0;
  for (int e0 = 0; e0 < n; e0 += S::kThreads) {
    const int e = e0 + tid;
    const uint64_t w = e < n ? weight_in(sh.sorted[e]) : 0, b = e < n ? sh.before[e] : 0;
    const bool may = e < n && (k == 0 || e < k) && w >= least;
    unsure = unsure || (may && b >= low && b < high);
    m += __syncthreads_count(e == 0 || (may && b < low));
  }
  if (__syncthreads_or(unsure)) return false;
  d.total = m < n ? sh.before[m] : sh.before[n - 1] + weight_in(sh.sorted[n - 1]);
  const uint64_t at = __umul64hi(draw, d.total);
  if (tid == 0) sh.cut = {sh.sorted[m - 1].x, int(sh.sorted[m - 1].y)};
  __syncthreads();  // (all have read what is before whom)
  masses_by_index(sh, m, V);
  for (int e = tid; e < m; e += S::kThreads) {
    const uint64_t w = weight_in(sh.sorted[e]), b = sh.before[e];
    if (b <= at && at < b + w) {
      sh.found = int(sh.sorted[e].y);
      sh.found_key = sh.sorted[e].x;
    }
  }
  __syncthreads();
  d.token = sh.found;
  d.value = value_of(sh.found_key);
  return true;
}

// ------------------------------------------------------------------ the row in general

// Where the draw falls, draw / 2^64 of the warps' sums (in sh.chunk, behind a row_sync): the run that passes it and the sum
// before it, to sh.pick and sh.pick_before; the sum of all to sh.total.
template <class S, class T>
__device__ __forceinline__ uint64_t find_run(S& sh, const Row<T>& r, uint64_t draw) {
  const int tid = threadIdx.x, runs = r.ctas * S::kWarps;
  const uint64_t mine = tid < runs ? ld_peer_u64(sh.chunk + tid % S::kWarps, tid / S::kWarps) : 0;
  const uint64_t incl = block_scan(mine, sh.room);
  if (tid == S::kThreads - 1) {
    sh.total = incl;
    sh.pick = 0;
  }
  __syncthreads();
  const uint64_t at = __umul64hi(draw, sh.total);
  if (tid < runs && incl > at && incl - mine <= at) {
    sh.pick = tid;
    sh.pick_before = incl - mine;
  }
  return at;
}

// The entry of run sh.pick that `at` falls into: to sh.found of the CTA that owns the run (-1: within `margin` of the
// entry's ends, or in none), read from there by all.  The run is shared out to the warps, the part that `at` falls into to
// the threads, a thread's vectors entry by entry.  run_sum(v0, v1): a warp's sum of the entries of vectors [v0, v1);
// vector_sum(vector, number); f(x, index): an entry's.
template <class S, class T, class Run, class Vector, class F>
__device__ __forceinline__ int find_entry(S& sh, const Row<T>& r, uint64_t at, uint64_t margin, Run run_sum,
                                          Vector vector_sum, F f) {
  const int tid = threadIdx.x, warp = tid / 32;
  if (tid == 0) {
    sh.found = -1;
    sh.pick_sum = 0;
  }
  __syncthreads();
  const int pick = sh.pick, owner = pick / S::kWarps;
  if (r.rank == owner) {
    const int v0 = r.run_start(owner, pick % S::kWarps), v1 = r.run_end(owner, pick % S::kWarps);
    uint64_t before = sh.pick_before;
    const int each = (v1 - v0 + S::kWarps - 1) / S::kWarps;
    const uint64_t own = run_sum(min(v0 + warp * each, v1), min(v0 + (warp + 1) * each, v1));
    if (tid % 32 == 0) sh.room2[warp] = own;
    __syncthreads();
    int part = 0;
    for (; part < S::kWarps - 1 && before + sh.room2[part] <= at; ++part) before += sh.room2[part];
    const int p0 = min(v0 + part * each, v1), p1 = min(p0 + each, v1), few = (p1 - p0 + S::kThreads - 1) / S::kThreads;
    {
      const int a = min(p0 + tid * few, p1), b = min(a + few, p1);
      uint64_t sum = 0;
      for (int v = a; v < b; v += 2) {
        const bool two = v + 1 < b;
        const uint4 w = load_vector(r, v), x = two ? load_vector(r, v + 1) : w;
        sum += vector_sum(w, v);
        if (two) sum += vector_sum(x, v + 1);
      }
      const uint64_t upto = before + block_scan(sum, sh.room);
      if (upto > at && upto - sum <= at) {
        sh.pick_sum = upto - sum;
        sh.pick = a;
        sh.found = -2;
      }
    }
    __syncthreads();
    if (sh.found == -2) {
      before = sh.pick_sum;
      const int a = sh.pick, i0 = max(a * kVec<T> - r.off, 0), i1 = min(min(a + few, p1) * kVec<T> - r.off, r.V);
      __syncthreads();
      if (tid == 0) sh.found = -1;
      for (int first = i0; first < i1 && before <= at; first += S::kThreads) {
        const int i = first + tid;
        const uint64_t own = i < i1 ? f(entry(r, i), i) : 0;
        const uint64_t upto = before + block_scan(own, sh.room);
        // (before the row's first weight there is nothing to be off by)
        if (upto > at && upto - own <= at && (upto == own || at - (upto - own) >= margin) && upto - at > margin) sh.found = i;
        if (tid == S::kThreads - 1) sh.pick_sum = upto;
        __syncthreads();
        before = sh.pick_sum;
      }
    }
  }
  row_sync();
  const int found = int(ld_peer_u32(&sh.found, owner));
  row_sync();
  return found;
}

// The index of the n-th entry with this key (n >= 1).  counted: the runs' counts are in sh.count already.
template <class S, class T>
__device__ __noinline__ int nth_equal(S& sh, const Row<T> r, uint32_t key, uint64_t n, bool counted) {
  uint64_t own = 0;
  auto count = [&](const uint4& w, int v) {
    float x[kVec<T>];
    unpack(w, x);
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const int i = v * kVec<T> - r.off + e;
      n += key_of(x[e]) == key && i >= 0 && i < r.V;
    }
    return uint64_t(n);
  };
  if (!counted) {
    stream(r, r.v0, r.v1, [&](const uint4& w, int v) { own += count(w, v); });
    own = warp_sum(own);
    if (threadIdx.x % 32 == 0) sh.count[threadIdx.x / 32] = own;
    row_sync();
  }
  // (the share n - 1 of the count, as find_run takes it: it is looked for in units, not in parts of 2^64)
  const int tid = threadIdx.x, runs = r.ctas * S::kWarps;
  const uint64_t mine = tid < runs ? ld_peer_u64(sh.count + tid % S::kWarps, tid / S::kWarps) : 0;
  const uint64_t incl = block_scan(mine, sh.room);
  if (tid == 0) sh.pick = 0;
  __syncthreads();
  if (tid < runs && incl >= n && incl - mine < n) {
    sh.pick = tid;
    sh.pick_before = incl - mine;
  }
  return find_entry(
      sh, r, n - 1, 0,
      [&](int v0, int v1) {
        own = 0;
        stream(r, v0, v1, [&](const uint4& w, int v) { own += count(w, v); });
        return warp_sum(own);
      },
      count, [&](float x, int) { return uint64_t(key_of(x) == key ? 1 : 0); });
}

// Where `target` = target_of(all) falls among bins, each CTA adding up a part of them over all CTAs (add_up(bin): to its own,
// in place; mass(bin): it again).  To all: the bin (-1: none), the mass before it (`above` and the bins'), its own.
struct Bin {
  int bin;
  uint64_t target, above, in, all;
};

template <class S, class T, class Add, class Mass, class G>
__device__ __forceinline__ Bin find_bin(S& sh, const Row<T>& r, int bins, uint64_t above, Add add_up, Mass mass,
                                        G target_of) {
  const int tid = threadIdx.x, lane = tid % 32;
  const int part = (bins + r.ctas - 1) / r.ctas, part0 = min(r.rank * part, bins), part1 = min(part0 + part, bins);
  row_sync();
  uint64_t sum = 0;
  for (int i = part0 + tid; i < part1; i += S::kThreads) sum += add_up(i);
  sum = block_scan(sum, sh.room);
  if (tid == S::kThreads - 1) sh.total = sum;
  if (tid == 0) sh.pick = -1;
  row_sync();
  const uint64_t mine = lane < r.ctas ? ld_peer_u64(&sh.total, lane) : 0;
  uint64_t upto = mine;
#pragma unroll
  for (int d = 1; d < kMaxCtas; d *= 2) {
    const uint64_t y = shfl_up_u64(upto, d);
    if (lane >= d) upto += y;
  }
  Bin found;
  found.all = __shfl_sync(0xffffffffu, upto, kMaxCtas - 1);
  const uint64_t target = found.target = target_of(found.all);
  upto += above;
  const uint32_t holds = __ballot_sync(0xffffffffu, lane < r.ctas && upto - mine < target && target <= upto);
  const int owner = max(__ffs(holds) - 1, 0);
  const uint64_t start = __shfl_sync(0xffffffffu, upto - mine, owner);
  if (r.rank == owner) {
    // the bin, each thread looking through a few
    const int few = (part + S::kThreads - 1) / S::kThreads, i0 = min(part0 + tid * few, part1), i1 = min(i0 + few, part1);
    uint64_t s = 0;
    for (int i = i0; i < i1; ++i) s += mass(i);
    uint64_t b = start + block_scan(s, sh.room) - s;
    if (b < target && target <= b + s) {
      for (int i = i0; i < i1; ++i) {
        const uint64_t own = mass(i);
        if (b < target && target <= b + own) {
          sh.pick = i;
          sh.pick_before = b;
          sh.pick_sum = own;
        }
        b += own;
      }
    }
  }
  row_sync();
  found.bin = int(ld_peer_u32(&sh.pick, owner));
  found.above = ld_peer_u64(&sh.pick_before, owner);
  found.in = ld_peer_u64(&sh.pick_sum, owner);
  row_sync();  // (all have read what the owner found)
  return found;
}

// The cut that keeps entries of `within`, in order, until their measures (MASS: weights; else one each) add up to
// target_of(all): the last is the first with target <= the inclusive sum.  Where that lies is estimated first: a histogram
// by value, each weight as its bin's times 4096 (1 - d ln 2 width), d its distance from the bin's middle, in 32 bits and
// without an exponential.  The bin (two, near a border) is a bracket, and one pass over the row weighs exactly: all, what is
// above the bracket, a sum for each warp; and collects what is in it.  The sums say whether the target is in the bracket;
// then the cut is among its entries, or, where they are more than the list holds and equal, the first so many of
// them by index.  False: it is not, or they are not.
// `sums`: the warps' masses of what is kept are left in sh.chunk (behind a row_sync).
// (64 flat fp32 rows of 151,936: an exact histogram, the bin's entries, and a draw by fast sums before the exact one took
// 116 us, this takes 80.)
template <bool MASS, class S, class T, class G>
__device__ __noinline__ bool search_near(S& sh, const Row<T> r, const Scale sc, const Cut within, G target_of, bool sums,
                                         Cut& cut) {
  constexpr int kNear = 2 * kBins;            // 32-bit ones; the last takes what counts for nothing
  constexpr float kSpan = 36.0f;              // log2 units down from the maximum (152 thousand entries below: 2^-18 of it)
  constexpr float kStep = kSpan / float(kNear - 1);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  uint32_t* bins = reinterpret_cast<uint32_t*>(sh.bins);
  const float width = float(kNear - 1) / kSpan * sc.c;
  const bool all = within.key == 0;
  auto place = [&](float x) { return __fmul_rn(sc.M - x, width); };  // (rounded alike in both passes)
  for (int i = tid; i < kNear; i += S::kThreads) bins[i] = 0;
  if (tid == 0) {
    sh.n_own = 0;
    sh.least_key = ~0u;
    sh.most_key = 0;
  }
  __syncthreads();
  stream(r, r.v0, r.v1, [&](const uint4& w, int v) {
    if (!(place(vector_max(w, static_cast<T*>(nullptr))) < float(kNear - 1))) return;
    float x[kVec<T>];
    unpack(w, x);
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const float t = fminf(place(x[e]), float(kNear - 1)), m = __fadd_rn(t, kMagic);
      const int bin = __float_as_int(m) - __float_as_int(kMagic);
      const float d = t - (m - kMagic);
      const float relative = fmaf(d, -4096.0f * kLn2Hi * kStep, kMagic + 4096.0f);
      const uint32_t q = MASS ? uint32_t(__float_as_int(relative) - __float_as_int(kMagic)) : 1u;
      bool counts = bin < kNear - 1;
      if (!all) counts = counts && within.keeps(key_of(x[e]), v * kVec<T> - r.off + e);
      if (counts && ASV_GUARD(r, bin >= 0 && bin < kNear)) atomicAdd(bins + bin, q);
    }
  });
  // (a bin's sum over all CTAs, 2^19 entries of 4109 at most, has room too)
  auto mass = [&](int i) {
    return MASS ? uint64_t(float(bins[i]) * ex2_approx(float(i) * -kStep) * 1048576.0f) : uint64_t(bins[i]);
  };
  const Bin near = find_bin(
      sh, r, kNear - 1, 0,
      [&](int i) {
        uint32_t own = 0;
#pragma unroll
        for (int c = 0; c < kMaxCtas; ++c)
          if (c < r.ctas) own += ld_peer_u32(bins + i, c);
        bins[i] = own;
        return mass(i);
      },
      mass, target_of);
  if (near.bin < 0) return false;
  const uint64_t margin = near.all >> 16;  // (counts have none: they are exact)
  const int b0 = max(near.bin - int(MASS && near.target - near.above <= margin), 0);
  const int b1 = min(near.bin + int(MASS && near.above + near.in - near.target < margin), kNear - 2);

  // ---- exactly
  const float m0 = kMagic + float(b0), m1 = kMagic + float(b1);
  const bool weigh = MASS || sums;
  uint64_t total = 0, above = 0;
  uint32_t count = 0, low = ~0u, high = 0;
  stream(r, r.v0, r.v1, [&](const uint4& w, int v) {
    const float most = vector_max(w, static_cast<T*>(nullptr));
    if (MASS ? !weighs(most, sc) : __fadd_rn(place(most), kMagic) > m1) return;
    pairs<T>(w, [&](float x0, float x1, int e) {
      const float x[2] = {x0, x1};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = v * kVec<T> - r.off + e + h;
        const float m = __fadd_rn(place(x[h]), kMagic);
        uint64_t u = weigh ? units_of(x[h], sc, sh.table) : 0;
        bool in = (m >= m0) & (m <= m1);  // (an entry that is not the row's is far below)
        if (!all) {
          const bool keeps = within.keeps(key_of(x[h]), i);
          u = keeps ? u : 0;
          in = in && keeps;
        }
        if (MASS) total += u;
        above += m < m0 ? u : 0;
        if (in) {
          const uint32_t key = key_of(x[h]);
          ++count;
          low = min(low, key);
          high = max(high, key);
          const int to = atomicAdd(&sh.n_own, 1);
          if (to < S::kList) sh.own[to] = make_uint2(key, uint32_t(i));
        }
      }
    });
  });
  total = warp_sum(total);
  above = warp_sum(above);
  count = __reduce_add_sync(0xffffffffu, count);
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    sh.run_mass[warp] = total;
    sh.chunk[warp] = above;
    sh.count[warp] = count;
    atomicMin(&sh.least_key, low);
    atomicMax(&sh.most_key, high);
  }
  row_sync();
  uint64_t before = near.above, target = near.target;  // (counts are exact)
  if (MASS) {
    uint64_t x = 0;
    for (int i = lane; i < r.ctas * S::kWarps; i += 32) x += ld_peer_u64(sh.run_mass + i % S::kWarps, i / S::kWarps);
    target = target_of(warp_sum(x));
    before = all_chunks(sh, r.ctas);
  }
  low = lane < r.ctas ? ld_peer_u32(&sh.least_key, lane) : ~0u;
  high = lane < r.ctas ? ld_peer_u32(&sh.most_key, lane) : 0;
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  const int n = share_out(sh, sc, r.ctas, true);
  const int runs = r.ctas * S::kWarps;
  const uint64_t mine = tid < runs ? ld_peer_u64(sh.count + tid % S::kWarps, tid / S::kWarps) : 0;
  row_sync();  // (all have read the masses above)
  if (target <= before || n == 0) return false;
  if (n > 0) {
    // each CTA has its own candidates, a group of threads for one: the mass before it, and whether it is the last
    const int first = sh.first_own, m = sh.n_own;
    if (tid == 0) sh.first = -1;
    __syncthreads();
    int g = 1;
    while (g < 32 && 2 * g * m <= S::kThreads) g *= 2;
    for (int e0 = 0; e0 < m; e0 += S::kThreads / g) {
      const int e = e0 + tid / g;
      const uint4 y = sh.list[first + min(e, m - 1)];
      uint64_t b = 0;
#pragma unroll 4
      for (int j = tid % g; j < n; j += g) {
        const uint4 z = sh.list[j];
        if ((z.x > y.x) | ((z.x == y.x) & (z.y < y.y))) b += MASS ? weight_in(z) : 1;
      }
      for (int o = 1; o < g; o *= 2) b += __shfl_xor_sync(0xffffffffu, b, o);
      b += before;
      if (tid % g == 0 && e < m && b < target && target <= b + (MASS ? weight_in(y) : 1)) {
        sh.cut = {y.x, int(y.y)};
        sh.first = e;
      }
    }
    row_sync();
    const int theirs = int(ld_peer_u32(&sh.first, min(lane, r.ctas - 1)));
    const uint32_t holds = __ballot_sync(0xffffffffu, lane < r.ctas && theirs >= 0);
    if (holds == 0) return false;
    const int owner = __ffs(holds) - 1;
    cut = {ld_peer_u32(&sh.cut.key, owner), int(ld_peer_u32(&sh.cut.index, owner))};
    for (int e = tid; e < m; e += S::kThreads) {
      const uint4 y = sh.list[first + e];
      const int v = int(y.y + uint32_t(r.off)) / kVec<T>, run = (v - r.rank * r.per_cta) / r.per_warp;
      if (cut.keeps(y.x, int(y.y)) && ASV_GUARD(r, run >= 0 && run < S::kWarps))
        atomicAdd(reinterpret_cast<unsigned long long*>(sh.chunk + run), (unsigned long long)weight_in(y));
    }
  } else {
    if (low != high) return false;
    const uint64_t each = weight(value_of(low), sc, sh.table), step = MASS ? each : 1;
    const uint64_t upto = block_scan(mine, sh.room);
    if (tid == S::kThreads - 1) sh.total = upto;
    __syncthreads();
    const uint64_t have = sh.total;
    if (step == 0 || target - before > have * step) return false;
    const uint64_t want = (target - before + step - 1) / step;
    if (tid / S::kWarps == r.rank && tid < runs)
      sh.chunk[tid % S::kWarps] += min(want - min(want, upto - mine), mine) * each;
    cut = {low, INT_MAX};
    if (want < have) cut.index = nth_equal(sh, r, low, want, true);
  }
  row_sync();
  return true;
}

// The same cut for rows that search_near does not settle.  A histogram of exact masses by value over the larger weights'
// range, then the bin's entries to the list; where there are more than it holds, a histogram by key within the bin, and so
// on.  The bins are added up a part by each CTA.
template <bool MASS, class S, class T, class G>
__device__ __noinline__ Cut search(S& sh, const Row<T> r, const Scale sc, const Cut within, G target_of) {
  const int tid = threadIdx.x, lane = tid % 32;
  // bins of equal width down to weights of 2^-24, the last takes the rest (7 % of a weight's width each: of 152 thousand
  // flat entries 250 at most fall into one)
  const float width = float(kBins - 1) / 24.0f * sc.c;
  auto bin_of = [&](float x) {
    return __float_as_int(fminf((sc.M - x) * width, float(kBins - 1)) + kMagic) - __float_as_int(kMagic);
  };
  auto add = [&](int bin, uint64_t m) {
    if (!ASV_GUARD(r, bin >= 0 && bin < kBins)) return;
    const uint32_t low = uint32_t(m), old = atomicAdd(&sh.bins[bin].x, low);
    const uint32_t high = uint32_t(m >> 32) + (old + low < old ? 1u : 0u);
    if (high) atomicAdd(&sh.bins[bin].y, high);
  };
  const bool all = within.key == 0;
  uint32_t lo = 1, hi = key_of(sc.M);
  int shift = 32, first_bin = 0;
  uint64_t above = 0, target = 0, in_bin = 0;
  for (int level = 0; shift > 0; ++level) {
    if (level > 0) {
      const uint32_t span = hi - lo;
      shift = 0;
      while ((span >> shift) >= uint32_t(kBins)) ++shift;
    }
    // what the entries of the bracket do
    auto each_entry = [&](auto f) {
      const float least = value_of(lo), most = value_of(hi);
      stream(r, r.v0, r.v1, [&](const uint4& w, int v) {
        float x[kVec<T>];
        unpack(w, x);
        uint32_t some = 0;
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) some |= uint32_t((x[e] >= least) & (x[e] <= most)) << e;
        for (; some != 0; some &= some - 1) {
          const int e = __ffs(some) - 1, i = v * kVec<T> - r.off + e;
          const float y = entry_of<T>(w, e);
          const uint32_t key = key_of(y);
          // (the keys are tested too: the one between 0's and the largest negative number's is no value's, and where the
          // bracket ends with it, 0 is not below its value, -0, but above it)
          if (key >= lo && key <= hi && bin_of(y) == first_bin && i >= 0 && i < r.V && within.keeps(key, i)) f(y, key, i);
        }
      });
    };
    if (level > 0) {
      if (tid == 0) sh.n_own = 0;
      __syncthreads();
      each_entry([&](float, uint32_t key, int i) {
        const int to = atomicAdd(&sh.n_own, 1);
        if (to < S::kList) sh.own[to] = make_uint2(key, uint32_t(i));
      });
      row_sync();
      const int n = share_out(sh, sc, r.ctas, MASS);
      if (n > 0) {
        sort_list(sh, n, value_of(hi), value_of(lo));
        for (int e = tid; e < n; e += S::kThreads) {
          const uint64_t m = MASS ? weight_in(sh.sorted[e]) : 1, b = above + (MASS ? sh.before[e] : uint64_t(e));
          if (b < target && target <= b + m) sh.cut = {sh.sorted[e].x, int(sh.sorted[e].y)};
        }
        row_sync();
        return sh.cut;
      }
    }
    for (int i = tid; i < kBins; i += S::kThreads) sh.bins[i] = make_uint2(0, 0);
    __syncthreads();
    if (level == 0) {
      uint64_t rest = 0;  // the last bin's, which most entries of a peaked row fall into
      stream(r, r.v0, r.v1, [&](const uint4& w, int v) {
        if (MASS && !weighs(vector_max(w, static_cast<T*>(nullptr)), sc)) return;
        pairs<T>(w, [&](float x0, float x1, int e) {
          const float x[2] = {x0, x1};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = v * kVec<T> - r.off + e + h;
            uint64_t m;
            if constexpr (MASS) m = units_of(x[h], sc, sh.table);
            else m = (i >= 0) & (i < r.V);
            if (!all) m = within.keeps(key_of(x[h]), i) ? m : 0;
            const int bin = m != 0 ? bin_of(x[h]) : kBins - 1;
            if (bin < kBins - 1) add(bin, m);
            else rest += m;
          }
        });
      });
      rest = warp_sum(rest);
      if (lane == 0 && rest != 0) add(kBins - 1, rest);
    } else {
      each_entry([&](float x, uint32_t key, int) {
        const uint64_t m = MASS ? weight(x, sc, sh.table) : 1;
        if (m != 0) add(int((hi - key) >> shift), m);
      });
    }
    auto mass = [&](int i) { return *reinterpret_cast<const uint64_t*>(sh.bins + i); };
    const Bin found = find_bin(
        sh, r, kBins, above,
        [&](int i) {
          uint64_t own = 0;
#pragma unroll
          for (int c = 0; c < kMaxCtas; ++c)
            if (c < r.ctas) own += ld_peer_u64(reinterpret_cast<const uint64_t*>(sh.bins + i), c);
          *reinterpret_cast<uint64_t*>(sh.bins + i) = own;
          return own;
        },
        mass, [&](uint64_t sum) { return level == 0 ? target_of(sum) : target; });
    const int bin = max(found.bin, 0);
    target = found.target;
    above = found.above;
    in_bin = found.in;
    if (level == 0) {
      // keys that the bin's values may have (its own test stays)
      first_bin = bin;
      const float from = sc.M - (float(bin) - 0.5f) / width, to = sc.M - (float(bin) + 0.5f) / width;
      const float slack = (fabsf(sc.M) + fabsf(to)) * 1e-5f;
      hi = min(hi, key_of(from + slack));
      lo = bin == kBins - 1 || !(to - slack > -INFINITY) ? key_of(-INFINITY) : key_of(to - slack);
    } else {
      hi -= uint32_t(bin) << shift;
      lo = max(lo, hi - ((1u << shift) - 1u));
    }
  }
  // one value, and more entries with it than the list holds: of equal values the lowest indices
  const uint64_t each = MASS ? weight(value_of(hi), sc, sh.table) : 1;
  const uint64_t want = (target - above + each - 1) / each;
  Cut cut = {hi, INT_MAX};
  if (want < in_bin / each) cut.index = nth_equal(sh, r, hi, want, false);
  return cut;
}

// Where the border of a nucleus of part / 2^64 of the mass is even: the next of the equal largest entries comes into the cut if
// what weighs less than a unit, of the entries in `within`, counts next to it.  True: one did.
template <class S, class T>
__device__ __noinline__ bool one_more(S& sh, const Row<T> r, const Scale sc, const Cut within, uint64_t part,
                                      uint64_t mass, Cut& cut) {
  const uint32_t top = key_of(sc.M);
  if (!even_border(part, mass) || cut.key != top) return false;
  if (threadIdx.x == 0) sh.least_key = ~0u;
  __syncthreads();
  uint64_t sum = 0;
  uint32_t next = ~0u;
  stream(r, r.v0, r.v1, [&](const uint4& w, int v) {
    pairs<T>(w, [&](float x0, float x1, int e) {
      const float x[2] = {x0, x1};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = v * kVec<T> - r.off + e + h;  // (an entry that is not the row's is -inf)
        if (!within.keeps(key_of(x[h]), i)) continue;
        sum += light_units(x[h], sc.M, sc.c);
        if (key_of(x[h]) == top && i > cut.index) next = min(next, uint32_t(i));
      }
    });
  });
  sum = warp_sum(sum);
  next = __reduce_min_sync(0xffffffffu, next);
  if (threadIdx.x % 32 == 0) {
    sh.run_mass[threadIdx.x / 32] = sum;  // (sh.chunk is still needed)
    atomicMin(&sh.least_key, next);
  }
  row_sync();
  const int lane = threadIdx.x % 32;
  sum = 0;
  for (int i = lane; i < r.ctas * S::kWarps; i += 32) sum += ld_peer_u64(sh.run_mass + i % S::kWarps, i / S::kWarps);
  next = __reduce_min_sync(0xffffffffu, lane < r.ctas ? ld_peer_u32(&sh.least_key, lane) : ~0u);
  row_sync();
  if (next == ~0u || !light_counts(warp_sum(sum), mass)) return false;
  cut.index = int(next);
  return true;
}

// The smallest key whose weight is at least `least`, by a warp: 32 candidates at a time.
template <class S>
__device__ __noinline__ uint32_t least_key(S& sh, const Scale sc, uint64_t least) {
  uint32_t lo = 1, hi = key_of(sc.M);
  __syncthreads();  // (sh.cut's last readers are done)
  if (threadIdx.x < 32) {
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32, key = min(lo + step * threadIdx.x, hi);
      const uint32_t reach = __ballot_sync(0xffffffffu, key == hi || weight(value_of(key), sc, sh.table) >= least);
      const int f = reach != 0 ? __ffs(reach) - 1 : 32;
      const uint32_t below = lo;
      if (f < 32) hi = min(below + step * f, hi);
      if (f > 0) lo = min(below + step * (f - 1) + 1, hi);
    }
    if (threadIdx.x == 0) sh.cut.key = hi;
  }
  __syncthreads();
  return sh.cut.key;
}

struct Kept {
  Cut cut;
  float value;  // the cut's
  __device__ __forceinline__ bool operator()(float x, int i) const { return (x > value) | ((x == value) & (i <= cut.index)); }
};

// The sum of a vector's kept entries.
template <class T>
__device__ __forceinline__ uint64_t kept_sum(const uint4& w, int v, const Row<T>& r, const Scale& sc, const Kept& keep,
                                             const uint32_t* table) {
  const float top = vector_max(w, static_cast<T*>(nullptr));
  if (top < keep.value || !weighs(top, sc)) return 0;
  uint64_t sum = 0;
  pairs<T>(w, [&](float a, float b, int e) {
    const uint64_t u = units_of(a, sc, table), w = units_of(b, sc, table);
    const int i = v * kVec<T> - r.off + e;
    sum += (keep(a, i) ? u : 0) + (keep(b, i + 1) ? w : 0);
  });
  return sum;
}

// A draw from the whole row by the warps' fast sums (finer ones of fp32; sh.chunk, behind a row_sync).  A token < 0: too near
// a border to say.
template <class S, class T>
__device__ __noinline__ Drawn draw_fast(S& sh, const Row<T> r, const Scale sc, uint64_t draw) {
  const uint64_t at = find_run(sh, r, draw);
  __syncthreads();
  Drawn d;
  d.total = sh.total;
  // Of sums b before a border and a behind it the draw u compares (1 - u) b with u a.  Next to the border both are u (1 - u)
  // of the mass, 1/4 at most, and each is off by 2^-20 (2^-18) of itself; the run's own sum counts once as the rows streamed
  // and once as it is taken apart here, each off by as much too.  (It is taken apart by the sums it was streamed with: the
  // finer ones' references do not hold for 16-bit rows, which come here from further than +-4000 too.)
  constexpr bool kFine = sizeof(T) == 4;
  constexpr int kBits = kFine ? kFineBits : kFastBits;
  const int run = sh.pick;
  const uint64_t margin = ((sh.total / 2 + 2 * ld_peer_u64(sh.chunk + run % S::kWarps, run / S::kWarps)) >> kBits) + 64;
  const Kept keep = {{0u, INT_MAX}, -INFINITY};
  d.token = find_entry(
      sh, r, at, margin,
      [&](int v0, int v1) {
        Partial s;
        stream(r, v0, v1, [&](const uint4& w, int v) {
          float x[kVec<T>];
          unpack(w, x);
          const float most = vector_max(w, static_cast<T*>(nullptr));
          if constexpr (kFine) add_weights_fine(s, x, most, sc.c, sc.c_lo);
          else add_weights(s, x, most, sc.c);
        });
        return warp_sum(units_of_sum(s, sc, kFine));
      },
      [&](const uint4& w, int v) { return kept_sum(w, v, r, sc, keep, kExp2Table); },
      [&](float x, int) { return weight(x, sc, kExp2Table); });
  d.value = d.token >= 0 ? entry(r, d.token) : -INFINITY;
  return d;
}

// A draw from the kept entries by exact sums.  summed: the warps' are in sh.chunk already.
template <class S, class T>
__device__ __noinline__ Drawn draw_exact(S& sh, const Row<T> r, const Scale sc, const Kept keep, bool summed, uint64_t draw) {
  uint64_t own = 0;
  auto sum = [&](const uint4& w, int v) { return kept_sum(w, v, r, sc, keep, sh.table); };
  if (!summed) {
    stream(r, r.v0, r.v1, [&](const uint4& w, int v) { own += sum(w, v); });
    own = warp_sum(own);
    if (threadIdx.x % 32 == 0) sh.chunk[threadIdx.x / 32] = own;
    row_sync();
  }
  const uint64_t at = find_run(sh, r, draw);
  __syncthreads();
  Drawn d;
  d.total = sh.total;
  d.token = find_entry(
      sh, r, at, 0,
      [&](int v0, int v1) {
        own = 0;
        stream(r, v0, v1, [&](const uint4& w, int v) { own += sum(w, v); });
        return warp_sum(own);
      },
      sum, [&](float x, int i) { return keep(x, i) ? weight(x, sc, sh.table) : uint64_t(0); });
  d.value = entry(r, d.token);
  return d;
}

// (x - max x) / T - ln(kept mass): from the logit, as its weight in whole units has few digits where it is light.  Neither
// part is above 0, so nothing cancels; the mass is the maximum's weight of 1 and the rest.
__device__ __forceinline__ float log_probability(const Drawn& d, const Scale& sc) {
  const Exponent t = exponent(d.value, sc);
  const float rest = float(d.total - min(d.total, kOne)) * (1.0f / float(kOne));
  return fmaf(t.hi, kLn2Hi, t.lo * kLn2Hi) - log1pf(rest);
}

// The kept entries' shares of the mass, 1 / inv, and 0 elsewhere (everywhere without a token).
template <class T>
__device__ __noinline__ void write_distribution(const SampleArgs& a, const Row<T> r, const Scale sc, const Cut cut, int token,
                                                float inv, int b, int n) {
  float* to = a.probs + b * a.probs_b + n * a.probs_n;
  // (what is further below the maximum than 2^-200 has no weight; of a row without a token nothing has)
  const float cut_at = cut.key == 0 ? -INFINITY : value_of(cut.key), least_value = sc.M - 200.0f / sc.c;
  const Kept keep = {{0u, token < 0 ? -1 : cut_at < least_value ? INT_MAX : cut.index},
                     token < 0 ? INFINITY : fmaxf(cut_at, least_value)};
  const bool vectors = (reinterpret_cast<uintptr_t>(to) / 4 + kVec<T> - r.off) % 4 == 0;
  const float2 cc = make_float2(sc.c, sc.c), cl = make_float2(sc.c_lo, sc.c_lo), mm = make_float2(-sc.M, -sc.M);
  const float2 minus = make_float2(-sc.c, -sc.c), ii = make_float2(inv, inv), ln2 = make_float2(kLn2Hi, kLn2Hi);
  stream<true>(r, r.v0, r.v1, [&](const uint4& w, int v) {
    float x[kVec<T>], p[kVec<T>];
    unpack(w, x);
    const int i0 = v * kVec<T> - r.off;
#pragma unroll
    for (int e = 0; e < kVec<T>; e += 2) {
      // exponents as sums of two floats, two entries at a time: x - M with its rounding (Knuth's TwoSum), its product with c
      const float2 y = make_float2(x[e], x[e + 1]), s = fadd2(y, mm), bb = fsub2(s, y);
      const float2 err = fadd2(fsub2(y, fsub2(s, bb)), fsub2(mm, bb)), down = fmul2(s, minus);
      const float2 lo = ffma2(err, cc, ffma2(s, cl, ffma2(s, cc, down)));
      const float2 q = fmul2(make_float2(ex2_approx(-down.x), ex2_approx(-down.y)), ii), more = ffma2(q, fmul2(lo, ln2), q);
      p[e] = keep(x[e], i0 + e) ? more.x : 0.0f;
      p[e + 1] = keep(x[e + 1], i0 + e + 1) ? more.y : 0.0f;
    }
    if (vectors && i0 >= 0 && i0 + kVec<T> <= a.V && ASV_GUARD(a, b < a.B && n < a.n)) {
#pragma unroll
      for (int e = 0; e < kVec<T>; e += 4)
        __stcs(reinterpret_cast<float4*>(to + i0 + e), make_float4(p[e], p[e + 1], p[e + 2], p[e + 3]));
    } else {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e)
        if (i0 + e >= 0 && i0 + e < a.V) to[i0 + e] = p[e];
    }
  });
}

// ------------------------------------------------------------------ the kernels

template <Part PART, class S, class T>
__device__ __forceinline__ void sample_row(const SampleArgs& a, S& sh, Row<T>& r, long long row) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int b = int(row / a.n), n = int(row - (long long)b * a.n);

  // ---- the request's parameters
  const float T_ = a.temperature != nullptr ? a.temperature[b] : a.one.temperature;
  const float top_p = a.top_p != nullptr ? a.top_p[b] : a.one.top_p;
  const float min_p = a.min_p != nullptr ? a.min_p[b] : a.one.min_p;
  int k = a.top_k != nullptr ? a.top_k[b] : a.one.top_k;
  const bool params_ok = sampling_ok(T_, k, top_p, min_p);
  float u = a.u[b * a.u_b + n * a.u_n];
  u = u >= 0.0f ? fminf(u, 0.99999994f) : 0.0f;
  const bool greedy = T_ == 0.0f;
  k = greedy ? 1 : k >= a.V ? 0 : k;

  const T* first = static_cast<const T*>(a.x) + b * a.x_b + n * a.x_n;
  r.off = int((reinterpret_cast<uintptr_t>(first) % 16) / sizeof(T));
  r.base = first - r.off;
  r.V = a.V;
#ifdef ASV_CHECKED
  r.check_log = a.check_log;
#endif
  r.vectors = (r.off + a.V + kVec<T> - 1) / kVec<T>;
  r.per_cta = (r.vectors + r.ctas - 1) / r.ctas;
  r.per_warp = (r.per_cta + S::kWarps - 1) / S::kWarps;
  r.v0 = r.run_start(r.rank, warp);
  r.v1 = r.run_end(r.rank, warp);
  const float c = greedy || !params_ok ? 1.0f : kLog2eHi / T_;
  const float c_lo = greedy || !params_ok ? 0.0f : (fmaf(-c, T_, kLog2eHi) + kLog2eLo) / T_;

  // ---- the row streams once: the threads' maxima, and the mass where it is needed
  constexpr int kFirstAhead = PART == kFirst ? kMostAhead : kAhead;  // (few CTAs to a row have more to do each)
  const bool nucleus = !greedy && top_p < 1.0f;
  const bool sums = PART != kRest && k == 0 && (nucleus || min_p == 0.0f);
  // (16-bit rows would be bound by it: 1024 of 151,936, drawn from whole, 235 us, 135 without; so 2 % of rows like Zipf's are
  // too near a border instead of 1 %, and 24 % of flat ones instead of 10)
  const bool fine = sizeof(T) == 4 && sums && !nucleus;
  float top = -INFINITY;
  Partial part;
  {
    const int per_group = Groups<T>(r).per_group;
    float most = -INFINITY;  // of the group
    int g = 0, left = per_group;
    auto one = [&](const uint4& w) {
      const float m = vector_max(w, static_cast<T*>(nullptr));
      if (sums) {
        float x[kVec<T>];
        unpack(w, x);
        if (fine) add_weights_fine(part, x, m, c, c_lo);
        else add_weights(part, x, m, c);
      }
      return m;
    };
    auto close = [&]() {  // (a group without vectors has no maximum)
      if (PART != kRest) sh.group[g * S::kThreads + tid] = left < per_group ? most : NAN;
      top = max_nan(top, most);
      most = -INFINITY;
      ++g;
      left = per_group;
    };
    const int w0 = r.off > 0 ? 1 : 0, w1 = (r.off + r.V) / kVec<T>, end = min(r.v1, w1);  // whole vectors
    const uint4* p = reinterpret_cast<const uint4*>(r.base);
    int v = max(r.v0, w0) + lane;
    for (; v - lane < end; v += 32 * kFirstAhead) {
      constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
      uint4 w[kFirstAhead];
#pragma unroll
      for (int i = 0; i < kFirstAhead; ++i)
        w[i] = v + 32 * i < end && ASV_GUARD(r, r.holds(v + 32 * i)) ? __ldg(p + v + 32 * i)
                                                                   : make_uint4(kNone, kNone, kNone, kNone);
#pragma unroll
      for (int i = 0; i < kFirstAhead; ++i) most = max_nan(most, one(w[i]));
      left -= kFirstAhead;
      if (left == 0) close();
    }
    while (g < kGroups) close();
    // the row's ends
    const int edge = lane == 0 && r.v0 == 0 && w0 == 1 && r.v1 > 0                                  ? 0
                     : lane == 1 && w1 >= w0 && w1 < r.vectors && w1 >= r.v0 && w1 < r.v1 ? w1
                                                                                            : -1;
    if (edge >= 0) {
      most = one(edge_vector(r, edge));
      --left;
    }
    close();
  }
  // Candidates are looked for from tau on: the row's k-th largest is at least the least of the CTAs' (k / ctas)-th
  // largest maxima of threads.
  const int nth = k > 0 ? (k + r.ctas - 1) / r.ctas : nucleus ? max(kNucleus / r.ctas, 1) : S::kThreads + 1;
  sh.tops[tid] = top;
  if (sums) {
    const float most = warp_max(top), s = most > -kFastRange ? part.next_to(most * c) : 0.0f;
    float all = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) sh.sums[warp] = make_float2(most, all);
  }
  bool bad = __syncthreads_or(!(top < INFINITY));
  // (a lower bound by the next warp, for a nucleus that the first does not hold: by half as many maxima as the list has
  // room, which 60 to 80 % as many candidates reach)
  if (warp < (PART != kRest && sums && nucleus ? 2 : 1)) {
    const int count = PART == kRest ? 1 : warp == 0 ? min(nth, S::kThreads) : min(S::kList / 2 / r.ctas, S::kThreads * 3 / 4);
    float least_top = -INFINITY, most = -INFINITY;
    nth_largest(sh, count, least_top, most);
    const float next_to = most > -INFINITY ? most : 0.0f;  // (next to a maximum of -inf nothing has a weight)
    float all = 0.0f;
    if (sums)
      for (int w = 0; w < S::kWarps; ++w) all += sh.sums[w].y * ex2_approx((sh.sums[w].x - next_to) * c);
    float lead = 0.0f;
    if (sums) {
#pragma unroll 4
      for (int i = lane; i < S::kThreads; i += 32)
        lead += sh.tops[i] >= least_top ? ex2_approx((sh.tops[i] - next_to) * c) : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lead += __shfl_xor_sync(0xffffffffu, lead, o);
    }
    if (lane == 0) sh.lead[warp] = make_float2(nth <= S::kThreads ? least_top : -INFINITY, lead);
    if (lane == 0 && warp == 0) sh.ends = make_float4(most, bad ? 1.0f : 0.0f, all, 0.0f);
  }
  row_sync();
  float tau, M, about, lead;  // about, lead: the row's mass and the largest maxima's, roughly
  {
    float4 e = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    float2 first = make_float2(INFINITY, 0.0f), second = first;
    auto pair = [&](const void* p) {
      const uint64_t x = ld_peer_u64(static_cast<const uint64_t*>(p), lane);
      return make_float2(__uint_as_float(uint32_t(x)), __uint_as_float(uint32_t(x >> 32)));
    };
    if (lane < r.ctas) {
      const float2 ab = pair(&sh.ends), cd = pair(&sh.ends.z);
      e = make_float4(ab.x, ab.y, cd.x, cd.y);
      first = pair(sh.lead);
      if (sums && nucleus) second = pair(sh.lead + 1);
    }
    bad = __any_sync(0xffffffffu, e.y != 0.0f);
    M = e.x;
#pragma unroll
    for (int o = 1; o < kMaxCtas; o *= 2) {
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      first.x = fminf(first.x, __shfl_xor_sync(0xffffffffu, first.x, o));
      second.x = fminf(second.x, __shfl_xor_sync(0xffffffffu, second.x, o));
    }
    M = __shfl_sync(0xffffffffu, M, 0);
    const float scale = e.z > 0.0f ? ex2_approx((e.x - M) * c) : 0.0f;
    about = e.z * scale;
    first.y *= scale;
    second.y *= scale;
#pragma unroll
    for (int o = 1; o < kMaxCtas; o *= 2) {
      about += __shfl_xor_sync(0xffffffffu, about, o);
      first.y += __shfl_xor_sync(0xffffffffu, first.y, o);
      second.y += __shfl_xor_sync(0xffffffffu, second.y, o);
    }
    if (sums && nucleus && top_p * about > first.y) first = second;
    about = __shfl_sync(0xffffffffu, about, 0);
    tau = __shfl_sync(0xffffffffu, first.x, 0);
    lead = __shfl_sync(0xffffffffu, first.y, 0);
  }
  bad = bad || M == -INFINITY;
  // (numbers, also where CTAs hold nothing but -inf: what follows chooses by them)
  (void)ASV_GUARD(r, !sums || bad || !(fabsf(M * c) < kFastRange) || (about >= 0.0f && lead >= 0.0f));
  const Scale sc = scale_of(M, c, c_lo);

  Drawn d = {-1, -INFINITY, 0};
  Cut cut = {0u, INT_MAX};
  uint64_t least = 0;
  if (params_ok && !bad) {  // (for all CTAs of the row)
    if (!greedy && min_p > 0.0f) {
      const uint64_t most = weight(M, sc, kExp2Table);
      least = min_p < 1.0f ? part_of(uint64_t(min_p * 18446744073709551616.0f), most) : most;
    }
    const uint64_t draw = greedy ? 0 : uint64_t(u * 18446744073709551616.0f);
    bool settled = false;
    if constexpr (PART != kRest) {
      if (sums) {
        const uint64_t w = warp_sum(units_of_sum(part, sc, fine));
        if (lane == 0) sh.chunk[warp] = w;
      }
      // Where nothing depends on the mass below min-p's border, candidates end there (a little below it, for the
      // roundings: of the maximum, the span, and of weights, as which exact ones decide).
      bool closed = false;
      if (greedy) {
        tau = sc.M;
      } else if (min_p > 0.0f && (k == 0 || !nucleus)) {
        const float span = T_ * logf(min_p), border = sc.M + span - 1e-5f * (fabsf(sc.M) - span + T_);
        if (!(tau > border) || nth > S::kThreads || (nucleus && top_p * about > lead)) {
          tau = border;
          closed = true;
        }
      }
      const bool trusted = !sums || (fine ? !sc.far : fabsf(sc.M * sc.c) < kFastRange - 128.0f);
      // (the candidates are half as many again as the maxima they are found by, but smaller ones: 1.0 to 1.2 times the mass,
      // and more where threads have few entries, several of them candidates)
      const float reach = 1.25f + 16.0f * float(S::kThreads * r.ctas) / float(a.V);
      const bool hopeless = sums && nucleus && !closed && top_p * about > reach * lead;
      const bool by_list = trusted && !hopeless && (nth <= S::kThreads || closed);
      if (by_list) {
        collect<PART == kFirst ? kAhead : 1>(sh, r, tau);
        row_sync();
        const int found = share_out(sh, sc, r.ctas, !greedy);
        const uint64_t mass = sums ? all_chunks(sh, r.ctas) : 0;
        if (found > 0)
          settled = settle(sh, found, k, greedy ? 1.0f : top_p, least, closed, mass, (mass >> kFastBits) + 1, draw, sc.M,
                           tau, a.V, d);
        if (settled) cut = sh.cut;
        else row_sync();  // (the peers have read the candidates)
      } else if (trusted && sums && !nucleus) {
        row_sync();
        d = draw_fast(sh, r, sc, draw);
        settled = d.token >= 0;
      }
    }
    if constexpr (PART != kFirst) {
      if (!settled) {
        for (int i = tid; i < 1024; i += S::kThreads) sh.table[i] = kExp2Table[i];
        __syncthreads();
        bool summed = false;  // what is kept, for each warp
        if (k > 0) {
          auto target = [&](uint64_t) { return uint64_t(k); };
          summed = search_near<false>(sh, r, sc, cut, target, !nucleus, cut);
          if (!summed) cut = search<false>(sh, r, sc, Cut{0u, INT_MAX}, target);
        }
        if (nucleus) {
          const Cut first_k = cut;
          const uint64_t part = uint64_t(top_p * 18446744073709551616.0f);
          uint64_t mass = 0;
          auto target = [&](uint64_t all) {
            mass = all;
            return max(part_of(part, all), uint64_t(1));
          };
          summed = search_near<true>(sh, r, sc, first_k, target, true, cut);
          if (!summed) cut = search<true>(sh, r, sc, first_k, target);
          if (one_more(sh, r, sc, first_k, part, mass, cut)) summed = false;
          if (cut.key == first_k.key) cut.index = min(cut.index, first_k.index);
        }
        if (least > 0) {
          const uint32_t key = least_key(sh, sc, least);
          if (key > cut.key) {
            cut = {key, INT_MAX};
            summed = false;
          }
        }
        d = draw_exact(sh, r, sc, Kept{cut, cut.key == 0 ? -INFINITY : value_of(cut.key)}, summed, draw);
      }
    } else if (!settled) {
      if (r.rank == 0 && tid == 0) a.tokens[b * a.tokens_b + n * a.tokens_n] = kLeft;
      row_sync();
      return;
    }
  }
  if (r.rank == 0 && tid == 0 && ASV_GUARD(a, b >= 0 && b < a.B && n >= 0 && n < a.n && d.token >= -1 && d.token < a.V)) {
    if (!params_ok) atomicOr(a.status + b, ASV_REQ_BAD_PARAM);
    if (bad) atomicOr(a.status + b, ASV_REQ_NONFINITE);
    a.tokens[b * a.tokens_b + n * a.tokens_n] = d.token;
    if (a.logprobs != nullptr)
      a.logprobs[b * a.logprobs_b + n * a.logprobs_n] = d.token < 0 ? -INFINITY : log_probability(d, sc);
  }

  // ---- the distribution
  if (a.probs != nullptr)
    write_distribution(a, r, sc, cut, d.token, d.token >= 0 ? float(kOne) / float(d.total) : 0.0f, b, n);
  row_sync();  // (no CTA goes on while its peers read its shared memory)
}

// A cluster for each row.
template <Part PART, class T, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ Shared<THREADS, PART> sh;
  Row<T> r;
  r.ctas = int(cluster_size());
  r.rank = int(cluster_rank());
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  sample_row<PART>(a, sh, r, blockIdx.x / r.ctas);
}

// The rows that the first way left.  Each cluster goes through all rows once, from a place of its own, and takes those
// that no other has taken (an exchange of the mark; by turns, two of a few rows often came to one cluster).
template <class T, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) sample_rest_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ Shared<THREADS, kRest> sh;
  Row<T> r;
  r.ctas = int(cluster_size());
  r.rank = int(cluster_rank());
  const int tid = threadIdx.x;
  const long long rows = (long long)a.B * a.n, clusters = gridDim.x / r.ctas, mine = blockIdx.x / r.ctas;
  const long long chunks = (rows + THREADS - 1) / THREADS, start = mine * chunks / clusters;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto token_of = [&](long long row) {
    const long long b = row / a.n;
    return a.tokens + b * a.tokens_b + (row - b * a.n) * a.tokens_n;
  };
  long long chunk = 0;
  for (;;) {
    if (r.rank == 0) {
      // the next row that can be taken, or none
      if (tid == 0) sh.row = -1;
      while (chunk < chunks) {
        const long long row = (start + chunk) % chunks * THREADS + tid;
        // (in an order of its own within the chunk too)
        const int place = int((tid + THREADS - mine * 13 % THREADS) % THREADS);
        const bool left = row < rows && __ldcg(token_of(row)) == kLeft;
        if (tid == 0) sh.first = THREADS;
        __syncthreads();
        if (left) atomicMin(&sh.first, place);
        __syncthreads();
        const int first = sh.first;
        if (first == THREADS) {
          ++chunk;
          __syncthreads();
          continue;
        }
        if (left && place == first && atomicCAS(token_of(row), kLeft, kTaken) == kLeft) sh.row = row;
        __syncthreads();
        if (sh.row >= 0) break;
      }
    }
    row_sync();
    const long long row = (long long)ld_peer_u64(reinterpret_cast<const uint64_t*>(&sh.row), 0);
    row_sync();
    if (row < 0) break;
    sample_row<kRest>(a, sh, r, row);
  }
}

constexpr int kAllThreads = 256, kAllCtas = 4, kFirstThreads = 128, kFirstCtas = 8;  // of a CTA; CTAs to an SM
constexpr int kRestThreads = 512, kRestCtas = 2;
constexpr int kSms = 152;

template <class Kernel>
cudaError_t launch(Kernel kernel, const SampleArgs& a, long long clusters, int ctas, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters * ctas), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class T>
cudaError_t launch_rows(const SampleArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.B * a.n;
  const int tuned = std::min(tuned_cluster(), kMaxCtas);
  // CTAs to a row: `share`, what all rows together leave room for, but no more than have enough of the row to be worth their
  // exchanges; where distributions are wanted, as many more as leave the rows in hand (of `room` CTAs) small enough to stay in L2
  // until they are written, about half of it (fp32 rows: 352 of 128,256 239 us with two, 169 with eight; 700 of 50,257 206 with
  // one, 145 with four, 161 with eight; 1500 of 16,384 109, 107 with two, 196; 4000 of 8192 143 with one, 430 with eight).
  auto ctas_of = [&](long long share, int least, int room) {
    if (tuned > 0) return tuned;
    auto in_hand = [&](long long ctas) { return std::min(rows, room / ctas) * a.V * (long long)sizeof(T); };
    long long ctas = std::min(share, (long long)kMaxCtas);
    if (a.probs != nullptr)
      while (in_hand(ctas) > (60ll << 20) && in_hand(kMaxCtas) < in_hand(ctas)) ++ctas;
    return int(std::clamp(std::min(ctas, (long long)a.V / least), 1ll, (long long)kMaxCtas));
  };
  if (rows <= kSms / 2) {
    // One CTA to an SM, six to a row at most, where no row can have a large kept set (64 rows of 151,936, top-k 50, in L2: 15.6 us
    // with two, 18.8 with eight, out of HBM 20.4, 18.4 with three and 20.2 with eight; 16 rows 12.9 with six, 14.2 with eight);
    // with a nucleus of any size four to an SM (64 flat rows: 80 with eight, 111 with three).  Not quite all there is room for:
    // 76 rows of eight take two turns, 33 us against 23.
    const bool nucleus = a.top_p != nullptr || a.one.top_p < 1.0f, min_p = a.min_p != nullptr || a.one.min_p > 0.0f;
    const bool few = (a.temperature == nullptr && a.one.temperature == 0.0f) ||
                     (a.top_k == nullptr && (a.one.top_k > 0 ? a.one.top_k <= 256 : !nucleus && !min_p));
    const long long share = few ? std::clamp(kSms / rows, 2ll, 6ll) : kSms * kAllCtas * 15 / 16 / rows;
    return launch(sample_kernel<kAll, T, kAllThreads, kAllCtas>, a, rows, ctas_of(share, 2048, kSms * kAllCtas), kAllThreads, s);
  }
  // Many rows: small CTAs whose chains of exchanges overlap, some half of those that there is room for, four to a row at
  // most (300 rows of 151,936, top-p: 39 us with three, 49 with four; 150 rows 28.6 with four, 39 with eight; 600 58 with
  // two, 68 with one and 70 with three); and the few rows that need it in general behind them, where large clusters have
  // them at once.
  const long long share = std::min((kSms * kFirstCtas * 9 / 16 + rows - 1) / rows, 4ll);
  const cudaError_t e = launch(sample_kernel<kFirst, T, kFirstThreads, kFirstCtas>, a, rows,
                               ctas_of(share, 1024, kSms * kFirstCtas), kFirstThreads, s);
  if (e != cudaSuccess) return e;
  return launch(sample_rest_kernel<T, kRestThreads, kRestCtas>, a, std::min(rows, (long long)kSms * kRestCtas / kMaxCtas),
                kMaxCtas, kRestThreads, s);
}

#ifdef ASV_CHECKED
__device__ uint32_t g_check_log[2];  // the sampling has no workspace to keep a log in
#endif

}  // namespace

cudaError_t launch_sample(const SampleArgs& args, int dtype, cudaStream_t s) {
  SampleArgs a = args;
#ifdef ASV_CHECKED
  void* log = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&log, g_check_log);
  if (e != cudaSuccess) return e;
  a.check_log = static_cast<uint32_t*>(log);
#endif
  return dtype == ASV_BF16 ? launch_rows<bf16_t>(a, s) : launch_rows<float>(a, s);
}

}  // namespace asv

#ifdef ASV_CHECKED
// The sampling's check log (the count and the line of the first failure), when the device's work is done.  Returns a
// cudaError.
extern "C" int asv_sample_check_log(uint32_t* out) {
  const cudaError_t e = cudaDeviceSynchronize();
  return int(e != cudaSuccess ? e : cudaMemcpyFromSymbol(out, asv::g_check_log, sizeof(asv::g_check_log)));
}
#endif
