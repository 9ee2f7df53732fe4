// asv_sample.cu -- sample_tokens: tokens drawn from rows of logits by given random numbers.
//
// Of a row x, with T > 0:  w_i = exp((x_i - max x) / T).  The entries in order (value descending, index ascending at
// equal values): top-k keeps the first k; top-p of these the ones with less than p of their mass before them; min-p those
// with w_i >= min_p.  All three keep a beginning of the order, so the kept set is a cut, the pair (value, index) of its last
// entry.  The token is the first kept index whose cumulative mass (over kept entries, by index) passes u times the
// kept mass; the distribution is w over the kept mass.
//
// Whole numbers come out, so a border must fall where exact arithmetic has it: weights are worked out as (hi, lo) pairs to
// about 2^-39 and summed in units of 2^-44 in 64-bit integers, which makes every sum exact in any order: the same token
// for any number of CTAs.
//
// A cluster of CTAs has a row; each a run of its vectors, each warp a run of the CTA's.  The row streams from HBM once
// for its maximum and is read again from L2.
#include <algorithm>
#include <climits>

#include "asv_device.cuh"
#include "asv_sample.h"

namespace asv {

namespace {

#include "exp2_table.inc"

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;
constexpr int kMaxCtas = 8;
constexpr uint64_t kOne = uint64_t(1) << kSampleUnitBits;  // the largest weight

template <class T>
constexpr int kVec = 16 / int(sizeof(T));  // entries of a 16-byte vector

struct Shared {
  float2 table[64];
  uint32_t bin_lo[kBins], bin_hi[kBins];   // a histogram's 64-bit sums
  uint64_t chunk[kWarps];                  // sums of the warps' runs
  uint64_t all[kMaxCtas * kWarps];         // ... of all CTAs'
  uint64_t room[kWarps], room2[kWarps];
  float top;
  int bad;
  int first;   // lowest index of the maximum
  int found;
  int pick;
  uint64_t pick_before, pick_sum;
};

// ------------------------------------------------------------------ a row

template <class T>
struct Row {
  const T* base;     // the 16-byte vector with the first entry
  int off;           // entries of it before the first
  int V, vectors;
  int v0, v1;        // this warp's vectors
  __device__ __forceinline__ bool whole(int v) const {
    return (v > 0 || off == 0) && (long long)(v + 1) * kVec<T> - off <= V;
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

template <class T>
__device__ __forceinline__ float entry(const Row<T>& r, int i) {
  return widen(r.base[r.off + i]);
}

// f(x, index) for the entries of the warp's vectors.
template <class T, class F>
__device__ __forceinline__ void sweep(const Row<T>& r, F f) {
  const int lane = threadIdx.x % 32;
  for (int v = r.v0 + lane; v < r.v1; v += 32) {
    const int i0 = v * kVec<T> - r.off;
    if (r.whole(v)) {
      float x[kVec<T>];
      unpack(__ldg(reinterpret_cast<const uint4*>(r.base) + v), x);
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) f(x[e], i0 + e);
    } else {
      for (int i = max(i0, 0); i < min(i0 + kVec<T>, r.V); ++i) f(entry(r, i), i);
    }
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

struct Scale {
  float M;         // the row's maximum
  float c, c_lo;   // log2(e) / T
};

// exp((x - M) / T) in units of 2^-44, rounded, to about 2^-39.  x - M as the sum s + err (Knuth's TwoSum), times
// log2(e) / T as the sum th + tl; 2^th by the table (k / 64 next to th, r the rest, |r| <= 2^-7) and Taylor's terms of
// exp(z) - 1, z = r ln 2; what is below fp32's last place is carried in a second float throughout.
__device__ __noinline__ uint64_t weight(float x, const Scale sc, const float2* table) {
  const float s = x - sc.M, bb = s - x, err = (x - (s - bb)) + (-sc.M - bb);
  const float th = s * sc.c;
  if (!(th > -float(kSampleUnitBits + 2))) return 0;
  const float tl = fmaf(s, sc.c, -th) + fmaf(s, sc.c_lo, err * sc.c);
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number
  const float m = fmaf(th, 64.0f, kMagic), kf = m - kMagic;
  const int k = __float_as_int(m) - __float_as_int(kMagic);
  const float r = fmaf(kf, -0.015625f, th);
  const float2 t = table[k & 63];
  const float zh = r * kLn2Hi;
  const float zl = fmaf(tl, kLn2Hi, fmaf(r, kLn2Lo, fmaf(r, kLn2Hi, -zh)));
  const float p = fmaf(fmaf(fmaf(zh, 1.0f / 120.0f, 1.0f / 24.0f), zh, 1.0f / 6.0f), zh, 0.5f) * (zh * zh);
  const float q = fmaf(zl, zh, zl) + p;
  const float mh = t.x * zh;
  const float ml = fmaf(t.y, zh, fmaf(t.x, q, fmaf(t.x, zh, -mh) + t.y));
  const float sh = t.x + mh, sl = (mh - (sh - t.x)) + ml;
  const float unit = __int_as_float(((k >> 6) + 22 + 127) << 23);  // 2^(e + 22)
  const float yh = sh * unit, a = (yh + kMagic) - kMagic;
  const float low = ((yh - a) + sl * unit) * 4194304.0f;
  return uint64_t((long long)(int(a)) * 4194304 + __float2int_rn(low));
}

// ------------------------------------------------------------------ sums over the row

__device__ __forceinline__ void row_sync() {  // all threads of the row's CTAs
  __syncwarp();
  cluster_sync();
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

// The sum f(x, index) of the whole row's entries passes target(total) at the returned index: the first whose inclusive
// sum, by index, is above it.  Every CTA returns it.
template <class T, class F, class G>
__device__ __noinline__ int locate(Shared& sh, const Row<T>& r, int rank, int ctas, int per_cta, int per_warp, F f, G target,
                                   uint64_t& total) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint64_t own = 0;
  sweep(r, [&](float x, int i) { own += f(x, i); });
  own = warp_sum(own);
  if (lane == 0) sh.chunk[warp] = own;
  row_sync();
  if (tid < ctas * kWarps) sh.all[tid] = ld_peer_u64(sh.chunk + tid % kWarps, tid / kWarps);
  const int chunks = ctas * kWarps;
  __syncthreads();
  uint64_t incl = tid < chunks ? sh.all[tid] : 0;
  const uint64_t mine = incl;
  incl = block_scan(incl, sh.room);
  if (tid == kThreads - 1) sh.pick_sum = incl;
  __syncthreads();
  total = sh.pick_sum;
  const uint64_t at = target(total);
  if (tid < chunks && incl > at && incl - mine <= at) {
    sh.pick = tid;
    sh.pick_before = incl - mine;
  }
  __syncthreads();
  const int pick = sh.pick, owner = pick / kWarps;
  if (rank == owner) {
    // the run of the warp that passes it, its entries shared out to all threads in order
    const int v0 = min(rank * per_cta + (pick % kWarps) * per_warp, r.vectors);
    const int v1 = min(min(v0 + per_warp, (rank + 1) * per_cta), r.vectors);
    const int i0 = max(v0 * kVec<T> - r.off, 0), i1 = min(v1 * kVec<T> - r.off, r.V);
    const int per = (i1 - i0 + kThreads - 1) / kThreads, a = min(i0 + tid * per, i1), b = min(a + per, i1);
    uint64_t sum = 0;
    for (int i = a; i < b; ++i) sum += f(entry(r, i), i);
    const uint64_t upto = sh.pick_before + block_scan(sum, sh.room2);
    if (upto > at && upto - sum <= at) {
      uint64_t before = upto - sum;
      for (int i = a; i < b; ++i) {
        before += f(entry(r, i), i);
        if (before > at) {
          sh.found = i;
          break;
        }
      }
    }
  }
  row_sync();
  const int found = int(ld_peer_u32(&sh.found, owner));
  row_sync();
  return found;
}

struct Cut {
  uint32_t key;   // entries with larger keys are kept, and those of this key up to the index
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

// The cut that keeps entries, in order, until their measures f(x, key, index) add up to target(total): the last is the
// first with target <= the inclusive sum.  A histogram by value over the weights' range, then by key within the bin, each
// level a sweep; then the index among equal values.
template <class T, class F, class G>
__device__ __noinline__ Cut search(Shared& sh, const Row<T>& r, const Scale& sc, int rank, int ctas, int per_cta,
                                   int per_warp, F f, G target_of) {
  const int tid = threadIdx.x;
  // bins of equal width down to where weights vanish; the last takes the rest
  const float width = float(kBins - 1) / float(kSampleUnitBits + 3) * sc.c;
  auto bin_of = [&](float x) { return min(int((sc.M - x) * width), kBins - 1); };
  uint32_t lo = 1, hi = key_of(sc.M);
  int level = 0, shift = 32, first_bin = 0;
  uint64_t above = 0, target = 0, in_bin = 0;
  while (shift > 0) {
    if (level > 0) {
      const uint32_t span = hi - lo;
      shift = 0;
      while ((span >> shift) >= uint32_t(kBins)) ++shift;
    }
    sh.bin_lo[tid] = 0;
    sh.bin_hi[tid] = 0;
    __syncthreads();
    sweep(r, [&](float x, int i) {
      const uint32_t key = key_of(x);
      int bin = bin_of(x);
      if (level > 0) {
        if (bin != first_bin || key < lo || key > hi) return;
        bin = int((hi - key) >> shift);
      }
      const uint64_t m = f(x, key, i);
      if (m == 0) return;
      const uint32_t low = uint32_t(m), old = atomicAdd(&sh.bin_lo[bin], low);
      const uint32_t high = uint32_t(m >> 32) + (old + low < old ? 1u : 0u);
      if (high) atomicAdd(&sh.bin_hi[bin], high);
    });
    row_sync();
    uint64_t own = 0;
    for (int c = 0; c < ctas; ++c)
      own += (uint64_t(ld_peer_u32(&sh.bin_hi[tid], c)) << 32) + ld_peer_u32(&sh.bin_lo[tid], c);
    uint64_t incl = block_scan(own, sh.room);
    if (tid == kThreads - 1) sh.pick_sum = incl;
    __syncthreads();
    if (level == 0) target = target_of(sh.pick_sum);
    if (own > 0 && above + incl >= target && above + incl - own < target) {
      sh.pick = tid;
      sh.pick_before = incl - own;
    }
    __syncthreads();
    const int bin = sh.pick;
    above += sh.pick_before;
    __syncthreads();
    if (tid == bin) sh.pick_sum = own;
    if (level == 0) {
      // keys that the bin's values may have (its own test stays)
      first_bin = bin;
      const float from = sc.M - float(bin) / width, to = sc.M - float(bin + 1) / width;
      const float slack = (fabsf(sc.M) + fabsf(to)) * 1e-5f;
      hi = min(hi, key_of(from + slack));
      lo = bin == kBins - 1 || !(to - slack > -INFINITY) ? 1u : key_of(to - slack);
    } else {
      hi -= uint32_t(bin) << shift;
      lo = max(lo, hi - ((1u << shift) - 1u));
    }
    ++level;
    row_sync();  // (the peers have read the bins)
    in_bin = sh.pick_sum;
  }
  const uint32_t key = hi;
  const float value = value_of(key);
  // of equal values the lowest indices
  const uint64_t each = f(value, key, 0);
  const uint64_t want = (target - above + each - 1) / each;
  Cut cut = {key, INT_MAX};
  if (want < in_bin / each) {
    uint64_t n;
    cut.index = locate(
        sh, r, rank, ctas, per_cta, per_warp, [&](float x, int) { return uint64_t(key_of(x) == key ? 1 : 0); },
        [&](uint64_t) { return want - 1; }, n);
  }
  return cut;
}

// ------------------------------------------------------------------ the kernel

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int ctas = int(cluster_size()), rank = int(cluster_rank());
  const long long row = blockIdx.x / ctas;
  const int b = int(row / a.n), n = int(row - (long long)b * a.n);
  if (tid < 64) sh.table[tid] = kExp2Table[tid];
  if (tid == 0) {
    sh.first = INT_MAX;
    sh.found = 0;
    sh.pick = 0;
    sh.pick_before = 0;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the request's parameters
  const float T_ = a.temperature != nullptr ? a.temperature[b] : a.one.temperature;
  const int top_k = a.top_k != nullptr ? a.top_k[b] : a.one.top_k;
  const float top_p = a.top_p != nullptr ? a.top_p[b] : a.one.top_p;
  const float min_p = a.min_p != nullptr ? a.min_p[b] : a.one.min_p;
  const bool params_ok = sampling_ok(T_, top_k, top_p, min_p);
  float u = a.u[b * a.u_b + n * a.u_n];
  u = u >= 0.0f ? fminf(u, 0.99999994f) : 0.0f;

  Row<T> r;
  const T* first = static_cast<const T*>(a.x) + b * a.x_b + n * a.x_n;
  r.off = int((reinterpret_cast<uintptr_t>(first) % 16) / sizeof(T));
  r.base = first - r.off;
  r.V = a.V;
  r.vectors = (r.off + a.V + kVec<T> - 1) / kVec<T>;
  const int per_cta = (r.vectors + ctas - 1) / ctas, per_warp = (per_cta + kWarps - 1) / kWarps;
  r.v0 = min(rank * per_cta + warp * per_warp, r.vectors);
  r.v1 = min(min(r.v0 + per_warp, (rank + 1) * per_cta), r.vectors);

  // ---- the maximum
  float top = -INFINITY;
  bool bad = false;
  sweep(r, [&](float x, int) {
    bad = bad || x != x;
    top = fmaxf(top, x);
  });
  bad = __syncthreads_or(bad || top == INFINITY);
  top = warp_max(top);
  if (lane == 0) sh.chunk[warp] = __float_as_uint(top);
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, __uint_as_float(uint32_t(sh.chunk[w])));
    sh.top = top;
    sh.bad = bad;
  }
  row_sync();
  Scale sc;
  sc.M = -INFINITY;
  for (int c = 0; c < ctas; ++c) {
    sc.M = fmaxf(sc.M, __uint_as_float(ld_peer_u32(&sh.top, c)));
    bad = bad || ld_peer_u32(&sh.bad, c) != 0;
  }
  bad = bad || sc.M == -INFINITY;
  int token = -1;
  float logprob = -INFINITY;
  uint64_t total = 0;
  Cut cut = {0u, INT_MAX};
  uint64_t least = 0;

  // (params_ok and bad are the whole cluster's)
  const bool greedy = T_ == 0.0f;
  if (params_ok && !bad) {
    if (greedy) {
      const uint32_t key = key_of(sc.M);
      token = locate(
          sh, r, rank, ctas, per_cta, per_warp, [&](float x, int) { return uint64_t(key_of(x) == key ? 1 : 0); },
          [&](uint64_t) { return uint64_t(0); }, total);
      cut = {key, token};
      logprob = 0.0f;
    } else {
      sc.c = kLog2eHi / T_;
      sc.c_lo = (fmaf(-sc.c, T_, kLog2eHi) + kLog2eLo) / T_;
      if (top_k > 0 && top_k < a.V)
        cut = search(
            sh, r, sc, rank, ctas, per_cta, per_warp, [&](float, uint32_t, int) { return uint64_t(1); },
            [&](uint64_t) { return uint64_t(top_k); });
      if (top_p < 1.0f) {
        const Cut k = cut;
        const uint64_t part = uint64_t(top_p * 18446744073709551616.0f);
        cut = search(
            sh, r, sc, rank, ctas, per_cta, per_warp,
            [&](float x, uint32_t key, int i) { return k.keeps(key, i) ? weight(x, sc, sh.table) : uint64_t(0); },
            [&](uint64_t all) {
              const uint64_t whole = __umul64hi(part, all) + (part * all != 0 ? 1 : 0);  // p times the mass, up
              return whole > 0 ? whole : uint64_t(1);
            });
        if (cut.key == k.key) cut.index = min(cut.index, k.index);
      }
      least = uint64_t(ceilf(min_p * float(kOne)));
      const uint64_t draw = uint64_t(u * 18446744073709551616.0f);
      token = locate(
          sh, r, rank, ctas, per_cta, per_warp,
          [&](float x, int i) {
            if (!cut.keeps(key_of(x), i)) return uint64_t(0);
            const uint64_t w = weight(x, sc, sh.table);
            return w >= least ? w : uint64_t(0);
          },
          [&](uint64_t all) { return __umul64hi(draw, all); }, total);
      const uint64_t w = weight(entry(r, token), sc, sh.table);
      logprob = -log1pf(float(total - w) / float(w));
    }
  }
  if (rank == 0 && tid == 0) {
    if (!params_ok) atomicOr(a.status + b, ASV_REQ_BAD_PARAM);
    if (bad) atomicOr(a.status + b, ASV_REQ_NONFINITE);
    a.tokens[b * a.tokens_b + n * a.tokens_n] = token;
    if (a.logprobs != nullptr) a.logprobs[b * a.logprobs_b + n * a.logprobs_n] = logprob;
  }

  // ---- the distribution
  if (a.probs != nullptr) {
    float* to = a.probs + b * a.probs_b + n * a.probs_n;
    const float inv = token >= 0 && !greedy ? float(kOne) / float(total) : 1.0f;
    sweep(r, [&](float x, int i) {
      float p = 0.0f;
      if (token >= 0 && cut.keeps(key_of(x), i)) {
        if (greedy) {
          p = 1.0f;
        } else {
          const uint64_t w = weight(x, sc, sh.table);
          if (w >= least) p = float(w) * (1.0f / float(kOne)) * inv;
        }
      }
      to[i] = p;
    });
  }
  row_sync();  // (no CTA leaves while its peers read its shared memory)
}

// CTAs to a row: enough that all rows' together fill the GPU, each with enough of the row to be worth its exchanges.
int sample_ctas(const SampleArgs& a) {
  int ctas = 1;
  while (ctas < kMaxCtas && 2ll * ctas * a.B * a.n <= 304 && a.V / (2 * ctas) >= 2048) ctas *= 2;
  return ctas;
}

template <class T>
cudaError_t launch(const SampleArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int ctas = sample_ctas(a);
  cfg.gridDim = dim3(unsigned((long long)a.B * a.n * ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
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
  return dtype == ASV_BF16 ? launch<bf16_t>(a, s) : launch<float>(a, s);
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
