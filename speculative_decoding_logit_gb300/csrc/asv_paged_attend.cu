// asv_paged_attend.cu -- paged_attention: attention of a chunk of new tokens over a paged cache.
//
//   s_ij = scale * (q_i . k_j),  out_i = sum_j 2^((s_ij - m_i) log2 e) v_j / sum_j 2^((s_ij - m_i) log2 e)
//
// over the positions j that token i attends to (causal, window), with a running reference m_i.
//
// Rows.  The query heads of a key head read the same keys, so a row tile of 128 rows holds
// floor(128 / G) tokens x G heads, and an item is (request, NT row tiles, key head): NT = 1 where a
// request's chunk fits one tile, NT = 2 for longer chunks (each key and value tile then serves 256 rows,
// which halves what a CTA reads from L2 per multiplication).  With at most 32 rows to an item the row tile is
// divided (DIV): it holds the 32 rows four times, and each softmax warp takes 32 of a tile's 128 positions
// instead of one warp all of them (a warp can only reach 32 rows of tensor memory).
//
// Split.  An item costs as many units as it has key tiles of 128 positions, and one or two for itself.  The
// units of all items, in order, are cut into equal runs, one for each CTA (one CTA per SM), so a batch of any
// lengths keeps every SM busy to the end; the prefix sums need only indptr and cache_len and a closed form per
// request, and a warp of every CTA computes them.  An item that a cut goes through is finished from partial
// results (unnormalised outputs, reference, sum) in the workspace by the CTA that files the last of them, in CTA
// order, so the result does not depend on timing.
//
// In a CTA, warps take roles that hand over through mbarriers:
//   scheduler  finds the CTA's run, walks it and describes its pieces in a queue
//   copies     (two warps: keys; queries and values) one box of the tensor map per page (part), 128-byte swizzled,
//              into a ring of key / value tiles; positions that no row of the item attends to are not read (zero
//              fill)
//   matrices   S = Q K^T into tensor memory; out += P V with P taken from tensor memory (NT = 1: a warp each)
//   softmax    one thread per row: S to registers, reference, 2^x, P back over S in the 16-bit type; the
//              outputs are rescaled only when the reference moves by more than 2^8, so seldom after the
//              first tiles; the epilogue divides and stores
// NT = 1 keeps two S and two output buffers, so the next tile's S is formed while the softmax runs; NT = 2
// gives each row tile one, and the two tiles alternate.
//
// Measured (bf16, heads of 128, one call among others): 64 requests x 3 tokens over 500 .. 12,000, 64 / 8 heads,
// 148 us, bound by HBM (6.2 TB/s); 256 x 1 token over 1 .. 4096 (fp16) 94 us, 507 MB; 4 x 2048 tokens over
// 8192, 32 / 8 heads, 715 - 721 us at the clock that the power limit leaves (1.34 PFLOP/s; a single launch 630), bound by
// each row tile's chain S, softmax, P V; 1 token over 4096, 10.5 us, all latency.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "asv_paged_device.cuh"
#include "asv_ring.h"
#include "asv_tcgen05.cuh"

namespace asv {

namespace {

using namespace tc;

constexpr int kTile = 128;  // rows of a row tile; positions of a key tile
constexpr int kQueue = 16;  // pieces ahead: of 4, short items left the copies waiting for the scheduler (2 % at 6 prompts)
constexpr uint32_t kTmemColumns = 512;  // S buffers at 0 and 128, outputs at 256 and 384
// Key tiles that an item's own work (queries in, outputs out, the pipeline's fill) is worth in the split: one for the
// divided row tile of many short items (256 requests, one token: 95.3 us, 100 with 1.75, 97.5 with 1.5; undivided it
// took 107 with two, 121 with one), else two (one request, one token: 10.6 us, 11.1 with one).
template <bool DIV>
__device__ int item_cost(const PagedView& c) {
  return DIV && (long long)c.B * c.kv_heads > gridDim.x ? 1 : 2;
}
constexpr float kLazy = 8.0f;  // log2 units the maximum may pass the reference by
// Weights are 2^kLift times 2^(s - reference).  fp16 has no step below 2^-24, so next to a largest weight of 1 those below
// 2^-25 would vanish from the product with the values (20 thousand of 2^-25.6 are 4e-4 of the sum); lifted by 2^7 the
// largest, 2^(kLazy + 7), is still in range and they vanish below 2^-32.  bf16 has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;

// Warps: four of softmax for each row tile, matrices, copies of keys, copies of values, scheduler; with one row tile
// the products P V have a warp of their own.
template <int NT>
constexpr int kThreadsOf = 32 * (4 * NT + 4 + (NT == 1 ? 1 : 0));

// Slots of the ring of keys and values.  Five of 32 KB are what shared memory holds next to two tiles of queries; where
// the copies are what bounds (NT = 1), two tiles ahead are enough and go faster (256 requests, one token: 102.6 us, 105
// with five; NT = 2, 4 x 2048 tokens: 5 % slower with four).
template <int DP, int NT>
constexpr int kRingSlots = (NT == 1 ? 4 : 5) * (128 / DP);
constexpr uint32_t kChunkBytes = 32 * 32 * 2;  // weights of 32 rows for 32 positions: [8 positions][row] vectors
template <bool DIV>
constexpr uint32_t kExchangeBytes = DIV ? 2 * 4 * kChunkBytes : 0;

// A run of key tiles of one item.
struct Piece {
  int request;
  int tok0, ntok;  // first row of the item's tokens and their number
  int head;        // key head
  int pos0;        // position of the first token
  int kv_lo;       // first position that any of the tokens attends to
  int t0, t1;      // key tiles [t0, t1); none: a request left out, whose outputs are zero
  int part;        // -1: the whole item; else the slot of its partial result
  int item_tiles;  // key tiles of the item
  int kind;        // 0: a piece; 1: the end of the run
  long long item;  // units before the item's first key tile
};

// a / b for a >= 0, b > 0; in 32 bits where that will do (all but always), at a fraction of the time.  (What is
// rare is out of line here and below: a short call runs most of its instructions for the first time, and fetching
// them is a good part of its time.)
__device__ __noinline__ long long quotient_64(long long a, long long b) { return a / b; }

__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)(uint32_t(a) / uint32_t(b)) : quotient_64(a, b);
}

// sum_{i < n} floor((a i + b) / m) for a, b >= 0: each round takes out the whole parts of a / m and b / m
// and counts the lattice points left under the line with the axes exchanged.
__device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  for (;;) {
    if (a >= m) {
      const long long q = quotient(a, m);
      sum += n * (n - 1) / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const long long q = quotient(b, m);
      sum += n * q;
      b -= q * m;
    }
    const long long top = a * n + b;
    if (top < m) return sum;
    n = quotient(top, m);
    b = top - n * m;
    const long long t = m;
    m = a;
    a = t;
  }
}

// sum_{i < n} floor((T i + b) / 128) for b >= 0; `shift` is log2 T where T is a power of two, else -1.
__device__ __noinline__ long long tile_sum(long long n, int T, int shift, long long b) {
  if (shift < 0) return floor_sum(n, kTile, T, b);
  if (shift >= 7) return n * (b >> 7) + ((n * (n - 1) / 2) << (shift - 7));
  // floor((floor(b / T) + i) / r), r = 128 / T: differences of sum_{m < x} floor(m / r)
  const int s = 7 - shift;
  auto below = [&](long long x) {
    const long long q = x >> s;
    return ((q * (q - 1) / 2) << s) + q * (x - (q << s));
  };
  const long long c = b >> shift;
  return below(c + n) - below(c);
}

// Key tiles of the first i items of T tokens behind `past` tokens.
__device__ __noinline__ long long sum_before(int past, int T, int shift, int window, int i) {
  long long sum = tile_sum(i, T, shift, (long long)past + T + kTile - 1);
  if (window > 0) {
    // items before z start at position 0
    const long long z = past >= window - 1 ? 0 : quotient((long long)window - 1 - past + T - 1, T);
    if (i > z) sum -= tile_sum(i - z, T, shift, past + z * T - window + 1);
  }
  return sum;
}

// A request's items of one key head: n of them, item r with the tokens from r * T.
struct Items {
  Request r;
  int T, shift, n;
  __device__ int lo(int window, int i) const { return window > 0 ? max(0, r.past + i * T - window + 1) : 0; }
  // key tiles (1 for a request that is left out)
  __device__ int tiles(int window, int i) const {
    if (!r.ok) return 1;
    const int hi = r.past + min((i + 1) * T, r.end - r.start);
    return (hi + kTile - 1) / kTile - lo(window, i) / kTile;
  }
  // key tiles of the items before i (i < n)
  __device__ long long tiles_before(int window, int i) const {
    return i == 0 ? 0 : r.ok ? sum_before(r.past, T, shift, window, i) : i;
  }
  // units of one key head before item i
  __device__ long long before(int window, int cost, int i) const { return tiles_before(window, i) + (long long)cost * i; }
  // units of all (most requests have one item to a key head, or none)
  __device__ long long units(int window, int cost, int kv_heads) const {
    const long long last = (long long)tiles(window, max(n - 1, 0)) + cost;
    return n == 0 ? 0 : kv_heads * (n == 1 ? last : last + before(window, cost, n - 1));
  }
};

__device__ Items load_items(const PagedView& c, int b, int T) {
  Items it;
  it.r = load_request(c, b, table_positions(c));
  it.T = T;
  it.shift = (T & (T - 1)) == 0 ? 31 - __clz(T) : -1;
  // the rows of a request that is left out are still zeroed, where they are rows
  const bool rows = it.r.start >= 0 && it.r.start <= it.r.end && it.r.end <= c.N;
  const int len = rows ? it.r.end - it.r.start : 0;
  it.n = len <= T ? (len > 0 ? 1 : 0) : it.shift >= 0 ? ((len - 1) >> it.shift) + 1 : (len - 1) / T + 1;
  return it;
}

struct Misc {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[4], pv_done[2], o_full[2], o_empty[2];
  uint64_t piece_full[kQueue], piece_empty[kQueue], wg_sync[2];
  Piece piece[kQueue];
  long long units;  // of all runs
  uint32_t tmem;
  int abort;
  int poison[2];  // a value that some rows of the item in this output buffer do not attend to is not finite
  int last[2][2];
  // for a launch that gives up: where the copies of keys, values and queries ended, the matrix instructions' end
  Ring copied[2], queries;
  uint64_t drained[2];
};

// What the warps of a divided row tile tell each other, for odd and even tiles: whether the reference has to move, the
// maxima; the sums of a piece.
struct Divided {
  int vote[2][4];
  float top[2][4][32], sum[4][32];
};

__device__ __forceinline__ uint32_t at(const uint64_t* bars, int i) { return smem_addr(bars + i); }

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// 0 * x + acc for both 16-bit elements: NaN from the first x that is not finite on.
template <bool BF16>
__device__ __forceinline__ uint32_t probe2(uint32_t x, uint32_t acc) {
  uint32_t r;
  if constexpr (BF16) {
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  } else {
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t finite_or_zero2(uint32_t w) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  if ((w & kExp) == kExp) w &= 0xffff0000u;
  if (((w >> 16) & kExp) == kExp) w &= 0x0000ffffu;
  return w;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// Rows [r0, r1) of a tile of keys or values, 16 bytes a time over the lanes of a warp: f(address).
template <int DP, class F>
__device__ __forceinline__ void each_vec(uint32_t tile, int r0, int r1, int lane, F f) {
  constexpr int kVecs = DP / 8, kRows = 32 / kVecs;  // vectors of a row, rows of a step
  const int vec = lane % kVecs;
  uint32_t p = tile + (vec / 8) * (kTile * 128) + (r0 + lane / kVecs) * 128 + (vec % 8) * 16;
  const uint32_t end = tile + (vec / 8) * (kTile * 128) + r1 * 128;
#pragma unroll 4
  for (; p < end; p += kRows * 128) f(p);
}

template <bool BF16, int DP>
__device__ __noinline__ void zero_nonfinite(uint32_t tile, int r0, int r1, int lane) {
  each_vec<DP>(tile, r0, r1, lane, [](uint32_t p) {
    const uint4 x = lds16(p);
    sts16(p, make_uint4(finite_or_zero2<BF16>(x.x), finite_or_zero2<BF16>(x.y), finite_or_zero2<BF16>(x.z),
                        finite_or_zero2<BF16>(x.w)));
  });
}

// Makes a tile of values (rows = positions base .. base + 127) safe to multiply by weights of zero.  The
// product takes rows in steps of 16, those that reach into [lo, hi): the rest of the first and the last
// step, which no row of the item attends to, is zeroed.  In the rows that only some attend to, [zone, hi)
// and [lo, wzone), elements that are not finite are zeroed and reported (the epilogue adds them to the rows
// that do attend to them).  By one warp.
template <bool BF16, int DP>
__device__ bool clean_values(uint32_t tile, int base, int lo, int hi, int zone, int wzone, int lane) {
  const int first = max(lo - base, 0), end = min(hi - base, kTile);
  auto zero = [](uint32_t p) { sts16(p, make_uint4(0, 0, 0, 0)); };
  each_vec<DP>(tile, first & ~15, first, lane, zero);
  each_vec<DP>(tile, end, (end + 15) & ~15, lane, zero);
  const int w1 = max(min(wzone - base, end), first), z0 = max(max(zone - base, first), w1);
  uint32_t acc[4] = {0, 0, 0, 0};
  auto probe = [&](uint32_t p) {
    const uint4 x = lds16(p);
    acc[0] = probe2<BF16>(x.x, acc[0]);
    acc[1] = probe2<BF16>(x.y, acc[1]);
    acc[2] = probe2<BF16>(x.z, acc[2]);
    acc[3] = probe2<BF16>(x.w, acc[3]);
  };
  each_vec<DP>(tile, first, w1, lane, probe);
  each_vec<DP>(tile, z0, end, lane, probe);
  // sums of products with zero: +-0 unless one was not finite
  const bool found = __any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0);
  if (found) {
    zero_nonfinite<BF16, DP>(tile, first, w1, lane);
    zero_nonfinite<BF16, DP>(tile, z0, end, lane);
  }
  fence_async_shared();
  __syncwarp();
  return found;
}

// Eight 16-byte vectors of each lane (its row) exchanged among groups of eight lanes, so that lane i of a
// group ends with vector i of the group's eight rows and a store covers whole 128-byte lines.
__device__ __forceinline__ void transpose8(uint32_t (&w)[32], int lane) {
#pragma unroll
  for (int m = 1; m < 8; m *= 2) {
    const bool up = lane & m;
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      if (a & m) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t mine = w[4 * a + e], theirs = w[4 * (a | m) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? mine : theirs, m);
        w[4 * a + e] = up ? got : mine;
        w[4 * (a | m) + e] = up ? theirs : got;
      }
    }
  }
}

// Adds to entries d0 .. d0 + N - 1 of a row's outputs the values that are not finite among those it attends
// to at positions [lo, hi) and the item's other rows may not (all but [skip_lo, skip_hi)).  Out of line: only
// rows next to such values come here.
template <bool BF16, int N>
__device__ __noinline__ void add_poison(const PagedView& c, int request, int head, int lo, int hi, int skip_lo,
                                        int skip_hi, int d0, float* o) {
  for (int k = lo; k < hi; ++k) {
    if (k >= skip_lo && k < skip_hi) continue;
    const int page = c.table[request * c.table_stride + k / c.page_size];
    if (page < 0 || page >= c.num_pages) continue;
    const uint16_t* v = c.v + page * c.v_page + (k % c.page_size) * c.v_slot + head * c.v_head;
    for (int d = 0; d < N && d0 + d < c.head_dim; ++d) {
      const float x = unpack1<BF16>(v[d0 + d]);
      if (!(fabsf(x) < INFINITY)) o[d] += x;
    }
  }
}

template <bool BF16, int DP, int NT, bool DIV>
__global__ void __launch_bounds__(kThreadsOf<NT>, 1)
    paged_attention_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  static_assert(NT == 1 || !DIV);
  constexpr int kRing = kRingSlots<DP, NT>;
  constexpr int kHalves = DP / 64;                // 64-element column blocks, 128 bytes a row
  constexpr uint32_t kTileBytes = kTile * DP * 2;
  constexpr uint32_t kHalfBytes = kTile * 128;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t smem0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_tiles = smem0, ring = smem0 + 2 * kTileBytes;
  const uint32_t exchange = ring + kRing * kTileBytes;
  unsigned char* rest = smem_raw + (smem0 - smem_addr(smem_raw)) + (2 + kRing) * kTileBytes + kExchangeBytes<DIV>;
  Misc& ms = *reinterpret_cast<Misc*>(rest);
  Divided& dv = *reinterpret_cast<Divided*>(rest + sizeof(Misc));  // (only where DIV)
  const PagedView& c = a.c;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr int kMmaWarp = 4 * NT, kCopyWarp = 4 * NT + 1, kWalkWarp = 4 * NT + 3;
  const int T = NT * a.tile_tokens;  // tokens of an item
  volatile int* abort = &ms.abort;

  // ---- set-up, and the run of this CTA
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&ms.tmem), kTmemColumns);
  } else if (warp == kCopyWarp && lane == 0) {
    for (int i = 0; i < kRing; ++i) {
      bar_init(at(ms.kv_full, i), 1);
      bar_init(at(ms.kv_empty, i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(at(ms.q_full, i), 1);
      bar_init(at(ms.q_empty, i), 1);
      bar_init(at(ms.s_full, i), 1);
      bar_init(at(ms.p_full, 2 * i), 4);
      bar_init(at(ms.p_full, 2 * i + 1), DIV ? 1 : 4);
      bar_init(at(ms.pv_done, i), 1);
      bar_init(at(ms.o_full, i), 1);
      bar_init(at(ms.o_empty, i), 4);
      bar_init(at(ms.wg_sync, i), 4);
      bar_init(at(ms.drained, i), 1);
      ms.poison[i] = 0;
    }
    for (int i = 0; i < kQueue; ++i) {
      bar_init(at(ms.piece_full, i), 1);
      bar_init(at(ms.piece_empty, i), 3 + 4 * NT + (NT == 1 ? 1 : 0));
    }
    ms.abort = 0;
    fence_barrier_init();
    prefetch_map(&map_q);
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ms.tmem;
  // What comes after on the stream may set itself up; what came before is needed from here on.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kWalkWarp) {
    const int cost = item_cost<DIV>(c);
    // ---- scheduler: the lanes sum up their shares of the requests, find where the run starts, and one walks it
    const int per_lane = (c.B + 31) / 32, b0 = min(lane * per_lane, c.B), b1 = min(b0 + per_lane, c.B);
    long long own = 0;
    Items it;
    for (int b = b0; b < b1; ++b) {
      it = load_items(c, b, T);
      if (!it.r.ok && blockIdx.x == 0) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
      own += it.units(a.window, cost, c.kv_heads);
    }
    long long before = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    const long long total = __shfl_sync(0xffffffffu, before, 31);
    before -= own;
    // The runs: c * units / grid up to (c + 1) * units / grid, rounded down.  Short ones are made of one length (units
    // rounded up), which cuts the items into fewer parts (one request, one token: 10.7 us, 11.8 with runs of one and
    // two units); long ones would leave the last CTAs idle (256 requests: 94.1 us, 95.4).
    const int grid = gridDim.x;
    const long long run = quotient(max(total, 1ll) + grid - 1, grid);
    long long units = run * grid, u0 = blockIdx.x * run, u1 = u0 + run;
    if (run > 16) {
      units = total;
      u0 = quotient(blockIdx.x * units, grid);
      u1 = quotient((blockIdx.x + 1) * units, grid);
    }
    u0 = min(u0, total);
    u1 = min(u1, total);
    if (lane == 0) ms.units = units;
    __syncwarp();
    // the request and the item that hold unit u0 (none: the end of the run)
    int b = c.B, i = 0, n = 0, h = 0;
    long long item0 = u0;
    const uint32_t has = __ballot_sync(0xffffffffu, u0 < u1 && u0 >= before && u0 < before + own);
    if (has != 0) {
      const int lane_of = __ffs(has) - 1;
      if (lane == lane_of) {
        for (b = b0; b + 1 < b1; ++b) {
          const long long units = load_items(c, b, T).units(a.window, cost, c.kv_heads);
          if (u0 < before + units) break;
          before += units;
        }
      }
      b = __shfl_sync(0xffffffffu, b, lane_of);
      before = __shfl_sync(0xffffffffu, before, lane_of);
      it = load_items(c, b, T);
      // the last item with no more than rel units before it: 32 candidates at a time
      const long long rel = u0 - before;
      for (int end = it.n; end - i > 1;) {
        const int step = (end - i + 31) / 32, k = i + lane * step;
        const bool below = k < end && c.kv_heads * it.before(a.window, cost, min(k, end - 1)) <= rel;
        i += (__popc(__ballot_sync(0xffffffffu, below)) - 1) * step;
        end = min(i + step, end);
      }
      n = it.tiles(a.window, i);
      item0 = before + c.kv_heads * it.before(a.window, cost, i);
      const long long units = (long long)n + cost;
      h = int(quotient(u0 - item0, units));
      item0 += h * units;
    }
    if (lane == 0) {
      Ring ring_p;
      for (;;) {
        // its first `cost` units are its own, then one for each key tile
        const int ta = int(max(u0 - item0 - cost, 0ll));
        const int tb = int(min(max(u1 - item0 - cost, 0ll), (long long)n));
        const bool end = b >= c.B || item0 >= u1;
        if (end || tb > ta) {
          if (!bar_wait(at(ms.piece_empty, ring_p.slot), ring_p.phase ^ 1, abort)) break;
          Piece& p = ms.piece[ring_p.slot];
          p.kind = end;
          if (!end) {
            p.request = b;
            p.tok0 = it.r.start + i * T;
            p.ntok = min(T, it.r.end - p.tok0);
            p.head = h;
            p.pos0 = it.r.past + i * T;
            p.kv_lo = it.lo(a.window, i);
            const int tile0 = p.kv_lo / kTile;
            p.t0 = it.r.ok ? tile0 + ta : 0;
            p.t1 = it.r.ok ? tile0 + tb : 0;
            p.part = tb - ta == n ? -1 : 2 * int(blockIdx.x) + (ta == 0 ? 1 : 0);
            p.item_tiles = n;
            p.item = item0 + cost;
          }
          bar_arrive(at(ms.piece_full, ring_p.slot));
          ring_p.next(kQueue);
        }
        if (end) break;
        item0 += n + cost;
        if (++h == c.kv_heads) {
          h = 0;
          if (++i == it.n) {
            i = 0;
            do {
              if (++b >= c.B) break;
              it = load_items(c, b, T);
            } while (it.n == 0);
          }
          if (b < c.B) n = it.tiles(a.window, i);
        }
      }
    }
  } else if (warp == kCopyWarp || warp == kCopyWarp + 1) {
    // ---- copies: one warp for keys, one for queries and values; a copy takes its warp about 50 cycles
    const bool values = warp == kCopyWarp + 1;
    // 32 lanes hold the pages of up to 32 boxes, a window of one or more tiles; the next window's entries of
    // the block table are on their way while this one's tiles are copied.
    Ring ring_p, ring_kv, ring_q;
    const int boxes = kTile / a.box, shift = 31 - __clz(boxes);
    const int group = lane >> shift, in_tile = (lane & (boxes - 1)) * a.box;  // this lane's tile and box
    struct Window {
      int head, tok0, ntok, request, t0, n, entry, slot;
      bool first, need;
    };
    Piece p;
    p.kind = p.t1 = 0;
    int t = 0;
    // the next window; `block`: wait for its piece.  n = 0: none (yet).
    auto next_window = [&](bool block, Window& w) {
      w.n = 0;
      while (t == p.t1) {
        if (p.kind == 1) return true;
        const uint32_t bar = at(ms.piece_full, ring_p.slot);
        if (block ? !warp_wait(bar, ring_p.phase, abort) : !__all_sync(0xffffffffu, bar_test(bar, ring_p.phase)))
          return !block;
        p = ms.piece[ring_p.slot];
        __syncwarp();
        if (lane == 0) bar_arrive(at(ms.piece_empty, ring_p.slot));
        ring_p.next(kQueue);
        if (p.kind == 1) {
          t = p.t1;
          return true;
        }
        t = p.t0;
      }
      w.head = p.head;
      w.tok0 = p.tok0;
      w.ntok = p.ntok;
      w.request = p.request;
      w.first = t == p.t0;
      w.t0 = t;
      w.n = min(32 >> shift, p.t1 - t);
      // what no row attends to is filled with zeros (a page past the last)
      const int pos = (t + group) * kTile + in_tile;
      w.need = group < w.n && pos < p.pos0 + p.ntok && pos + a.box > p.kv_lo;
      const int page = pos / c.page_size;
      w.slot = pos - page * c.page_size;
      w.entry = w.need && ASV_GUARD(a, page >= 0 && page < c.max_pages && p.request < c.B)
                    ? c.table[p.request * c.table_stride + page]
                    : -1;
      t += w.n;
      return true;
    };
    // A tile's keys and values take two slots of the ring, one after the other.
    if (values) ring_kv.next(kRing);
    const CUtensorMap* map = values ? &map_v : &map_k;
    // one tile of keys (or values) into its slot: the lanes of `g` copy their boxes
    auto copy_tile = [&](int head, int g, int page, int slot) {
      if (!warp_wait(at(ms.kv_empty, ring_kv.slot), ring_kv.phase ^ 1, abort)) return false;
      const uint32_t bar = at(ms.kv_full, ring_kv.slot);
      if (lane == 0) bar_expect(bar, kTileBytes);
      __syncwarp();
      if (group == g) {
        const uint32_t dst = ring + ring_kv.slot * kTileBytes + in_tile * 128;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) copy_4d(dst + h * kHalfBytes, map, h * 64, head, slot, page, bar);
      }
      __syncwarp();
      ring_kv.next(kRing, 2);
      return true;
    };
    auto copy_queries = [&](const Window& w) {
      if (!warp_wait(at(ms.q_empty, ring_q.slot), ring_q.phase ^ 1, abort)) return false;
      if (lane == 0) {
        const int tiles = NT == 1 || w.ntok <= a.tile_tokens ? 1 : 2;
        const uint32_t bar = at(ms.q_full, ring_q.slot);
        bar_expect(bar, (DIV ? 4 : tiles) * kHalves * a.tile_tokens * a.group * 128);
        for (int i = 0; i < (DIV ? 4 : tiles); ++i)
          for (int h = 0; h < kHalves; ++h)
            copy_3d(q_tiles + (NT == 1 ? ring_q.slot * kTileBytes + i * 32 * 128 : i * kTileBytes) + h * kHalfBytes, &map_q,
                    h * 64, w.head * a.group, w.tok0 + (DIV ? 0 : i * a.tile_tokens), bar);
      }
      __syncwarp();
      ring_q.next(3 - NT);
      return true;
    };
    Window w, ahead;
    ahead.n = 0;
    bool run = true;
    for (int late = 1; run; late = 0) {
      if (ahead.n == 0 && (!next_window(true, ahead) || ahead.n == 0)) break;
      w = ahead;
      ahead.n = 0;
      if (values && w.first) run = copy_queries(w);
      const bool ok = w.need && w.entry >= 0 && w.entry < c.num_pages;
      if (w.need && !ok && !values) atomicOr(a.status + w.request, ASV_REQ_BAD_PAGE);
      const int page = ok ? w.entry : c.num_pages;
      for (int i = 0; i < w.n && run; ++i) {
        if (i == late) next_window(false, ahead);
        run = copy_tile(w.head, i, page, w.slot);
      }
    }
    if (lane == 0) {
      ms.copied[values] = ring_kv;
      if (values) ms.queries = ring_q;
    }
  } else if (warp == kMmaWarp || warp > kWalkWarp) {
    // ---- matrices
    Ring ring_p, ring_k, ring_v, ring_q;  // a tile's keys and values take two slots of the ring, one after the other
    ring_v.next(kRing);
    const uint32_t id_qk = instr_desc(BF16, false, kTile);
    const uint32_t id_pv = instr_desc(BF16, true, (c.head_dim + 15) / 16 * 16);
    const int k_steps = (c.head_dim + 15) / 16;

    // An instruction runs 64 cycles and blocks its issue until there is room, so its operands must be there
    // by then: descriptors are those of the first tiles plus constants (in 16-byte units), unrolled, in a
    // branch of one elected lane (formed by a lane picked by its number, from vector registers, an
    // instruction took about 130 cycles).
    const uint64_t q_desc = smem_desc(q_tiles, 16, 1024), k_desc = smem_desc(ring, 16, 1024);
    const uint64_t v_desc = smem_desc(ring, kHalfBytes, 1024);
    // S (buffer sb) of the queries of Q tile q and the keys at `slot`
    auto qk = [&](int sb, int q, int slot) {
      const uint64_t qd = q_desc + q * (kTileBytes / 16), kd = k_desc + slot * (kTileBytes / 16);
      auto step = [&](int i) {
        const uint32_t off = ((i / 4) * kHalfBytes + (i % 4) * 32) / 16;
        mma_ss(tmem + sb * 128, qd + off, kd + off, id_qk, i > 0);
      };
      if (k_steps == DP / 16) {
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) step(i);
      } else {
#pragma unroll 1
        for (int i = 0; i < k_steps; ++i) step(i);
      }
    };
    // out (buffer ob) += P V over N of the tile's 16-position steps from i0, or over those of [i0, i1)
    auto pv_run = [&](int ob, int sb, int slot, int i0, bool first, auto n) {
      const uint64_t vd = v_desc + slot * (kTileBytes / 16) + i0 * (2048 / 16);
#pragma unroll
      for (int i = 0; i < decltype(n)::value; ++i)
        mma_ts(tmem + 256 + ob * 128, tmem + sb * 128 + (i0 + i) * 8, vd + i * (2048 / 16), id_pv, i > 0 || !first);
    };
    auto pv_steps = [&](int ob, int sb, int slot, bool first, int i0, int i1) {
      const uint64_t vd = v_desc + slot * (kTileBytes / 16);
#pragma unroll 1
      for (int i = i0; i < i1; ++i)
        mma_ts(tmem + 256 + ob * 128, tmem + sb * 128 + i * 8, vd + i * (2048 / 16), id_pv, !(first && i == i0));
    };
    // A tile's values: there, and safe to multiply by weights of zero.
    struct Span {
      int base, pos0, lo, hi;  // the tile's first position; the item's first token's, and the bounds of its rows'
      __device__ bool whole() const { return lo <= base && base + kTile <= hi; }
      __device__ int first_step() const { return max(lo - base, 0) / 16; }
      __device__ int end_step() const { return (min(hi - base, kTile) + 15) / 16; }
    };
    auto take_values = [&](const Ring& value, const Span& g, int poison0, int poison1) {
      if (!warp_wait(at(ms.kv_full, value.slot), value.phase, abort)) return false;
      const int last_lo = a.window > 0 ? max(0, g.hi - a.window) : 0;
      if (g.base + kTile > g.pos0 + 1 || g.base < last_lo) {
        if (clean_values<BF16, DP>(ring + value.slot * kTileBytes, g.base, g.lo, g.hi, g.pos0 + 1, last_lo, lane)) {
          if (lane >= poison0 && lane <= poison1) *reinterpret_cast<volatile int*>(&ms.poison[lane]) = 1;
          __threadfence_block();
          __syncwarp();
        }
      }
      return true;
    };
    auto next_piece = [&](Piece& p) {
      if (!warp_wait(at(ms.piece_full, ring_p.slot), ring_p.phase, abort)) return false;
      p = ms.piece[ring_p.slot];
      __syncwarp();
      if (lane == 0) bar_arrive(at(ms.piece_empty, ring_p.slot));
      ring_p.next(kQueue);
      return true;
    };

    if constexpr (NT == 2) {
      // Piece by piece; the two row tiles in turn, each tile's product and then its next S, which goes where the
      // weights were.
      uint32_t p_phase[2] = {0, 0}, o_phase[2] = {1, 1};
      Piece p;
      for (bool ok = true; ok && next_piece(p) && p.kind == 0;) {
        if (p.t0 == p.t1) continue;
        const int tiles = p.ntok <= a.tile_tokens ? 1 : 2;
        Span g = {p.t0 * kTile, p.pos0, p.kv_lo, p.pos0 + p.ntok};
        ok = warp_wait(at(ms.kv_full, ring_k.slot), ring_k.phase, abort) && warp_wait(at(ms.q_full, 0), ring_q.phase, abort);
        if (!ok) break;
        fence_after();
        if (elect()) {
          for (int x = 0; x < tiles; ++x) {
            qk(x, x, ring_k.slot);
            commit(at(ms.s_full, x));
          }
          commit(at(ms.kv_empty, ring_k.slot));
          if (p.t0 + 1 == p.t1) commit(at(ms.q_empty, 0));
        }
        __syncwarp();
        ring_k.next(kRing, 2);
        for (int x = 0; x < tiles && ok; ++x) {  // the output buffers (and their poison marks) are free
          ok = warp_wait(at(ms.o_empty, x), o_phase[x], abort);
          o_phase[x] ^= 1;
        }
        // What a tile's instructions need is waited for behind the ones before (a wait that is over takes about a
        // hundred cycles, the pipe holds three instructions): the values after the first row tile's, the keys after
        // the last's.
        auto keys_there = [&]() { return warp_wait(at(ms.kv_full, ring_k.slot), ring_k.phase, abort); };
        ok = ok && take_values(ring_v, g, 0, tiles - 1) && (p.t0 + 1 == p.t1 || keys_there());
        Ring next_v = ring_v;
        Span next_g = g;
        for (int left = p.t1 - p.t0, first = 1; left > 0 && ok; --left, first = 0) {
          const bool more = left > 1, whole = g.whole();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x == tiles || !ok) break;
            ok = warp_wait(at(ms.p_full, 2 * x + 1), p_phase[x], abort);
            p_phase[x] ^= 1;
            if (!ok) break;
            fence_after();
            if (elect()) {
              if (whole) pv_run(x, x, ring_v.slot, 0, first, std::integral_constant<int, kTile / 16>());
              else pv_steps(x, x, ring_v.slot, first, g.first_step(), g.end_step());
              if (more) {
                qk(x, x, ring_k.slot);
                commit(at(ms.s_full, x));
              } else {
                commit(at(ms.o_full, x));
              }
              if (x == tiles - 1) {
                commit(at(ms.kv_empty, ring_v.slot));
                if (more) commit(at(ms.kv_empty, ring_k.slot));
                if (left == 2) commit(at(ms.q_empty, 0));
              }
            }
            __syncwarp();
            if (x == 0) {
              next_v = ring_v;
              next_v.next(kRing, 2);
              next_g = g;
              next_g.base += kTile;
              if (more) ok = take_values(next_v, next_g, 0, tiles - 1);
            }
          }
          ring_v = next_v;
          g = next_g;
          if (more) ring_k.next(kRing, 2);
          if (ok && left > 2) ok = keys_there();
        }
        ring_q.next(1);
      }
    } else {
      // One warp forms S of every tile, the other its product: a tile costs a warp three waits and as many signals
      // next to its instructions (one warp in turn for both: 2100 cycles a tile, of which instructions run 1024).
      Piece p;
      uint32_t tiles = 0, pieces = 0;
      if (warp == kMmaWarp) {
        for (bool ok = true; ok && next_piece(p) && p.kind == 0;) {
          for (int t = p.t0; t < p.t1; ++t) {
            const int sb = tiles & 1;
            ok = warp_wait(at(ms.kv_full, ring_k.slot), ring_k.phase, abort) &&
                 (t > p.t0 || warp_wait(at(ms.q_full, ring_q.slot), ring_q.phase, abort)) &&
                 warp_wait(at(ms.pv_done, sb), ((tiles >> 1) & 1) ^ 1, abort);  // the weights there before are used
            if (!ok) break;
            fence_after();
            if (elect()) {
              qk(sb, ring_q.slot, ring_k.slot);
              commit(at(ms.s_full, sb));
              commit(at(ms.kv_empty, ring_k.slot));
              if (t == p.t1 - 1) commit(at(ms.q_empty, ring_q.slot));
            }
            __syncwarp();
            ++tiles;
            ring_k.next(kRing, 2);
          }
          if (p.t0 < p.t1) ring_q.next(2);
        }
      } else {
        for (bool ok = true; ok && next_piece(p) && p.kind == 0;) {
          const int ob = pieces & 1;
          // the output buffer (and its poison mark) is free
          if (p.t0 < p.t1) {
            ok = warp_wait(at(ms.o_empty, ob), ((pieces >> 1) & 1) ^ 1, abort);
            ++pieces;
          }
          for (int t = p.t0; t < p.t1 && ok; ++t) {
            const int sb = tiles & 1;
            const bool first = t == p.t0;
            const Span g = {t * kTile, p.pos0, p.kv_lo, p.pos0 + p.ntok};
            constexpr int kFirst = DIV ? 0 : 4;  // steps taken with the first half of the weights
            const bool whole = g.whole();
            ok = take_values(ring_v, g, ob, ob);
            if constexpr (!DIV) {
              ok = ok && warp_wait(at(ms.p_full, 2 * sb), (tiles >> 1) & 1, abort);
              if (!ok) break;
              fence_after();
              if (whole && elect()) pv_run(ob, sb, ring_v.slot, 0, first, std::integral_constant<int, kFirst>());
              __syncwarp();
            }
            ok = ok && warp_wait(at(ms.p_full, 2 * sb + 1), (tiles >> 1) & 1, abort);
            if (!ok) break;
            fence_after();
            if (elect()) {
              if (whole) pv_run(ob, sb, ring_v.slot, kFirst, DIV && first, std::integral_constant<int, 8 - kFirst>());
              else pv_steps(ob, sb, ring_v.slot, first, g.first_step(), g.end_step());
              commit(at(ms.pv_done, sb));
              commit(at(ms.kv_empty, ring_v.slot));
              if (t == p.t1 - 1) commit(at(ms.o_full, ob));
            }
            __syncwarp();
            ++tiles;
            ring_v.next(kRing, 2);
          }
        }
      }
    }
  } else {
    // ---- softmax: thread = row
    const int wg = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t lanes = uint32_t((warp % 4) * 32) << 16;
    const int part32 = DIV ? warp % 4 : 0;  // the warp's 32 positions of a tile, where it is divided by positions
    const int tok = (DIV ? lane : row) / a.group, g = (DIV ? lane : row) - tok * a.group;
    const bool stores = part32 == 0;  // the warp has outputs in its rows
    const float scale2 = a.scale * kLog2e;
    Ring ring_p;
    uint32_t used = 0, pieces = 0, sync_phase = 0;
    bool run = true;
    // the four warps of this row tile meet (bounded, like every wait)
    auto wg_sync = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(at(ms.wg_sync, wg));
      const bool ok = warp_wait(at(ms.wg_sync, wg), sync_phase, abort);
      sync_phase ^= 1;
      return ok;
    };
    while (run) {
      if (!warp_wait(at(ms.piece_full, ring_p.slot), ring_p.phase, abort)) break;
      const Piece p = ms.piece[ring_p.slot];
      __syncwarp();
      if (lane == 0) bar_arrive(at(ms.piece_empty, ring_p.slot));
      ring_p.next(kQueue);
      if (p.kind == 1) break;
      const int first_tok = wg * a.tile_tokens;
      const int ntok = min(a.tile_tokens, p.ntok - first_tok);
      if (NT == 2 && ntok <= 0) continue;
      const bool valid = tok < ntok;
      const int pos = p.pos0 + first_tok + tok;
      const int hi = valid ? pos + 1 : 0, lo = valid && a.window > 0 ? max(0, pos - a.window + 1) : 0;
      const bool any = __any_sync(0xffffffffu, valid);
      // positions that every valid row of the warp attends to
      int all_hi = valid ? hi : 0x7fffffff, all_lo = lo;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
      }
      const int ob = NT == 1 ? int(pieces & 1) : wg;
      const uint32_t o_addr = tmem + 256 + ob * 128 + lanes;
      float ref = -INFINITY, sum = 0.0f;
      // the outputs so far, once the previous product is in them
      auto rescale = [&](float keep) {
        __syncwarp();
        if (NT == 1) {
          const uint32_t w = used - 1;
          if (!warp_wait(at(ms.pv_done, int(w & 1)), (w >> 1) & 1, abort)) return false;
          fence_after();
        }
#pragma unroll 1
        for (int i = 0; i < DP / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(o_addr + i * 32, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
          tmem_st32(o_addr + i * 32, o);
        }
        return true;
      };
      for (int t = p.t0; t < p.t1; ++t) {
        const int sb = NT == 1 ? int(used & 1) : wg;
        const uint32_t s_addr = tmem + sb * 128 + lanes;
        if (!warp_wait(at(ms.s_full, sb), NT == 1 ? (used >> 1) & 1 : used & 1, abort)) {
          run = false;
          break;
        }
        if constexpr (DIV) {
          fence_after();
          __syncwarp();
          const int base = t * kTile + part32 * 32, buf = used & 1;
          uint32_t s[32];
          tmem_ld32(s_addr + part32 * 32, s);
          tmem_wait_ld(s);
          fence_before();
          if (base + 32 > all_hi || base < all_lo) {
            const int b0 = lo - base, b1 = hi - base;
            const uint32_t from = b0 <= 0 ? ~0u : b0 >= 32 ? 0u : ~0u << b0;
            const uint32_t keep = b1 >= 32 ? from : b1 <= 0 ? 0u : from & ((1u << b1) - 1);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((keep >> j) & 1u)) s[j] = 0xff800000u;
          }
          float m[4] = {__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[30]), __uint_as_float(s[31])};
#pragma unroll
          for (int j = 2; j < 30; j += 2) m[(j / 2) & 3] = max3(m[(j / 2) & 3], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          const float top = valid ? fmaxf(max3(m[0], m[1], m[2]), m[3]) * scale2 : -INFINITY;
          // The weights by the reference so far, which holds for most tiles; should a row have passed it (and for a
          // piece's first tile), once more by the reference that the warps' maxima give.
          const uint32_t mine = exchange + (buf * 4 + part32) * kChunkBytes + lane * 16;
          float2 part = make_float2(0.0f, 0.0f);
#pragma unroll 1
          for (int pass = t == p.t0 ? 1 : 0; pass < 2; ++pass) {
            if (pass == 1) {
              dv.top[buf][part32][lane] = top;
              if (!wg_sync()) {
                run = false;
                break;
              }
              const float all = fmaxf(max3(dv.top[buf][0][lane], dv.top[buf][1][lane], dv.top[buf][2][lane]), dv.top[buf][3][lane]);
              const bool move = all > ref + kLazy;
              const float keep = move ? ex2_approx(ref - all) : 1.0f;
              if (move) {
                ref = all;
                sum *= keep;
              }
              if (t > p.t0 && stores && !rescale(keep)) {
                run = false;
                break;
              }
            }
            const float shift = ref == -INFINITY ? 0.0f : kLift<BF16> - ref;
            const float2 sc = make_float2(scale2, scale2), sh = make_float2(shift, shift);
            part = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 x = ffma2(make_float2(__uint_as_float(s[8 * v + 2 * j]), __uint_as_float(s[8 * v + 2 * j + 1])), sc, sh);
                x.x = ex2_approx(x.x);
                x.y = ex2_approx(x.y);
                part = fadd2(part, x);
                w[j] = pack2<BF16>(x.x, x.y);
              }
              sts16(mine + v * 512, make_uint4(w[0], w[1], w[2], w[3]));
            }
            const bool passed = __any_sync(0xffffffffu, top > ref + kLazy);
            if (lane == 0) dv.vote[buf][part32] = passed;
            if (!wg_sync()) {
              run = false;
              break;
            }
            if (pass == 0 && (dv.vote[buf][0] | dv.vote[buf][1] | dv.vote[buf][2] | dv.vote[buf][3]) == 0) break;
          }
          if (!run) break;
          sum += part.x + part.y;
          if (stores) {
            // all of the rows' weights, from the four warps
            const uint32_t theirs = exchange + buf * 4 * kChunkBytes + lane * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t w[32];
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                const uint4 x = lds16(theirs + (half * 8 + v) * 512);
                w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
              }
              tmem_st32(s_addr + half * 32, w);
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(at(ms.p_full, 2 * sb + 1));
          }
        } else if (any) {
          fence_after();
          __syncwarp();
          const int base = t * kTile;
          const bool masked = base + kTile > all_hi || base < all_lo;
          const int h = hi - base, l = lo - base;
          // Both passes over the row read S from tensor memory, 64 columns at a time: reading it twice costs
          // less than holding 128 registers of it, and the loops are kept rolled and the masks short because the
          // warps' roles together are about as much code as the instruction cache holds.
          auto load_s = [&](int half, uint32_t (&s)[64]) {
            tmem_ld32(s_addr + half * 64, reinterpret_cast<uint32_t(&)[32]>(s[0]));
            tmem_ld32(s_addr + half * 64 + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
            tmem_wait_ld(s);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int b0 = l - half * 64 - i * 32, b1 = h - half * 64 - i * 32;  // columns [b0, b1) stay
                const uint32_t from = b0 <= 0 ? ~0u : b0 >= 32 ? 0u : ~0u << b0;
                const uint32_t keep = b1 >= 32 ? from : b1 <= 0 ? 0u : from & ((1u << b1) - 1);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((keep >> j) & 1u)) s[i * 32 + j] = 0xff800000u;
              }
            }
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t s[64];
            load_s(half, s);
            float m[4] = {top, __uint_as_float(s[61]), __uint_as_float(s[62]), __uint_as_float(s[63])};
#pragma unroll
            for (int j = 0; j < 60; j += 2)
              m[(j / 2) & 3] = max3(m[(j / 2) & 3], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            top = fmaxf(max3(m[0], m[1], __uint_as_float(s[60])), fmaxf(m[2], m[3]));
          }
          top *= scale2;
          const bool move = top > ref + kLazy;
          if (__any_sync(0xffffffffu, move)) {
            const float keep = move ? ex2_approx(ref - top) : 1.0f;
            if (move) {
              ref = top;
              sum *= keep;
            }
            if (t > p.t0 && !rescale(keep)) {
              run = false;
              break;
            }
          }
          __syncwarp();
          const float shift = ref == -INFINITY ? 0.0f : kLift<BF16> - ref;
          const float2 sc = make_float2(scale2, scale2), sh = make_float2(shift, shift);
          float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t s[64], w[32];
            load_s(half, s);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float2 x = ffma2(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), sc, sh);
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              part[j & 1] = fadd2(part[j & 1], x);
              w[j] = pack2<BF16>(x.x, x.y);
            }
            tmem_st32(s_addr + half * 32, w);
            if (NT == 1 || half == 1) {
              tmem_wait_st();
              fence_before();
              __syncwarp();
              if (lane == 0) bar_arrive(at(ms.p_full, 2 * sb + half));
            }
          }
          const float2 both = fadd2(part[0], part[1]);
          sum += both.x + both.y;
        } else if (lane == 0) {
          if (NT == 1) bar_arrive(at(ms.p_full, 2 * sb));
          bar_arrive(at(ms.p_full, 2 * sb + 1));
        }
        ++used;
      }
      if (!run) break;

      if constexpr (DIV) {
        if (p.t1 > p.t0) {
          dv.sum[part32][lane] = sum;
          if (!wg_sync()) break;
          sum = dv.sum[0][lane] + dv.sum[1][lane] + (dv.sum[2][lane] + dv.sum[3][lane]);
        }
      }

      // ---- epilogue
      int first_cta = 0, n_parts = 1;  // the CTAs that have parts of the item
      if (p.part >= 0) {
        const long long units = ms.units;
        first_cta = int(quotient((p.item + 1) * gridDim.x - 1, units));
        n_parts = int(quotient((p.item + p.item_tiles) * gridDim.x - 1, units)) - first_cta + 1;
      }
      const int n_rows = ntok * a.group;
      const int tok_row = p.tok0 + first_tok + tok;
      const int head = p.head * a.group + g;
      if (p.t1 > p.t0) {
        if (!warp_wait(at(ms.o_full, ob), NT == 1 ? (pieces >> 1) & 1 : pieces & 1, abort)) break;
        fence_after();
      }
      // values that are not finite and that not all rows attend to: this row's own
      const bool poison = p.t1 > p.t0 && *reinterpret_cast<volatile int*>(&ms.poison[ob]) != 0;
      auto poisoned = [&](auto& y, int d0) {
        constexpr int kN = sizeof(y) / sizeof(float);
        float z[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) z[j] = y[j];
        const int hi_all = p.pos0 + p.ntok;
        if (valid)
          add_poison<BF16, kN>(c, p.request, p.head, max(lo, p.t0 * kTile), min(hi, p.t1 * kTile),
                               a.window > 0 ? max(0, hi_all - a.window) : 0, p.pos0 + 1, d0, z);
#pragma unroll
        for (int j = 0; j < kN; ++j) y[j] = z[j];
        __syncwarp();
      };
      const size_t part_floats = size_t(kTile) * DP + 2 * kTile;
      if (p.part < 0) {
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        const bool store = valid && stores && ASV_GUARD(a, tok_row >= 0 && tok_row < c.N && head < a.q_heads);
        uint16_t* out = a.out.p + tok_row * a.out.tok + head * a.out.head;
        if (any && stores) {
          constexpr int kCols = NT == 1 ? 32 : 64;
#pragma unroll 1
          for (int i = 0; i < DP; i += kCols) {
            __syncwarp();
            float y[kCols];
            if (p.t1 > p.t0) {
              uint32_t o[kCols];
#pragma unroll
              for (int j = 0; j < kCols; j += 32) tmem_ld32(o_addr + i + j, reinterpret_cast<uint32_t(&)[32]>(o[j]));
              tmem_wait_ld(o);
#pragma unroll
              for (int j = 0; j < kCols; ++j) y[j] = __uint_as_float(o[j]) * inv;
            } else {
#pragma unroll
              for (int j = 0; j < kCols; ++j) y[j] = 0.0f;
            }
            if (poison) poisoned(y, i);
            uint32_t v[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) v[j] = pack2<BF16>(y[2 * j], y[2 * j + 1]);
            if constexpr (NT == 1) {
#pragma unroll
              for (int j = 0; j < kCols / 8; ++j)
                if (store && i + j * 8 < c.head_dim)
                  *reinterpret_cast<uint4*>(out + i + j * 8) =
                      make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
              // full tiles: a lane's own row to 16 bytes of 32 lines a store took 512 cycles of the L1 each
              transpose8(v, lane);
              const int d = i + (lane & 7) * 8;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const unsigned long long to = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), (lane & ~7) + j);
                const bool ok = __shfl_sync(0xffffffffu, int(store), (lane & ~7) + j) != 0;
                if (ok && d < c.head_dim)
                  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(to) + d) =
                      make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
              }
            }
          }
          if (store && a.lse != nullptr)
            a.lse[(long long)tok_row * a.q_heads + head] = sum == 0.0f ? -INFINITY : (ref + (log2f(sum) - kLift<BF16>)) * kLn2f;
        }
      } else {
        // file the partial result: [column / 4][row] float4, then (reference, sum) per row
        float* part = a.parts + (size_t(p.part) * 2 + wg) * part_floats;
        if (any && stores) {
#pragma unroll 1
          for (int i = 0; i < DP / 32; ++i) {
            __syncwarp();
            uint32_t o[32];
            tmem_ld32(o_addr + i * 32, o);
            tmem_wait_ld(o);
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(o[j]);
            if (poison) poisoned(y, i * 32);
            if (valid && ASV_GUARD(a, p.part < kPagedSlots)) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                __stcg(reinterpret_cast<float4*>(part) + (i * 8 + j) * kTile + row,
                       make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]));
            }
          }
          if (valid && stores && ASV_GUARD(a, p.part < kPagedSlots))
            __stcg(reinterpret_cast<float2*>(part + kTile * DP) + row, make_float2(ref, sum));
        }
      }
      if (p.t1 > p.t0) {
        // the output buffer is free again
        fence_before();
        if (poison) {
          if (!wg_sync()) break;
          if (row == 0) ms.poison[ob] = 0;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(at(ms.o_empty, ob));
        ++pieces;
      }
      if (p.part < 0) continue;

      // The last to file joins the parts, in CTA order.  The warps' writes come before the ticket through the
      // barrier and the ticket's release, the other CTAs' before the reads through its acquire and the barrier.
      // (Rows of the first warp alone need no barrier.)
      if (n_rows > 32 && !wg_sync()) break;
      __syncwarp();
      if (row == 0 && ASV_GUARD(a, first_cta + n_parts <= int(gridDim.x))) {
        const uint32_t old = atom_add_acq_rel_gpu(a.tickets + 2 * first_cta + wg, 1u);
        ms.last[wg][sync_phase] = old == uint32_t(n_parts - 1);
      }
      const uint32_t which = sync_phase;
      if (!wg_sync()) break;
      if (*reinterpret_cast<volatile int*>(&ms.last[wg][which]) == 0) continue;
      if (row == 0) a.tickets[2 * first_cta + wg] = 0;
      // A thread keeps one row: `span` threads side by side have the rows, the others further columns.
      const int span = n_rows <= 1 ? 1 : 1 << (32 - __clz(n_rows - 1)), r = row & (span - 1);
      const int cols4 = c.head_dim / 4, step = kTile / span;
      if (r >= n_rows) continue;
      auto part_of = [&](int k) {
        const int slot = k == 0 ? 2 * first_cta + 1 : 2 * (first_cta + k);
        return a.parts + (size_t(slot) * 2 + wg) * part_floats;
      };
      auto stats_of = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(part_of(k) + kTile * DP) + r); };
      const int tk = r / a.group, hd = p.head * a.group + (r - tk * a.group);
      const int dst = p.tok0 + first_tok + tk;
      if (!ASV_GUARD(a, dst >= 0 && dst < c.N && hd < a.q_heads)) continue;
      uint16_t* out = a.out.p + dst * a.out.tok + hd * a.out.head;
      const int col0 = row / span;
      auto put = [&](int col, float4 y) {
        *reinterpret_cast<uint2*>(out + col * 4) = make_uint2(pack2<BF16>(y.x, y.y), pack2<BF16>(y.z, y.w));
      };
      auto add = [](float4 acc, float4 o, float w) {
        return make_float4(fmaf(o.x, w, acc.x), fmaf(o.y, w, acc.y), fmaf(o.z, w, acc.z), fmaf(o.w, w, acc.w));
      };
      const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float m = -INFINITY, l = 0.0f;
      // The parts in order, `kIn` at a time with all their loads in flight.  Few rows: a thread has one vector of
      // four columns and everything of a part at once.  Many: the rows' sums first, then eight vectors a time.
      constexpr int kIn = 16, kCols = 8;
      if (cols4 <= step) {
        float4 acc = zero;
        for (int k0 = 0; k0 < n_parts; k0 += kIn) {
          float2 ml[kIn];
          float4 o[kIn];
#pragma unroll
          for (int k = 0; k < kIn; ++k) {
            ml[k] = make_float2(-INFINITY, 0.0f);
            o[k] = zero;
            if (k0 + k < n_parts && col0 < cols4) {
              ml[k] = stats_of(k0 + k);
              o[k] = __ldcg(reinterpret_cast<const float4*>(part_of(k0 + k)) + col0 * kTile + r);
            }
          }
          float top = m;
#pragma unroll
          for (int k = 0; k < kIn; ++k) top = fmaxf(top, ml[k].x);
          const float base = top == -INFINITY ? 0.0f : top, keep = ex2_approx(m - base);
          m = top;
          l *= keep;
          acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
          for (int k = 0; k < kIn; ++k) {
            const float w = ex2_approx(ml[k].x - base);
            l = fmaf(ml[k].y, w, l);
            acc = add(acc, o[k], w);
          }
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (col0 < cols4) put(col0, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      } else {
#pragma unroll 8
        for (int k = 0; k < n_parts; ++k) {
          const float2 ml = stats_of(k);
          const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.0f : top;
          l = l * ex2_approx(m - base) + ml.y * ex2_approx(ml.x - base);
          m = top;
        }
        const float base = m == -INFINITY ? 0.0f : m, inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        for (int c0 = col0 * kCols; c0 < cols4; c0 += kCols * step) {
          float4 acc[kCols];
#pragma unroll
          for (int i = 0; i < kCols; ++i) acc[i] = zero;
          for (int k = 0; k < n_parts; k += 2) {
            float4 o[2][kCols];
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (what is past the last is read again and left out)
              const int at = min(k + e, n_parts - 1);
              const float4* part = reinterpret_cast<const float4*>(part_of(at)) + r;
              w[e] = stats_of(at).x;
#pragma unroll
              for (int i = 0; i < kCols; ++i) o[e][i] = ld_cg_f4(part + min(c0 + i, cols4 - 1) * kTile);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (k + e >= n_parts) break;  // (not a weight of zero: the outputs may be infinite)
              w[e] = ex2_approx(w[e] - base) * inv;
#pragma unroll
              for (int i = 0; i < kCols; ++i) acc[i] = add(acc[i], o[e][i], w[e]);
            }
          }
#pragma unroll
          for (int i = 0; i < kCols; i += 2)
            if (c0 + i < cols4)
              *reinterpret_cast<uint4*>(out + (c0 + i) * 4) =
                  make_uint4(pack2<BF16>(acc[i].x, acc[i].y), pack2<BF16>(acc[i].z, acc[i].w),
                             pack2<BF16>(acc[i + 1].x, acc[i + 1].y), pack2<BF16>(acc[i + 1].z, acc[i + 1].w));
        }
      }
      if (row < span && a.lse != nullptr)
        a.lse[(long long)dst * a.q_heads + hd] = l == 0.0f ? -INFINITY : (m + (log2f(l) - kLift<BF16>)) * kLn2f;
    }
    if (*abort && lane == 0) {
      for (int b = 0; b < c.B; ++b) atomicOr(a.status + b, ASV_REQ_TIMEOUT);
    }
  }
  fence_before();
  __syncthreads();
  if (*abort) {
    // A wait ran out.  Nothing waits any more, so all warps see it: leave with no copy, matrix instruction or store to
    // tensor memory in flight (each waited for, a while).
    if (warp == kCopyWarp || warp == kCopyWarp + 1) {
      // Its last tiles: before it copied them, the ones before were used.
      Ring r = ms.copied[warp - kCopyWarp];
      for (int i = 0; i < (kRing + 1) / 2; ++i) {
        r.back(kRing, 2);
        wait_a_while(at(ms.kv_full, r.slot), r.phase);
      }
      r = ms.queries;
      for (int i = 0; warp != kCopyWarp && i < 3 - NT; ++i) {
        r.back(3 - NT);
        wait_a_while(at(ms.q_full, r.slot), r.phase);
      }
    } else if (warp == kMmaWarp || warp > kWalkWarp) {
      const int which = warp == kMmaWarp ? 0 : 1;
      if (elect()) commit(at(ms.drained, which));
      __syncwarp();
      wait_a_while(at(ms.drained, which), 0);
    } else if (warp != kWalkWarp) {
      tmem_wait_st();
    }
    fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) tmem_free(tmem, kTmemColumns);
}

// ------------------------------------------------------------------ launch

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A map of `rank` dimensions of 16-bit elements, the first contiguous; strides in elements (0: the
// dimension has extent 1, any stride will do).
cudaError_t make_map(CUtensorMap* m, bool bf16, void* base, int rank, const cuuint64_t* dims, const long long* strides,
                     const cuuint32_t* box) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t bytes[4];
  cuuint32_t unit[5] = {1, 1, 1, 1, 1};
  // What L2 fetches at a time: 256 bytes where they are one row of a head, else they would bring in the next head's
  // (151 requests of one token, 2 key heads of 64: 118 us with 256, 87 with 128; 64 x 3 tokens, heads of 128: 148, 150).
  const CUtensorMapL2promotion fetch = dims[0] == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] > 0 ? cuuint64_t(strides[i]) * 2 : 256;
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, base, dims,
                        bytes, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool BF16, int DP, int NT, bool DIV>
cudaError_t launch(const AttendArgs& a, const CUtensorMap* maps, int grid, int dev, cudaStream_t s) {
  auto kernel = paged_attention_kernel<BF16, DP, NT, DIV>;
  constexpr int kSmem = 1024 + (2 + kRingSlots<DP, NT>) * kTile * DP * 2 + int(kExchangeBytes<DIV>) +
                        int(sizeof(Misc) + (DIV ? sizeof(Divided) : 0));
  static_assert(kSmem <= 232448, "shared memory");
  // a programmatic launch: the set-up runs while the launch before it ends
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(kThreadsOf<NT>, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // the limit is raised once per device, and again should a launch fail (a device reset forgets it)
  static std::atomic<uint64_t> raised{0};
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (raised.load(std::memory_order_relaxed) & bit) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, maps[0], maps[1], maps[2]);
    if (e != cudaErrorInvalidValue) return e;
    cudaGetLastError();
  }
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  raised.fetch_or(bit, std::memory_order_relaxed);
  return cudaLaunchKernelEx(&cfg, kernel, a, maps[0], maps[1], maps[2]);
}

}  // namespace

cudaError_t launch_paged_attention(const AttendArgs& args, int dtype, cudaStream_t s) {
  AttendArgs a = args;
  const PagedView& c = a.c;
  const bool bf16 = dtype == ASV_BF16;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  // Two row tiles to an item where the average chunk has more rows than one tile holds; a divided one where (as far as
  // the host can tell: the same number of tokens to each request, if they are alike) every chunk has at most 32 rows.
  // With four ring tiles undivided / divided: 256 requests, one token 102.6 / 100.6 us; 64 x 3 tokens, 24 rows, 151.5 /
  // 150.3; one request, one token 10.72 / 10.64.  A longer chunk among them is right, in more items.
  const bool two = (long long)c.N * a.group > (long long)kTile * c.B;
  const bool div = c.N % c.B == 0 && (long long)c.N * a.group <= 32ll * c.B;
  a.tile_tokens = (div ? 32 : kTile) / a.group;
  a.box = std::min(kTile, c.page_size & -c.page_size);
  CUtensorMap maps[3];
  const cuuint64_t qd[3] = {cuuint64_t(c.head_dim), cuuint64_t(a.q_heads), cuuint64_t(c.N)};
  const long long qs[2] = {a.q.head, a.q.tok};
  const cuuint32_t qb[3] = {64, cuuint32_t(a.group), cuuint32_t(a.tile_tokens)};
  const cuuint64_t kd[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.kv_heads), cuuint64_t(c.page_size),
                            cuuint64_t(c.num_pages)};
  const long long ks[3] = {c.k_head, c.k_slot, c.k_page}, vs[3] = {c.v_head, c.v_slot, c.v_page};
  const cuuint32_t kb[4] = {64, 1, cuuint32_t(a.box), 1};
  if ((e = make_map(&maps[0], bf16, a.q.p, 3, qd, qs, qb)) != cudaSuccess) return e;
  if ((e = make_map(&maps[1], bf16, c.k, 4, kd, ks, kb)) != cudaSuccess) return e;
  if ((e = make_map(&maps[2], bf16, c.v, 4, kd, vs, kb)) != cudaSuccess) return e;
  const int grid = std::min(sms, kPagedMaxGrid);
  const int which = (bf16 ? 6 : 0) + (c.head_dim > 64 ? 3 : 0) + (two ? 1 : div ? 2 : 0);
  switch (which) {
    case 0: return launch<false, 64, 1, false>(a, maps, grid, dev, s);
    case 1: return launch<false, 64, 2, false>(a, maps, grid, dev, s);
    case 2: return launch<false, 64, 1, true>(a, maps, grid, dev, s);
    case 3: return launch<false, 128, 1, false>(a, maps, grid, dev, s);
    case 4: return launch<false, 128, 2, false>(a, maps, grid, dev, s);
    case 5: return launch<false, 128, 1, true>(a, maps, grid, dev, s);
    case 6: return launch<true, 64, 1, false>(a, maps, grid, dev, s);
    case 7: return launch<true, 64, 2, false>(a, maps, grid, dev, s);
    case 8: return launch<true, 64, 1, true>(a, maps, grid, dev, s);
    case 9: return launch<true, 128, 1, false>(a, maps, grid, dev, s);
    case 10: return launch<true, 128, 2, false>(a, maps, grid, dev, s);
    default: return launch<true, 128, 1, true>(a, maps, grid, dev, s);
  }
}

}  // namespace asv
