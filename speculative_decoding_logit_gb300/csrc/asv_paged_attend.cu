// asv_paged_attend.cu -- paged_attention: attention of a chunk of new tokens over a paged cache.
//
//   s_ij = scale * (q_i . k_j),  out_i = sum_j 2^((s_ij - m_i) log2 e) v_j / sum_j 2^((s_ij - m_i) log2 e)
//
// over the positions j that token i attends to (causal, window), with a running reference m_i.
//
// Rows.  The query heads of a key head read the same keys, so a row tile of 128 rows holds
// floor(128 / G) tokens x G heads, and an item is (request, NT row tiles, key head): NT = 1 where a
// request's chunk fits one tile, NT = 2 for longer chunks (each key and value tile then serves 256 rows,
// which halves what a CTA reads from L2 per multiplication).
//
// Split.  An item costs as many units as it has key tiles of 128 positions.  The units of all items, in
// order, are cut into equal runs, one for each CTA (one CTA per SM), so a batch of any lengths keeps every
// SM busy to the end; the prefix sums need only indptr and cache_len and a closed form per request, and
// every CTA computes them.  An item that a cut goes through is finished from partial results (unnormalised
// outputs, reference, sum) in the workspace by the CTA that files the last of them, in CTA order, so the
// result does not depend on timing.
//
// In a CTA, warps take roles that hand over through mbarriers:
//   scheduler  walks the CTA's run and describes its pieces in a queue
//   copies     one box of the tensor map per page (part), 128-byte swizzled, into a ring of key / value
//              tiles; positions that no row of the item attends to are not read (zero fill)
//   matrices   S = Q K^T into tensor memory; out += P V with P taken from tensor memory
//   softmax    one thread per row: S to registers, reference, 2^x, P back over S in the 16-bit type; the
//              outputs are rescaled only when the reference moves by more than 2^8, so seldom after the
//              first tiles; the epilogue divides and stores
// NT = 1 keeps two S and two output buffers, so the next tile's S is formed while the softmax runs; NT = 2
// gives each row tile one, and the two tiles alternate.
#include <algorithm>

#include "asv_paged_device.cuh"
#include "asv_tcgen05.cuh"

namespace asv {

namespace {

using namespace tc;

constexpr int kTile = 128;  // rows of a row tile; positions of a key tile
constexpr int kQueue = 4;
constexpr uint32_t kTmemColumns = 512;  // S buffers at 0 and 128, outputs at 256 and 384
constexpr float kLazy = 8.0f;           // log2 units the maximum may pass the reference by

template <int DP>
constexpr int kRingSlots = DP == 128 ? 5 : 10;

// A run of key tiles of one item.
struct Piece {
  int request;
  int tok0, ntok;  // first row of the item's tokens and their number
  int head;        // key head
  int pos0;        // position of the first token
  int kv_lo;       // first position that any of the tokens attends to
  int t0, t1;      // key tiles [t0, t1); none: a request left out, whose outputs are zero
  int part;        // -1: the whole item; else the slot of its partial result
  int first_cta, n_parts;
  int kind;        // 0: a piece; 1: the end of the run
};

struct Misc {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], o_full[2], o_empty[2];
  uint64_t piece_full[kQueue], piece_empty[kQueue], wg_sync[2];
  Piece piece[kQueue];
  long long warp_sum[12];
  long long start_units;  // units before the run's first request
  int start_request;
  uint32_t tmem;
  int abort;
  int poison[2];  // a value that some rows of the item in this output buffer do not attend to is not finite
  int last[2];
};

// sum_{i < n} floor((a i + b) / m) for a, b >= 0: each round takes out the whole parts of a / m and b / m
// and counts the lattice points left under the line with the axes exchanged.
__device__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  for (;;) {
    if (a >= m) {
      sum += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const long long top = a * n + b;
    if (top < m) return sum;
    n = top / m;
    b = top % m;
    const long long t = m;
    m = a;
    a = t;
  }
}

// A request's items of one key head: n of them, item r with the tokens from r * T.
struct Items {
  Request r;
  int T, n;
  __device__ int lo(int window, int i) const { return window > 0 ? max(0, r.past + i * T - window + 1) : 0; }
  // key tiles (1 for a request that is left out)
  __device__ int tiles(int window, int i) const {
    if (!r.ok) return 1;
    const int hi = r.past + min((i + 1) * T, r.end - r.start);
    return (hi + kTile - 1) / kTile - lo(window, i) / kTile;
  }
  // key tiles of the items before i (i < n)
  __device__ long long tiles_before(int window, int i) const {
    if (i == 0) return 0;
    if (!r.ok) return i;
    long long sum = floor_sum(i, kTile, T, (long long)r.past + T + kTile - 1);
    if (window > 0) {
      // items before z start at position 0
      const long long z = r.past >= window - 1 ? 0 : ((long long)window - 1 - r.past + T - 1) / T;
      if (i > z) sum -= floor_sum(i - z, kTile, T, r.past + z * T - window + 1);
    }
    return sum;
  }
  __device__ long long units(int window, int kv_heads) const {
    return n == 0 ? 0 : kv_heads * (tiles_before(window, n - 1) + tiles(window, n - 1));
  }
};

__device__ Items load_items(const PagedView& c, int b, int T) {
  Items it;
  it.r = load_request(c, b, table_positions(c));
  it.T = T;
  // the rows of a request that is left out are still zeroed, where they are rows
  const bool rows = it.r.start >= 0 && it.r.start <= it.r.end && it.r.end <= c.N;
  it.n = rows ? (it.r.end - it.r.start + T - 1) / T : 0;
  return it;
}

// Counters of a ring of `n` barriers: slot and phase of the i-th use.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ uint32_t at(const uint64_t* bars, int i) { return smem_addr(bars + i); }

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Any 16-bit element of the words with all exponent bits set.
template <bool BF16>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  return (w & kExp) == kExp || ((w >> 16) & kExp) == kExp;
}

template <bool BF16>
__device__ __forceinline__ uint32_t finite_or_zero2(uint32_t w) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  if ((w & kExp) == kExp) w &= 0xffff0000u;
  if (((w >> 16) & kExp) == kExp) w &= 0x0000ffffu;
  return w;
}

// Makes a tile of values (rows = positions base .. base + 127) safe to multiply by weights of zero: rows
// outside [lo, hi), which no row of the item attends to, are zeroed where a copied box reaches past the
// bounds; in the rows that only some attend to, [zone, hi) and [lo, wzone), elements that are not finite
// are zeroed and reported (the epilogue adds them to the rows that do attend to them).  By one warp.
template <bool BF16, int DP>
__device__ bool clean_values(uint32_t tile, int base, int lo, int hi, int zone, int wzone, int box, int lane) {
  constexpr int kVecs = DP / 8;
  auto addr = [&](int row, int vec) { return tile + (vec / 8) * (kTile * 128) + row * 128 + (vec % 8) * 16; };
  bool touched = false, found = false;
  auto zero = [&](int r0, int r1) {
    for (int i = r0 * kVecs + lane; i < r1 * kVecs; i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr(i / kVecs, i % kVecs)), "r"(0) : "memory");
    touched |= r1 > r0;
  };
  auto scan = [&](int r0, int r1) {
    for (int i = r0 * kVecs + lane; i < r1 * kVecs; i += 32) {
      const uint32_t p = addr(i / kVecs, i % kVecs);
      uint4 x;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(p));
      if (nonfinite2<BF16>(x.x) || nonfinite2<BF16>(x.y) || nonfinite2<BF16>(x.z) || nonfinite2<BF16>(x.w)) {
        found = true;
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(finite_or_zero2<BF16>(x.x)),
                     "r"(finite_or_zero2<BF16>(x.y)), "r"(finite_or_zero2<BF16>(x.z)), "r"(finite_or_zero2<BF16>(x.w))
                     : "memory");
      }
    }
  };
  const int first = max(lo - base, 0), end = min(hi - base, kTile);
  zero(first / box * box, first);
  zero(end, min(kTile, (end + box - 1) / box * box));
  const int w1 = min(wzone - base, end);
  scan(first, w1);
  scan(max(max(zone - base, first), w1), end);
  found = __any_sync(0xffffffffu, found);
  if (found || touched) {
    fence_async_shared();
    __syncwarp();
  }
  return found;
}

template <bool BF16, int DP, int NT>
__global__ void __launch_bounds__(32 * (4 * NT + 3), 1)
    paged_attention_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr int kThreads = 32 * (4 * NT + 3);
  constexpr int kRing = kRingSlots<DP>;
  constexpr int kHalves = DP / 64;                // 64-element column blocks, 128 bytes a row
  constexpr uint32_t kTileBytes = kTile * DP * 2;
  constexpr uint32_t kHalfBytes = kTile * 128;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t smem0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_tiles = smem0, ring = smem0 + 2 * kTileBytes;
  Misc& ms = *reinterpret_cast<Misc*>(smem_raw + (smem0 - smem_addr(smem_raw)) + (2 + kRing) * kTileBytes);
  const PagedView& c = a.c;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr int kMmaWarp = 4 * NT, kCopyWarp = 4 * NT + 1, kWalkWarp = 4 * NT + 2;
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
      bar_init(at(ms.p_full, i), 4);
      bar_init(at(ms.pv_done, i), 1);
      bar_init(at(ms.o_full, i), 1);
      bar_init(at(ms.o_empty, i), 4);
      bar_init(at(ms.wg_sync, i), 4);
      ms.poison[i] = 0;
    }
    for (int i = 0; i < kQueue; ++i) {
      bar_init(at(ms.piece_full, i), 1);
      bar_init(at(ms.piece_empty, i), 2 + 4 * NT);
    }
    ms.abort = 0;
    fence_barrier_init();
    prefetch_map(&map_q);
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  // units of this thread's requests, and of all
  const int per_thread = (c.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per_thread, c.B), b1 = min(b0 + per_thread, c.B);
  long long own = 0;
  for (int b = b0; b < b1; ++b) {
    const Items it = load_items(c, b, T);
    if (!it.r.ok && blockIdx.x == 0) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
    own += it.units(a.window, c.kv_heads);
  }
  long long incl = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) ms.warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - own, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += ms.warp_sum[w];
    total += ms.warp_sum[w];
  }
  const long long per_cta = max((total + gridDim.x - 1) / (long long)gridDim.x, 1ll);
  const long long u0 = blockIdx.x * per_cta, u1 = min(u0 + per_cta, total);
  if (u0 >= before && u0 < before + own) {
    long long x = before;
    for (int b = b0; b < b1; ++b) {
      const long long n = load_items(c, b, T).units(a.window, c.kv_heads);
      if (u0 < x + n) {
        ms.start_request = b;
        ms.start_units = x;
        break;
      }
      x += n;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ms.tmem;
  const bool idle = u0 >= u1;

  if (idle) {
  } else if (warp == kWalkWarp) {
    // ---- scheduler
    if (lane == 0) {
      int b = ms.start_request;
      Items it = load_items(c, b, T);
      const long long rel = u0 - ms.start_units;
      int i = 0;  // the item that holds unit u0: the last with no more than rel units before it
      for (int hi = it.n; hi - i > 1;) {
        const int mid = (i + hi) / 2;
        if (c.kv_heads * it.tiles_before(a.window, mid) <= rel) i = mid;
        else hi = mid;
      }
      int n = it.tiles(a.window, i);
      const long long off = rel - c.kv_heads * it.tiles_before(a.window, i);
      int h = int(off / n), t = int(off % n);
      Ring ring_p;
      for (long long u = u0;;) {
        if (!bar_wait(at(ms.piece_empty, ring_p.slot), ring_p.phase ^ 1, abort)) break;
        Piece& p = ms.piece[ring_p.slot];
        if (u >= u1) {
          p.kind = 1;
          bar_arrive(at(ms.piece_full, ring_p.slot));
          break;
        }
        const int take = int(min((long long)(n - t), u1 - u));
        const long long item0 = u - t;
        p.kind = 0;
        p.request = b;
        p.tok0 = it.r.start + i * T;
        p.ntok = min(T, it.r.end - p.tok0);
        p.head = h;
        p.pos0 = it.r.past + i * T;
        p.kv_lo = it.lo(a.window, i);
        const int tile0 = p.kv_lo / kTile;
        p.t0 = it.r.ok ? tile0 + t : 0;
        p.t1 = it.r.ok ? tile0 + t + take : 0;
        p.first_cta = int(item0 / per_cta);
        p.n_parts = int((item0 + n - 1) / per_cta) - p.first_cta + 1;
        p.part = p.n_parts == 1 ? -1 : 2 * int(blockIdx.x) + (item0 >= u0 ? 1 : 0);
        bar_arrive(at(ms.piece_full, ring_p.slot));
        ring_p.next(kQueue);
        u += take;
        t = 0;
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
  } else if (warp == kCopyWarp) {
    // ---- copies
    Ring ring_p, ring_kv, ring_q;
    const int boxes = kTile / a.box;
    Piece prev = {};
    int prev_tile = 0, prev_page = 0;
    bool have_prev = false, run = true;
    // this lane's box of a tile of keys (or values) into the next slot of the ring
    auto copy_tile = [&](const CUtensorMap* map, int head, int tile, int page) {
      if (!warp_wait(at(ms.kv_empty, ring_kv.slot), ring_kv.phase ^ 1, abort)) return false;
      const uint32_t bar = at(ms.kv_full, ring_kv.slot);
      if (lane == 0) bar_expect(bar, kTileBytes);
      __syncwarp();
      if (lane < boxes) {
        const int slot = (tile * kTile + lane * a.box) % c.page_size;
        const uint32_t dst = ring + ring_kv.slot * kTileBytes + lane * a.box * 128;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) copy_4d(dst + h * kHalfBytes, map, h * 64, head, slot, page, bar);
      }
      ring_kv.next(kRing);
      return true;
    };
    while (run) {
      if (!warp_wait(at(ms.piece_full, ring_p.slot), ring_p.phase, abort)) break;
      const Piece p = ms.piece[ring_p.slot];
      __syncwarp();
      if (lane == 0) bar_arrive(at(ms.piece_empty, ring_p.slot));
      ring_p.next(kQueue);
      if (p.kind == 1) break;
      const int kv_hi = p.pos0 + p.ntok;
      for (int t = p.t0; t < p.t1; ++t) {
        // this lane's page; what no row attends to is filled with zeros (a page past the last)
        int page = c.num_pages;
        const int pos = t * kTile + lane * a.box;
        if (lane < boxes && pos < kv_hi && pos + a.box > p.kv_lo) {
          const int id = c.table[p.request * c.table_stride + pos / c.page_size];
          if (id >= 0 && id < c.num_pages) page = id;
          else atomicOr(a.status + p.request, ASV_REQ_BAD_PAGE);
        }
        if (NT == 2 && have_prev) run = run && copy_tile(&map_v, prev.head, prev_tile, prev_page);
        run = run && copy_tile(&map_k, p.head, t, page);
        if (run && t == p.t0) {
          if (!warp_wait(at(ms.q_empty, ring_q.slot), ring_q.phase ^ 1, abort)) {
            run = false;
          } else if (lane == 0) {
            const int tiles = NT == 1 ? 1 : (p.ntok + a.tile_tokens - 1) / a.tile_tokens;
            const uint32_t bar = at(ms.q_full, ring_q.slot);
            bar_expect(bar, tiles * kHalves * a.tile_tokens * a.group * 128);
            for (int i = 0; i < tiles; ++i)
              for (int h = 0; h < kHalves; ++h)
                copy_3d(q_tiles + (NT == 1 ? ring_q.slot : i) * kTileBytes + h * kHalfBytes, &map_q, h * 64,
                        p.head * a.group, p.tok0 + i * a.tile_tokens, bar);
          }
          ring_q.next(3 - NT);
        }
        if (NT == 1 && have_prev) run = run && copy_tile(&map_v, prev.head, prev_tile, prev_page);
        if (!run) break;
        prev = p;
        prev_tile = t;
        prev_page = page;
        have_prev = true;
      }
    }
    if (have_prev && run) copy_tile(&map_v, prev.head, prev_tile, prev_page);
    if (*abort) {  // leave with no copy in flight: every slot of the ring once more
      for (int i = 0; i < kRing; ++i) {
        const unsigned long long t0 = now_ns();
        const uint32_t parity = i < ring_kv.slot ? ring_kv.phase : ring_kv.phase ^ 1;
        while (!bar_try(at(ms.kv_full, i), parity) && now_ns() - t0 < kWaitNs / 100) {
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- matrices
    Ring ring_p, ring_kv, ring_q;
    const uint32_t id_qk = instr_desc(BF16, false, kTile);
    const uint32_t id_pv = instr_desc(BF16, true, (c.head_dim + 15) / 16 * 16);
    const int k_steps = (c.head_dim + 15) / 16;
    int used[2] = {0, 0};   // S / P buffer uses so far
    int items[2] = {0, 0};  // output buffer uses so far
    int cur_ob = 0, next_ob = 0;
    int tile_no = 0;  // NT = 1: tiles so far
    Piece prev = {};
    int prev_tile = 0, prev_ob = 0, prev_sb = 0, prev_tiles = 0;
    bool have_prev = false, prev_first = false, prev_last = false;
    bool run = true;

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
        for (int i = 0; i < k_steps; ++i) step(i);
      }
    };
    auto pv = [&](int ob, int sb, int slot, bool first) {
      const uint64_t vd = v_desc + slot * (kTileBytes / 16);
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i)
        mma_ts(tmem + 256 + ob * 128, tmem + sb * 128 + i * 8, vd + i * (2048 / 16), id_pv, !(first && i == 0));
    };
    // out += P V of the previous tile, row tile x
    auto pv_tile = [&](int x, int v_slot, bool last_tile) {
      const int sb = NT == 1 ? prev_sb : x, ob = NT == 1 ? prev_ob : x;
      if (!warp_wait(at(ms.p_full, sb), (used[sb] & 1) ^ 1, abort)) return false;
      fence_after();
      if (elect()) {
        pv(ob, sb, v_slot, prev_first);
        if (NT == 1) commit(at(ms.pv_done, sb));
        if (last_tile) commit(at(ms.kv_empty, v_slot));
        if (prev_last) commit(at(ms.o_full, ob));
      }
      __syncwarp();
      if (prev_last) ++items[ob];
      return true;
    };
    // the values of the previous tile are next in the ring: wait for them, make them safe
    auto take_values = [&](int* v_slot) {
      if (prev_first)  // its output buffers (and their poison marks) are free
        for (int x = 0; x < prev_tiles; ++x) {
          const int ob = NT == 1 ? prev_ob : x;
          if (!warp_wait(at(ms.o_empty, ob), (items[ob] & 1) ^ 1, abort)) return false;
        }
      if (!warp_wait(at(ms.kv_full, ring_kv.slot), ring_kv.phase, abort)) return false;
      *v_slot = ring_kv.slot;
      ring_kv.next(kRing);
      const int base = prev_tile * kTile, hi = prev.pos0 + prev.ntok;
      const int last_lo = a.window > 0 ? max(0, hi - a.window) : 0;
      if (base + kTile > prev.pos0 + 1 || base < last_lo) {
        if (clean_values<BF16, DP>(ring + *v_slot * kTileBytes, base, prev.kv_lo, hi, prev.pos0 + 1, last_lo, a.box,
                                   lane)) {
          if (lane < 2 && (NT == 2 || lane == prev_ob)) *reinterpret_cast<volatile int*>(&ms.poison[lane]) = 1;
          __threadfence_block();
          __syncwarp();
        }
      }
      return true;
    };

    Piece p;
    int t = 0;
    p.t0 = p.t1 = 0;
    p.kind = 0;
    for (; run;) {
      // the next tile of the run
      bool more = true;
      while (t == p.t1) {
        if (!warp_wait(at(ms.piece_full, ring_p.slot), ring_p.phase, abort)) {
          run = false;
          break;
        }
        p = ms.piece[ring_p.slot];
        __syncwarp();
        if (lane == 0) bar_arrive(at(ms.piece_empty, ring_p.slot));
        ring_p.next(kQueue);
        t = p.t0;
        if (p.kind == 1) {
          more = false;
          break;
        }
      }
      if (!run) break;
      const int tiles = NT == 1 ? 1 : (p.ntok + a.tile_tokens - 1) / a.tile_tokens;
      int k_slot = 0, v_slot = 0;
      int q = 0;
      auto begin_tile = [&]() {  // keys (and queries) of the next tile are there
        if (!warp_wait(at(ms.kv_full, ring_kv.slot), ring_kv.phase, abort)) return false;
        k_slot = ring_kv.slot;
        ring_kv.next(kRing);
        if (t == p.t0) {
          if (!warp_wait(at(ms.q_full, ring_q.slot), ring_q.phase, abort)) return false;
          cur_ob = next_ob;
          if (NT == 1) next_ob ^= 1;
        }
        if (NT == 1) q = ring_q.slot;
        fence_after();
        return true;
      };
      auto qk_tile = [&](int x) {
        const int sb = NT == 1 ? tile_no & 1 : x;
        if (elect()) {
          qk(sb, NT == 2 ? x : q, k_slot);
          commit(at(ms.s_full, sb));
          if (x == tiles - 1) {
            commit(at(ms.kv_empty, k_slot));
            if (t == p.t1 - 1) commit(at(ms.q_empty, ring_q.slot));
          }
        }
        __syncwarp();
        ++used[sb];
        if (x == tiles - 1 && t == p.t1 - 1) ring_q.next(3 - NT);
      };
      if (NT == 1) {
        const int sb = tile_no & 1;
        if (more) {
          if (!begin_tile()) break;
          qk_tile(0);
        }
        // `used` of the other buffer is not moved by the line above, so prev's parity is its own
        if (have_prev) {
          if (!take_values(&v_slot) || !pv_tile(0, v_slot, true)) break;
        }
        prev_sb = sb;
        if (more) ++tile_no;
      } else {
        if (have_prev && !take_values(&v_slot)) break;
        if (more && !begin_tile()) break;
        bool ok = true;
        for (int x = 0; x < 2 && ok; ++x) {
          if (have_prev && x < prev_tiles) ok = pv_tile(x, v_slot, x == prev_tiles - 1);
          if (ok && more && x < tiles) qk_tile(x);
        }
        if (!ok) break;
      }
      if (!more) break;
      prev = p;
      prev_tile = t;
      prev_tiles = tiles;
      prev_ob = cur_ob;
      prev_first = t == p.t0;
      prev_last = t == p.t1 - 1;
      have_prev = true;
      ++t;
    }
  } else {
    // ---- softmax: thread = row
    const int wg = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t lanes = uint32_t((warp % 4) * 32) << 16;
    const int tok = row / a.group, g = row - tok * a.group;
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
      for (int t = p.t0; t < p.t1; ++t) {
        const int sb = NT == 1 ? int(used & 1) : wg;
        const uint32_t s_addr = tmem + sb * 128 + lanes;
        if (!warp_wait(at(ms.s_full, sb), NT == 1 ? (used >> 1) & 1 : used & 1, abort)) {
          run = false;
          break;
        }
        if (any) {
          fence_after();
          __syncwarp();
          const int base = t * kTile;
          const bool masked = base + kTile > all_hi || base < all_lo;
          const int h = hi - base, l = lo - base;
          // Both passes over the row read S from tensor memory, 64 columns at a time: reading it twice costs
          // less than holding 128 registers of it, and the loops' code stays small.
          auto load_s = [&](int half, uint32_t (&s)[64]) {
            tmem_ld32(s_addr + half * 64, reinterpret_cast<uint32_t(&)[32]>(s[0]));
            tmem_ld32(s_addr + half * 64 + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int j = 0; j < 64; ++j) {
                const int col = half * 64 + j;
                if (col >= h || col < l) s[j] = 0xff800000u;
              }
            }
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t s[64];
            load_s(half, s);
            float m[2] = {top, __uint_as_float(s[63])};
#pragma unroll
            for (int j = 0; j < 62; j += 2) m[(j / 2) & 1] = max3(m[(j / 2) & 1], __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            top = max3(m[0], m[1], __uint_as_float(s[62]));
          }
          top *= scale2;
          const bool move = top > ref + kLazy;
          if (__any_sync(0xffffffffu, move)) {
            const float keep = move ? ex2_approx(ref - top) : 1.0f;
            if (move) {
              ref = top;
              sum *= keep;
            }
            if (t > p.t0) {
              // the outputs so far, once the previous product is in them
              __syncwarp();
              if (NT == 1) {
                const uint32_t w = used - 1;
                if (!warp_wait(at(ms.pv_done, int(w & 1)), (w >> 1) & 1, abort)) {
                  run = false;
                  break;
                }
                fence_after();
              }
#pragma unroll
              for (int i = 0; i < DP / 32; ++i) {
                uint32_t o[32];
                tmem_ld32(o_addr + i * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                tmem_st32(o_addr + i * 32, o);
              }
            }
          }
          __syncwarp();
          const float shift = ref == -INFINITY ? 0.0f : -ref;
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
          }
          const float2 both = fadd2(part[0], part[1]);
          sum += both.x + both.y;
          tmem_wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) bar_arrive(at(ms.p_full, sb));
        ++used;
      }
      if (!run) break;

      // ---- epilogue
      const int n_rows = ntok * a.group;
      const int tok_row = p.tok0 + first_tok + tok;
      const int head = p.head * a.group + g;
      if (p.t1 > p.t0) {
        if (!warp_wait(at(ms.o_full, ob), NT == 1 ? (pieces >> 1) & 1 : pieces & 1, abort)) break;
        fence_after();
      }
      // values that are not finite and that not all rows attend to: this row's own
      const bool poison = p.t1 > p.t0 && *reinterpret_cast<volatile int*>(&ms.poison[ob]) != 0;
      auto add_poison = [&](float* o, int d0, int n) {
        if (!valid) return;
        const int hi_all = p.pos0 + p.ntok;
        const int last_lo = a.window > 0 ? max(0, hi_all - a.window) : 0;
        for (int k = max(lo, p.t0 * kTile); k < min(hi, p.t1 * kTile); ++k) {
          if (k < p.pos0 + 1 && k >= last_lo) continue;
          const int page = c.table[p.request * c.table_stride + k / c.page_size];
          if (page < 0 || page >= c.num_pages) continue;
          const uint16_t* v = c.v + page * c.v_page + (k % c.page_size) * c.v_slot + p.head * c.v_head;
          for (int d = 0; d < n && d0 + d < c.head_dim; ++d) {
            const float x = unpack1<BF16>(v[d0 + d]);
            if (!(fabsf(x) < INFINITY)) o[d] += x;
          }
        }
      };
      const size_t part_floats = size_t(kTile) * DP + 2 * kTile;
      if (p.part < 0) {
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        const bool store = valid && ASV_GUARD(a, tok_row >= 0 && tok_row < c.N && head < a.q_heads);
        uint16_t* out = a.out.p + tok_row * a.out.tok + head * a.out.head;
        if (any) {
#pragma unroll 1
          for (int i = 0; i < DP / 32; ++i) {
            __syncwarp();
            uint32_t o[32];
            if (p.t1 > p.t0) {
              tmem_ld32(o_addr + i * 32, o);
              tmem_wait_ld();
            }
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = p.t1 > p.t0 ? __uint_as_float(o[j]) * inv : 0.0f;
            if (poison) add_poison(y, i * 32, 32);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (store && i * 32 + j * 8 < c.head_dim)
                *reinterpret_cast<uint4*>(out + i * 32 + j * 8) =
                    make_uint4(pack2<BF16>(y[8 * j], y[8 * j + 1]), pack2<BF16>(y[8 * j + 2], y[8 * j + 3]),
                               pack2<BF16>(y[8 * j + 4], y[8 * j + 5]), pack2<BF16>(y[8 * j + 6], y[8 * j + 7]));
            }
          }
          if (store && a.lse != nullptr)
            a.lse[(long long)tok_row * a.q_heads + head] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2f;
        }
      } else {
        // file the partial result: [column / 4][row] float4, then (reference, sum) per row
        float* part = a.parts + (size_t(p.part) * 2 + wg) * part_floats;
        if (any) {
#pragma unroll 1
          for (int i = 0; i < DP / 32; ++i) {
            __syncwarp();
            uint32_t o[32];
            tmem_ld32(o_addr + i * 32, o);
            tmem_wait_ld();
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(o[j]);
            if (poison) add_poison(y, i * 32, 32);
            if (valid) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                __stcg(reinterpret_cast<float4*>(part) + (i * 8 + j) * kTile + row,
                       make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]));
            }
          }
          if (valid) __stcg(reinterpret_cast<float2*>(part + kTile * DP) + row, make_float2(ref, sum));
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

      // the last to file joins the parts, in CTA order
      __threadfence();
      if (!wg_sync()) break;
      if (row == 0) {
        const uint32_t old = atom_add_acq_rel_gpu(a.tickets + 2 * p.first_cta + wg, 1u);
        ms.last[wg] = old == uint32_t(p.n_parts - 1);
      }
      if (!wg_sync()) break;
      const bool last = *reinterpret_cast<volatile int*>(&ms.last[wg]) != 0;
      if (!wg_sync()) break;
      if (!last) continue;
      __threadfence();
      if (row == 0) a.tickets[2 * p.first_cta + wg] = 0;
      const int cols4 = c.head_dim / 4;
      for (int i = row; i < n_rows * cols4; i += kTile) {
        const int c4 = i / n_rows, r = i - c4 * n_rows;
        float m = -INFINITY, l = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < p.n_parts; ++k) {
          const int slot = k == 0 ? 2 * p.first_cta + 1 : 2 * (p.first_cta + k);
          const float* part = a.parts + (size_t(slot) * 2 + wg) * part_floats;
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(part + kTile * DP) + r);
          const float4 o = __ldcg(reinterpret_cast<const float4*>(part) + c4 * kTile + r);
          const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.0f : top;
          const float wa = ex2_approx(m - base), wb = ex2_approx(ml.x - base);
          m = top;
          l = l * wa + ml.y * wb;
          acc = make_float4(acc.x * wa + o.x * wb, acc.y * wa + o.y * wb, acc.z * wa + o.z * wb, acc.w * wa + o.w * wb);
        }
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int tk = r / a.group, hd = p.head * a.group + (r - tk * a.group);
        const int dst = p.tok0 + first_tok + tk;
        if (!ASV_GUARD(a, dst >= 0 && dst < c.N && hd < a.q_heads)) continue;
        *reinterpret_cast<uint2*>(a.out.p + dst * a.out.tok + hd * a.out.head + c4 * 4) =
            make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
        if (c4 == 0 && a.lse != nullptr)
          a.lse[(long long)dst * a.q_heads + hd] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2f;
      }
    }
    if (*abort && lane == 0) {
      for (int b = 0; b < c.B; ++b) atomicOr(a.status + b, ASV_REQ_TIMEOUT);
    }
  }
  fence_before();
  __syncthreads();
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
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] > 0 ? cuuint64_t(strides[i]) * 2 : 256;
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, base, dims,
                        bytes, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool BF16, int DP, int NT>
cudaError_t launch(const AttendArgs& a, const CUtensorMap* maps, int grid, cudaStream_t s) {
  auto kernel = paged_attention_kernel<BF16, DP, NT>;
  constexpr int kSmem = 1024 + (2 + kRingSlots<DP>) * kTile * DP * 2 + int(sizeof(Misc));
  static_assert(kSmem <= 232448, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * (4 * NT + 3), kSmem, s>>>(a, maps[0], maps[1], maps[2]);
  return cudaGetLastError();
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
  a.tile_tokens = kTile / a.group;
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
  // two row tiles to an item where the average chunk has more rows than one tile holds
  const bool two = (long long)c.N * a.group > (long long)kTile * c.B;
  const int which = (bf16 ? 4 : 0) + (c.head_dim > 64 ? 2 : 0) + (two ? 1 : 0);
  switch (which) {
    case 0: return launch<false, 64, 1>(a, maps, grid, s);
    case 1: return launch<false, 64, 2>(a, maps, grid, s);
    case 2: return launch<false, 128, 1>(a, maps, grid, s);
    case 3: return launch<false, 128, 2>(a, maps, grid, s);
    case 4: return launch<true, 64, 1>(a, maps, grid, s);
    case 5: return launch<true, 64, 2>(a, maps, grid, s);
    case 6: return launch<true, 128, 1>(a, maps, grid, s);
    default: return launch<true, 128, 2>(a, maps, grid, s);
  }
}

}  // namespace asv
