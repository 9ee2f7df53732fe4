// asv_paged_plan.cu -- paged_plan: pages for a step's new tokens out of a pool on the device, block tables, and the slot,
// position and request of every packed row.
//
// With sums over the requests in order (a released request counts back_b pages, any request need_b = max(0,
// ceil((cache_len + new) / page) - held) and new_b rows):
//   push   the j-th page of released request b goes to free[count + sum_{c < b} back_c + j]
//   serve  b is served when sum_{c <= b} need_c fits the pool (or need_b = 0) and sum_{c <= b} new_c fits the rows
//   pop    the i-th page of a served request comes from free[count' - 1 - sum_{c < b} need_c - i]
//   place  row r belongs to the last request that starts at or before it; its position and slot follow
// so four prefix sums place every write by itself, and the result does not depend on timing.
//
// A launch of one cluster (CTAs of 512 threads; one of them where there is little to write): every CTA works the
// sums out for itself from the requests' lengths (a few KB, from L2), the CTAs share the pages and the rows, and two
// cluster barriers keep them in step: between pushes and pops (a released request's old entries are read before its new
// ones are written, and pushed pages may be popped), and before the lengths, which all have read, are brought up to date.
// Long steps' rows are placed by a second launch over as many CTAs as they need.
// Next to nothing is moved (16 bytes a row), so the launch is bound by its chain of dependent loads and barriers: 64
// requests of 3 tokens take 4.5 us, 8 prompts of 1000 to 8192 tokens 8.2 and 1024 requests, 6 % of them new prompts, 14.0 (two
// launches each).
#include <algorithm>
#include <climits>

#include "asv_paged_device.cuh"

namespace asv {

namespace {

constexpr int kThreads = 512;
constexpr int kKept = 4;  // requests of a thread whose lengths stay in registers
constexpr int kRows = 4;  // rows of a thread at a time
constexpr int kRowThreads = 128;
constexpr int kWarps = kThreads / 32;

// Sums that stay at the largest number of 31 bits once they reach it: none of the limits they are held against is larger.
struct Sums {
  uint32_t back, need, rows;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  constexpr uint32_t kMost = 0x7fffffffu;
  return {min(a.back + b.back, kMost), min(a.need + b.need, kMost), min(a.rows + b.rows, kMost)};
}

// The sums of the lanes up to this one.
__device__ __forceinline__ Sums warp_scan(Sums x) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Sums y = {__shfl_up_sync(0xffffffffu, x.back, d), __shfl_up_sync(0xffffffffu, x.need, d),
                    __shfl_up_sync(0xffffffffu, x.rows, d)};
    if (lane >= d) x = x + y;
  }
  return x;
}

__device__ __forceinline__ Sums lane_before(Sums x) {
  const Sums y = {__shfl_up_sync(0xffffffffu, x.back, 1), __shfl_up_sync(0xffffffffu, x.need, 1),
                  __shfl_up_sync(0xffffffffu, x.rows, 1)};
  return threadIdx.x % 32 == 0 ? Sums{0, 0, 0} : y;
}

// The sums of the threads before this one, and of all; `room` is [kWarps].
__device__ __forceinline__ Sums scan(Sums own, Sums* room, Sums& all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Sums upto = warp_scan(own), inner = lane_before(upto);
  __syncthreads();  // (the room's last readers are done)
  if (lane == 31) room[warp] = upto;
  __syncthreads();
  const Sums warps = warp_scan(lane < kWarps ? room[lane] : Sums{0, 0, 0}), outer = lane_before(warps);
  auto of = [&](const Sums& x, int l) {
    return Sums{__shfl_sync(0xffffffffu, x.back, l), __shfl_sync(0xffffffffu, x.need, l), __shfl_sync(0xffffffffu, x.rows, l)};
  };
  all = of(warps, 31);
  return of(outer, warp) + inner;
}

// What a request asks for.
struct Want {
  int past, grow, held, back, need;  // held: without the pages given back
  bool ok;
};

__device__ __forceinline__ Want load_want(const PlanArgs& a, int b) {
  Want w;
  w.past = a.cache_len[b];
  w.grow = a.new_len[b];
  const int held = a.held[b];
  const bool released = a.release != nullptr && a.release[b] != 0;
  const bool held_ok = held >= 0 && held <= a.max_pages;
  w.back = released && held_ok ? held : 0;
  w.held = held_ok && !released ? held : 0;
  const long long end = (long long)w.past + w.grow;
  w.ok = held_ok && w.past >= 0 && w.grow >= 0 && w.past <= (long long)w.held * a.page_size &&
         end <= (long long)a.max_pages * a.page_size;
  w.need = w.ok ? max(0, int((end + a.page_size - 1) / a.page_size) - w.held) : 0;
  if (!w.ok) w.grow = 0;
  return w;
}

// The rows' requests, positions and slots; `first` [B + 1] the requests' first rows.  A few of a thread at a time (the
// searches one behind the other took most of the launch).
__device__ __forceinline__ void place_rows(const PlanArgs& a, const int* first, int total, int tid, int threads) {
  int steps = 0;
  while ((1 << steps) < a.B) ++steps;
  for (int x0 = tid; x0 < a.N; x0 += kRows * threads) {
    int lo[kRows], hi[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      lo[i] = 0;
      hi[i] = a.B;
    }
    for (int s = 0; s < steps; ++s) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int mid = (lo[i] + hi[i]) / 2;
        const bool up = first[mid] <= x0 + i * threads;
        lo[i] = up ? mid : lo[i];
        hi[i] = up ? hi[i] : mid;
      }
    }
    int pos[kRows], page[kRows], slot[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int x = x0 + i * threads;
      page[i] = pos[i] = -1;
      if (x < total) {
        pos[i] = a.cache_len[lo[i]] + (x - first[lo[i]]);
        const int entry = pos[i] / a.page_size;
        slot[i] = pos[i] - entry * a.page_size;
        if (ASV_GUARD(a, entry >= 0 && entry < a.max_pages)) page[i] = __ldcg(a.table + lo[i] * a.table_stride + entry);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int x = x0 + i * threads;
      if (x >= a.N) break;
      if (x < total && page[i] < 0) atomicOr(a.status + lo[i], ASV_REQ_BAD_PAGE);
      if (a.slots != nullptr) a.slots[x] = page[i] >= 0 ? (long long)page[i] * a.page_size + slot[i] : -1;
      if (a.positions != nullptr) a.positions[x] = pos[i];
      if (a.requests != nullptr) a.requests[x] = x < total ? lo[i] : -1;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ __align__(16) int s_dyn[];
  __shared__ Sums s_room[kWarps];
  // Of the requests, in order: the first row; pages given back, pages taken (exclusive sums).  (Ends behind the last.)
  int* s_row = s_dyn;
  int* s_back = s_row + a.B + 1;
  int* s_take = s_back + a.B + 1;
  const int tid = threadIdx.x;
  const int rank = int(cluster_rank()), ctas = int(cluster_size());
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the sums: a thread has consecutive requests
  const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  Want kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (b0 + i < b1) kept[i] = load_want(a, b0 + i);
  // f(request, what it asks for) for the thread's requests
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (b0 + i < b1) f(b0 + i, kept[i]);
    for (int b = b0 + kKept; b < b1; ++b) f(b, load_want(a, b));
  };
  const int count0 = a.free_count[0];
  const bool pool_ok = count0 >= 0 && count0 <= a.pool;
  Sums own = {0, 0, 0}, all;
  each([&](int b, const Want& w) {
    own = own + Sums{uint32_t(w.back), uint32_t(w.need), uint32_t(w.grow)};
    if (rank == 0 && !w.ok) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
    if (rank == 0 && !pool_ok) atomicOr(a.status + b, ASV_REQ_BAD_PAGE);
  });
  const Sums first = scan(own, s_room, all);
  const uint32_t given_all = all.back;
  // (pages beyond the pool's end are not there: the pool was handed more pages than it holds)
  const long long count = pool_ok ? min((long long)count0 + all.back, (long long)a.pool) : 0;
  auto served = [&](const Sums& at, const Want& w) {
    return pool_ok && (w.need == 0 || (long long)at.need + w.need <= count) && (long long)at.rows + w.grow <= a.N;
  };
  Sums at = first, got = {0, 0, 0};
  each([&](int, const Want& w) {
    if (served(at, w)) got = got + Sums{0, uint32_t(w.need), uint32_t(w.grow)};
    at = at + Sums{uint32_t(w.back), uint32_t(w.need), uint32_t(w.grow)};
  });
  got = scan(got, s_room, all);  // the served requests' own sums before this thread's
  at = first;
  each([&](int b, const Want& w) {
    const bool is = served(at, w);
    s_back[b] = int(at.back);
    s_take[b] = int(got.need);
    s_row[b] = int(got.rows);
    if (rank == 0) {
      a.indptr[b] = int(got.rows);
      if (w.ok && pool_ok && !is) atomicOr(a.status + b, ASV_REQ_NO_ROOM);
    }
    at = at + Sums{uint32_t(w.back), uint32_t(w.need), uint32_t(w.grow)};
    if (is) got = got + Sums{0, uint32_t(w.need), uint32_t(w.grow)};
  });
  if (tid == 0) {
    s_row[a.B] = int(all.rows);
    s_take[a.B] = int(all.need);
    s_back[a.B] = int(given_all);
    if (rank == 0) a.indptr[a.B] = int(all.rows);
  }
  __syncthreads();
  const int total = s_row[a.B], taken = s_take[a.B];

  // The last request that starts at or before place x of one of the sums, in [0, B).
  auto owner = [&](const int* sum, int x) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sum[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };

  // ---- pages given back (numbers of 32 bits without a sign: there may be almost 2^31 pages, and a thread's next is past them)
  const uint32_t tid_all = rank * kThreads + tid, threads = ctas * kThreads, given = pool_ok ? uint32_t(s_back[a.B]) : 0;
  for (uint32_t x = tid_all; x < given; x += threads) {
    const int b = owner(s_back, int(x));
    int32_t* entry = a.table + b * a.table_stride + (int(x) - s_back[b]);
    const int page = *entry;
    const bool room = x < uint32_t(a.pool - count0);
    if (room) a.free_pages[count0 + int(x)] = page;
    if (!room || page < 0) atomicOr(a.status + b, ASV_REQ_BAD_PAGE);
    *entry = -1;
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();

  // ---- pages taken
  for (uint32_t x = tid_all; x < uint32_t(taken); x += threads) {
    const int b = owner(s_take, int(x)), i = int(x) - s_take[b];
    const Want w = load_want(a, b);
    if (ASV_GUARD(a, x < count && w.held + i < a.max_pages))
      a.table[b * a.table_stride + w.held + i] = __ldcg(a.free_pages + (count - 1 - x));
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();

  // ---- rows
  if (!a.rows_behind) place_rows(a, s_row, total, int(tid_all), int(threads));

  // ---- what is held now (nobody reads it any more)
  if (rank == 0) {
    for (int b = tid; b < a.B; b += kThreads) {
      const Want w = load_want(a, b);
      if (pool_ok && (w.ok || w.back > 0)) a.held[b] = w.held + (s_take[b + 1] - s_take[b]);
    }
    if (tid == 0 && pool_ok) a.free_count[0] = int(count) - taken;
  }
}

// The rows of a long step, by a launch of their own.
__global__ void __launch_bounds__(kRowThreads) paged_rows_kernel(const __grid_constant__ PlanArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  place_rows(a, a.indptr, a.indptr[a.B], blockIdx.x * kRowThreads + threadIdx.x, gridDim.x * kRowThreads);
}

#ifdef ASV_CHECKED
__device__ uint32_t g_check_log[2];  // the plan has no workspace to keep a log in
#endif

cudaError_t launch(const PlanArgs& args, cudaStream_t s) {
  PlanArgs a = args;
  // More CTAs where there are rows for them (192 rows: 4.5 us with one; 24 thousand: 26 with one, 12 with eight), and for
  // many rows a launch behind this one, of as many CTAs as they need.
  a.rows_behind = a.N > 8192;
  const int ctas = a.N > 2048 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = 3 * sizeof(int) * size_t(a.B + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cfg.dynamicSmemBytes > 48 * 1024 - 1024) {
    // (always to the most: the limit is the function's, not the launch's, and another host thread may be between the two)
    constexpr int kMost = 3 * int(sizeof(int)) * (kPlanMaxRequests + 1);
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
  if (e != cudaSuccess || !a.rows_behind) return e;
  cfg.gridDim = dim3(unsigned((a.N + kRows * kRowThreads - 1) / (kRows * kRowThreads)), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_rows_kernel, a);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& args, cudaStream_t s) {
#ifdef ASV_CHECKED
  PlanArgs a = args;
  void* log = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&log, g_check_log);
  if (e != cudaSuccess) return e;
  a.check_log = static_cast<uint32_t*>(log);
  return launch(a, s);
#else
  return launch(args, s);
#endif
}

}  // namespace asv

#ifdef ASV_CHECKED
// The plan's check log (the count and the line of the first failure), when the device's work is done.  Returns a
// cudaError.
extern "C" int asv_paged_plan_check_log(uint32_t* out) {
  const cudaError_t e = cudaDeviceSynchronize();
  return int(e != cudaSuccess ? e : cudaMemcpyFromSymbol(out, asv::g_check_log, sizeof(asv::g_check_log)));
}
#endif
