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
// One launch of one cluster (CTAs of 512 threads; one of them where there is little to write): every CTA works the
// sums out for itself from the requests' lengths (a few KB, from L2), the CTAs share the pages and the rows, and two
// cluster barriers keep them in step: between pushes and pops (a released request's old entries are read before its new
// ones are written, and pushed pages may be popped), and before the lengths, which all have read, are brought up to date.
// Next to nothing is moved (16 bytes a row), so the launch is bound by its chain of dependent loads and barriers.
#include <algorithm>
#include <climits>

#include "asv_paged_device.cuh"

namespace asv {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Sums {
  long long back, need, rows;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.back + b.back, a.need + b.need, a.rows + b.rows}; }

__device__ __forceinline__ long long shfl_up(long long x, int d) { return __shfl_up_sync(0xffffffffu, x, d); }

// The sums of the threads before this one, and of all; `room` is [kWarps].
__device__ __forceinline__ Sums scan(Sums own, Sums* room, Sums& all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Sums incl = own;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Sums x = {shfl_up(incl.back, d), shfl_up(incl.need, d), shfl_up(incl.rows, d)};
    if (lane >= d) incl = incl + x;
  }
  __syncthreads();  // (the room's last readers are done)
  if (lane == 31) room[warp] = incl;
  __syncthreads();
  Sums before = {0, 0, 0};
  all = before;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before = before + room[w];
    all = all + room[w];
  }
  return before + Sums{incl.back - own.back, incl.need - own.need, incl.rows - own.rows};
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

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
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
  const int count0 = a.free_count[0];
  const bool pool_ok = count0 >= 0 && count0 <= a.pool;
  Sums own = {0, 0, 0}, all;
  for (int b = b0; b < b1; ++b) {
    const Want w = load_want(a, b);
    own = own + Sums{w.back, w.need, w.grow};
    if (rank == 0 && !w.ok) atomicOr(a.status + b, ASV_REQ_BAD_LEN);
    if (rank == 0 && !pool_ok) atomicOr(a.status + b, ASV_REQ_BAD_PAGE);
  }
  Sums before = scan(own, s_room, all);
  // (pages beyond the pool's end are not there: the pool was handed more pages than it holds)
  const long long count = pool_ok ? min((long long)count0 + all.back, (long long)a.pool) : 0;
  Sums take = {0, 0, 0};
  const Sums first = before;
  for (int pass = 0; pass < 2; ++pass) {
    Sums at = first, got = take;  // (second pass: the served requests' own sums before this thread's)
    for (int b = b0; b < b1; ++b) {
      const Want w = load_want(a, b);
      const bool served = pool_ok && (w.need == 0 || at.need + w.need <= count) && at.rows + w.grow <= a.N;
      if (pass == 1) {
        s_back[b] = int(min(at.back, (long long)INT_MAX));
        s_take[b] = int(got.need);
        s_row[b] = int(got.rows);
        if (rank == 0) {
          a.indptr[b] = int(got.rows);
          if (w.ok && pool_ok && !served) atomicOr(a.status + b, ASV_REQ_NO_ROOM);
        }
      }
      at = at + Sums{w.back, w.need, w.grow};
      if (served) got = got + Sums{0, w.need, w.grow};
    }
    if (pass == 0) take = scan(got, s_room, all);
  }
  if (tid == 0) {
    s_row[a.B] = int(all.rows);
    s_take[a.B] = int(all.need);
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

  // ---- pages given back, by warps in turn (few requests have any)
  const int warp = rank * kWarps + tid / 32, warps = ctas * kWarps, lane = tid % 32;
  if (a.release != nullptr && pool_ok) {
    for (int g = warp; g * 32 < a.B; g += warps) {
      const int mine = g * 32 + lane;
      const int back = mine < a.B ? load_want(a, mine).back : 0;
      for (uint32_t some = __ballot_sync(0xffffffffu, back > 0); some != 0; some &= some - 1) {
        const int b = g * 32 + __ffs(some) - 1, n = __shfl_sync(0xffffffffu, back, __ffs(some) - 1);
        int32_t* row = a.table + b * a.table_stride;
        for (int j = lane; j < n; j += 32) {
          const long long to = (long long)count0 + s_back[b] + j;
          if (to < a.pool) a.free_pages[to] = row[j];
          else atomicOr(a.status + b, ASV_REQ_BAD_PAGE);
          row[j] = -1;
        }
      }
    }
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();

  // ---- pages taken
  const int tid_all = rank * kThreads + tid, threads = ctas * kThreads;
  for (int x = tid_all; x < taken; x += threads) {
    const int b = owner(s_take, x), i = x - s_take[b];
    const Want w = load_want(a, b);
    if (ASV_GUARD(a, x < count && w.held + i < a.max_pages)) a.table[b * a.table_stride + w.held + i] = __ldcg(a.free_pages + (count - 1 - x));
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();

  // ---- rows
  for (int x = tid_all; x < a.N; x += threads) {
    int request = -1, pos = -1;
    long long slot = -1;
    if (x < total) {
      request = owner(s_row, x);
      pos = a.cache_len[request] + (x - s_row[request]);
      const int entry = pos / a.page_size;
      const int page = ASV_GUARD(a, entry >= 0 && entry < a.max_pages) ? __ldcg(a.table + request * a.table_stride + entry) : -1;
      if (page >= 0) slot = (long long)page * a.page_size + (pos - entry * a.page_size);
      else atomicOr(a.status + request, ASV_REQ_BAD_PAGE);
    }
    if (a.slots != nullptr) a.slots[x] = slot;
    if (a.positions != nullptr) a.positions[x] = pos;
    if (a.requests != nullptr) a.requests[x] = request;
  }

  // ---- what is held now (nobody reads it any more)
  if (rank == 0) {
    for (int b = tid; b < a.B; b += kThreads) {
      const Want w = load_want(a, b);
      if (pool_ok && (w.ok || w.back > 0)) a.held[b] = w.held + (s_take[b + 1] - s_take[b]);
    }
    if (tid == 0 && pool_ok) a.free_count[0] = int(count) - taken;
  }
}

#ifdef ASV_CHECKED
__device__ uint32_t g_check_log[2];  // the plan has no workspace to keep a log in
#endif

// More CTAs where there are rows for them.
int plan_ctas(const PlanArgs& a) { return a.N > 2048 ? 8 : 1; }

cudaError_t launch(const PlanArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int ctas = plan_ctas(a);
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
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(cfg.dynamicSmemBytes));
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
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
