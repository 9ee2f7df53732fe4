// asv_paged.h -- host-side declarations shared by the paged-cache entry points and their kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "asv.h"
#include "asv_internal.h"

namespace asv {

struct RowsView {
  uint16_t* p;
  long long tok, head;  // strides in elements
};

// The cache and the batch as the kernels take them (strides of extent-1 dimensions zeroed).
struct PagedView {
  uint16_t* k;
  uint16_t* v;
  int num_pages, page_size, kv_heads, head_dim;
  long long k_page, k_slot, k_head, v_page, v_slot, v_head;
  int B, N;
  const int32_t* indptr;
  const int32_t* cache_len;
  const int32_t* table;
  int max_pages;
  long long table_stride;
};

struct AppendArgs {
  PagedView c;
  RowsView k, v, q, out_q;  // q.p == nullptr: keys and values only
  int q_heads;
  const float* rotary;  // nullptr: no rotation
  int rot_dim, max_position, interleaved;
  uint32_t* status;
  uint32_t* check_log;  // of the checked build: the append has no workspace, its log is the library's
};

// The same with positions of their own for the rotation.
struct PlacedArgs : AppendArgs {
  const int32_t* positions;  // [axes, N]; nullptr: the slots' positions
  int axes;
  long long axis_stride;
  uint8_t axis[64];  // axis of each pair
};

struct AttendArgs {
  PagedView c;
  RowsView q, out;
  int q_heads, group;
  float scale;
  int window;
  float* lse;
  uint32_t* status;
  int box;             // slots one copy of keys or values takes (a power of two that divides the page)
  int tile_tokens;     // tokens of one row tile
  uint32_t* tickets;   // workspace: [kMaxGrid * 2], zero between calls
  float* parts;        // workspace: partial results of split items
  uint32_t* check_log;
};

struct PlanArgs {
  const int32_t* cache_len;
  const int32_t* new_len;
  int B, N;
  int32_t* table;
  int max_pages;
  long long table_stride;
  int page_size;
  int32_t* held;
  int32_t* free_pages;
  int pool;  // entries of free_pages
  int32_t* free_count;
  const uint8_t* release;  // nullptr: none
  int32_t* indptr;
  int64_t* slots;       // these three: nullptr, not wanted
  int32_t* positions;
  int32_t* requests;
  bool rows_behind;  // the rows are placed by the launch behind
  uint32_t* status;
  uint32_t* check_log;  // of the checked build: the plan has no workspace, its log is the library's
};

// paged_attention's workspace: tickets (zero between calls), then each CTA's two partial results of up
// to two row tiles (unnormalised outputs, then row maxima and sums).
constexpr int kPagedMaxGrid = 152;
constexpr int kPagedTicketBytes = ASV_PAGED_WORKSPACE_ZEROED;
constexpr int kPagedSlots = 2 * kPagedMaxGrid;
inline size_t paged_part_floats(int dim_padded) { return size_t(128) * dim_padded + 2 * 128; }
inline size_t paged_workspace_bytes(int head_dim) {
  return kPagedTicketBytes + kPagedSlots * 2 * paged_part_floats(head_dim <= 64 ? 64 : 128) * sizeof(float);
}

constexpr int kPlanMaxRequests = 16384;  // three words each in one CTA's shared memory
constexpr int kPlanMaxRows = 1 << 30;  // (a thread's next rows are still numbers of 32 bits)
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s);
cudaError_t launch_paged_append(const PlacedArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_paged_attention(const AttendArgs& a, int dtype, cudaStream_t s);

// ASV_ERR_CUDA, with `e` kept for asv_last_cuda_error (asv_api.cu).
asv_status record_cuda_error(cudaError_t e);

}  // namespace asv
