// Host-side interface of the page plan (not part of the public ABI); the fields as in g4attn_page_group.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace g4 {

constexpr int kPlanGroups = 2;        // layer kinds with a pool of their own
constexpr int kPlanRequests = 4096;   // requests at most (40 bytes of shared memory each)

struct PlanGroup {
  int32_t window, num_pages, max_pages;
  int32_t* free_pages;
  const int32_t* pool;
  int32_t* out_pool;
  int32_t* page_table;
  const int32_t* first_page;
  int32_t* out_first_page;
  const int32_t* lost;
  int32_t* out_lost;
  const int32_t* freed;
  const int32_t* n_freed;
  int32_t* seq_len;
  int64_t* slots;
  int32_t* out_n_freed;
};

struct PlanArgs {
  PlanGroup group[kPlanGroups];
  int n_groups, B, T;
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* out_ctx_len;
  int32_t* q_start;
  int32_t* q_len;
  int32_t* ctx_start;
  int32_t* positions;
  uint32_t* err;
};

cudaError_t launch_plan_pages(const PlanArgs& p, cudaStream_t s);

}  // namespace g4
