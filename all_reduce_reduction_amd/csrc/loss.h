// loss.h -- argument blocks and launchers of the routing and distillation
// kernels (k_route.hip, k_distill.hip), shared with their entry points
// (api_loss.cpp).
//
// Row t of a logit matrix starts at element t * stride of its base; only the
// alignment of single elements is assumed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "simar.h"

namespace simar {

// api.cpp: whether sim_init has run; making the library's device current; its
// number of compute units
bool library_ready();
int library_device();
int library_cus();
// A word of device memory that holds 0 between the launches of `stream`, for
// those launches alone; NULL where there is none: a captured stream (its graph
// may run on any other), the per-thread stream (one handle for many), more
// streams than there are words.
uint32_t* library_turn(hipStream_t stream);

struct RouteArgs {
  const void* x;
  int64_t stride;
  const uint8_t* keep;
  int64_t tokens;
  int experts, topk, normalize;
  int32_t* chosen;
  float* weights;
  int32_t* counts;
  float* sums;
  uint32_t* partial;  // per workgroup: experts + 1 counts, then experts sums
  int workgroups;
  uint32_t* turn;     // 0 before and after the launch: the workgroups add up their own sums
};

struct RouteGradArgs {
  const void* x;
  int64_t stride;
  const uint8_t* keep;
  int64_t tokens;
  int experts, topk, normalize;
  const int32_t* chosen;
  const float* dweights;
  const int32_t* counts;
  const float* sums;
  float coef;
  void* dx;
  int64_t dstride;
  float* loss;
};

// The slots of a row and the softmax they are compared with.
struct DistillArgs {
  const void* x;
  int64_t stride;
  int64_t rows, cols, first, vocab;
  const int32_t* ids;
  const void* teacher;
  int teacher_dtype, topk;
  float tau;
  const float* row_scale;
  float coef;
  void* dx;
  int64_t dstride;
  float* loss;
  float* parts;       // [splits][4][rows]: written by the statistics, read by join and gradient
  float* norm;        // [2][rows]
  int splits;         // workgroups per row, each over a run of columns
  int64_t span;       // columns per workgroup
  int look_first;     // rows without slots are left unread
};

int route_workgroups(int64_t tokens, int experts, int dtype);
bool route_sums_itself(int workgroups, int experts);
hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s);
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s);

int distill_splits(int64_t rows, int64_t cols, int64_t least);
int64_t distill_span(int64_t cols, int splits);
hipError_t launch_distill_stats(const DistillArgs& a, int dtype, hipStream_t s);
hipError_t launch_distill_join(const DistillArgs& a, float* loss, float* norm, hipStream_t s);
hipError_t launch_distill_grad(const DistillArgs& a, int dtype, hipStream_t s);
// one workgroup per row: statistics and gradient in one launch
bool distill_whole_rows(int64_t rows, int64_t cols, int dtype);
hipError_t launch_distill_row_fp32(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_row_fp16(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_row_bf16(const DistillArgs& a, hipStream_t s);
// a shard's parts from those of its splits
hipError_t launch_distill_merge(const DistillArgs& a, float* out, hipStream_t s);

}  // namespace simar
