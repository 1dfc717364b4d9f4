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
// A word of device memory for one launch alone.  Each of its workgroups adds 1
// to it, and the last one reports `call` to `done`, in host memory; only then is
// the word handed out again, so that no two launches can meet in it, on whatever
// streams they are.  A launch that should ever end without its report keeps its
// word for good.
struct Turn {
  uint32_t* word;  // NULL: none
  uint32_t base;   // what the word holds before the launch
  uint32_t* done;
  uint32_t call;
};
// A word for the next launch on `stream`; none for a captured one (its graph is
// replayed with the same arguments) or while the next word is still in use.
Turn library_turn(hipStream_t stream);
// That launch was made, of `workgroups` workgroups and with `launches` kernels
// in all.
void library_turn_used(const Turn& t, int workgroups, int launches);

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
  Turn turn;          // with a word: the workgroups add up their own sums
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
