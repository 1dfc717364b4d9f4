// api_loss.cpp -- entry points of the routing and distillation operators:
// argument checks, workspace sizes and launches.  Nothing is enqueued when a
// check fails.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_checks.h"
#include "loss.h"

namespace simar {
namespace {

// a gradient (array 1) may lie on its logits (array 0)
constexpr Over kGradOnLogits[] = {{1, 0}};

int check_route(int64_t tokens, int experts, int topk, int dtype) {
  if (!float_dtype(dtype)) return SIM_ERR_INVALID_ARG;
  if (experts < 1 || experts > SIM_ROUTE_MAX_EXPERTS || topk < 1 || topk > SIM_ROUTE_MAX_TOPK || topk > experts)
    return SIM_ERR_INVALID_ARG;
  return tokens < 0 || tokens > kMaxGrid ? SIM_ERR_INVALID_ARG : SIM_OK;
}

int64_t route_work_bytes(int64_t tokens, int experts, int dtype) {
  const int64_t wg = route_workgroups(tokens, experts, dtype);
  return wg > 1 ? wg * (2 * (int64_t)experts + 1) * 4 : 0;
}

// Everything of a distillation call but its outputs.
int check_distill(int64_t rows, int64_t cols, int64_t stride, int dtype, int64_t first, int64_t vocab, int tdtype,
                  int topk, float tau) {
  if (!float_dtype(dtype) || !float_dtype(tdtype)) return SIM_ERR_INVALID_ARG;
  if (topk < 1 || topk > SIM_DISTILL_MAX_TOPK) return SIM_ERR_INVALID_ARG;
  if (!(tau >= 1e-20f && tau <= 1e20f)) return SIM_ERR_INVALID_ARG;
  if (!rows_fit(rows, cols, stride)) return SIM_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > INT32_MAX || first < 0 || first > vocab - cols) return SIM_ERR_INVALID_ARG;
  return rows > kMaxGrid ? SIM_ERR_INVALID_ARG : SIM_OK;
}

// Least columns per workgroup where a row is split.  A shard's parts need one
// more launch to merge splits, so a row's statistics are split no finer than
// 256 KiB (64 rows x 32,768 bf16 whole 5.2 us, in two 9.1; 400 rows x 131,072
// whole 20.7, in two 24.2); a gradient and a step's two launches, which need
// none, split down to 8 KiB.
int64_t stats_least(int dtype) { return (256 << 10) / size_of(dtype); }
int64_t grad_least(int dtype) { return (8 << 10) / size_of(dtype); }
// A gradient's workgroup takes one chunk of 16 KiB at most: with more, its
// loads would wait for its stores (1,024 rows x 65,536 bf16: 97 us in four
// chunks, 49 in one).
int grad_splits(int64_t rows, int64_t cols, int dtype) {
  const int64_t chunk = (16 << 10) / size_of(dtype);
  return std::max(distill_splits(rows, cols, grad_least(dtype)), (int)((cols + chunk - 1) / chunk));
}

int64_t distill_work_bytes(int64_t rows, int64_t cols, int dtype) {
  const int64_t step = distill_whole_rows(rows, cols, dtype) ? 0 : grad_splits(rows, cols, dtype);
  const int64_t parts = distill_splits(rows, cols, stats_least(dtype));
  return std::max<int64_t>(step, parts > 1 ? parts : 0) * 4 * rows * 4;
}

}  // namespace
}  // namespace simar

using namespace simar;

extern "C" {

int sim_route_work(int64_t tokens, int experts, int topk, int dtype, size_t* bytes) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  const int rc = check_route(tokens, experts, topk, dtype);
  if (rc) return rc;
  if (!bytes) return SIM_ERR_INVALID_ARG;
  *bytes = (size_t)route_work_bytes(tokens, experts, dtype);
  return SIM_OK;
}

int sim_route(const void* logits, int64_t row_stride, int dtype, const uint8_t* keep, int64_t tokens, int experts,
              int topk, int normalize, int32_t* chosen, float* weights, int32_t* counts, float* prob_sums,
              void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_route(tokens, experts, topk, dtype);
  if (rc) return rc;
  if (!rows_fit(tokens, experts, row_stride)) return SIM_ERR_INVALID_ARG;
  if (!counts || !prob_sums || (tokens > 0 && (!logits || !chosen || !weights))) return SIM_ERR_INVALID_ARG;
  const int64_t need = route_work_bytes(tokens, experts, dtype);
  if ((rc = check_work(work, work_bytes, need))) return rc;
  const Array all[] = {rows_of(logits, tokens, experts, row_stride, dtype, false),
                       {keep, tokens, 1, false},
                       {chosen, tokens * topk * 4, 4, true},
                       {weights, tokens * topk * 4, 4, true},
                       {counts, ((int64_t)experts + 1) * 4, 4, true},
                       {prob_sums, (int64_t)experts * 4, 4, true},
                       {need ? work : nullptr, need, 4, true}};
  if ((rc = check_arrays(all))) return rc;
  if ((rc = library_device())) return rc;
  const int wg = route_workgroups(tokens, experts, dtype);
  const Turn turn = route_sums_itself(wg, experts) ? library_turn((hipStream_t)stream) : Turn{};
  const RouteArgs a{logits, row_stride, keep, tokens, experts, topk, normalize != 0, chosen, weights, counts, prob_sums,
                    (uint32_t*)work, wg, turn};
  const hipError_t e = launch_route(a, dtype, (hipStream_t)stream);
  if (e == hipSuccess) library_turn_used(turn, wg, wg == 1 || turn.word ? 1 : 2);
  return hip_status(e);
}

int sim_route_grad(const void* logits, int64_t row_stride, int dtype, const uint8_t* keep, int64_t tokens,
                   int experts, int topk, int normalize, const int32_t* chosen, const float* dweights,
                   const int32_t* counts, const float* prob_sums, float coef, void* dlogits, int64_t drow_stride,
                   float* loss, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_route(tokens, experts, topk, dtype);
  if (rc) return rc;
  if (!rows_fit(tokens, experts, row_stride) || !rows_fit(tokens, experts, drow_stride)) return SIM_ERR_INVALID_ARG;
  if ((counts == nullptr) != (prob_sums == nullptr) || (counts && !loss)) return SIM_ERR_INVALID_ARG;
  if (tokens > 0 && (!logits || !dlogits || (dweights && !chosen))) return SIM_ERR_INVALID_ARG;
  const Array all[] = {rows_of(logits, tokens, experts, row_stride, dtype, false),
                       rows_of(dlogits, tokens, experts, drow_stride, dtype, true),
                       {keep, tokens, 1, false},
                       {chosen, tokens * topk * 4, 4, false},
                       {dweights, tokens * topk * 4, 4, false},
                       {counts, ((int64_t)experts + 1) * 4, 4, false},
                       {prob_sums, (int64_t)experts * 4, 4, false},
                       {loss, 4, 4, true}};
  if ((rc = check_arrays(all, kGradOnLogits))) return rc;
  if ((rc = library_device())) return rc;
  const RouteGradArgs a{logits, row_stride, keep, tokens, experts, topk, normalize != 0, chosen, dweights, counts,
                        prob_sums, coef, dlogits, drow_stride, loss};
  return hip_status(launch_route_grad(a, dtype, (hipStream_t)stream));
}

int sim_distill_work(int64_t rows, int64_t columns, int dtype, size_t* bytes) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  if (!float_dtype(dtype) || rows < 0 || rows > kMaxGrid || columns < 1 || columns > INT32_MAX || !bytes)
    return SIM_ERR_INVALID_ARG;
  *bytes = (size_t)distill_work_bytes(rows, columns, dtype);
  return SIM_OK;
}

int sim_distill_step(const void* logits, int64_t row_stride, int dtype, int64_t rows, int64_t vocab,
                     const int32_t* ids, const void* teacher, int teacher_dtype, int topk, float temperature,
                     const float* row_scale, float coef, void* dlogits, int64_t drow_stride, float* loss,
                     void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_distill(rows, vocab, row_stride, dtype, 0, vocab, teacher_dtype, topk, temperature);
  if (rc) return rc;
  if (!rows_fit(rows, vocab, drow_stride)) return SIM_ERR_INVALID_ARG;
  if (rows == 0) return SIM_OK;
  if (!logits || !ids || !teacher || !dlogits || !loss) return SIM_ERR_INVALID_ARG;
  const int64_t need = distill_work_bytes(rows, vocab, dtype);
  if ((rc = check_work(work, work_bytes, need))) return rc;
  const Array all[] = {rows_of(logits, rows, vocab, row_stride, dtype, false),
                       rows_of(dlogits, rows, vocab, drow_stride, dtype, true),
                       {ids, rows * topk * 4, 4, false},
                       {teacher, rows * topk * size_of(teacher_dtype), size_of(teacher_dtype), false},
                       {row_scale, rows * 4, 4, false},
                       {loss, rows * 4, 4, true},
                       {need ? work : nullptr, need, 4, true}};
  if ((rc = check_arrays(all, kGradOnLogits))) return rc;
  if ((rc = library_device())) return rc;
  DistillArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.rows = rows;
  a.cols = a.vocab = vocab;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_dtype = teacher_dtype;
  a.topk = topk;
  a.tau = temperature;
  a.row_scale = row_scale;
  a.coef = coef;
  a.dx = dlogits;
  a.dstride = drow_stride;
  a.loss = loss;
  a.parts = (float*)work;
  a.splits = grad_splits(rows, vocab, dtype);
  a.span = distill_span(vocab, a.splits);
  if ((int64_t)a.splits * rows > kMaxGrid) return SIM_ERR_INVALID_ARG;
  const hipStream_t s = (hipStream_t)stream;
  if (distill_whole_rows(rows, vocab, dtype))
    return hip_status(dtype == SIM_FP32   ? launch_distill_row_fp32(a, s)
                      : dtype == SIM_FP16 ? launch_distill_row_fp16(a, s)
                                          : launch_distill_row_bf16(a, s));
  const hipError_t e = launch_distill_stats(a, dtype, s);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(launch_distill_grad(a, dtype, s));
}

int sim_distill_parts(const void* logits, int64_t row_stride, int dtype, int64_t rows, int64_t columns,
                      int64_t first, int64_t vocab, const int32_t* ids, const void* teacher, int teacher_dtype,
                      int topk, float temperature, float* parts, void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_distill(rows, columns, row_stride, dtype, first, vocab, teacher_dtype, topk, temperature);
  if (rc) return rc;
  if (rows == 0) return SIM_OK;
  if (!logits || !ids || !teacher || !parts) return SIM_ERR_INVALID_ARG;
  const int64_t need = distill_work_bytes(rows, columns, dtype);
  if ((rc = check_work(work, work_bytes, need))) return rc;
  const Array all[] = {rows_of(logits, rows, columns, row_stride, dtype, false),
                       {ids, rows * topk * 4, 4, false},
                       {teacher, rows * topk * size_of(teacher_dtype), size_of(teacher_dtype), false},
                       {parts, rows * 16, 4, true},
                       {need ? work : nullptr, need, 4, true}};
  if ((rc = check_arrays(all))) return rc;
  if ((rc = library_device())) return rc;
  DistillArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.rows = rows;
  a.cols = columns;
  a.first = first;
  a.vocab = vocab;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_dtype = teacher_dtype;
  a.topk = topk;
  a.tau = temperature;
  a.splits = distill_splits(rows, columns, stats_least(dtype));
  a.span = distill_span(columns, a.splits);
  if ((int64_t)a.splits * rows > kMaxGrid) return SIM_ERR_INVALID_ARG;
  a.parts = a.splits > 1 ? (float*)work : parts;
  const hipError_t e = launch_distill_stats(a, dtype, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e);
  return a.splits > 1 ? hip_status(launch_distill_merge(a, parts, (hipStream_t)stream)) : SIM_OK;
}

int sim_distill_join(const float* parts, int nparts, int64_t rows, int64_t vocab, const int32_t* ids,
                     const void* teacher, int teacher_dtype, int topk, float temperature, float* loss, float* norm,
                     void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_distill(rows, 1, 1, SIM_FP32, 0, vocab, teacher_dtype, topk, temperature);
  if (rc) return rc;
  if (nparts < 1 || nparts > (1 << 20) || rows > kMaxBytes / 16 / nparts) return SIM_ERR_INVALID_ARG;
  if (rows == 0) return SIM_OK;
  if (!parts || !ids || !teacher || !loss || !norm) return SIM_ERR_INVALID_ARG;
  const Array all[] = {{parts, (int64_t)nparts * rows * 16, 4, false},
                       {ids, rows * topk * 4, 4, false},
                       {teacher, rows * topk * size_of(teacher_dtype), size_of(teacher_dtype), false},
                       {loss, rows * 4, 4, true},
                       {norm, rows * 8, 4, true}};
  if ((rc = check_arrays(all))) return rc;
  if ((rc = library_device())) return rc;
  DistillArgs a{};
  a.rows = rows;
  a.vocab = vocab;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_dtype = teacher_dtype;
  a.topk = topk;
  a.tau = temperature;
  a.parts = const_cast<float*>(parts);
  a.splits = nparts;
  return hip_status(launch_distill_join(a, loss, norm, (hipStream_t)stream));
}

int sim_distill_grad(const void* logits, int64_t row_stride, int dtype, int64_t rows, int64_t columns,
                     int64_t first, int64_t vocab, const int32_t* ids, const void* teacher, int teacher_dtype,
                     int topk, float temperature, const float* norm, const float* row_scale, float coef,
                     void* dlogits, int64_t drow_stride, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_distill(rows, columns, row_stride, dtype, first, vocab, teacher_dtype, topk, temperature);
  if (rc) return rc;
  if (!rows_fit(rows, columns, drow_stride)) return SIM_ERR_INVALID_ARG;
  if (rows == 0) return SIM_OK;
  if (!logits || !ids || !teacher || !norm || !dlogits) return SIM_ERR_INVALID_ARG;
  const Array all[] = {rows_of(logits, rows, columns, row_stride, dtype, false),
                       rows_of(dlogits, rows, columns, drow_stride, dtype, true),
                       {ids, rows * topk * 4, 4, false},
                       {teacher, rows * topk * size_of(teacher_dtype), size_of(teacher_dtype), false},
                       {norm, rows * 8, 4, false},
                       {row_scale, rows * 4, 4, false}};
  if ((rc = check_arrays(all, kGradOnLogits))) return rc;
  if ((rc = library_device())) return rc;
  DistillArgs a{};
  a.x = logits;
  a.stride = row_stride;
  a.rows = rows;
  a.cols = columns;
  a.first = first;
  a.vocab = vocab;
  a.ids = ids;
  a.teacher = teacher;
  a.teacher_dtype = teacher_dtype;
  a.topk = topk;
  a.tau = temperature;
  a.row_scale = row_scale;
  a.coef = coef;
  a.dx = dlogits;
  a.dstride = drow_stride;
  a.norm = const_cast<float*>(norm);
  a.splits = grad_splits(rows, columns, dtype);
  a.span = distill_span(columns, a.splits);
  if ((int64_t)a.splits * rows > kMaxGrid) return SIM_ERR_INVALID_ARG;
  return hip_status(launch_distill_grad(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
