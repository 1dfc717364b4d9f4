// api_layer.cpp -- entry points of the norm, expert and clipping operators:
// argument checks, workspace sizes and launches.  Nothing is enqueued when a
// check fails.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "api_checks.h"
#include "layer.h"

namespace simar {
namespace {

// (a launch has fewer than 2^32 threads, a workgroup for a piece 256)
constexpr int64_t kMaxPieces = ((int64_t)1 << 24) - 1;
constexpr int64_t kMaxColumns = (int64_t)1 << 30;

bool eps_fits(float eps) { return eps >= 1e-30f && eps <= 1e30f; }

// rows of bytes
Array bytes_of(const void* p, int64_t rows, int64_t width, int64_t pitch, int64_t align, bool output) {
  return {p, rows > 0 && width > 0 ? (rows - 1) * pitch + width : 0, align, output, width, pitch};
}
bool pitch_fits(int64_t rows, int64_t width, int64_t pitch) {
  return rows >= 0 && width >= 0 && width <= INT32_MAX && pitch >= width && pitch <= kMaxBytes &&
         (rows == 0 || pitch == 0 || rows <= kMaxBytes / pitch);
}

int check_norm(int64_t rows, int64_t cols, int dtype, int gain_dtype, float eps) {
  if (!float_dtype(dtype) || !float_dtype(gain_dtype) || !eps_fits(eps)) return SIM_ERR_INVALID_ARG;
  return rows < 0 || rows > kMaxGrid || cols < 1 || cols > SIM_NORM_MAX_COLUMNS ? SIM_ERR_INVALID_ARG : SIM_OK;
}
int64_t norm_grad_work_bytes(int64_t rows, int64_t cols, int dtype) {
  const int64_t wg = norm_grad_workgroups(rows, cols, dtype, true);
  return wg > 1 ? wg * cols * 4 : 0;
}

int check_slots(int64_t tokens, int topk) {
  return tokens < 0 || topk < 1 || topk > SIM_ROUTE_MAX_TOPK || tokens > INT32_MAX / topk ? SIM_ERR_INVALID_ARG : SIM_OK;
}
int64_t dispatch_work_bytes(int64_t tokens, int topk, int experts) {
  int64_t chunk;
  const int64_t chunks = dispatch_chunks(tokens * topk, experts, &chunk);
  return dispatch_counts(tokens * topk, experts) ? chunks * experts * 4 : 0;
}

// Up to so many pieces the workgroups that scale them each add up the squares'
// sums (322 pieces 12.9 us, 15.8 with a launch for it; 1,000 12.7, 14.4; 2,000 23.2,
// 24.4); with more, that costs them more than a launch (3,000 pieces 33.9, 31.8; 8,000
// 77, 67; 98,824 864, 747).
constexpr int64_t kJoinPieces = 2048;

// ---- lists of tensors ---------------------------------------------------------
int check_list(const void* const* grads, const int64_t* counts, const int* dtypes, int n) {
  if (n < 0 || n > SIM_CLIP_MAX_TENSORS) return SIM_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !counts || !dtypes)) return SIM_ERR_INVALID_ARG;
  int64_t all = 0;
  for (int i = 0; i < n; i++) {
    if (!float_dtype(dtypes[i]) || counts[i] < 0 || counts[i] > kMaxBytes / 4) return SIM_ERR_INVALID_ARG;
    if ((all += counts[i]) > kMaxBytes / 4 || clip_pieces(counts[i], dtypes[i]) > kMaxPieces) return SIM_ERR_INVALID_ARG;
    if (counts[i] > 0 && !grads[i]) return SIM_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; i++)
    if (counts[i] > 0 && ((uintptr_t)grads[i] & (uintptr_t)(size_of(dtypes[i]) - 1))) return SIM_ERR_ALIGN;
  return SIM_OK;
}

// The tensors of one launch, from `i` on: fills `l` and moves `i` on.  Tensors
// without elements are left out.
void take(ClipList& l, int& i, const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes, int n) {
  l.tensors = 0;
  int64_t pieces = 0;
  for (; i < n && l.tensors < kClipTensors; i++) {
    if (counts[i] == 0) continue;
    const int64_t p = clip_pieces(counts[i], dtypes[i]);
    if (l.tensors > 0 && pieces + p > kMaxPieces) break;
    const int t = l.tensors++;
    l.first[t] = (uint32_t)pieces;
    l.in[t] = grads ? grads[i] : nullptr;
    l.out[t] = outs ? outs[i] : grads ? const_cast<void*>(grads[i]) : nullptr;
    l.count[t] = counts[i];
    l.dtype[t] = (uint8_t)dtypes[i];
    pieces += p;
  }
  l.pieces = (uint32_t)pieces;
}
struct Sizes {
  int launches, squares;
  int64_t pieces;
};
Sizes sizes_of(const int64_t* counts, const int* dtypes, int n) {
  Sizes s{0, 0, 0};
  for (int i = 0; i < n;) {
    ClipList l;
    take(l, i, nullptr, nullptr, counts, dtypes, n);
    if (l.tensors == 0) break;
    s.launches++;
    s.pieces += l.pieces;
    s.squares += clip_workgroups(l.pieces);
  }
  return s;
}
int64_t clip_work_bytes(const Sizes& s) { return 8 * (int64_t)s.squares; }

struct Extent {
  uintptr_t lo, hi;
  bool output;
};
// Whether an output shares a byte with anything else.  A tensor that is scaled in
// place is one extent.
bool any_overlap(std::vector<Extent>& v) {
  std::sort(v.begin(), v.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  uintptr_t any = 0, out = 0;
  for (const Extent& e : v) {
    if (e.lo < (e.output ? any : out)) return true;
    any = std::max(any, e.hi);
    if (e.output) out = std::max(out, e.hi);
  }
  return false;
}
void add_extent(std::vector<Extent>& v, const void* p, int64_t bytes, bool output) {
  if (p && bytes > 0) v.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, output});
}

hipError_t squares_of_list(const void* const* grads, const int64_t* counts, const int* dtypes, int n, double* squares,
                           hipStream_t s) {
  int at = 0;
  for (int i = 0; i < n;) {
    ClipList l;
    take(l, i, grads, nullptr, counts, dtypes, n);
    if (l.tensors == 0) break;
    const hipError_t e = launch_clip_squares(l, squares + at, s);
    if (e != hipSuccess) return e;
    at += clip_workgroups(l.pieces);
  }
  return hipSuccess;
}

}  // namespace
}  // namespace simar

using namespace simar;

extern "C" {

int sim_norm(const void* x, int64_t x_stride, int dtype, const void* residual, int64_t residual_stride, int64_t rows,
             int64_t columns, const void* gain, int gain_dtype, float eps, void* sum, int64_t sum_stride, void* out,
             int64_t out_stride, float* scales, int group, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_norm(rows, columns, dtype, gain_dtype, eps);
  if (rc) return rc;
  if (scales && group != 0 && group != 32 && group != 64 && group != 128) return SIM_ERR_INVALID_ARG;
  if (!rows_fit(rows, columns, x_stride) || !rows_fit(rows, columns, out_stride)) return SIM_ERR_INVALID_ARG;
  if (residual && !rows_fit(rows, columns, residual_stride)) return SIM_ERR_INVALID_ARG;
  if (sum && (!residual || !rows_fit(rows, columns, sum_stride))) return SIM_ERR_INVALID_ARG;
  if (rows == 0) return SIM_OK;
  if (!x || !out) return SIM_ERR_INVALID_ARG;
  const int64_t groups = scales && group ? (columns + group - 1) / group : 1;
  const Array all[] = {rows_of(x, rows, columns, x_stride, dtype, false),
                       rows_of(residual, rows, columns, residual_stride, dtype, false),
                       {gain, columns * size_of(gain_dtype), size_of(gain_dtype), false},
                       rows_of(sum, rows, columns, sum_stride, dtype, true),
                       scales ? bytes_of(out, rows, columns, out_stride, 1, true)
                              : rows_of(out, rows, columns, out_stride, dtype, true),
                       {scales, rows * groups * 4, 4, true}};
  const Over may[] = {{3, 0}, {3, 1}, {4, 0}, {4, 1}};
  if ((rc = check_arrays(all, may))) return rc;
  if ((rc = library_device())) return rc;
  const NormArgs a{x, x_stride, residual, residual_stride, rows, (int)columns, gain, gain_dtype, eps, sum, sum_stride,
                   out, out_stride, scales, scales ? group : 0, groups};
  return hip_status(launch_norm(a, dtype, (hipStream_t)stream));
}

int sim_norm_grad_work(int64_t rows, int64_t columns, int dtype, size_t* bytes) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  const int rc = check_norm(rows, columns, dtype, SIM_FP32, 1.0f);
  if (rc) return rc;
  if (!bytes) return SIM_ERR_INVALID_ARG;
  *bytes = (size_t)norm_grad_work_bytes(rows, columns, dtype);
  return SIM_OK;
}

int sim_norm_grad(const void* h, int64_t h_stride, int dtype, int64_t rows, int64_t columns, const void* gain,
                  int gain_dtype, float eps, const void* dy, int64_t dy_stride, const void* dsum, int64_t dsum_stride,
                  void* dx, int64_t dx_stride, float* dgain, void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_norm(rows, columns, dtype, gain_dtype, eps);
  if (rc) return rc;
  if (!rows_fit(rows, columns, h_stride) || !rows_fit(rows, columns, dy_stride) || !rows_fit(rows, columns, dx_stride))
    return SIM_ERR_INVALID_ARG;
  if (dsum && !rows_fit(rows, columns, dsum_stride)) return SIM_ERR_INVALID_ARG;
  if (rows == 0 && !dgain) return SIM_OK;
  if (rows > 0 && (!h || !dy || !dx)) return SIM_ERR_INVALID_ARG;
  const int64_t need = dgain ? norm_grad_work_bytes(rows, columns, dtype) : 0;
  if ((rc = check_work(work, work_bytes, need))) return rc;
  const Array all[] = {rows_of(h, rows, columns, h_stride, dtype, false),
                       rows_of(dy, rows, columns, dy_stride, dtype, false),
                       rows_of(dsum, rows, columns, dsum_stride, dtype, false),
                       {gain, columns * size_of(gain_dtype), size_of(gain_dtype), false},
                       rows_of(dx, rows, columns, dx_stride, dtype, true),
                       {dgain, columns * 4, 4, true},
                       {need ? work : nullptr, need, 4, true}};
  const Over may[] = {{4, 0}, {4, 1}, {4, 2}};
  if ((rc = check_arrays(all, may))) return rc;
  if ((rc = library_device())) return rc;
  const NormGradArgs a{h, h_stride, rows, (int)columns, gain, gain_dtype, eps, dy, dy_stride, dsum, dsum_stride, dx,
                       dx_stride, dgain, (float*)work, norm_grad_workgroups(rows, columns, dtype, dgain != nullptr)};
  return hip_status(launch_norm_grad(a, dtype, (hipStream_t)stream));
}

int sim_dispatch_work(int64_t tokens, int topk, int experts, size_t* bytes) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  const int rc = check_slots(tokens, topk);
  if (rc) return rc;
  if (experts < 1 || experts > SIM_ROUTE_MAX_EXPERTS || !bytes) return SIM_ERR_INVALID_ARG;
  *bytes = (size_t)dispatch_work_bytes(tokens, topk, experts);
  return SIM_OK;
}

int sim_dispatch(const void* x, int64_t x_pitch, int64_t row_bytes, const float* scales, int64_t groups,
                 const int32_t* chosen, int64_t tokens, int topk, int experts, void* rows, int64_t rows_pitch,
                 float* row_scales, int32_t* place, int32_t* offsets, void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_slots(tokens, topk);
  if (rc) return rc;
  if (experts < 1 || experts > SIM_ROUTE_MAX_EXPERTS) return SIM_ERR_INVALID_ARG;
  const int64_t slots = tokens * topk;
  if (!pitch_fits(tokens, row_bytes, x_pitch) || !pitch_fits(slots, row_bytes, rows_pitch)) return SIM_ERR_INVALID_ARG;
  if (groups < 0 || groups > INT32_MAX / 4 || !pitch_fits(slots, groups * 4, groups * 4)) return SIM_ERR_INVALID_ARG;
  if (!offsets || (slots > 0 && (!chosen || !place))) return SIM_ERR_INVALID_ARG;
  if (slots > 0 && row_bytes > 0 && (!x || !rows)) return SIM_ERR_INVALID_ARG;
  if (slots > 0 && groups > 0 && (!scales || !row_scales)) return SIM_ERR_INVALID_ARG;
  const int64_t need = dispatch_work_bytes(tokens, topk, experts);
  if ((rc = check_work(work, work_bytes, need))) return rc;
  const Array all[] = {bytes_of(x, tokens, row_bytes, x_pitch, 1, false),
                       {scales, tokens * groups * 4, 4, false},
                       {chosen, slots * 4, 4, false},
                       bytes_of(rows, slots, row_bytes, rows_pitch, 1, true),
                       {row_scales, slots * groups * 4, 4, true},
                       {place, slots * 4, 4, true},
                       {offsets, ((int64_t)experts + 1) * 4, 4, true},
                       {need ? work : nullptr, need, 4, true}};
  if ((rc = check_arrays(all))) return rc;
  if ((rc = library_device())) return rc;
  DispatchArgs a{x, x_pitch, row_bytes, groups > 0 ? scales : nullptr, groups * 4, chosen, tokens, topk, experts, rows,
                 rows_pitch, row_scales, place, offsets, need ? (uint32_t*)work : nullptr, 0, 0};
  a.chunks = dispatch_chunks(slots, experts, &a.chunk);
  return hip_status(launch_dispatch(a, (hipStream_t)stream));
}

int sim_combine(const void* rows, int64_t rows_stride, int dtype, int64_t nrows, int64_t columns, const int32_t* place,
                const float* weights, int64_t tokens, int topk, void* out, int64_t out_stride, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_slots(tokens, topk);
  if (rc) return rc;
  if (!float_dtype(dtype) || columns > kMaxColumns) return SIM_ERR_INVALID_ARG;
  if (!rows_fit(nrows, columns, rows_stride) || !rows_fit(tokens, columns, out_stride)) return SIM_ERR_INVALID_ARG;
  if (tokens == 0) return SIM_OK;
  if (!place || !out || (nrows > 0 && !rows)) return SIM_ERR_INVALID_ARG;
  const Array all[] = {rows_of(rows, nrows, columns, rows_stride, dtype, false),
                       {place, tokens * topk * 4, 4, false},
                       {weights, tokens * topk * 4, 4, false},
                       rows_of(out, tokens, columns, out_stride, dtype, true)};
  if ((rc = check_arrays(all))) return rc;
  if ((rc = library_device())) return rc;
  const CombineArgs a{rows, rows_stride, nrows, columns, place, weights, tokens, topk, out, out_stride};
  return hip_status(launch_combine(a, dtype, (hipStream_t)stream));
}

int sim_combine_grad(const void* dy, int64_t dy_stride, int dtype, const void* rows, int64_t rows_stride,
                     int64_t nrows, int64_t columns, const int32_t* place, const float* weights, int64_t tokens,
                     int topk, void* drows, int64_t drows_stride, float* dweights, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_slots(tokens, topk);
  if (rc) return rc;
  if (!float_dtype(dtype) || columns > kMaxColumns) return SIM_ERR_INVALID_ARG;
  if (!rows_fit(tokens, columns, dy_stride)) return SIM_ERR_INVALID_ARG;
  if (dweights && !rows_fit(nrows, columns, rows_stride)) return SIM_ERR_INVALID_ARG;
  if (drows && !rows_fit(nrows, columns, drows_stride)) return SIM_ERR_INVALID_ARG;
  if (tokens == 0) return SIM_OK;
  // (a pointer to no rows may be NULL)
  if (!drows && !dweights) return nrows == 0 ? SIM_OK : SIM_ERR_INVALID_ARG;
  if (!dy || !place || (dweights && nrows > 0 && !rows)) return SIM_ERR_INVALID_ARG;
  const Array all[] = {rows_of(dy, tokens, columns, dy_stride, dtype, false),
                       rows_of(dweights ? rows : nullptr, nrows, columns, rows_stride, dtype, false),
                       {place, tokens * topk * 4, 4, false},
                       {weights, tokens * topk * 4, 4, false},
                       rows_of(drows, nrows, columns, drows_stride, dtype, true),
                       {dweights, tokens * topk * 4, 4, true}};
  const Over may[] = {{4, 1}};
  if ((rc = check_arrays(all, may))) return rc;
  if ((rc = library_device())) return rc;
  const CombineGradArgs a{dy, dy_stride, rows, rows_stride, nrows, columns, place, weights, tokens, topk, drows,
                          drows_stride, dweights};
  return hip_status(launch_combine_grad(a, dtype, (hipStream_t)stream));
}

int sim_clip_work(const int64_t* counts, const int* dtypes, int ntensors, size_t* bytes) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  if (ntensors < 0 || ntensors > SIM_CLIP_MAX_TENSORS || !bytes) return SIM_ERR_INVALID_ARG;
  if (ntensors > 0 && (!counts || !dtypes)) return SIM_ERR_INVALID_ARG;
  for (int i = 0; i < ntensors; i++)
    if (!float_dtype(dtypes[i]) || counts[i] < 0 || counts[i] > kMaxBytes / 4 ||
        clip_pieces(counts[i], dtypes[i]) > kMaxPieces)
      return SIM_ERR_INVALID_ARG;
  *bytes = (size_t)clip_work_bytes(sizes_of(counts, dtypes, ntensors));
  return SIM_OK;
}

int sim_clip_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int ntensors, float* norm,
                  void* work, size_t work_bytes, void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_list(grads, counts, dtypes, ntensors);
  if (rc) return rc;
  if (!norm) return SIM_ERR_INVALID_ARG;
  if ((uintptr_t)norm & 3u) return SIM_ERR_ALIGN;
  const Sizes sizes = sizes_of(counts, dtypes, ntensors);
  const int64_t need = clip_work_bytes(sizes);
  if ((rc = check_work(work, work_bytes, need, 8))) return rc;
  try {
    std::vector<Extent> v;
    v.reserve((size_t)ntensors + 2);
    for (int i = 0; i < ntensors; i++) add_extent(v, grads[i], counts[i] * size_of(dtypes[i]), false);
    add_extent(v, norm, 4, true);
    add_extent(v, work, need, true);
    if (any_overlap(v)) return SIM_ERR_ALIAS;
  } catch (const std::bad_alloc&) {
    return SIM_ERR_NOMEM;
  }
  if ((rc = library_device())) return rc;
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = squares_of_list(grads, counts, dtypes, ntensors, (double*)work, s);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(launch_clip_join(ClipNorm{(const double*)work, sizes.squares, nullptr, 0, 0.0f, norm, 0, nullptr, nullptr}, s));
}

int sim_clip(const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes, int ntensors,
             const float* parts, int nparts, float max_norm, float* norm, void* work, size_t work_bytes,
             void* stream) {
  if (!library_ready()) return SIM_ERR_NOT_INIT;
  int rc = check_list(grads, counts, dtypes, ntensors);
  if (rc) return rc;
  if (!norm || !(max_norm >= 0.0f) || (parts ? nparts < 1 || nparts > (1 << 20) : nparts != 0)) return SIM_ERR_INVALID_ARG;
  if (((uintptr_t)norm | (uintptr_t)parts) & 3u) return SIM_ERR_ALIGN;
  bool in_place = true;
  for (int i = 0; outs && i < ntensors; i++) {
    if (counts[i] == 0) continue;
    if (!outs[i]) return SIM_ERR_INVALID_ARG;
    if ((uintptr_t)outs[i] & (uintptr_t)(size_of(dtypes[i]) - 1)) return SIM_ERR_ALIGN;
    in_place = in_place && outs[i] == grads[i];
  }
  const Sizes sizes = sizes_of(counts, dtypes, ntensors);
  const int64_t need = parts ? 0 : clip_work_bytes(sizes);
  if ((rc = check_work(work, work_bytes, need, 8))) return rc;
  try {
    std::vector<Extent> v;
    v.reserve(2 * (size_t)ntensors + 3);
    for (int i = 0; i < ntensors; i++) {
      const int64_t bytes = counts[i] * size_of(dtypes[i]);
      const bool same = !outs || outs[i] == grads[i];
      add_extent(v, grads[i], bytes, same);
      if (!same) add_extent(v, outs[i], bytes, true);
    }
    add_extent(v, parts, 4 * (int64_t)nparts, false);
    add_extent(v, norm, 4, true);
    add_extent(v, need ? work : nullptr, need, true);
    if (any_overlap(v)) return SIM_ERR_ALIAS;
  } catch (const std::bad_alloc&) {
    return SIM_ERR_NOMEM;
  }
  if ((rc = library_device())) return rc;
  const hipStream_t s = (hipStream_t)stream;
  double* squares = (double*)work;
  hipError_t e = hipSuccess;
  ClipNorm n{squares, parts ? 0 : sizes.squares, parts, nparts, max_norm, norm, in_place, nullptr, nullptr};
  if (!parts && (e = squares_of_list(grads, counts, dtypes, ntensors, squares, s)) != hipSuccess) return hip_status(e);
  if (sizes.launches != 1 || sizes.pieces > kJoinPieces) {
    // the norm by itself, read by every workgroup that scales
    n.keep = parts || sizes.squares == 0 ? nullptr : squares;
    if ((e = launch_clip_join(n, s)) != hipSuccess) return hip_status(e);
    n = n.keep ? ClipNorm{squares, 0, nullptr, 0, max_norm, nullptr, in_place, squares, nullptr}
               : ClipNorm{nullptr, 0, norm, 1, max_norm, nullptr, in_place, nullptr, nullptr};
  }
  for (int i = 0; i < ntensors;) {
    ClipList l;
    take(l, i, grads, outs, counts, dtypes, ntensors);
    if (l.tensors == 0) break;
    if ((e = launch_clip_scale(l, n, s)) != hipSuccess) return hip_status(e);
  }
  return SIM_OK;
}

}  // extern "C"
