// k_distill.hip -- distillation from a teacher's top logits (gfx950).
//
// With q the softmax of the teacher's slots and p the softmax of the
// student's row x (both at temperature tau),
//   loss = sum_k q_k (log q_k - log p[id_k])
//        = sum_k q_k log q_k + A log S - sum_k q_k (x[id_k] - M) / tau,
//   dx_v = coef row_scale / tau (p_v - sum over slots with id v of q_k),
// where M is the row's largest logit, S the sum of exp((x - M) / tau) and A
// the sum of q (1, or 0 for a row without slots).  A run of columns leaves its
// part: its own maximum m, its sum s against m, the slots' mass a in it and
// d = sum q (x - m) / tau over them; parts join by rebasing to the largest m,
// in the order of the columns.  All of it in fp32; a gradient is rounded once.
#include "distill_device.h"
#include "launch.h"

namespace simar {
namespace {

template <int DT>
__global__ void __launch_bounds__(kBlock) k_distill_stats(DistillArgs a) {
  constexpr int V = epv<DT>(), W = kBlock / 64;
  __shared__ Running run[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int64_t lo = split * a.span, hi = min(a.cols, lo + a.span);
  const void* x = row_at(a.x, row, a.stride, Ty<DT>::E);
  const float c = kLog2e / a.tau;
  Slots sl;
  float at[kSlotsPerLane];
  if (wave == 0) {
    sl = load_slots(a, row, lane);
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++) {
      const int64_t col = (int64_t)sl.id[i] - a.first;
      const bool here = sl.id[i] >= 0 && col >= lo && col < hi;
      at[i] = here ? load_elem<DT>(x, col) : 0.0f;
      if (!here) sl.q[i] = 0.0f;
    }
  }
  Running r{kNegInf, 0.0f};
  for (int64_t col = lo + (int64_t)tid * V; col < hi; col += kBlock * V) {
    float v[V];
    load_cols<DT>(x, col, hi, v);
    running_add(r, v, c);
  }
  r = wave_running(r, c);
  if (lane == 0) run[wave] = r;
  __syncthreads();
  if (wave == 0) {
    r = run[0];
#pragma unroll
    for (int w = 1; w < W; w++) r = running_join(r, run[w], c);
    float mass = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++) {
      if (sl.q[i] == 0.0f) continue;
      mass += sl.q[i];
      dot += at[i] == kNegInf ? sl.q[i] * kNegInf : sl.q[i] * ((at[i] - r.m) / a.tau);
    }
    mass = wave_sum(mass);
    dot = wave_sum(dot);
    if (lane == 0) {
      a.parts[part_index(split, 0, a.rows, row)] = r.m;
      a.parts[part_index(split, 1, a.rows, row)] = r.s;
      a.parts[part_index(split, 2, a.rows, row)] = mass;
      a.parts[part_index(split, 3, a.rows, row)] = dot;
    }
  }
}

// one wave per row
__global__ void __launch_bounds__(kBlock) k_distill_join(DistillArgs a, float* loss, float* norm) {
  const int64_t row = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63;
  const Slots s = load_slots(a, row, lane);
  const Part t = join_parts(a.parts, a.splits, a.rows, row, a.tau);
  if (lane == 0) {
    loss[row] = loss_of(s, t);
    norm[row] = t.m;
    norm[a.rows + row] = t.s;
  }
}

// one thread per row
__global__ void __launch_bounds__(kBlock) k_distill_merge(DistillArgs a, float* out) {
  const int64_t row = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (row >= a.rows) return;
  const Part t = join_parts(a.parts, a.splits, a.rows, row, a.tau);
  out[row] = t.m;
  out[a.rows + row] = t.s;
  out[2 * a.rows + row] = t.a;
  out[3 * a.rows + row] = t.d;
}

// The gradient of a run of columns.  First the slots' own logits are read
// (the gradient may lie on the logits), then every column gets scale * p,
// and last each slot's column its full value; slots with one id each write
// the same one.
template <int DT>
__global__ void __launch_bounds__(kBlock) k_distill_grad(DistillArgs a) {
  constexpr int V = epv<DT>();
  __shared__ int id_s[SIM_DISTILL_MAX_TOPK];
  __shared__ float q_s[SIM_DISTILL_MAX_TOPK];
  __shared__ int live_s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int64_t lo = split * a.span, hi = min(a.cols, lo + a.span);
  const void* x = row_at(a.x, row, a.stride, Ty<DT>::E);
  void* dx = row_at(a.dx, row, a.dstride, Ty<DT>::E);
  const float c = kLog2e / a.tau;
  Part t{};
  if (a.norm) {
    t.m = a.norm[row];
    t.s = a.norm[a.rows + row];
  } else {
    t = join_parts(a.parts, a.splits, a.rows, row, a.tau);
  }
  if (wave == 0) {
    const Slots sl = load_slots(a, row, lane);
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++)
      if (lane + 64 * i < a.topk) {
        id_s[lane + 64 * i] = sl.id[i];
        q_s[lane + 64 * i] = sl.q[i];
      }
    if (lane == 0) {
      live_s = sl.live;
      if (a.loss && split == 0) a.loss[row] = loss_of(sl, t);
    }
  }
  __syncthreads();
  const bool live = live_s;
  const float scale = live ? (a.row_scale ? a.row_scale[row] : 1.0f) * (a.coef / a.tau) : 0.0f;
  const float inv = live ? scale / t.s : 0.0f;
  int64_t own = -1;
  float value = 0.0f;
  if (tid < a.topk && live) {
    const int64_t col = (int64_t)id_s[tid] - a.first;
    if (id_s[tid] >= 0 && col >= lo && col < hi) {
      own = col;
      float q = 0.0f;
      for (int k = 0; k < a.topk; k++)
        if (id_s[k] == id_s[tid]) q += q_s[k];
      value = scale * (exp2_hw((load_elem<DT>(x, col) - t.m) * c) / t.s - q);
    }
  }
  __syncthreads();
  for (int64_t col = lo + (int64_t)tid * V; col < hi; col += kBlock * V) {
    float v[V];
    if (live) {
      load_cols<DT>(x, col, hi, v);
#pragma unroll
      for (int i = 0; i < V; i++) v[i] = exp2_hw((v[i] - t.m) * c) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) v[i] = 0.0f;
    }
    if (col + V <= hi) {
      st_row<DT>(dx, col, pack<DT>(v));
    } else {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (col + i < hi) store_elem<DT>(dx, col + i, v[i]);
    }
  }
  __syncthreads();
  if (own >= 0) store_elem<DT>(dx, own, value);
}

}  // namespace

bool distill_whole_rows(int64_t rows, int64_t cols, int dtype) {
  (void)cols;
  (void)dtype;
  return rows >= library_cus();
}
int distill_splits(int64_t rows, int64_t cols, int dtype) {
  (void)dtype;
  const int64_t most = (cols + kBlock * 8 - 1) / (kBlock * 8);
  const int64_t want = rows > 0 ? (2 * (int64_t)library_cus() + rows - 1) / rows : 1;
  return (int)(want < most ? want : most);
}
int64_t distill_span(int64_t cols, int splits) {
  const int64_t v = (cols + splits - 1) / splits;
  return (v + 7) / 8 * 8;
}

#define BY_DTYPE(K, ...)                                          \
  switch (dtype) {                                                \
    case SIM_FP32: return launch<K<SIM_FP32>>(__VA_ARGS__);       \
    case SIM_FP16: return launch<K<SIM_FP16>>(__VA_ARGS__);       \
    default: return launch<K<SIM_BF16>>(__VA_ARGS__);             \
  }

hipError_t launch_distill_stats(const DistillArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)(a.rows * a.splits)), block(kBlock);
  BY_DTYPE(k_distill_stats, grid, block, s, a)
}
hipError_t launch_distill_grad(const DistillArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)(a.rows * a.splits)), block(kBlock);
  BY_DTYPE(k_distill_grad, grid, block, s, a)
}
hipError_t launch_distill_join(const DistillArgs& a, float* loss, float* norm, hipStream_t s) {
  return launch<k_distill_join>(dim3((unsigned)((a.rows + 3) / 4)), dim3(kBlock), s, a, loss, norm);
}
hipError_t launch_distill_merge(const DistillArgs& a, float* out, hipStream_t s) {
  return launch<k_distill_merge>(dim3((unsigned)((a.rows + kBlock - 1) / kBlock)), dim3(kBlock), s, a, out);
}

}  // namespace simar
