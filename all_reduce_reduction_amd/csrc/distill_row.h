// distill_row.h -- a distillation step with one workgroup per row (gfx950):
// the row is read once, stays in registers while its maximum and sum are
// found, and its gradient is written from there, so that a step moves the
// logits' bytes twice instead of three times.
//
// A workgroup of NT threads holds R 16-byte vectors per thread: 16 vectors
// are 64 of the 128 VGPRs that four waves per SIMD leave, and 1024 threads of
// them hold a row of 256 KiB (131,072 16-bit logits).  What a row has beyond
// NT * R vectors is read a second time for its gradient.
//
// While the row's loads are in flight, wave 0 reads the slots and their own
// logits.
#pragma once

#include "distill_device.h"
#include "launch.h"

namespace simar {

// of the R vectors of a thread, the last GUARD may lie past the row's end
template <int DT, int NT, int R, int GUARD>
__global__ void __launch_bounds__(NT, 4) k_distill_row(DistillArgs a) {
  constexpr int V = epv<DT>(), W = NT / 64, PAIR = R % 2 ? 1 : 2;
  constexpr bool STREAM = NT < 1024;
  __shared__ SlotLists<NT> slots;
  __shared__ float m_s[W], s_s[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const void* x = row_at(a.x, row, a.stride, Ty<DT>::E);
  void* dx = row_at(a.dx, row, a.dstride, Ty<DT>::E);
  const float c = kLog2e / a.tau;
  const float up = (a.row_scale ? a.row_scale[row] : 1.0f) * (a.coef / a.tau);
  u32x4 v[R];
#pragma unroll
  for (int i = 0; i < R; i++) {
    if (i < R - GUARD) v[i] = ld_row_lane<DT, STREAM>(x, i * NT * V, tid * V);
    else v[i] = ld_guarded<DT>(x, (int64_t)(i * NT + tid) * V, a.cols);
  }
  slots.head[tid] = -1;
  Slots sl;
  if (wave == 0) {
    sl = load_slots(a, row, lane);
    gather_slots<DT>(a, slots, sl, x, 0, a.cols, lane);
  }
  Running r{kNegInf, 0.0f};
#pragma unroll
  for (int i = 0; i < R; i += PAIR) {
    float f[PAIR * V];
#pragma unroll
    for (int j = 0; j < PAIR; j++) unpack<DT>(v[i + j], f + j * V);
    running_add(r, f, c);
  }
  for (int64_t col = (int64_t)(R * NT + tid) * V; col < a.cols; col += NT * V) {
    float f[V];
    load_cols<DT>(x, col, a.cols, f);
    running_add(r, f, c);
  }
  r = wave_running(r, c);
  if (lane == 0) {
    m_s[wave] = r.m;
    s_s[wave] = r.s;
  }
  __syncthreads();
  r.m = lane < W ? m_s[lane] : kNegInf;
  r.s = lane < W ? s_s[lane] : 0.0f;
  r = wave_running(r, c);
  const bool live = slots.live;
  if (wave == 0) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++) {
      if (sl.id[i] < 0 || sl.q[i] == 0.0f) continue;
      const float at = slots.x[lane + 64 * i];
      dot += at == kNegInf ? sl.q[i] * kNegInf : sl.q[i] * ((at - r.m) / a.tau);
    }
    dot = wave_sum(dot);
    if (lane == 0) a.loss[row] = live ? sl.entropy + __logf(r.s) - dot : 0.0f;
    hang_slots<DT>(a, slots, sl, 0, a.cols, r.m, r.s, c, lane);
  }
  const float k2 = live ? up / r.s : 0.0f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; i++) {
    // widened again here: kept from above, the fp32 values would take the
    // registers of two more rows
    asm volatile("" : "+v"(v[i]));
    float f[V];
    unpack<DT>(v[i], f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = live ? exp2_hw((f[j] - r.m) * c) * k2 : 0.0f;
    if (i < R - GUARD) st_row_lane<DT, STREAM>(dx, i * NT * V, tid * V, pack<DT>(f));
    else st_guarded<DT>(dx, (int64_t)(i * NT + tid) * V, a.cols, f);
  }
  for (int64_t col = (int64_t)(R * NT + tid) * V; col < a.cols; col += NT * V) {
    float f[V];
    load_cols<DT>(x, col, a.cols, f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = live ? exp2_hw((f[j] - r.m) * c) * k2 : 0.0f;
    st_guarded<DT>(dx, col, a.cols, f);
  }
  write_slots<DT>(a, slots, dx, up, tid);
}

// The workgroup and the vectors per thread for a row of n vectors: the
// smallest workgroup that holds it in 16 vectors per thread.  R comes in
// steps of 2 from 4 on, so the last two vectors of a thread may lie past the
// row's end.
template <int DT, int NT, int R>
hipError_t launch_row_as(const DistillArgs& a, hipStream_t s) {
  constexpr int G = R < 4 ? 1 : 2;
  return launch<k_distill_row<DT, NT, R, G>>(dim3((unsigned)a.rows), dim3(NT), s, a);
}
template <int DT, int NT, bool SHORT>
hipError_t launch_row_with(const DistillArgs& a, int64_t vectors, hipStream_t s) {
  const int r = (int)((vectors + NT - 1) / NT);
  if constexpr (SHORT) {
    if (r <= 1) return launch_row_as<DT, NT, 1>(a, s);
    if (r <= 2) return launch_row_as<DT, NT, 2>(a, s);
    if (r <= 3) return launch_row_as<DT, NT, 3>(a, s);
  }
  if (r <= 4) return launch_row_as<DT, NT, 4>(a, s);
  if (r <= 6) return launch_row_as<DT, NT, 6>(a, s);
  if (r <= 8) return launch_row_as<DT, NT, 8>(a, s);
  if (r <= 10) return launch_row_as<DT, NT, 10>(a, s);
  if (r <= 12) return launch_row_as<DT, NT, 12>(a, s);
  if (r <= 14) return launch_row_as<DT, NT, 14>(a, s);
  return launch_row_as<DT, NT, 16>(a, s);
}
template <int DT>
hipError_t launch_row(const DistillArgs& a, hipStream_t s) {
  const int64_t n = (a.cols + epv<DT>() - 1) / epv<DT>();
  if (n <= 64 * 16) return launch_row_with<DT, 64, true>(a, n, s);
  if (n <= 256 * 16) return launch_row_with<DT, 256, false>(a, n, s);
  if (n <= 512 * 16) return launch_row_with<DT, 512, false>(a, n, s);
  return launch_row_with<DT, 1024, false>(a, n, s);
}

}  // namespace simar
