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
// Wave 0 asks for the slots before it asks for its share of the row, and works
// them out and reads their own logits while the row is in flight.
//
// Bound by memory that reads and writes at once: 785 us for 8,192 rows x
// 131,072 bf16 (5.5 TB/s; a copy of as many bytes 666), 95 us for 2,048 x 65,536
// (5.6 TB/s; 83); the vector units take 330 us of the 785.  Tried and slower:
// the whole grid meeting between reading and writing (1,040 us: the exponentials
// then overlap with neither), the next row's loads among this row's stores
// (858), the rows' starts rotated against each other (803).
#pragma once

#include "distill_device.h"
#include "launch.h"

namespace simar {

// of the R vectors of a thread, the last GUARD may lie past the row's end; a
// row is longer than one vector
template <int DT, int NT, int R, int GUARD, bool STREAM>
__global__ void __launch_bounds__(NT, 4) k_distill_row(DistillArgs a) {
  constexpr int V = epv<DT>(), W = NT / 64, PAIR = R % 2 ? 1 : 2;
  static_assert((R - GUARD) % PAIR == 0, "a pair lies wholly before the guarded vectors or among them");
  __shared__ SlotLists<NT> slots;
  __shared__ float m_s[W], s_s[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const void* row_x = row_at(a.x, row, a.stride, Ty<DT>::E);
  void* row_dx = row_at(a.dx, row, a.dstride, Ty<DT>::E);
  const uint32_t lone = lone_columns<DT>(row_x), cols = (uint32_t)a.cols - lone;
  const void* x = (const char*)row_x + lone * Ty<DT>::E;
  void* dx = (char*)row_dx + lone * Ty<DT>::E;
  const float c = kLog2e / a.tau;
  const float up = (a.row_scale ? a.row_scale[row] : 1.0f) * (a.coef / a.tau);
  const SlotLoads asked = ask_slots(a, row, lane, wave == 0);
  u32x4 v[R];
  auto load = [&](int i) __attribute__((always_inline)) {
    if (i < R - GUARD) v[i] = ld_row_lane<DT, STREAM>(x, i * NT * V, tid * V);
    else v[i] = Tail<DT>(i * NT * V + tid * V, cols).load(x);
  };
  // The first EARLY vectors are asked for before it is known whether the row
  // has slots, so that this costs no time; the others only if it has.
  constexpr int EARLY = R < 8 ? R : 4;
#pragma unroll
  for (int i = 0; i < EARLY; i++) load(i);
  if (!has_slots(a, asked)) {
    const float f[V] = {};
    for (uint32_t col = tid * V; col < cols; col += NT * V) Tail<DT>(col, cols).store(dx, f);
    if (tid == 0) a.loss[row] = 0.0f;
    if (tid == 0 && lone) store_elem<DT>(row_dx, 0, 0.0f);
    return;
  }
#pragma unroll
  for (int i = EARLY; i < R; i++) load(i);
  slots.head[tid] = -1;
  Slots sl;
  if (wave == 0) {
    sl = make_slots(a, asked);
    gather_slots<DT>(a, slots, sl, row_x, 0, a.cols, lane);
  }
  Scan scan;
  const float alone = lone && tid == 0 ? load_elem<DT>(row_x, 0) : kNegInf;
#pragma unroll
  for (int i = 0; i < R; i += PAIR) {
    if (i < R - GUARD) {
      float f[PAIR * V];
#pragma unroll
      for (int j = 0; j < PAIR; j++) unpack<DT>(v[i + j], f + j * V);
      scan.add(f, c);
    } else {
#pragma unroll
      for (int j = 0; j < PAIR; j++) {
        float f[V];
        unpack<DT>(v[i + j], f);
        Tail<DT>((i + j) * NT * V + lane_offset(tid * V), cols).mask(f);
        scan.add(f, c);
      }
    }
  }
  for (uint32_t col = (uint32_t)(R * NT + tid) * V; col < cols; col += NT * V) {
    const Tail<DT> t(col, cols);
    float f[V];
    unpack<DT>(t.load(x), f);
    t.mask(f);
    scan.add(f, c);
  }
  if (lone) scan.add({alone}, c);
  Running r = wave_running(scan.done(c), c);
  if (lane == 0) {
    m_s[wave] = r.m;
    s_s[wave] = r.s;
  }
  __syncthreads();
  r.m = lane < W ? m_s[lane] : kNegInf;
  r.s = lane < W ? s_s[lane] : 0.0f;
  r = wave_running(r, c);
  if (__builtin_expect(far(r.m, c), 0)) {
    float n = alone == r.m ? 1.0f : 0.0f;
#pragma unroll 1
    for (uint32_t col = tid * V; col < cols; col += NT * V) {
      const Tail<DT> t(col, cols);
      float f[V];
      unpack<DT>(t.load(x), f);
      t.mask(f);
      n += count_of(f, r.m);
    }
    n = wave_sum(n);
    __syncthreads();
    if (lane == 0) s_s[wave] = n;
    __syncthreads();
    r.s += wave_sum(lane < W ? s_s[lane] : 0.0f);
  }
  const bool live = slots.live;
  const Against top = against(r.m, c);
  const float sum = r.s * exp2_hw(at_max(r.m, top));  // against top.t
  if (wave == 0) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++) {
      if (64 * i >= a.topk) break;
      if (sl.id[i] < 0 || sl.q[i] == 0.0f) continue;
      const float at = slots.x[lane + 64 * i];
      dot += at == kNegInf ? sl.q[i] * kNegInf : times_distance(sl.q[i], at, r.m, a.tau);
    }
    dot = wave_sum(dot);
    if (lane == 0) a.loss[row] = live ? sl.entropy + __logf(r.s) - dot : 0.0f;
    hang_slots<DT>(a, slots, sl, 0, a.cols, lone, top, sum, lane);
  }
  const float k2 = up / sum;
  __syncthreads();
  if (!live) {
    // (0 * p would keep the NaN of a row that does not count)
    const float f[V] = {};
    for (uint32_t col = tid * V; col < cols; col += NT * V) Tail<DT>(col, cols).store(dx, f);
    if (tid == 0 && lone) store_elem<DT>(row_dx, 0, 0.0f);
    return;
  }
  if (tid == 0 && lone) store_elem<DT>(row_dx, 0, exp_against(alone, top) * k2);
#pragma unroll
  for (int i = 0; i < R; i++) {
    // widened again here: kept from above, the fp32 values would take the
    // registers of two more rows
    asm volatile("" : "+v"(v[i]));
    float f[V];
    unpack<DT>(v[i], f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = exp_against(f[j], top) * k2;
    if (i < R - GUARD) st_row_lane<DT, STREAM>(dx, i * NT * V, tid * V, pack_rounded<DT>(f));
    else Tail<DT>(i * NT * V + lane_offset(tid * V), cols).store(dx, f);
  }
  for (uint32_t col = (uint32_t)(R * NT + tid) * V; col < cols; col += NT * V) {
    const Tail<DT> t(col, cols);
    float f[V];
    unpack<DT>(t.load(x), f);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = exp_against(f[j], top) * k2;
    t.store(dx, f);
  }
  write_slots<DT>(a, slots, row_dx, up, tid);
}

// The workgroup, the vectors per thread (R, in steps of 2 from 4 on, so that
// the last two of a thread may lie past the row's end) and the cache policy
// for a row of n vectors, measured on MI355X (us, bf16):
//   - fewer rows than compute units: the largest workgroup, as a row's own time
//     counts (256 rows x 32,768: 1024 threads 11.8, 256 threads 18.3);
//   - rows of up to 32 KiB, any number: cached accesses, small workgroups
//     (32,768 x 8,192: 193, streaming 264), of one wave up to 8 KiB, as a
//     row's steps wait for each other and more rows are then under way
//     (16,384 x 2,560: 38.5, 256 threads 54; 8,192 x 8,000 in 64 threads of
//     16 vectors 54.7, in 256 50.2);
//   - longer rows, less than 512 MiB of them: streaming accesses and the
//     smallest workgroup that holds a row in 16 vectors per thread, so that
//     several share a compute unit and one reads while another computes or
//     writes (2,048 x 65,536: 93, cached 107, 1024 threads 104);
//   - 512 MiB and more, which the 256 MiB memory-side cache helps little:
//     cached accesses and one workgroup per compute unit, whose reads and
//     writes come in long runs (16,384 x 32,768: 407, cached in small
//     workgroups 444, streaming in them 494).
template <int DT, int NT, int R, bool STREAM>
hipError_t launch_row_as(const DistillArgs& a, hipStream_t s) {
  constexpr int G = R % 2 ? 1 : 2;
  // the kernel reads the first R - G vectors of every thread unchecked
  if (a.cols <= (int64_t)(R - G) * NT * epv<DT>() || a.cols <= epv<DT>()) return hipErrorInvalidValue;
  return launch<k_distill_row<DT, NT, R, G, STREAM>>(dim3((unsigned)a.rows), dim3(NT), s, a);
}
// the smallest R of LEAST, ..., MOST that holds the row (MOST where none does)
template <int DT, int NT, bool STREAM, int LEAST, int MOST>
hipError_t launch_row_with(const DistillArgs& a, int64_t vectors, hipStream_t s) {
  if constexpr (LEAST < MOST) {
    constexpr int NEXT = LEAST < 4 ? LEAST + 1 : LEAST + 2;
    if (vectors > (int64_t)NT * LEAST) return launch_row_with<DT, NT, STREAM, NEXT, MOST>(a, vectors, s);
  }
  return launch_row_as<DT, NT, LEAST, STREAM>(a, s);
}
template <int DT>
hipError_t launch_row(const DistillArgs& a, hipStream_t s) {
  const int64_t n = (a.cols + epv<DT>() - 1) / epv<DT>();
  const bool few = a.rows <= library_cus();
  if (n <= 2048) {
    if (few && n > 512) return launch_row_with<DT, 1024, false, 1, 2>(a, n, s);
    if (!few && n <= 512) return launch_row_with<DT, 64, false, 1, 8>(a, n, s);
    return launch_row_with<DT, 256, false, 1, 8>(a, n, s);
  }
  if (!few && a.rows * a.cols * Ty<DT>::E >= ((int64_t)512 << 20))
    return launch_row_with<DT, 1024, false, 3, 16>(a, n, s);
  if (few || n > 8192) return launch_row_with<DT, 1024, true, 3, 16>(a, n, s);
  return n <= 4096 ? launch_row_with<DT, 256, true, 10, 16>(a, n, s) : launch_row_with<DT, 512, true, 10, 16>(a, n, s);
}

}  // namespace simar
