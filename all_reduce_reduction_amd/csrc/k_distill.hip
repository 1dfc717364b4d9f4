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
#include <type_traits>

#include "distill_device.h"
#include "launch.h"

namespace simar {
namespace {

// A workgroup's columns [lo, hi) of a row come in chunks of kHeld vectors per
// thread, whose loads are all in flight together: whole chunks (WHOLE), then
// one that ends at hi.  There each vector is the row's last where its own
// would reach past the row (see Tail), so that no load waits for a branch.
// TINY: rows of a vector or less, element by element.  Four vectors: a
// gradient's workgroup of 16 KiB ends sooner, so that fewer reads and writes of
// different runs meet in memory (4,096 x 50,021 bf16: 145 us; with eight 157,
// with two 155).
constexpr int kHeld = 4;
template <int DT, int B> constexpr uint32_t chunk_cols() { return kHeld * B * epv<DT>(); }
// `lone`: column 0 by itself before lo, thread 0's (see lone_columns).
struct Columns {
  uint32_t lo, hi, cols;
  bool lone;
  __device__ __forceinline__ int64_t first() const { return lone ? 0 : lo; }
};
template <int DT, bool TINY>
__device__ __forceinline__ Columns columns_of(const DistillArgs& a, const void* row, int64_t split) {
  const int64_t off = TINY ? 0 : lone_columns<DT>(row);
  const int64_t lo = min(a.cols, split * a.span + off), hi = min(a.cols, (split + 1) * a.span + off);
  return {(uint32_t)lo, (uint32_t)hi, (uint32_t)a.cols, off != 0 && split == 0};
}
// (a thread's place is worked out at each use: kept for all vectors of a chunk,
// it would take more registers than the vectors)
template <int DT, int B>
__device__ __forceinline__ Tail<DT> tail(uint32_t col, int i, int tid, const Columns& r) {
  constexpr int V = epv<DT>();
  return Tail<DT>(col + i * B * V + lane_offset(tid * V), r.hi, r.cols);
}
template <int DT, int B, bool WHOLE, bool TINY>
__device__ __forceinline__ void load_chunk(const void* x, uint32_t col, int tid, const Columns& r,
                                           u32x4 (&v)[kHeld]) {
  constexpr int V = epv<DT>();
#pragma unroll
  for (int i = 0; i < kHeld; i++) {
    if constexpr (TINY) v[i] = ld_guarded<DT>(x, (i * B + tid) * V, r.cols);
    else if constexpr (WHOLE) v[i] = ld_row_lane<DT, true>(x, col + i * B * V, tid * V);
    else v[i] = tail<DT, B>(col, i, tid, r).load(x);
  }
}
// All chunks: load, `first` behind the first loads, use(v, col, whole).  A
// last chunk of one vector per thread or less is asked for with the first, so
// that it costs no wait of its own.
template <int DT, int B, bool TINY, class First, class Use>
__device__ __forceinline__ void each_chunk(const void* x, int tid, const Columns& r, First first, Use use) {
  constexpr uint32_t chunk = chunk_cols<DT, B>();
  uint32_t col = r.lo;
  u32x4 v[kHeld];
  if (!TINY && col + chunk <= r.hi) {
    const uint32_t last = r.hi - (r.hi - r.lo) % chunk;
    load_chunk<DT, B, true, false>(x, col, tid, r, v);
    u32x4 few[1] = {tail<DT, B>(last, 0, tid, r).load(x)};
    first();
    use(v, col, std::true_type());
#pragma unroll 1
    for (col += chunk; col < last; col += chunk) {
      load_chunk<DT, B, true, false>(x, col, tid, r, v);
      use(v, col, std::true_type());
    }
    if (last + B * epv<DT>() >= r.hi) {
      use(few, last, std::false_type());
      return;
    }
    load_chunk<DT, B, false, TINY>(x, last, tid, r, v);
  } else {
    load_chunk<DT, B, false, TINY>(x, col, tid, r, v);
    first();
  }
  use(v, col, std::false_type());
}

// Bound by the read: 24 to 27 us for 4,096 rows x 16,384 bf16 (5.0 to 5.6 TB/s),
// 67 us for 4,096 x 50,021 (6.1 TB/s).  Workgroups of B threads: 256, as many of
// them share a compute unit (512: 47 us for 4,096 x 16,385 against 30), unless
// the rows are few or short (see stats_dtype).
template <int DT, int B, bool TINY>
__global__ void __launch_bounds__(B) k_distill_stats(DistillArgs a) {
  constexpr int V = epv<DT>(), W = B / 64;
  __shared__ float m_s[W], s_s[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const void* x = row_at(a.x, row, a.stride, Ty<DT>::E);
  const Columns range = columns_of<DT, TINY>(a, x, split);
  const float c = kLog2e / a.tau;
  const SlotLoads asked = ask_slots(a, row, lane, wave == 0);
  if (a.look_first && !has_slots(a, asked)) {
    if (tid < 4) a.parts[part_index(split, tid, a.rows, row)] = tid == 0 ? kNegInf : 0.0f;
    return;
  }
  Slots sl;
  float at[kSlotsPerLane];
  Scan scan;
  const float alone = range.lone && tid == 0 ? load_elem<DT>(x, 0) : kNegInf;
  each_chunk<DT, B, TINY>(
      x, tid, range,
      [&]() __attribute__((always_inline)) {
        if (wave != 0) return;
        sl = make_slots(a, asked);
#pragma unroll
        for (int i = 0; i < kSlotsPerLane; i++) {
          if (64 * i >= a.topk) break;
          const int64_t col = (int64_t)sl.id[i] - a.first;
          const bool here = sl.id[i] >= 0 && col >= range.first() && col < range.hi;
          at[i] = here ? load_elem<DT>(x, col) : 0.0f;
          if (!here) sl.q[i] = 0.0f;
        }
      },
      [&](auto& v, uint32_t col, auto whole) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof v / sizeof v[0]); i++) {
          if (!whole() && col + i * B * V >= range.hi) break;
          float f[V];
          unpack<DT>(v[i], f);
          if (!whole() && !TINY && col + (i + 1) * B * V > range.hi) tail<DT, B>(col, i, tid, range).mask(f);
          scan.add(f, c);
        }
      });
  if (range.lone) scan.add({alone}, c);
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
    float top = alone == r.m ? 1.0f : 0.0f;
    for (int64_t col = range.lo + tid * V; col < range.hi; col += B * V) {
      float f[V];
      load_cols<DT>(x, col, range.hi, f);
      top += count_of(f, r.m);
    }
    top = wave_sum(top);
    __syncthreads();
    if (lane == 0) s_s[wave] = top;
    __syncthreads();
    r.s += wave_sum(lane < W ? s_s[lane] : 0.0f);
  }
  if (wave == 0) {
    float mass = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlotsPerLane; i++) {
      if (64 * i >= a.topk) break;
      if (sl.q[i] == 0.0f) continue;
      mass += sl.q[i];
      dot += at[i] == kNegInf ? sl.q[i] * kNegInf : times_distance(sl.q[i], at[i], r.m, a.tau);
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

// One wave per row, a lane per part: 3.8 us for 333 rows, 5.0 for 4,096, most
// of it the launch and one round trip to memory (a loop over the parts: 11).
__global__ void __launch_bounds__(kBlock) k_distill_join(DistillArgs a, float* loss, float* norm) {
  const int64_t row = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63;
  const Slots s = make_slots(a, ask_slots(a, row, lane, true));
  const Part t = join_parts(a.parts, a.splits, a.rows, row, a.tau, lane);
  if (lane == 0) {
    loss[row] = loss_of(s, t);
    norm[row] = t.m;
    norm[a.rows + row] = t.s;
  }
}

// one wave per row
__global__ void __launch_bounds__(kBlock) k_distill_merge(DistillArgs a, float* out) {
  const int64_t row = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int lane = threadIdx.x & 63;
  const Part t = join_parts(a.parts, a.splits, a.rows, row, a.tau, lane);
  if (lane != 0) return;
  out[row] = t.m;
  out[a.rows + row] = t.s;
  out[2 * a.rows + row] = t.a;
  out[3 * a.rows + row] = t.d;
}

// The gradient of a run of columns, from the row's joined parts or its norm.
// Bound by reading and writing at once: 48 us for 4,096 rows x 16,384 bf16 (5.5
// TB/s; a copy of as many bytes 42).
template <int DT, int B, bool TINY>
__global__ void __launch_bounds__(B) k_distill_grad(DistillArgs a) {
  constexpr int V = epv<DT>();
  __shared__ SlotLists<B> slots;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const void* x = row_at(a.x, row, a.stride, Ty<DT>::E);
  const Columns range = columns_of<DT, TINY>(a, x, split);
  void* dx = row_at(a.dx, row, a.dstride, Ty<DT>::E);
  const float c = kLog2e / a.tau;
  const float up = (a.row_scale ? a.row_scale[row] : 1.0f) * (a.coef / a.tau);
  const SlotLoads asked = ask_slots(a, row, lane, wave == 0);
  if (a.look_first && !has_slots(a, asked)) {
    const float f[V] = {};
    for (uint32_t col = range.lo + tid * V; col < range.hi; col += B * V) st_guarded<DT>(dx, col, range.hi, f);
    if (range.lone && tid == 0) store_elem<DT>(dx, 0, 0.0f);
    if (a.loss && split == 0 && tid == 0) a.loss[row] = 0.0f;
    return;
  }
  slots.head[tid] = -1;
  Part t{};
  if (a.norm) {
    t.m = a.norm[row];
    t.s = a.norm[a.rows + row];
  } else {
    t = join_parts(a.parts, a.splits, a.rows, row, a.tau, lane);
  }
  const Against top = against(t.m, c);
  const float sum = t.s * exp2_hw(at_max(t.m, top));  // against top.t
  const float k2 = up / sum;
  bool live = true;
  const float alone = range.lone && tid == 0 ? load_elem<DT>(x, 0) : kNegInf;
  each_chunk<DT, B, TINY>(
      x, tid, range,
      [&]() __attribute__((always_inline)) {
        __syncthreads();
        if (wave == 0) {
          const Slots sl = make_slots(a, asked);
          gather_slots<DT>(a, slots, sl, x, range.first(), range.hi, lane);
          wave_fence();
          if (lane == 0 && a.loss && split == 0) a.loss[row] = loss_of(sl, t);
          hang_slots<DT>(a, slots, sl, range.first(), range.hi, range.lo, top, sum, lane);
        }
        __syncthreads();
        live = slots.live;
      },
      [&](auto& v, uint32_t col, auto whole) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof v / sizeof v[0]); i++) {
          if (!whole() && col + i * B * V >= range.hi) break;
          float f[V];
          unpack<DT>(v[i], f);
          // (0 * p would keep the NaN of a row that does not count)
#pragma unroll
          for (int j = 0; j < V; j++) f[j] = live ? exp_against(f[j], top) * k2 : 0.0f;
          if (whole()) st_row_lane<DT, true>(dx, col + i * B * V, tid * V, pack_rounded<DT>(f));
          else if (!TINY) tail<DT, B>(col, i, tid, range).store(dx, f);
          else st_guarded<DT>(dx, (i * B + tid) * V, range.cols, f);
        }
      });
  if (range.lone && tid == 0) store_elem<DT>(dx, 0, live ? exp_against(alone, top) * k2 : 0.0f);
  write_slots<DT>(a, slots, dx, up, tid);
}

}  // namespace

// A step takes one workgroup per row where that holds the row in registers, or
// where half the compute units have a row each; two launches over runs of
// columns otherwise (they read the row twice, but by more workgroups).  Measured
// (us, bf16, whole / runs): 1 row x 32,768 6.2 / 9.2, 160 x 200,003 31.8 / 46.4,
// 64 x 200,003 27.6 / 21.6.  Both limits are round numbers, and near them the
// other side can be the faster one: 1 x 131,072 14.2 / 9.5, 64 x 131,072 16.6 /
// 15.5, 127 x 200,003 29.4 / 35.6.
bool distill_whole_rows(int64_t rows, int64_t cols, int dtype) {
  const int v = dtype == SIM_FP32 ? 4 : 8;
  if (cols <= v) return false;
  return (cols + v - 1) / v <= 16 * 1024 || rows >= library_cus() / 2;
}
// Workgroups per row: enough for two per compute unit, each with at least
// `least` columns.
int distill_splits(int64_t rows, int64_t cols, int64_t least) {
  const int64_t most = (cols + least - 1) / least;
  const int64_t want = rows > 0 ? (2 * (int64_t)library_cus() + rows - 1) / rows : 1;
  return (int)(want < most ? want : most);
}
int64_t distill_span(int64_t cols, int splits) {
  const int64_t v = (cols + splits - 1) / splits;
  return (v + 7) / 8 * 8;
}

// Many short runs, of at most `chunks` chunks of one wave, take a workgroup of
// one wave each: a run's steps wait for each other, and more runs are then under
// way (8,192 rows x 1,000 bf16: statistics 8.8 us, gradient 11.7; 256 threads
// 19.5 and 21.2).  A run that is only read pays longer (8,192 x 8,192: 25.9, 256
// threads 32.5; 4,096 x 16,384: 25.7 and 26.2) than one that is written too
// (4,096 x 8,192: 27.1 and 25.7).
template <int DT>
bool one_wave(const DistillArgs& a, int chunks) {
  return a.span <= chunks * (int64_t)chunk_cols<DT, 64>() && a.rows * a.splits >= 4 * (int64_t)library_cus();
}
template <int DT>
hipError_t stats_dtype(const DistillArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.rows * a.splits));
  if (a.cols <= epv<DT>()) return launch<k_distill_stats<DT, 64, true>>(grid, dim3(64), s, a);
  if (one_wave<DT>(a, 8)) return launch<k_distill_stats<DT, 64, false>>(grid, dim3(64), s, a);
  // Few rows of more than a chunk: workgroups as wide as they can all be under
  // way at once, so that a row takes fewer waits in a row (64 rows x 32,768
  // bf16: 5.2 us; two splits of 256 threads and a launch to merge them 9.1).
  const int64_t n = a.rows * a.splits, cus = library_cus();
  if (n <= cus && a.span > chunk_cols<DT, 512>())
    return launch<k_distill_stats<DT, 1024, false>>(grid, dim3(1024), s, a);
  if (n <= 2 * cus && a.span > chunk_cols<DT, kBlock>())
    return launch<k_distill_stats<DT, 512, false>>(grid, dim3(512), s, a);
  return launch<k_distill_stats<DT, kBlock, false>>(grid, dim3(kBlock), s, a);
}
template <int DT>
hipError_t grad_dtype(const DistillArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.rows * a.splits));
  if (a.cols <= epv<DT>()) return launch<k_distill_grad<DT, 64, true>>(grid, dim3(64), s, a);
  if (one_wave<DT>(a, 2)) return launch<k_distill_grad<DT, 64, false>>(grid, dim3(64), s, a);
  return launch<k_distill_grad<DT, kBlock, false>>(grid, dim3(kBlock), s, a);
}

// Whether a workgroup waits for the slots before it reads its columns, to
// leave out rows without any: where eight or more workgroups share a compute
// unit, others fill the wait (statistics and gradient, us, looking / not: 4,096
// rows x 16,384 bf16, half of them empty, 18.5 and 34.5 / 24.2 and 46.3, none
// empty 25.1 and 47.4 / 24.8 and 47.3).  With fewer, little is to be gained: 400
// x 12,505, half of them empty, 5.2 and 7.3 / 5.3 and 8.1.
DistillArgs with_look(const DistillArgs& in) {
  DistillArgs a = in;
  a.look_first = a.rows * a.splits >= 8 * (int64_t)library_cus();
  return a;
}
hipError_t launch_distill_stats(const DistillArgs& in, int dtype, hipStream_t s) {
  const DistillArgs a = with_look(in);
  if (dtype == SIM_FP32) return stats_dtype<SIM_FP32>(a, s);
  return dtype == SIM_FP16 ? stats_dtype<SIM_FP16>(a, s) : stats_dtype<SIM_BF16>(a, s);
}
hipError_t launch_distill_grad(const DistillArgs& in, int dtype, hipStream_t s) {
  const DistillArgs a = with_look(in);
  if (dtype == SIM_FP32) return grad_dtype<SIM_FP32>(a, s);
  return dtype == SIM_FP16 ? grad_dtype<SIM_FP16>(a, s) : grad_dtype<SIM_BF16>(a, s);
}
hipError_t launch_distill_join(const DistillArgs& a, float* loss, float* norm, hipStream_t s) {
  return launch<k_distill_join>(dim3((unsigned)((a.rows + 3) / 4)), dim3(kBlock), s, a, loss, norm);
}
hipError_t launch_distill_merge(const DistillArgs& a, float* out, hipStream_t s) {
  return launch<k_distill_merge>(dim3((unsigned)((a.rows + 3) / 4)), dim3(kBlock), s, a, out);
}

}  // namespace simar
