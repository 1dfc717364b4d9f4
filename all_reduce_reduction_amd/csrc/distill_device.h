// distill_device.h -- what the distillation kernels share: a row's slots, its
// columns, and the parts that runs of columns leave (formulas: k_distill.hip).
#pragma once

#include "device_common.h"
#include "loss.h"
#include "loss_device.h"

namespace simar {

constexpr int kSlotsPerLane = SIM_DISTILL_MAX_TOPK / 64;

// A row's slots as wave 0 holds them: slot lane + 64 i.
struct Slots {
  int id[kSlotsPerLane];   // -1: empty
  float q[kSlotsPerLane];  // 0 where empty
  float entropy;           // sum q log q
  bool live;               // the row has a teacher
};

__device__ __forceinline__ float teacher_at(const void* p, int dtype, int64_t i) {
  if (dtype == SIM_FP32) return load_elem<SIM_FP32>(p, i);
  return dtype == SIM_FP16 ? load_elem<SIM_FP16>(p, i) : load_elem<SIM_BF16>(p, i);
}

// The slots' ids and logits on their way from memory: a wave asks for them
// before it asks for anything else and works on them once the rest is in
// flight.  `all`: the logits too, not only the ids.
struct SlotLoads {
  int id[kSlotsPerLane];
  float z[kSlotsPerLane];
};
__device__ __forceinline__ SlotLoads ask_slots(const DistillArgs& a, int64_t row, int lane, bool all) {
  SlotLoads s;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    const int k = lane + 64 * i;
    s.id[i] = -1;
    s.z[i] = 0.0f;
    if (k < a.topk) {
      s.id[i] = a.ids[row * a.topk + k];
      if (all) s.z[i] = teacher_at(a.teacher, a.teacher_dtype, row * a.topk + k);
    }
  }
  return s;
}
// Whether the row has a slot at all: a row without one (a prompt's, padding)
// need not be read.  One whole wave calls this.
__device__ __forceinline__ bool has_slots(const DistillArgs& a, const SlotLoads& in) {
  bool some = false;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    some = some || (in.id[i] >= 0 && in.id[i] < a.vocab);
  }
  return __any(some);
}
// one whole wave calls this
__device__ __forceinline__ Slots make_slots(const DistillArgs& a, const SlotLoads& in) {
  Slots s;
  float z[kSlotsPerLane];
  float top = kNegInf;
  bool some = false;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    const bool ok = in.id[i] >= 0 && in.id[i] < a.vocab;
    s.id[i] = ok ? in.id[i] : -1;
    z[i] = ok ? in.z[i] : kNegInf;
    some = some || !(z[i] == kNegInf);
    top = fmaxf(top, z[i]);
  }
  top = wave_max(top);
  s.live = __any(some);
  const float c = kLog2e / a.tau;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    s.q[i] = z[i] == kNegInf ? 0.0f : exp2_hw((z[i] - top) * c + 8.0f);  // (8: see Against)
    sum += s.q[i];
  }
  sum = wave_sum(sum);
  sum *= 0x1p-8f;
  const float log_sum = __logf(sum);
  float h = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    s.q[i] = s.live ? s.q[i] * 0x1p-8f / sum : 0.0f;
    if (!(s.q[i] == 0.0f)) h += s.q[i] * ((z[i] - top) / a.tau - log_sum);
  }
  s.entropy = s.live ? wave_sum(h) : 0.0f;
  return s;
}

// q (a - b) / tau for q <= 1, of which the difference, or the difference over
// tau, may lie past fp32's range where the whole does not (a masked logit of the
// type's lowest value); halves are exact
__device__ __forceinline__ float times_distance(float q, float a, float b, float tau) {
  return 2.0f * (q * (0.5f * a - 0.5f * b) / tau);
}

__device__ __forceinline__ void* row_at(const void* base, int64_t row, int64_t stride, int esize) {
  return (char*)base + row * stride * esize;
}

// part (m, s, a, d) `part` of row `row`
__device__ __forceinline__ int64_t part_index(int64_t part, int which, int64_t rows, int64_t row) {
  return (part * 4 + which) * rows + row;
}

// A row's slots as the threads of a workgroup of NT use them.  Slot k hangs on
// the thread that holds its column (list head[thread], then next[k]); after
// its vectors a thread writes the full values of its slots' columns.  Its own
// stores to one address stay in order, so no barrier is needed in between.
template <int NT>
struct SlotLists {
  int head[NT];
  int next[SIM_DISTILL_MAX_TOPK], id[SIM_DISTILL_MAX_TOPK];
  float q[SIM_DISTILL_MAX_TOPK], x[SIM_DISTILL_MAX_TOPK];  // x: the slot's logit, then its probability
  int live;
};
// Wave 0, before anything is written (the gradient may lie on the logits):
// the slots and the logits of those in the columns [lo, hi) of `x`.
template <int DT, int NT>
__device__ __forceinline__ void gather_slots(const DistillArgs& a, SlotLists<NT>& s, const Slots& sl, const void* x,
                                             int64_t lo, int64_t hi, int lane) {
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    const int k = lane + 64 * i;
    if (k >= a.topk) continue;
    const int64_t col = (int64_t)sl.id[i] - a.first;
    s.id[k] = sl.id[i];
    s.q[k] = sl.q[i];
    if (sl.id[i] >= 0 && col >= lo && col < hi) s.x[k] = load_elem<DT>(x, col);
  }
  if (lane == 0) s.live = sl.live;
}
// 1 where a row of 16-bit logits starts in the middle of a word.  Its first
// column then goes by itself and the vectors start behind it: 16-byte accesses
// that are not even word-aligned take two passes each (4,096 rows x 50,021
// bf16, every other one such: 182 us against 157 with 50,022 columns).
template <int DT>
__device__ __forceinline__ uint32_t lone_columns(const void* row) {
  return Ty<DT>::E == 2 ? (uint32_t)((uintptr_t)row >> 1) & 1u : 0u;
}
// Wave 0, once the row's maximum and its sum against `top` are known: each
// slot's probability, and its place in its thread's list (a slot of q = 0
// changes nothing of its column).  `base`: the first vector's column (the
// column before it is thread 0's).
template <int DT, int NT>
__device__ __forceinline__ void hang_slots(const DistillArgs& a, SlotLists<NT>& s, const Slots& sl, int64_t lo,
                                           int64_t hi, int64_t base, const Against& top, float sum, int lane) {
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    if (64 * i >= a.topk) break;
    const int k = lane + 64 * i;
    const int64_t col = (int64_t)sl.id[i] - a.first;
    if (!sl.live || sl.id[i] < 0 || sl.q[i] == 0.0f || col < lo || col >= hi) continue;
    s.x[k] = exp_against(s.x[k], top) / sum;
    s.next[k] = atomicExch(&s.head[col < base ? 0 : (col - base) / epv<DT>() % NT], k);
  }
}
// Each slot's column gets up (p - the sum of q over the slots with its id).
// Slots with one id hang on one thread, so it sees in its own list, whose
// order depends on timing, whether there are others; the first of them then
// adds them in the order of the slots (79 rows x 2,263 with 101 slots, some
// of one id: 14.9 us; every slot adding, one load after the other: 27.4).
template <int DT, int NT>
__device__ __forceinline__ void write_slots(const DistillArgs& a, const SlotLists<NT>& s, void* dx, float up, int tid) {
  const int head = s.head[tid];
  for (int k = head; k >= 0; k = s.next[k]) {
    const int id = s.id[k];
    bool more = false, first = true;
    auto other = [&](int j) {
      if (s.id[j] != id) return;
      more = true;
      first = j > k;
    };
    for (int j = s.next[k]; j >= 0 && first; j = s.next[j]) other(j);
    for (int j = head; j != k && first; j = s.next[j]) other(j);
    if (!first) continue;
    float q = s.q[k];
    if (more) {
      q = 0.0f;
      constexpr int N = 8;  // a batch of loads at a time
      for (int j0 = 0; j0 < a.topk; j0 += N) {
        int ids[N];
        float qs[N];
#pragma unroll
        for (int j = 0; j < N; j++) {
          ids[j] = s.id[j0 + j];
          qs[j] = s.q[j0 + j];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < N; j++) q += j0 + j < a.topk && ids[j] == id ? qs[j] : 0.0f;
      }
    }
    store_elem<DT>(dx, (int64_t)id - a.first, up * (s.x[k] - q));
  }
}

// The parts of a row as one, in the order of the columns.
struct Part {
  float m, s, a, d;
};
__device__ __forceinline__ Part join_two(const Part& p, const Part& q, float tau, float c) {
  Part t;
  t.m = fmaxf(p.m, q.m);
  t.s = p.s * rebase(p.m, t.m, c) + q.s * rebase(q.m, t.m, c);
  t.a = p.a + q.a;
  // (a part without slots moves nothing, wherever its own maximum is)
  const float dp = p.a == 0.0f || p.m == t.m ? 0.0f : times_distance(p.a, p.m, t.m, tau);
  const float dq = q.a == 0.0f || q.m == t.m ? 0.0f : times_distance(q.a, q.m, t.m, tau);
  t.d = (p.d + dp) + (q.d + dq);
  return t;
}
// A whole wave joins a row's n parts: lane k takes parts k, k + 64, ..., so
// that all loads are in flight together.
__device__ __forceinline__ Part join_parts(const float* parts, int n, int64_t rows, int64_t row, float tau, int lane) {
  const float c = kLog2e / tau;
  Part t{kNegInf, 0.0f, 0.0f, 0.0f};
  for (int k = lane; k < n; k += 64) {
    const Part p{parts[part_index(k, 0, rows, row)], parts[part_index(k, 1, rows, row)],
                 parts[part_index(k, 2, rows, row)], parts[part_index(k, 3, rows, row)]};
    t = join_two(t, p, tau, c);
  }
  const float top = wave_max(t.m);
  t = join_two(t, Part{top, 0.0f, 0.0f, 0.0f}, tau, c);
  t.s = wave_sum(t.s);
  t.a = wave_sum(t.a);
  t.d = wave_sum(t.d);
  return t;
}
__device__ __forceinline__ float loss_of(const Slots& s, const Part& t) {
  return s.live ? s.entropy + t.a * __logf(t.s) - t.d : 0.0f;
}

}  // namespace simar
