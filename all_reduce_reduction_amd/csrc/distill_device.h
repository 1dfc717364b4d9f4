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

// one whole wave calls this
__device__ __forceinline__ Slots load_slots(const DistillArgs& a, int64_t row, int lane) {
  Slots s;
  float z[kSlotsPerLane];
  float top = kNegInf;
  bool some = false;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    const int k = lane + 64 * i;
    s.id[i] = -1;
    z[i] = kNegInf;
    if (k < a.topk) {
      const int id = a.ids[row * a.topk + k];
      if (id >= 0 && id < a.vocab) {
        s.id[i] = id;
        z[i] = teacher_at(a.teacher, a.teacher_dtype, row * a.topk + k);
      }
    }
    some = some || !(z[i] == kNegInf);
    top = fmaxf(top, z[i]);
  }
  top = wave_max(top);
  s.live = __any(some);
  const float c = kLog2e / a.tau;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    s.q[i] = z[i] == kNegInf ? 0.0f : exp2_hw((z[i] - top) * c);
    sum += s.q[i];
  }
  sum = wave_sum(sum);
  const float log_sum = __logf(sum), inv = 1.0f / sum;
  float h = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlotsPerLane; i++) {
    s.q[i] = s.live ? s.q[i] * inv : 0.0f;
    if (!(s.q[i] == 0.0f)) h += s.q[i] * ((z[i] - top) / a.tau - log_sum);
  }
  s.entropy = s.live ? wave_sum(h) : 0.0f;
  return s;
}

__device__ __forceinline__ void* row_at(const void* base, int64_t row, int64_t stride, int esize) {
  return (char*)base + row * stride * esize;
}

// part (m, s, a, d) `part` of row `row`
__device__ __forceinline__ int64_t part_index(int64_t part, int which, int64_t rows, int64_t row) {
  return (part * 4 + which) * rows + row;
}

// The parts of a row as one, in the order of the columns.
struct Part {
  float m, s, a, d;
};
__device__ __forceinline__ Part join_parts(const float* parts, int n, int64_t rows, int64_t row, float tau) {
  const float c = kLog2e / tau;
  Part t{kNegInf, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < n; k++) t.m = fmaxf(t.m, parts[part_index(k, 0, rows, row)]);
  for (int k = 0; k < n; k++) {
    const float m = parts[part_index(k, 0, rows, row)], mass = parts[part_index(k, 2, rows, row)];
    t.s += parts[part_index(k, 1, rows, row)] * rebase(m, t.m, c);
    if (mass == 0.0f) continue;
    t.a += mass;
    t.d += parts[part_index(k, 3, rows, row)] + (m == t.m ? 0.0f : mass * ((m - t.m) / tau));
  }
  return t;
}
__device__ __forceinline__ float loss_of(const Slots& s, const Part& t) {
  return s.live ? s.entropy + t.a * __logf(t.s) - t.d : 0.0f;
}

}  // namespace simar
