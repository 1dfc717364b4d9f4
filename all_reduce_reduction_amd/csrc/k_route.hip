// k_route.hip -- softmax gate with per-expert statistics, and the gradient of
// its balance loss and combine weights (gfx950).
//
// Forward, row x: m = max x, Z = sum exp(x - m), p = exp(x - m) / Z; the topk
// largest logits by value, ties to the lowest index, taken from the logits
// themselves, so that the choice does not depend on any rounding.  Counts are
// integers; probability sums are taken per lane over the rows of a wave, then
// over the waves of a workgroup, then over the workgroups, in that order, so
// they do not depend on timing.
//
// Gradient: with g_e = coef f_e / N,
//   dx_e = p_e (g_e + u_e - sum_j p_j (g_j + u_j)),  u = dweights at chosen e,
// for raw weights; for normalised ones w = p / (their sum over the chosen),
//   dx_e = p_e (g_e - sum_j p_j g_j) + [e chosen] w_e (dw_e - sum_i w_i dw_i).
#include "device_common.h"
#include "launch.h"
#include "loss.h"
#include "loss_device.h"

namespace simar {
namespace {

constexpr int kWaves = kBlock / 64;

// One wave per row; lane l holds the experts l, l + 64, ...: N of them.
template <int DT, int N>
__device__ __forceinline__ bool load_row(const void* base, int64_t row, int64_t stride, int experts,
                                         const uint8_t* keep, int lane, float (&x)[N]) {
  const char* r = (const char*)base + row * stride * Ty<DT>::E;
  const bool kept = !keep || keep[row];
  bool some = false;
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int e = lane + 64 * i;
    x[i] = kept && e < experts ? load_elem<DT>(r, e) : kNegInf;
    some = some || !(x[i] == kNegInf);
  }
  return __any(some);
}

template <int N>
__device__ __forceinline__ float softmax(const float (&x)[N], float (&p)[N]) {
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < N; i++) top = fmaxf(top, x[i]);
  top = wave_max(top);
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) {
    p[i] = exp2_hw((x[i] - top) * kLog2e);
    z += p[i];
  }
  z = wave_sum(z);
#pragma unroll
  for (int i = 0; i < N; i++) p[i] = p[i] / z;
  return z;
}

template <int DT, int N>
__global__ void __launch_bounds__(kBlock) k_route(RouteArgs a) {
  __shared__ uint32_t count_s[SIM_ROUTE_MAX_EXPERTS + 1];
  __shared__ float sum_s[kWaves][64 * N];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.experts; e += kBlock) count_s[e] = 0;
  __syncthreads();
  float sums[N];
#pragma unroll
  for (int i = 0; i < N; i++) sums[i] = 0.0f;
  const int64_t step = (int64_t)a.workgroups * kWaves;
  for (int64_t row = (int64_t)blockIdx.x * kWaves + wave; row < a.tokens; row += step) {
    float x[N], p[N];
    const bool live = load_row<DT, N>(a.x, row, a.stride, a.experts, a.keep, lane, x);
    int mine = -1;
    float w = 0.0f;
    if (live) {
      const float z = softmax(x, p);
      for (int j = 0; j < a.topk; j++) {
        float best = kNegInf;
        int at = -1;
#pragma unroll
        for (int i = 0; i < N; i++)
          if (x[i] > best) {
            best = x[i];
            at = lane + 64 * i;
          }
        const float top = wave_max(best);
        // the lowest index among the lanes that hold the maximum
        int e = best == top && at >= 0 ? at : INT32_MAX;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) e = min(e, __shfl_xor(e, d, 64));
        if (e == INT32_MAX) break;
        float pe = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i++)
          if (lane + 64 * i == e) {
            pe = p[i];
            x[i] = kNegInf;
          }
        pe = __shfl(pe, e & 63, 64);
        if (lane == j) {
          mine = e;
          w = pe;
        }
      }
      if (a.normalize) {
        const float total = wave_sum(w);
        if (mine >= 0) w = z != z ? z : w / total;
      }
      if (mine >= 0) atomicAdd(&count_s[mine], 1u);
      if (lane == 0) atomicAdd(&count_s[a.experts], 1u);
#pragma unroll
      for (int i = 0; i < N; i++) sums[i] += p[i];
    }
    if (lane < a.topk) {
      a.chosen[row * a.topk + lane] = mine;
      a.weights[row * a.topk + lane] = w;
    }
  }
#pragma unroll
  for (int i = 0; i < N; i++) sum_s[wave][lane + 64 * i] = sums[i];
  __syncthreads();
  uint32_t* part = a.partial + (int64_t)blockIdx.x * (2 * a.experts + 1);
  for (int e = tid; e <= a.experts; e += kBlock) {
    float s = 0.0f;
    if (e < a.experts) {
#pragma unroll
      for (int w = 0; w < kWaves; w++) s += sum_s[w][e];
    }
    if (a.workgroups == 1) {
      a.counts[e] = (int32_t)count_s[e];
      if (e < a.experts) a.sums[e] = s;
    } else {
      part[e] = count_s[e];
      if (e < a.experts) part[a.experts + 1 + e] = __builtin_bit_cast(uint32_t, s);
    }
  }
}

// one thread per counted value, over all workgroups in order
__global__ void __launch_bounds__(kBlock) k_route_sum(RouteArgs a) {
  const int e = blockIdx.x * kBlock + threadIdx.x, all = 2 * a.experts + 1;
  if (e >= all) return;
  uint32_t n = 0;
  float s = 0.0f;
  for (int w = 0; w < a.workgroups; w++) {
    const uint32_t v = a.partial[(int64_t)w * all + e];
    n += v;
    s += __builtin_bit_cast(float, v);
  }
  if (e <= a.experts) a.counts[e] = (int32_t)n;
  else a.sums[e - a.experts - 1] = s;
}

template <int DT, int N>
__global__ void __launch_bounds__(kBlock) k_route_grad(RouteGradArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float n = a.counts ? (float)a.counts[a.experts] : 0.0f;
  const float unit = n > 0.0f ? a.coef * ((float)a.experts / (float)a.topk) / n / n : 0.0f;
  float g[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int e = lane + 64 * i;
    g[i] = n > 0.0f && e < a.experts ? unit * (float)a.counts[e] : 0.0f;
  }
  if (blockIdx.x == 0 && wave == 0 && a.loss) {
    float loss = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = lane + 64 * i;
      if (n > 0.0f && e < a.experts) loss += g[i] * a.sums[e];
    }
    loss = wave_sum(loss);
    if (lane == 0) *a.loss = loss;
  }
  const int64_t row = (int64_t)blockIdx.x * kWaves + wave;
  if (row >= a.tokens) return;
  float x[N], p[N], d[N];
  const bool live = load_row<DT, N>(a.x, row, a.stride, a.experts, a.keep, lane, x);
#pragma unroll
  for (int i = 0; i < N; i++) d[i] = 0.0f;
  if (live) {
    softmax(x, p);
    int mine = -1;
    float dw = 0.0f, w = 0.0f;
    if (a.dweights && lane < a.topk) {
      mine = a.chosen[row * a.topk + lane];
      if (mine < 0 || mine >= a.experts) mine = -1;
      if (mine >= 0) dw = a.dweights[row * a.topk + lane];
    }
    float u[N];
#pragma unroll
    for (int i = 0; i < N; i++) u[i] = 0.0f;
    if (a.dweights) {
      // the probability of this lane's slot
#pragma unroll
      for (int i = 0; i < N; i++) {
        const float v = __shfl(p[i], mine & 63, 64);
        if (mine >= 0 && (mine >> 6) == i) w = v;
      }
      float slot = dw;
      if (a.normalize) {
        const float total = wave_sum(w);
        w = mine >= 0 ? w / total : 0.0f;
        const float mean = wave_sum(w * dw);
        slot = mine >= 0 ? w * (dw - mean) : 0.0f;
      }
      for (int j = 0; j < a.topk; j++) {
        const int e = __shfl(mine, j, 64);
        const float v = __shfl(slot, j, 64);
#pragma unroll
        for (int i = 0; i < N; i++)
          if (lane + 64 * i == e) u[i] += v;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float up = a.normalize ? g[i] : g[i] + u[i];
      dot += p[i] * up;
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float up = a.normalize ? g[i] : g[i] + u[i];
      d[i] = p[i] * (up - dot) + (a.normalize ? u[i] : 0.0f);
    }
  }
  char* out = (char*)a.dx + row * a.dstride * Ty<DT>::E;
#pragma unroll
  for (int i = 0; i < N; i++)
    if (lane + 64 * i < a.experts) store_elem<DT>(out, lane + 64 * i, d[i]);
}

template <int DT>
hipError_t route_dtype(const RouteArgs& a, hipStream_t s) {
  const dim3 grid(a.workgroups), block(kBlock);
  if (a.experts <= 64) return launch<k_route<DT, 1>>(grid, block, s, a);
  if (a.experts <= 256) return launch<k_route<DT, 4>>(grid, block, s, a);
  return launch<k_route<DT, 16>>(grid, block, s, a);
}
template <int DT>
hipError_t grad_dtype(const RouteGradArgs& a, hipStream_t s) {
  const int64_t wg = (a.tokens + kWaves - 1) / kWaves;
  const dim3 grid((unsigned)(wg > 0 ? wg : 1)), block(kBlock);
  if (a.experts <= 64) return launch<k_route_grad<DT, 1>>(grid, block, s, a);
  if (a.experts <= 256) return launch<k_route_grad<DT, 4>>(grid, block, s, a);
  return launch<k_route_grad<DT, 16>>(grid, block, s, a);
}

}  // namespace

int route_workgroups(int64_t tokens, int experts) {
  (void)experts;
  const int64_t wg = (tokens + kWaves - 1) / kWaves, most = 4 * (int64_t)library_cus();
  return (int)(wg < 1 ? 1 : wg < most ? wg : most);
}

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
  const hipError_t e = dtype == SIM_FP32   ? route_dtype<SIM_FP32>(a, s)
                       : dtype == SIM_FP16 ? route_dtype<SIM_FP16>(a, s)
                                           : route_dtype<SIM_BF16>(a, s);
  if (e != hipSuccess || a.workgroups == 1) return e;
  return launch<k_route_sum>(dim3((2 * a.experts + kBlock) / kBlock), dim3(kBlock), s, a);
}
hipError_t launch_route_grad(const RouteGradArgs& a, int dtype, hipStream_t s) {
  if (dtype == SIM_FP32) return grad_dtype<SIM_FP32>(a, s);
  return dtype == SIM_FP16 ? grad_dtype<SIM_FP16>(a, s) : grad_dtype<SIM_BF16>(a, s);
}

}  // namespace simar
