// k_norm_grad.hip -- gradient of the root-mean-square norm for the normed sum
// h and for the gain (gfx950).
//
// With u = h r and d = dy g:  dx = r (d - u mean(d u)) + dsum, and dgain = the
// sum over the rows of dy u.  A workgroup takes rows in turn, each kept in
// registers from its read to its write, with the gain and the columns' share of
// dgain in registers from the first row to the last; the workgroups' shares are
// added up by a second launch, in the workgroups' order.
#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

template <int DT, int NT, int R, bool TINY>
__global__ void __launch_bounds__(NT) k_norm_grad(NormGradArgs a) {
  constexpr int V = epv<DT>(), W = NT / 64;
  __shared__ float ss_s[2][W], dot_s[2][W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t cols = (uint32_t)a.cols;
  const float n = (float)cols;
  float g[R][V], acc[R][V];
#pragma unroll
  for (int i = 0; i < R; i++) {
    load_gain(a.gain, a.gain_dtype, RowPart<DT, TINY>((i * NT + tid) * V, cols), g[i]);
#pragma unroll
    for (int t = 0; t < V; t++) acc[i][t] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const char* hp = (const char*)a.h + row * a.h_stride * Ty<DT>::E;
    const char* dp = (const char*)a.dy + row * a.dy_stride * Ty<DT>::E;
    u32x4 hv[R], dv[R], sv[R];
#pragma unroll
    for (int i = 0; i < R; i++) hv[i] = RowPart<DT, TINY>((i * NT + tid) * V, cols).load(hp);
#pragma unroll
    for (int i = 0; i < R; i++) dv[i] = RowPart<DT, TINY>((i * NT + tid) * V, cols).load(dp);
    if (a.dsum) {
      const char* sp = (const char*)a.dsum + row * a.dsum_stride * Ty<DT>::E;
#pragma unroll
      for (int i = 0; i < R; i++) sv[i] = RowPart<DT, TINY>((i * NT + tid) * V, cols).load(sp);
    } else {
#pragma unroll
      for (int i = 0; i < R; i++) sv[i] = u32x4{0, 0, 0, 0};
    }
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < R; i++) {
      const RowPart<DT, TINY> p((i * NT + tid) * V, cols);
      float h[V], d[V];
      unpack<DT>(hv[i], h);
      unpack<DT>(dv[i], d);
#pragma unroll
      for (int t = 0; t < V; t++) {
        const float f = p.own(t) ? h[t] : 0.0f, e = p.own(t) ? d[t] * g[i][t] : 0.0f;
        ss = __builtin_fmaf(f, f, ss);
        dot = __builtin_fmaf(f, e, dot);
      }
    }
    ss = wave_sum(ss);
    dot = wave_sum(dot);
    if constexpr (W > 1) {
      if (lane == 0) {
        ss_s[turn][wave] = ss;
        dot_s[turn][wave] = dot;
      }
      __syncthreads();
      ss = wave_sum(lane < W ? ss_s[turn][lane] : 0.0f);
      dot = wave_sum(lane < W ? dot_s[turn][lane] : 0.0f);
    }
    const float r = 1.0f / __builtin_sqrtf(ss / n + a.eps);
    const float mean = r * (dot / n);  // of d u
    char* to = (char*)a.dx + row * a.dx_stride * Ty<DT>::E;
#pragma unroll
    for (int i = 0; i < R; i++) {
      const RowPart<DT, TINY> p((i * NT + tid) * V, cols);
      float h[V], d[V], s[V];
      unpack<DT>(hv[i], h);
      unpack<DT>(dv[i], d);
      unpack<DT>(sv[i], s);
#pragma unroll
      for (int t = 0; t < V; t++) {
        const float u = h[t] * r;
        acc[i][t] = __builtin_fmaf(d[t], u, acc[i][t]);
        s[t] = __builtin_fmaf(r, __builtin_fmaf(-u, mean, d[t] * g[i][t]), s[t]);
      }
      if (p.any()) p.store(to, s);
    }
  }
  if (!a.dgain) return;
  // (one workgroup's share is the whole sum)
  float* to = a.workgroups > 1 ? a.partial + (int64_t)blockIdx.x * cols : a.dgain;
#pragma unroll
  for (int i = 0; i < R; i++) {
    const RowPart<DT, TINY> p((i * NT + tid) * V, cols);
    if (!p.any()) continue;
#pragma unroll
    for (int t = 0; t < V; t++)
      if (p.own(t)) to[p.column(t)] = acc[i][t];
  }
}

// dgain[c] = the sum of partial[w][c]: 64 columns per workgroup, a wave takes
// every fourth row of them.
__global__ void __launch_bounds__(256) k_gain_sum(const float* partial, int workgroups, int cols, float* dgain) {
  __shared__ float s[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (c < cols) {
    int w = wave;
    for (; w + 28 < workgroups; w += 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = partial[(int64_t)(w + 4 * i) * cols + c];
#pragma unroll
      for (int i = 0; i < 8; i++) sum += v[i];
    }
    for (; w < workgroups; w += 4) sum += partial[(int64_t)w * cols + c];
  }
  s[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && c < cols) dgain[c] = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
}

template <int DT, int NT, int R, bool TINY = false>
hipError_t go(const NormGradArgs& a, hipStream_t s) {
  return launch<k_norm_grad<DT, NT, R, TINY>>(dim3(a.workgroups), dim3(NT), s, a);
}

template <int DT>
hipError_t pick(const NormGradArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = ((int64_t)a.cols + V - 1) / V;
  if (a.cols < V) return go<DT, 64, 1, true>(a, s);
  if (nv <= 64) return go<DT, 64, 1>(a, s);
  if (nv <= 256) return go<DT, 256, 1>(a, s);
  if (nv <= 512) return go<DT, 256, 2>(a, s);
  if (nv <= 1024) return go<DT, 1024, 1>(a, s);
  if (nv <= 2048) return go<DT, 1024, 2>(a, s);
  if (nv <= 4096) return go<DT, 1024, 4>(a, s);
  if constexpr (V == 4) return go<DT, 1024, 8>(a, s);
  return hipErrorInvalidValue;  // (rows of more than SIM_NORM_MAX_COLUMNS are refused before)
}

}  // namespace

hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s) {
  const hipError_t e = dtype == SIM_FP32   ? pick<SIM_FP32>(a, s)
                       : dtype == SIM_FP16 ? pick<SIM_FP16>(a, s)
                                           : pick<SIM_BF16>(a, s);
  if (e != hipSuccess || !a.dgain || a.workgroups == 1) return e;
  return launch<k_gain_sum>(dim3((unsigned)((a.cols + 63) / 64)), dim3(256), s, (const float*)a.partial, a.workgroups,
                            a.cols, a.dgain);
}

}  // namespace simar
