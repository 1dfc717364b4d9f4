// k_norm_grad.hip -- gradient of the root-mean-square norm for the normed sum
// h and for the gain (gfx950).
//
// With u = h r and d = dy g:  dx = r (d - u mean(d u)) + dsum, and dgain = the
// sum over the rows of dy u.  A workgroup takes rows in turn, each kept in
// registers from its read to its write, with the gain and the columns' share of
// dgain in registers from the first row to the last; the workgroups' shares are
// added up by a second launch, in the workgroups' order.
//
// Bound by memory that reads and writes at once: 183 us for 16,384 rows x 8,192
// bf16 with dsum (1,074 MB; a copy of as many bytes 161; without the next row's loads
// ahead 186), of which the second launch and its gap are 6; 1,003 rows x 2,261 fp32 11
// us, where a workgroup's four rows follow each other; 2 rows x 4,096 bf16 4.1 us, in one
// workgroup and one launch.  Four vectors of 16 bits or eight of fp32 per thread spill
// (fp32 84 registers, fp16 68, bf16 32): 1,024 x 32,768 without dsum fp32 169 us, fp16
// 133, bf16 82.
#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

// A row's vectors of a thread.  With eight elements each, the next row's are asked
// for before this one's are used; with four vectors or more the gain and dsum are loaded where they
// are needed, as they do not fit in the registers beside the others.
template <int DT, int R>
__global__ void __launch_bounds__(1024) k_norm_grad(NormGradArgs a) {
  constexpr int V = epv<DT>();
  constexpr bool AHEAD = R * V <= 8, HOLD = R <= 2;
  __shared__ float ss_s[2][16], dot_s[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const RowVectors<DT, R, false> vectors{threadIdx.x, blockDim.x, (uint32_t)a.cols};
  const bool exact = vectors.exact();
  const float n = (float)a.cols;
  float g[HOLD ? R : 1][V], acc[R][V];
  vectors([&](auto i, auto p) __attribute__((always_inline)) {
    if constexpr (HOLD) load_gain(a.gain, a.gain_dtype, p, g[i]);
#pragma unroll
    for (int t = 0; t < V; t++) acc[i][t] = 0.0f;
  });
  // d g
  const auto gained = [&](auto i, auto p, const float (&d)[V], float (&x)[V]) __attribute__((always_inline)) {
    if constexpr (!HOLD) load_gain(a.gain, a.gain_dtype, p, x);
#pragma unroll
    for (int t = 0; t < V; t++) x[t] = d[t] * (HOLD ? g[HOLD ? decltype(i)::value : 0][t] : x[t]);
  };
  u32x4 hv[R], dv[R], sv[HOLD ? R : 1];
  const auto ask = [&](int64_t row) __attribute__((always_inline)) {
    const char* hp = (const char*)a.h + row * a.h_stride * Ty<DT>::E;
    const char* dp = (const char*)a.dy + row * a.dy_stride * Ty<DT>::E;
    vectors([&](auto i, auto p) __attribute__((always_inline)) { hv[i] = p.load(hp); });
    vectors([&](auto i, auto p) __attribute__((always_inline)) { dv[i] = p.load(dp); });
    if constexpr (HOLD) {
      if (a.dsum) {
        const char* sp = (const char*)a.dsum + row * a.dsum_stride * Ty<DT>::E;
        vectors([&](auto i, auto p) __attribute__((always_inline)) { sv[i] = p.load(sp); });
      } else {
#pragma unroll
        for (int i = 0; i < R; i++) sv[i] = u32x4{0, 0, 0, 0};
      }
    }
  };
  if (AHEAD && (int64_t)blockIdx.x < a.rows) ask(blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    if constexpr (!AHEAD) ask(row);
    u32x4 hr[R], dr[R], sr[HOLD ? R : 1];
#pragma unroll
    for (int i = 0; i < R; i++) {
      hr[i] = hv[i];
      dr[i] = dv[i];
      if constexpr (HOLD) sr[i] = sv[i];
    }
    if (AHEAD && row + gridDim.x < a.rows) ask(row + gridDim.x);
    float ss = 0.0f, dot = 0.0f;
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
      float h[V], d[V], dg[V];
      unpack<DT>(hr[i], h);
      unpack<DT>(dr[i], d);
      if (i == R - 1 && !exact) {
        p.mask(h);
        p.mask(d);
      }
      gained(i, p, d, dg);
#pragma unroll
      for (int t = 0; t < V; t++) {
        ss = __builtin_fmaf(h[t], h[t], ss);
        dot = __builtin_fmaf(h[t], dg[t], dot);
      }
    });
    ss = wave_sum(ss);
    dot = wave_sum(dot);
    if (waves > 1) {
      if (lane == 0) {
        ss_s[turn][wave] = ss;
        dot_s[turn][wave] = dot;
      }
      __syncthreads();
      ss = group_sum<16>((lane & 15) < waves ? ss_s[turn][lane & 15] : 0.0f);
      dot = group_sum<16>((lane & 15) < waves ? dot_s[turn][lane & 15] : 0.0f);
    }
    if constexpr (!HOLD) {
      // (unpacked again below: kept from above, the fp32 values would not fit)
#pragma unroll
      for (int i = 0; i < R; i++) asm volatile("" : "+v"(hr[i]), "+v"(dr[i]));
    }
    const float r = 1.0f / __builtin_sqrtf(ss / n + a.eps);
    const float mean = r * (dot / n);  // of d u
    char* to = (char*)a.dx + row * a.dx_stride * Ty<DT>::E;
    const char* sp = (const char*)a.dsum + row * a.dsum_stride * Ty<DT>::E;
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
      float h[V], d[V], dg[V], s[V];
      unpack<DT>(hr[i], h);
      unpack<DT>(dr[i], d);
      gained(i, p, d, dg);
      if constexpr (HOLD) unpack<DT>(sr[i], s);
      else unpack<DT>(a.dsum ? p.load(sp) : u32x4{0, 0, 0, 0}, s);
#pragma unroll
      for (int t = 0; t < V; t++) {
        const float u = h[t] * r;
        acc[i][t] = __builtin_fmaf(d[t], u, acc[i][t]);
        s[t] = __builtin_fmaf(r, __builtin_fmaf(-u, mean, dg[t]), s[t]);
      }
      if (p.any()) p.store(to, s);
    });
  }
  if (!a.dgain) return;
  // (one workgroup's share is the whole sum)
  float* to = a.workgroups > 1 ? a.partial + (int64_t)blockIdx.x * a.cols : a.dgain;
  vectors([&](auto i, auto p) __attribute__((always_inline)) {
    if (p.any()) p.store_floats(to, acc[i]);
  });
}

// Short rows: L lanes take a row, R vectors each, and kShortThreads / L rows share
// a workgroup, whose waves add up their shares of dgain through shared memory: as
// many partial sums as long rows make, however many rows a wave takes at once.
template <int DT, int L, int R, bool TINY>
__global__ void __launch_bounds__(kNormShortThreads) k_norm_grad_short(NormGradArgs a) {
  constexpr int V = epv<DT>(), ROWS = kNormShortThreads / L, W = kNormShortThreads / 64;
  __shared__ float share_s[W][64 * R * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = threadIdx.x % L;
  const RowVectors<DT, R, TINY> vectors{(uint32_t)l, L, (uint32_t)a.cols};
  const float n = (float)a.cols;
  float g[R][V], acc[R][V];
  vectors([&](auto i, auto p) __attribute__((always_inline)) {
    load_gain(a.gain, a.gain_dtype, p, g[i]);
#pragma unroll
    for (int t = 0; t < V; t++) acc[i][t] = 0.0f;
  });
  u32x4 hv[R], dv[R], sv[R];
  const auto ask = [&](int64_t row) __attribute__((always_inline)) {
    const char* hp = (const char*)a.h + row * a.h_stride * Ty<DT>::E;
    const char* dp = (const char*)a.dy + row * a.dy_stride * Ty<DT>::E;
    vectors([&](auto i, auto p) __attribute__((always_inline)) { hv[i] = p.load(hp); });
    vectors([&](auto i, auto p) __attribute__((always_inline)) { dv[i] = p.load(dp); });
    if (a.dsum) {
      const char* sp = (const char*)a.dsum + row * a.dsum_stride * Ty<DT>::E;
      vectors([&](auto i, auto p) __attribute__((always_inline)) { sv[i] = p.load(sp); });
    } else {
#pragma unroll
      for (int i = 0; i < R; i++) sv[i] = u32x4{0, 0, 0, 0};
    }
  };
  const int64_t first = (int64_t)blockIdx.x * ROWS + threadIdx.x / L, step = (int64_t)gridDim.x * ROWS;
  if (first < a.rows) ask(first);
  for (int64_t row = first; row < a.rows; row += step) {
    float h[R][V], d[R][V], s[R][V];
    float ss = 0.0f, dot = 0.0f;
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
      unpack<DT>(hv[i], h[i]);
      unpack<DT>(dv[i], d[i]);
      unpack<DT>(sv[i], s[i]);
      if (i == R - 1) {
        p.mask(h[i]);
        p.mask(d[i]);
      }
    });
    if (row + step < a.rows) ask(row + step);
#pragma unroll
    for (int i = 0; i < R; i++) {
#pragma unroll
      for (int t = 0; t < V; t++) {
        ss = __builtin_fmaf(h[i][t], h[i][t], ss);
        dot = __builtin_fmaf(h[i][t], d[i][t] * g[i][t], dot);
      }
    }
    ss = group_sum<L>(ss);
    dot = group_sum<L>(dot);
    const float r = 1.0f / __builtin_sqrtf(ss / n + a.eps);
    const float mean = r * (dot / n);  // of d u
    char* to = (char*)a.dx + row * a.dx_stride * Ty<DT>::E;
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < V; t++) {
        const float u = h[i][t] * r;
        acc[i][t] = __builtin_fmaf(d[i][t], u, acc[i][t]);
        s[i][t] = __builtin_fmaf(r, __builtin_fmaf(-u, mean, d[i][t] * g[i][t]), s[i][t]);
      }
      if (p.any()) p.store(to, s[i]);
    });
  }
  if (!a.dgain) return;
  // a wave's rows, then the waves
#pragma unroll
  for (int i = 0; i < R; i++) {
#pragma unroll
    for (int t = 0; t < V; t++) {
      float v = acc[i][t];
      for (int m = L; m < 64; m *= 2) v += __shfl_xor(v, m);
      if (lane < L) share_s[wave][(i * L + lane) * V + t] = v;
    }
  }
  __syncthreads();
  float* to = a.workgroups > 1 ? a.partial + (int64_t)blockIdx.x * a.cols : a.dgain;
  // where a column is: (vector i * L + l, element t), the row's last vector moved
  // back to end with the row
  const int whole = TINY ? 0 : a.cols / V * V;
  for (int c = threadIdx.x; c < a.cols; c += kNormShortThreads) {
    const int at = c < whole || TINY ? c : c - a.cols + whole + V;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w++) v += share_s[w][at];
    to[c] = v;
  }
}

// dgain[c] = the sum of partial[w][c]: 16 columns per workgroup, a quarter wave
// takes every 64th of them.
constexpr int kSumThreads = 1024, kSumColumns = 16;
__global__ void __launch_bounds__(kSumThreads) k_gain_sum(const float* partial, int workgroups, int cols, float* dgain) {
  constexpr int N = 8, ROWS = kSumThreads / kSumColumns;
  __shared__ float s[ROWS][kSumColumns + 1];
  const int k = threadIdx.x % kSumColumns, q = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + k;
  float sum = 0.0f;
  if (c < cols) {
    for (int w0 = q; w0 < workgroups; w0 += N * ROWS) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; i++) {
        v[i] = 0.0f;
        if (w0 + i * ROWS < workgroups) v[i] = partial[(int64_t)(w0 + i * ROWS) * cols + c];
      }
#pragma unroll
      for (int i = 0; i < N; i++) sum += v[i];
    }
  }
  s[q][k] = sum;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  // four threads per column, 16 rows each, then the four
  const int col = threadIdx.x / 4, part = threadIdx.x % 4;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < ROWS / 4; i++) sum += s[part * (ROWS / 4) + i][col];
  sum = group_sum<4>(sum);
  if (part == 0 && blockIdx.x * kSumColumns + col < cols) dgain[blockIdx.x * kSumColumns + col] = sum;
}

template <int DT, int R>
hipError_t go(const NormGradArgs& a, int threads, hipStream_t s) {
  if (!row_vectors_fit(a.cols, epv<DT>(), threads, R)) return hipErrorInvalidValue;
  return launch<k_norm_grad<DT, R>>(dim3(a.workgroups), dim3(threads), s, a);
}
template <int DT, int L, int R, bool TINY = false>
hipError_t go_short(const NormGradArgs& a, hipStream_t s) {
  if (!TINY && !row_vectors_fit(a.cols, epv<DT>(), L, R)) return hipErrorInvalidValue;
  return launch<k_norm_grad_short<DT, L, R, TINY>>(dim3(a.workgroups), dim3(kNormShortThreads), s, a);
}

template <int DT>
hipError_t pick(const NormGradArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  if (a.cols < V) return go_short<DT, 8, 1, true>(a, s);
  const NormGradShape f = norm_grad_shape(a.cols, V);
  if (f.lanes == 8) return go_short<DT, 8, 1>(a, s);
  if (f.lanes == 16) return go_short<DT, 16, 1>(a, s);
  if (f.lanes == 32) return go_short<DT, 32, 1>(a, s);
  if (f.lanes == 64) return f.per_thread == 1 ? go_short<DT, 64, 1>(a, s) : go_short<DT, 64, 2>(a, s);
  if constexpr (V == 8)
    if (f.per_thread == 1) return go<DT, 1>(a, f.threads, s);
  if (f.per_thread == 2) return go<DT, 2>(a, f.threads, s);
  if (f.per_thread == 4) return go<DT, 4>(a, f.threads, s);
  if constexpr (V == 4) return go<DT, 8>(a, f.threads, s);
  return hipErrorInvalidValue;  // (rows of more than SIM_NORM_MAX_COLUMNS are refused before)
}

}  // namespace

hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s) {
  const hipError_t e = dtype == SIM_FP32   ? pick<SIM_FP32>(a, s)
                       : dtype == SIM_FP16 ? pick<SIM_FP16>(a, s)
                                           : pick<SIM_BF16>(a, s);
  if (e != hipSuccess || !a.dgain || a.workgroups == 1) return e;
  return launch<k_gain_sum>(dim3((unsigned)((a.cols + kSumColumns - 1) / kSumColumns)), dim3(kSumThreads), s,
                            (const float*)a.partial, a.workgroups, a.cols, a.dgain);
}

}  // namespace simar
