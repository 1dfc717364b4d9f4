// k_norm.hip -- root-mean-square norm of x + residual, in the activations' type
// or in e4m3 with scales (gfx950).
//
// Row h = x + residual in fp32: r = (sum h^2 / n + eps)^(-1/2), y = g h r.  The
// sum is rounded to the activations' type only as it is written; y is taken of
// the unrounded one.  In 8 bits, with m the largest |g h| of a scale's columns:
// scale = m r / 448 and q = e4m3(g h * 448 / m), so that q needs no r and y is
// not rounded in between.
//
// A row stays in the registers of a wave or a workgroup from its one read to
// its writes.
#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

// e4m3 of V floats of at most 448
template <int V>
__device__ __forceinline__ void to_e4m3(const float (&x)[V], uint32_t (&w)[V / 4]) {
#pragma unroll
  for (int i = 0; i < V / 4; i++) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], v, true);
  }
}
template <int DT, bool TINY>
__device__ __forceinline__ void store_e4m3(void* row, const RowPart<DT, TINY>& p, const float (&x)[epv<DT>()]) {
  constexpr int V = epv<DT>();
  typedef uint32_t Words __attribute__((ext_vector_type(V / 4), aligned(1)));
  uint32_t w[V / 4];
  to_e4m3(x, w);
  uint8_t* at = (uint8_t*)row + p.column(0);
  if (p.own(0) && p.own(V - 1)) {
    Words v;
    if constexpr (V == 8) v = Words{w[0], w[1]};
    else v = Words{w[0]};
    *(__attribute__((address_space(1))) Words*)at = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (p.own(i)) at[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// the largest of `lanes` (4 to 32) neighbouring lanes
__device__ __forceinline__ float max_of(float v, int lanes) {
  v = fmaxf(v, dpp<kDppPair>(v));
  v = fmaxf(v, dpp<kDppQuad>(v));
  if (lanes >= 8) v = fmaxf(v, dpp<kDppHalfRow>(v));
  if (lanes >= 16) v = fmaxf(v, dpp<kDppRow>(v));
  if (lanes >= 32) v = across_rows(v, [](float a, float b) { return fmaxf(a, b); });
  return v;
}

// factors of g h on its way to e4m3: q = e4m3(g h * up * inv).  A largest value
// near the type's smallest ones is scaled up first, so that 448 over it is finite.
struct Quant {
  float up, inv;
  __device__ __forceinline__ explicit Quant(float top) {
    up = top < 0x1p-80f ? 0x1p80f : 1.0f;
    inv = top > 0.0f ? 448.0f / (top * up) : 0.0f;
  }
};

// NT threads hold a row, R vectors each; four rows share a workgroup where a
// wave holds one.
template <int DT, int NT, int R, bool TINY>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_norm(NormArgs a) {
  constexpr int V = epv<DT>(), W = NT / 64, ROWS = NT < 256 ? 256 / NT : 1;
  __shared__ float sum_s[2][W], top_s[2][W];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = NT == 64 ? 0 : tid >> 6, l = NT == 64 ? lane : tid;
  const uint32_t cols = (uint32_t)a.cols;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + (NT == 64 ? tid >> 6 : 0); row < a.rows;
       row += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    const char* x = (const char*)a.x + row * a.x_stride * Ty<DT>::E;
    float h[R][V], g[R][V];
    u32x4 v[R];
#pragma unroll
    for (int i = 0; i < R; i++) v[i] = RowPart<DT, TINY>((i * NT + l) * V, cols).load(x);
    if (a.residual) {
      const char* res = (const char*)a.residual + row * a.residual_stride * Ty<DT>::E;
      u32x4 w[R];
#pragma unroll
      for (int i = 0; i < R; i++) w[i] = RowPart<DT, TINY>((i * NT + l) * V, cols).load(res);
#pragma unroll
      for (int i = 0; i < R; i++) load_gain(a.gain, a.gain_dtype, RowPart<DT, TINY>((i * NT + l) * V, cols), g[i]);
#pragma unroll
      for (int i = 0; i < R; i++) {
        float f[V];
        unpack<DT>(v[i], h[i]);
        unpack<DT>(w[i], f);
#pragma unroll
        for (int t = 0; t < V; t++) h[i][t] += f[t];
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; i++) load_gain(a.gain, a.gain_dtype, RowPart<DT, TINY>((i * NT + l) * V, cols), g[i]);
#pragma unroll
      for (int i = 0; i < R; i++) unpack<DT>(v[i], h[i]);
    }
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int i = 0; i < R; i++) {
      const RowPart<DT, TINY> p((i * NT + l) * V, cols);
#pragma unroll
      for (int t = 0; t < V; t++) {
        const float f = p.own(t) ? h[i][t] : 0.0f;
        sum = __builtin_fmaf(f, f, sum);
        g[i][t] *= h[i][t];
      }
    }
    if (a.scales && a.group == 0) {
#pragma unroll
      for (int i = 0; i < R; i++) {
        const RowPart<DT, TINY> p((i * NT + l) * V, cols);
#pragma unroll
        for (int t = 0; t < V; t++) top = fmaxf(top, p.own(t) ? fabsf(g[i][t]) : 0.0f);
      }
      top = wave_max(top);
    }
    sum = wave_sum(sum);
    if constexpr (W > 1) {
      if (lane == 0) {
        sum_s[turn][wave] = sum;
        top_s[turn][wave] = top;
      }
      __syncthreads();
      sum = wave_sum(lane < W ? sum_s[turn][lane] : 0.0f);
      if (a.scales && a.group == 0) top = wave_max(lane < W ? top_s[turn][lane] : 0.0f);
    }
    const float r = 1.0f / __builtin_sqrtf(sum / (float)cols + a.eps);
    if (a.sum) {
      char* to = (char*)a.sum + row * a.sum_stride * Ty<DT>::E;
#pragma unroll
      for (int i = 0; i < R; i++) {
        const RowPart<DT, TINY> p((i * NT + l) * V, cols);
        if (p.any()) p.store(to, h[i]);
      }
    }
    if (!a.scales) {
      char* to = (char*)a.out + row * a.out_stride * Ty<DT>::E;
#pragma unroll
      for (int i = 0; i < R; i++) {
        const RowPart<DT, TINY> p((i * NT + l) * V, cols);
#pragma unroll
        for (int t = 0; t < V; t++) g[i][t] *= r;
        if (p.any()) p.store(to, g[i]);
      }
      continue;
    }
    char* to = (char*)a.out + row * a.out_stride;
    float* scales = a.scales + row * a.groups;
#pragma unroll
    for (int i = 0; i < R; i++) {
      const RowPart<DT, TINY> p((i * NT + l) * V, cols);
      float m = top;
      if (a.group) {
        m = 0.0f;
#pragma unroll
        for (int t = 0; t < V; t++) m = fmaxf(m, p.own(t) ? fabsf(g[i][t]) : 0.0f);
        m = max_of(m, a.group / V);
        if (p.any() && p.col % (uint32_t)a.group == 0) scales[p.col / (uint32_t)a.group] = m * r / 448.0f;
      } else if (p.col == 0) {
        scales[0] = m * r / 448.0f;
      }
      const Quant q(m);
#pragma unroll
      for (int t = 0; t < V; t++) g[i][t] = g[i][t] * q.up * q.inv;
      if (p.any()) store_e4m3(to, p, g[i]);
    }
  }
}

template <int DT, int NT, int R, bool TINY = false>
hipError_t go(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = NT < 256 ? 256 / NT : 1;
  const int64_t wg = (a.rows + ROWS - 1) / ROWS;
  const int64_t most = (int64_t)1 << 21;  // (a launch has fewer than 2^32 threads)
  return launch<k_norm<DT, NT, R, TINY>>(dim3((unsigned)(wg < most ? wg : most)), dim3(NT < 256 ? 256 : NT), s, a);
}

template <int DT>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = ((int64_t)a.cols + V - 1) / V;
  if (a.cols < V) return go<DT, 64, 1, true>(a, s);
  if (nv <= 64) return go<DT, 64, 1>(a, s);
  if (nv <= 128) return go<DT, 64, 2>(a, s);
  if (a.rows >= 4 * library_cus()) {
    if (nv <= 256) return go<DT, 256, 1>(a, s);
    if (nv <= 512) return go<DT, 256, 2>(a, s);
    if (nv <= 768) return go<DT, 256, 3>(a, s);
    if (nv <= 1024) return go<DT, 256, 4>(a, s);
    if constexpr (V == 4)
      if (nv <= 2048) return go<DT, 256, 8>(a, s);
  }
  if (nv <= 256) return go<DT, 256, 1>(a, s);
  if (nv <= 1024) return go<DT, 1024, 1>(a, s);
  if (nv <= 2048) return go<DT, 1024, 2>(a, s);
  if (nv <= 4096) return go<DT, 1024, 4>(a, s);
  if constexpr (V == 4) return go<DT, 1024, 8>(a, s);
  return hipErrorInvalidValue;  // (rows of more than SIM_NORM_MAX_COLUMNS are refused before)
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  return dtype == SIM_FP32 ? pick<SIM_FP32>(a, s) : dtype == SIM_FP16 ? pick<SIM_FP16>(a, s) : pick<SIM_BF16>(a, s);
}

}  // namespace simar
