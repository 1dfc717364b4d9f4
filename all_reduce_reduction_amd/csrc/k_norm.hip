// k_norm.hip -- root-mean-square norm of x + residual, in the activations' type
// or in e4m3 with scales (gfx950).
//
// Row h = x + residual in fp32: r = (sum h^2 / n + eps)^(-1/2), y = g (h r): |h r| is
// at most sqrt n, so that no product on the way is past fp32's range if y is not.  The
// sum is rounded to the activations' type only as it is written; y is taken of the
// unrounded one.  In 8 bits, with m the largest |g h| of a scale's columns:
// scale = m r / 448 and q = e4m3(g h * 448 / m), so that q needs no r and y is
// not rounded in between: of 16-bit values q is the nearest code, of two the even one.
//
// A row stays in the registers of its lanes (8 to 64) or of its workgroup from its
// one read to its writes; a workgroup is cut to the row's length in whole waves, so
// that only a thread's last vector may lie at the row's end.
//
// Bound by memory that reads and writes at once: 151 us for 16,384 rows x 8,192
// bf16 with residual to e4m3 (944 MB at 6.3 TB/s; a copy of as many bytes 142), the
// vector units beside it busy for 65 % of that.  fp32 and fp16 rows of more than 16,384
// columns spill registers (44, 8): 1,024 x 32,768 fp32 134 us, fp16 52, bf16 47.5.  One
// row of 8,192: 3.7 us on the GPU (load, sum over eight waves, store), 4.2 a call.
#include "launch.h"
#include "layer.h"
#include "row_device.h"

namespace simar {
namespace {

constexpr float kE4m3Max = 448.0f;

// e4m3 of V floats of at most 448 (and its rounding error), four to a word
template <int DT, Where K>
__device__ __forceinline__ void store_e4m3(void* row, const RowPart<DT, K>& p, const float (&x)[epv<DT>()]) {
  constexpr int V = epv<DT>();
  typedef uint32_t Words __attribute__((ext_vector_type(V / 4), aligned(1)));
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; i++) {
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], v, true);
  }
  uint8_t* at = (uint8_t*)row + p.at();
  if (K == kInside || (K == kEnd && p.t.skip == 0)) {
    Words v;
    if constexpr (V == 8) v = Words{w[0], w[1]};
    else v = Words{w[0]};
    __builtin_nontemporal_store(v, (__attribute__((address_space(1))) Words*)at);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (p.own(i)) at[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// the largest of `lanes` (4, 8, 16 or 32) neighbouring lanes
__device__ __forceinline__ float max_of(float v, int lanes) {
  v = fmaxf(v, dpp<kDppPair>(v));
  v = fmaxf(v, dpp<kDppQuad>(v));
  if (lanes >= 8) v = fmaxf(v, dpp<kDppHalfRow>(v));
  if (lanes >= 16) v = fmaxf(v, dpp<kDppRow>(v));
  if (lanes >= 32) v = across_rows(v, [](float a, float b) { return fmaxf(a, b); });
  return v;
}
template <int V>
__device__ __forceinline__ float largest(const float (&x)[V]) {
  float m = 0.0f;
#pragma unroll
  for (int t = 0; t < V; t++) m = fmaxf(m, fabsf(x[t]));
  return m;
}

// g h on its way to e4m3: g h * 448 / m, rounded once.  Values in 16 bits often lie
// halfway between two codes exactly, and go to the even one only if the quotient has
// no error of its own: 448 / m as the hardware's reciprocal (1 ulp) and what it
// leaves, together off by 2^-44, so that the fused sum is the nearest float and a
// halfway value stays one.
template <int V>
__device__ __forceinline__ void quantise(float (&x)[V], float m) {
  const float inv = __builtin_amdgcn_rcpf(m), hi = kE4m3Max * inv, lo = __builtin_fmaf(-hi, m, kE4m3Max) * inv;
#pragma unroll
  for (int t = 0; t < V; t++) x[t] = __builtin_fmaf(x[t], hi, x[t] * lo);
}

// Near the ends of fp32's range (m = max |g h| outside [2^-100, 2^100)) g h may have
// overflowed or lost bits although g (h r) is a normal number, and 448 / m be one that
// the reciprocal takes for 0.  There g h is formed again, as a multiple of `unit`: the
// smaller of both by 2^126, or the larger by 2^-126.  (Groups of zeros go that way too,
// for those that g h alone made so.)
__device__ __forceinline__ bool mid_range(float m) { return m >= 0x1p-100f && m < 0x1p100f; }
struct Range {
  float by, unit;
  bool low;
  __device__ __forceinline__ explicit Range(float m)
      : by(mid_range(m) ? 1.0f : m < 1.0f ? 0x1p126f : 0x1p-126f),
        unit(mid_range(m) ? 1.0f : m < 1.0f ? 0x1p-126f : 0x1p126f), low(m < 1.0f) {}
  __device__ __forceinline__ float operator()(float g, float h) const {
    const bool first = (fabsf(g) < fabsf(h)) == low;
    return (first ? g : h) * by * (first ? h : g);
  }
};
// A group without a largest value that quantise could divide by: zeros stay, and
// finite values beside an infinite one become 0.
template <int V>
__device__ __forceinline__ void settle(float (&x)[V], float& m) {
  const bool sane = m > 0.0f && m < __builtin_inff();
#pragma unroll
  for (int t = 0; t < V; t++) x[t] = sane ? x[t] : x[t] * 0.0f;
  m = sane ? m : kE4m3Max;
}

// L lanes (8, 16, 32 or 64; several rows share a workgroup of 256 threads) or, with
// L = 0, a workgroup take a row, R vectors per thread.
template <int DT, int L, int R, bool TINY>
__global__ void __launch_bounds__(L ? 256 : 1024) k_norm(NormArgs a) {
  constexpr int V = epv<DT>(), G = L ? L : 64;
  // With one vector the gain stays in registers; with more the gain is loaded again, so
  // that two workgroups have room (16,384 x 8,192 bf16 151 us, 184 held).
  constexpr bool HOLD = R == 1;
  __shared__ float sum_s[2][16], top_s[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int waves = blockDim.x >> 6;
  const RowVectors<DT, R, TINY> vectors{L ? threadIdx.x % G : threadIdx.x, L ? L : blockDim.x, (uint32_t)a.cols};
  const bool exact = vectors.exact(), one_scale = a.scales && a.group == 0;
  // (a group of more columns than the row has is the row)
  const int scale_lanes = L && a.group / V > L ? L : a.group / V;
  int turn = 0;
  for (int64_t row = L ? (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G : (int64_t)blockIdx.x; row < a.rows;
       row += L ? (int64_t)gridDim.x * (256 / G) : (int64_t)gridDim.x, turn ^= 1) {
    const char* x = (const char*)a.x + row * a.x_stride * Ty<DT>::E;
    float h[R][V], held[HOLD ? R : 1][V];
    u32x4 v[R], w[R];
    vectors([&](auto i, auto p) __attribute__((always_inline)) { v[i] = p.load(x); });
    if (a.residual) {
      const char* res = (const char*)a.residual + row * a.residual_stride * Ty<DT>::E;
      vectors([&](auto i, auto p) __attribute__((always_inline)) { w[i] = p.load(res); });
    } else {
#pragma unroll
      for (int i = 0; i < R; i++) w[i] = u32x4{0, 0, 0, 0};
    }
    if constexpr (HOLD)
      vectors([&](auto i, auto p) __attribute__((always_inline)) { load_gain(a.gain, a.gain_dtype, p, held[i]); });
    float sum = 0.0f, top = 0.0f;
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
      float f[V];
      unpack<DT>(v[i], h[i]);
      unpack<DT>(w[i], f);
#pragma unroll
      for (int t = 0; t < V; t++) h[i][t] += f[t];
      if (i == R - 1 && !exact) p.mask(h[i]);
#pragma unroll
      for (int t = 0; t < V; t++) sum = __builtin_fmaf(h[i][t], h[i][t], sum);
    });
    const auto gains = [&](auto i, auto p, float (&g)[V]) __attribute__((always_inline)) {
      if constexpr (HOLD) {
#pragma unroll
        for (int t = 0; t < V; t++) g[t] = held[i][t];
      } else {
        load_gain(a.gain, a.gain_dtype, p, g);
      }
    };
    // g h
    const auto gained = [&](auto i, auto p, float (&x)[V]) __attribute__((always_inline)) {
      gains(i, p, x);
#pragma unroll
      for (int t = 0; t < V; t++) x[t] *= h[i][t];
    };
    const auto ranged = [&](auto i, auto p, const Range& in, float (&x)[V]) __attribute__((always_inline)) {
      gains(i, p, x);
#pragma unroll
      for (int t = 0; t < V; t++) x[t] = in(x[t], h[i][t]);
    };
    sum = group_sum<G>(sum);
    if (one_scale) {
      vectors([&](auto i, auto p) __attribute__((always_inline)) {
        float x[V];
        gained(i, p, x);
        top = fmaxf(top, largest(x));
      });
      top = group_max<G>(top);
    }
    if (!L && waves > 1) {
      if (lane == 0) {
        sum_s[turn][wave] = sum;
        top_s[turn][wave] = top;
      }
      __syncthreads();
      sum = group_sum<16>((lane & 15) < waves ? sum_s[turn][lane & 15] : 0.0f);
      if (one_scale) top = group_max<16>((lane & 15) < waves ? top_s[turn][lane & 15] : 0.0f);
    }
    const float r = 1.0f / __builtin_sqrtf(sum / (float)a.cols + a.eps);
    if (a.sum) {
      char* to = (char*)a.sum + row * a.sum_stride * Ty<DT>::E;
      vectors([&](auto i, auto p) __attribute__((always_inline)) {
        if (p.any()) p.store(to, h[i]);
      });
    }
    if (!a.scales) {
      char* to = (char*)a.out + row * a.out_stride * Ty<DT>::E;
      vectors([&](auto i, auto p) __attribute__((always_inline)) {
        float x[V];
        gains(i, p, x);
#pragma unroll
        for (int t = 0; t < V; t++) x[t] *= h[i][t] * r;
        if (p.any()) p.store(to, x);
      });
      continue;
    }
    char* to = (char*)a.out + row * a.out_stride;
    float* scales = a.scales + row * a.groups;
    const float unit = r * (1.0f / kE4m3Max);
    // (all threads of a workgroup have one `top`)
    const Range row_in(one_scale ? top : 1.0f);
    const bool row_far = one_scale && __ballot(!mid_range(top)) != 0;
    if (__builtin_expect(row_far, 0)) {
      top = 0.0f;
      vectors([&](auto i, auto p) __attribute__((always_inline)) {
        float x[V];
        ranged(i, p, row_in, x);
        top = fmaxf(top, largest(x));
      });
      top = group_max<G>(top);
      if (!L && waves > 1) {
        __syncthreads();  // (the first one's maxima have been read)
        if (lane == 0) top_s[turn][wave] = top;
        __syncthreads();
        top = group_max<16>((lane & 15) < waves ? top_s[turn][lane & 15] : 0.0f);
      }
    }
    vectors([&](auto i, auto p) __attribute__((always_inline)) {
      float x[V], m = top;
      gained(i, p, x);
      if (a.group) m = max_of(largest(x), scale_lanes);
      float scale = m * unit;
      if (__builtin_expect(a.group ? __ballot(p.any() && !mid_range(m)) != 0 : row_far, 0)) {
        const Range in = a.group ? Range(m) : row_in;
        ranged(i, p, in, x);
        if (a.group) m = max_of(largest(x), scale_lanes);
        scale = m * unit * in.unit;
        settle(x, m);
      }
      if (a.group) {
        if (p.any() && p.col % (uint32_t)a.group == 0) scales[p.col / (uint32_t)a.group] = scale;
      } else if (p.col == 0) {
        scales[0] = scale;
      }
      quantise(x, m);
      if (p.any()) store_e4m3(to, p, x);
    });
  }
}

template <int DT, int L, int R, bool TINY = false>
hipError_t go(const NormArgs& a, int threads, hipStream_t s) {
  if (!TINY && !row_vectors_fit(a.cols, epv<DT>(), threads, R)) return hipErrorInvalidValue;
  const int64_t each = L ? 256 / L : 1, wg = (a.rows + each - 1) / each;
  const int64_t most = (int64_t)1 << 21;  // (a launch has fewer than 2^32 threads)
  return launch<k_norm<DT, L, R, TINY>>(dim3((unsigned)(wg < most ? wg : most)), dim3(L ? 256 : threads), s, a);
}

template <int DT>
hipError_t pick(const NormArgs& a, hipStream_t s) {
  constexpr int V = epv<DT>();
  const int64_t nv = ((int64_t)a.cols + V - 1) / V;
  if (a.cols < V) return go<DT, 8, 1, true>(a, 8, s);
  if (nv <= 8) return go<DT, 8, 1>(a, 8, s);
  if (nv <= 16) return go<DT, 16, 1>(a, 16, s);
  if (nv <= 32) return go<DT, 32, 1>(a, 32, s);
  if (nv <= 64) return go<DT, 64, 1>(a, 64, s);
  if (nv <= 128) return go<DT, 64, 2>(a, 64, s);
  // Two vectors per thread leave room for another row's workgroup on the same
  // compute unit (16,384 x 8,192 bf16 151 us, 220 with one; a few rows by
  // themselves take the same with either, 1 x 8,192 3.7 us).
  if (nv <= 2048) return go<DT, 0, 2>(a, row_threads(nv, 2), s);
  if (nv <= 4096) return go<DT, 0, 4>(a, row_threads(nv, 4), s);
  if constexpr (V == 4) return go<DT, 0, 8>(a, row_threads(nv, 8), s);
  return hipErrorInvalidValue;  // (rows of more than SIM_NORM_MAX_COLUMNS are refused before)
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  return dtype == SIM_FP32 ? pick<SIM_FP32>(a, s) : dtype == SIM_FP16 ? pick<SIM_FP16>(a, s) : pick<SIM_BF16>(a, s);
}

}  // namespace simar
