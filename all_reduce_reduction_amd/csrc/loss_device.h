// loss_device.h -- device helpers shared by the routing and distillation
// kernels: rows of 16-byte vectors of any alignment, wave reductions, the
// base-2 exponential.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace simar {

constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// A row of logits may start at any element (a column slice, an odd stride):
// its 16-byte accesses are typed with the alignment of one element.  gfx950
// serves them from the same global_load/store_dwordx4.
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
template <int E> struct RowVec;
template <> struct RowVec<2> {
  typedef u32x4_at2 V;
  typedef __attribute__((address_space(1))) const u32x4_at2 CG;
  typedef __attribute__((address_space(1))) u32x4_at2 G;
};
template <> struct RowVec<4> {
  typedef u32x4_at4 V;
  typedef __attribute__((address_space(1))) const u32x4_at4 CG;
  typedef __attribute__((address_space(1))) u32x4_at4 G;
};
template <int DT>
__device__ __forceinline__ u32x4 ld_row(const void* row, int64_t elem) {
  return *(typename RowVec<Ty<DT>::E>::CG*)((const char*)row + elem * Ty<DT>::E);
}
template <int DT>
__device__ __forceinline__ void st_row(void* row, int64_t elem, u32x4 v) {
  *(typename RowVec<Ty<DT>::E>::G*)((char*)row + elem * Ty<DT>::E) = v;
}

// The same with a workgroup-uniform element offset (kept in scalar registers)
// and a lane's own, which has 32 bits; NT: streaming (nontemporal).
template <int DT, bool NT>
__device__ __forceinline__ u32x4 ld_row_lane(const void* row, int64_t elem, uint32_t lane_elem) {
  const char* p = (const char*)row + elem * Ty<DT>::E;
  typename RowVec<Ty<DT>::E>::CG* q = (typename RowVec<Ty<DT>::E>::CG*)(p + lane_elem * (uint32_t)Ty<DT>::E);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  else return *q;
}
template <int DT, bool NT>
__device__ __forceinline__ void st_row_lane(void* row, int64_t elem, uint32_t lane_elem, u32x4 v) {
  char* p = (char*)row + elem * Ty<DT>::E;
  typename RowVec<Ty<DT>::E>::G* q = (typename RowVec<Ty<DT>::E>::G*)(p + lane_elem * (uint32_t)Ty<DT>::E);
  if constexpr (NT) __builtin_nontemporal_store((typename RowVec<Ty<DT>::E>::V)v, q);
  else *q = v;
}

// fp32 values rounded to storage, two at a time.
template <int DT>
__device__ __forceinline__ u32x4 pack_rounded(const float (&f)[epv<DT>()]) {
  if constexpr (Ty<DT>::E == 4) {
    return pack<DT>(f);
  } else {
    typedef float F2 __attribute__((ext_vector_type(2)));
    typedef _Float16 H2 __attribute__((ext_vector_type(2)));
    typedef __bf16 B2 __attribute__((ext_vector_type(2)));
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const F2 p = {f[2 * i], f[2 * i + 1]};
      if constexpr (DT == SIM_FP16) v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, H2));
      else v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, B2));
    }
    return v;
  }
}

template <int DT> constexpr uint32_t neg_inf_bits() {
  return DT == SIM_FP32 ? 0xff800000u : DT == SIM_FP16 ? 0xfc00fc00u : 0xff80ff80u;
}
// The vector at column `col` of a row that ends at column `cols`: what lies
// past the end reads as -inf (which changes no maximum and no sum) and is not
// written.
template <int DT>
__device__ __forceinline__ u32x4 ld_guarded(const void* row, int64_t col, int64_t cols) {
  constexpr int V = epv<DT>();
  const uint32_t n = neg_inf_bits<DT>();
  u32x4 v = {n, n, n, n};
  if (col + V <= cols) {
    v = ld_row<DT>(row, col);
  } else if (col < cols) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = col + i < cols ? load_elem<DT>(row, col + i) : kNegInf;
    v = pack<DT>(x);
  }
  return v;
}
template <int DT>
__device__ __forceinline__ void load_cols(const void* row, int64_t col, int64_t cols, float (&x)[epv<DT>()]) {
  unpack<DT>(ld_guarded<DT>(row, col, cols), x);
}
template <int DT>
__device__ __forceinline__ void st_guarded(void* row, int64_t col, int64_t cols, const float (&x)[epv<DT>()]) {
  constexpr int V = epv<DT>();
  if (col + V <= cols) {
    st_row<DT>(row, col, pack_rounded<DT>(x));
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (col + i < cols) store_elem<DT>(row, col + i, x[i]);
  }
}

// The vector at column `col` of a row of `cols` >= V columns, without a branch:
// past cols - V it is the row's last vector instead, which other columns'
// threads have too.  The first `skip` elements are not this thread's; none is
// from column `hi` on.
template <int DT>
struct Tail {
  uint32_t at;  // (a row has fewer than 2^31 columns)
  int skip;
  __device__ __forceinline__ Tail(uint32_t col, uint32_t hi, uint32_t cols) {
    constexpr uint32_t V = epv<DT>();
    at = col < cols - V ? col : cols - V;
    skip = (int)(col < hi ? col - at : V);
  }
  __device__ __forceinline__ Tail(uint32_t col, uint32_t cols) : Tail(col, cols, cols) {}
  __device__ __forceinline__ u32x4 load(const void* row) const { return ld_row<DT>(row, at); }
  // the others' elements as -inf
  __device__ __forceinline__ void mask(float (&x)[epv<DT>()]) const {
#pragma unroll
    for (int i = 0; i < epv<DT>(); i++) x[i] = i >= skip ? x[i] : kNegInf;
  }
  __device__ __forceinline__ void store(void* row, const float (&x)[epv<DT>()]) const {
    if (skip == 0) {
      st_row<DT>(row, at, pack_rounded<DT>(x));
    } else {
#pragma unroll
      for (int i = 0; i < epv<DT>(); i++)
        if (i >= skip) store_elem<DT>(row, (int64_t)at + i, x[i]);
    }
  }
};

// 2^x (v_exp_f32: 1 ulp; results below the normal range are flushed, far
// under what a sum that holds 1 can see)
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Reductions over groups of L = 4, 8, 16, 32 or 64 neighbouring lanes without
// LDS: with the partner in the pair, in the quad, in the mirrored half row and
// in the mirrored row by DPP, then between the two rows of 16 of a half wave
// and between the half waves by lane swaps.  Both partners combine the same
// two values, so all lanes of a group end with the same bits, and the order of
// a sum is fixed.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
constexpr int kDppPair = 0xB1, kDppQuad = 0x4E, kDppHalfRow = 0x141, kDppRow = 0x140;
// (the even rows' value, the odd rows' value) of each pair of rows
template <class T, class F>
__device__ __forceinline__ T across_rows(T v, F f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t lo = r[0], hi = r[1];
  return f(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
}
template <class T, class F>
__device__ __forceinline__ T across_halves(T v, F f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t lo = r[0], hi = r[1];
  return f(__builtin_bit_cast(T, lo), __builtin_bit_cast(T, hi));
}
template <int L, class T, class F>
__device__ __forceinline__ T group_reduce(T v, F f) {
  v = f(v, dpp<kDppPair>(v));
  v = f(v, dpp<kDppQuad>(v));
  if constexpr (L >= 8) v = f(v, dpp<kDppHalfRow>(v));
  if constexpr (L >= 16) v = f(v, dpp<kDppRow>(v));
  if constexpr (L >= 32) v = across_rows(v, f);
  if constexpr (L >= 64) v = across_halves(v, f);
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) { return group_sum<64>(v); }
__device__ __forceinline__ float wave_max(float v) { return group_max<64>(v); }

// LDS accesses of a wave before this line and after it stay apart
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Exponentials against a maximum m as one multiply-add: 2^(x c - t) with
// t = m c - 8, so that what lies up to 2^-134 below the maximum is still a
// normal number (the hardware's 2^x flushes others; a larger distance would
// cost the exponents near the maximum their last bits).  t's own rounding is
// no error of the sums, which are taken against t, not m; at_max() is the
// exact distance m c - t (at most 72, as |m c| stays below 2^31) for what has
// to be taken against m.  Where a finite m has |m c| >= 2^31 (far()), c is cut to a
// power of two, which makes t = m c exact: neighbouring floats lie 128 / c
// apart there or more, so the result is 1 at m and 0 below it with either.
// For m = -inf, t is 0 (2^-inf is 0); for +inf the results are NaN.  c lies
// below 2^67.
constexpr float kFar = 2147483648.0f;
__device__ __forceinline__ bool far(float m, float c) { return fabsf(m) < __builtin_inff() && !(fabsf(m * c) < kFar); }
struct Against {
  float c, t;
};
__device__ __forceinline__ Against against(float m, float c) {
  Against r{c, m == kNegInf ? 0.0f : m * c - 8.0f};
  if (__builtin_expect(far(m, c), 0)) {
    r.c = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, c) & 0xff800000u);
    if (fabsf(m) >= 0x1p60f) r.c = fminf(r.c, 1.0f);
    r.t = m * r.c;
  }
  return r;
}
__device__ __forceinline__ float exp_against(float x, const Against& r) {
  return exp2_hw(__builtin_fmaf(x, r.c, -r.t));
}
__device__ __forceinline__ float at_max(float m, const Against& r) {
  return m == kNegInf ? 0.0f : __builtin_fmaf(m, r.c, -r.t);
}

// A softmax's running maximum m and sum s of 2^((x - m) c), over the x seen
// so far (m = -inf, s = 0 for none).  A NaN never enters m and makes s NaN;
// so does +inf.
struct Running {
  float m, s;
};
// factor that brings a sum taken against m over to the maximum top >= m
__device__ __forceinline__ float rebase(float m, float top, float c) {
  return m == top ? 1.0f : exp2_hw((m - top) * c);
}
__device__ __forceinline__ Running wave_running(Running r, float c) {
  const float top = wave_max(r.m);
  r.s = wave_sum(r.s * rebase(r.m, top, c));
  r.m = top;
  return r;
}
// One thread's sum on its way, taken against t = m c.  A maximum that is -inf
// or far() leaves the sum 0: below zero that is what it is worth against any
// other maximum, and a row whose own maximum is far() is counted again.
struct Scan {
  float m = kNegInf, s = 0.0f, t = -kFar;
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N], float c) {
#pragma unroll
    for (int i = 0; i < N; i++) m = fmaxf(m, x[i]);
    float next = fmaxf(m * c, -kFar);
    next = next < kFar ? next : __builtin_inff();
    s *= exp2_hw(fminf(t - next, 0.0f));
    t = next;
#pragma unroll
    for (int i = 0; i < N; i++) s += exp2_hw(__builtin_fmaf(x[i], c, -t));
  }
  // against m; a NaN stays one
  __device__ __forceinline__ Running done(float c) const {
    return Running{m, s * (fabsf(m * c) < kFar ? exp2_hw(-__builtin_fmaf(m, c, -t)) : 0.0f)};
  }
};
// how many of the values are the maximum, in a row where it is far()
template <int N>
__device__ __forceinline__ float count_of(const float (&x)[N], float m) {
  float n = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) n += x[i] == m ? 1.0f : 0.0f;
  return n;
}

}  // namespace simar
