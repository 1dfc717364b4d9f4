// row_device.h -- device helpers of the kernels that keep a row's vectors in
// registers and write them back: vectors with zeros for what is not a thread's
// own, gains of any type.
#pragma once

#include <utility>

#include "loss_device.h"

namespace simar {

// Where a thread's V columns lie in a row: wholly inside; wherever the row ends
// (past cols - V the row's last vector is loaded in place of the thread's own,
// without a branch; the first `skip` elements are another thread's); or in a row
// of fewer than V columns.
enum Where { kInside, kEnd, kTiny };

template <int DT, Where K>
struct RowPart {
  static constexpr int V = epv<DT>();
  uint32_t col, cols;
  Tail<DT> t;
  __device__ __forceinline__ RowPart(uint32_t c, uint32_t n)
      : col(c), cols(n), t(K == kEnd ? c : 0, K == kEnd ? n : (uint32_t)V) {}
  __device__ __forceinline__ uint32_t at() const { return K == kEnd ? t.at : col; }
  // whether any column, and whether element i, is this thread's
  __device__ __forceinline__ bool any() const { return K == kInside || col < cols; }
  __device__ __forceinline__ bool own(int i) const {
    return K == kInside ? true : K == kEnd ? i >= t.skip : col + i < cols;
  }
  // STREAM: of rows that are read once
  template <bool STREAM = true>
  __device__ __forceinline__ u32x4 load(const void* row) const {
    if constexpr (K == kTiny) {
      float x[V];
#pragma unroll
      for (int i = 0; i < V; i++) x[i] = col + i < cols ? load_elem<DT>(row, col + i) : 0.0f;
      return pack<DT>(x);
    } else {
      return ld_row_lane<DT, STREAM>(row, 0, at());
    }
  }
  template <bool STREAM = true>
  __device__ __forceinline__ void store(void* row, const float (&x)[V]) const {
    if (K == kInside || (K == kEnd && t.skip == 0)) {
      st_row_lane<DT, STREAM>(row, 0, at(), pack_rounded<DT>(x));
    } else {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (own(i)) store_elem<DT>(row, (int64_t)at() + i, x[i]);
    }
  }
  // this thread's elements of a row of floats
  __device__ __forceinline__ void store_floats(float* row, const float (&x)[V]) const {
    if (K == kInside || (K == kEnd && t.skip == 0)) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float f[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
        st_row<SIM_FP32>(row, (int64_t)at() + i, pack<SIM_FP32>(f));
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (own(i)) row[at() + i] = x[i];
    }
  }
  // others' elements as zeros
  __device__ __forceinline__ void mask(float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = own(i) ? x[i] : 0.0f;
  }
};

// V floats of a gain at this part's columns; a NULL gain is all 1.
template <int DT, Where K>
__device__ __forceinline__ void load_gain(const void* gain, int gain_dtype, const RowPart<DT, K>& p,
                                          float (&g)[epv<DT>()]) {
  constexpr int V = epv<DT>();
#pragma unroll
  for (int i = 0; i < V; i++) g[i] = 1.0f;
  if (!gain) return;
  if constexpr (K == kTiny) {
#pragma unroll
    for (int i = 0; i < V; i++) {
      if (!p.own(i)) continue;
      const int64_t c = p.at() + i;
      g[i] = gain_dtype == SIM_FP32   ? load_elem<SIM_FP32>(gain, c)
             : gain_dtype == SIM_FP16 ? load_elem<SIM_FP16>(gain, c)
                                      : load_elem<SIM_BF16>(gain, c);
    }
  } else if (gain_dtype == SIM_FP32) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      float f[4];
      unpack<SIM_FP32>(ld_row<SIM_FP32>(gain, p.at() + j), f);
#pragma unroll
      for (int i = 0; i < 4; i++) g[j + i] = f[i];
    }
  } else if constexpr (V == 8) {
    const u32x4 v = ld_row<SIM_BF16>(gain, p.at());
    if (gain_dtype == SIM_FP16) unpack<SIM_FP16>(v, g);
    else unpack<SIM_BF16>(v, g);
  } else {
    // four 16-bit gains beside four fp32 elements
    typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
    const u32x2_at2 w = *(__attribute__((address_space(1))) const u32x2_at2*)((const char*)gain + (int64_t)p.at() * 2);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t word = w[i / 2], bits = i & 1 ? word >> 16 : word & 0xffffu;
      g[i] = gain_dtype == SIM_FP16 ? widen_bits<SIM_FP16>(bits) : widen_bits<SIM_BF16>(bits);
    }
  }
}

// f(integral_constant 0), ..., f(integral_constant R - 1)
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
// A row's R vectors of a thread: vector i of thread l is the row's vector
// i * threads + l.  Only the last one may lie at the row's end or past it.
template <int DT, int R, bool TINY>
struct RowVectors {
  uint32_t l, threads, cols;
  template <class F>
  __device__ __forceinline__ void operator()(F f) const {
    each_of(std::make_integer_sequence<int, R>(), [&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      f(i, RowPart<DT, TINY ? kTiny : I == R - 1 ? kEnd : kInside>((I * threads + l) * epv<DT>(), cols));
    });
  }
  // every thread's vectors lie wholly inside
  __device__ __forceinline__ bool exact() const { return !TINY && cols == threads * (uint32_t)(R * epv<DT>()); }
};
}  // namespace simar
