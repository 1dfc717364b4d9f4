// row_device.h -- device helpers of the kernels that keep a row's vectors in
// registers and write them back: vectors at a row's end with zeros for what is
// not a thread's own, gains of any type, sums over a workgroup.
#pragma once

#include "loss_device.h"

namespace simar {

// V elements of a row from column `col` on, as floats; what lies past the end,
// and what another column's thread has too (a row's last vector is loaded where
// it ends with the row), is 0.  TINY: rows of fewer than V columns.
template <int DT, bool TINY>
struct RowPart {
  static constexpr int V = epv<DT>();
  Tail<DT> t;
  uint32_t col, cols;
  __device__ __forceinline__ RowPart(uint32_t c, uint32_t n) : t(TINY ? 0 : c, TINY ? V : n), col(c), cols(n) {}
  __device__ __forceinline__ bool any() const { return col < cols; }
  __device__ __forceinline__ u32x4 load(const void* row) const {
    if constexpr (TINY) {
      float x[V];
#pragma unroll
      for (int i = 0; i < V; i++) x[i] = col + i < cols ? load_elem<DT>(row, col + i) : 0.0f;
      return pack<DT>(x);
    } else {
      return t.load(row);
    }
  }
  // whether element i is this thread's
  __device__ __forceinline__ bool own(int i) const {
    if constexpr (TINY) return col + i < cols;
    else return i >= t.skip;
  }
  // the column of element i
  __device__ __forceinline__ uint32_t column(int i) const { return (TINY ? col : t.at) + i; }
  __device__ __forceinline__ void store(void* row, const float (&x)[V]) const {
    if constexpr (TINY) {
#pragma unroll
      for (int i = 0; i < V; i++)
        if (col + i < cols) store_elem<DT>(row, col + i, x[i]);
    } else {
      t.store(row, x);
    }
  }
};

// V floats of the gain at this part's columns; a NULL gain is all 1.
template <int DT, bool TINY>
__device__ __forceinline__ void load_gain(const void* gain, int gain_dtype, const RowPart<DT, TINY>& p,
                                          float (&g)[epv<DT>()]) {
  constexpr int V = epv<DT>();
#pragma unroll
  for (int i = 0; i < V; i++) g[i] = 1.0f;
  if (!gain) return;
  if constexpr (TINY) {
#pragma unroll
    for (int i = 0; i < V; i++) {
      if (!p.own(i)) continue;
      const int64_t c = p.column(i);
      g[i] = gain_dtype == SIM_FP32   ? load_elem<SIM_FP32>(gain, c)
             : gain_dtype == SIM_FP16 ? load_elem<SIM_FP16>(gain, c)
                                      : load_elem<SIM_BF16>(gain, c);
    }
  } else if (gain_dtype == SIM_FP32) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      float f[4];
      unpack<SIM_FP32>(ld_row<SIM_FP32>(gain, p.t.at + j), f);
#pragma unroll
      for (int i = 0; i < 4; i++) g[j + i] = f[i];
    }
  } else if constexpr (V == 8) {
    const u32x4 v = ld_row<SIM_BF16>(gain, p.t.at);
    if (gain_dtype == SIM_FP16) unpack<SIM_FP16>(v, g);
    else unpack<SIM_BF16>(v, g);
  } else {
    // four 16-bit gains beside four fp32 elements
    typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
    const u32x2_at2 w = *(__attribute__((address_space(1))) const u32x2_at2*)((const char*)gain + (int64_t)p.t.at * 2);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t word = w[i / 2], bits = i & 1 ? word >> 16 : word & 0xffffu;
      g[i] = gain_dtype == SIM_FP16 ? widen_bits<SIM_FP16>(bits) : widen_bits<SIM_BF16>(bits);
    }
  }
}

}  // namespace simar
