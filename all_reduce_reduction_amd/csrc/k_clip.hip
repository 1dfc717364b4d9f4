// k_clip.hip -- the norm over many tensors, and the tensors scaled down to a
// largest norm (gfx950).
//
// norm = sqrt(sum g^2) over all elements of all tensors, rounded to fp32;
// g' = g * min(1, max_norm / norm).  The sums are held in 64 bits: fp32 and bf16
// gradients of 1e-25 or 1e25 are within their types' range, their squares are
// not within fp32's.  Tensors are cut into pieces of 16 KiB, and the workgroups'
// sums are added up in their order, so that the same list gives the same bits.
//
// Bound by memory: 747 us for 809 M bf16 and 33 K fp32 gradients (read, then read and
// written: 4,857 MB at 6.5 TB/s; a copy of as many bytes 730).  2.6 M halves in nine
// tensors take 10.3 us a call: two launches of 3.6 and 5.2 us at least, their gap, and
// what of the helper's 3 us the first one does not hide.
#include "launch.h"
#include "layer.h"
#include "loss_device.h"

namespace simar {
namespace {

// 16-byte vectors of a piece, and of one of a workgroup's threads
constexpr int kVectors = kClipPieceBytes / 16, kEach = kVectors / kBlock;

__device__ __forceinline__ double wave_sum64(double v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// the sum over the workgroup, in every thread
__device__ __forceinline__ double block_sum64(double v) {
  __shared__ double s[kBlock / 64];
  v = wave_sum64(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < kBlock / 64; i++) sum += s[i];
  return sum;
}

// Which tensor a piece is of: every lane holds two tensors' first pieces, and the
// number of those that are not after the piece is one more than its index.
struct Tensors {
  static_assert(kClipTensors <= 128, "two tensors per lane");
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Tensors(const ClipList& l) {
    const int lane = threadIdx.x & 63;
    lo = lane < l.tensors ? l.first[lane] : 0xffffffffu;
    hi = lane + 64 < l.tensors ? l.first[lane + 64] : 0xffffffffu;
  }
  __device__ __forceinline__ int of(uint32_t piece) const {
    return __popcll(__ballot(lo <= piece)) + __popcll(__ballot(hi <= piece)) - 1;
  }
};
// a piece: its tensor, its first byte and its elements
struct Piece {
  int t, n, dtype;
  int64_t byte;
  __device__ __forceinline__ Piece(const ClipList& l, const Tensors& all, uint32_t piece) : t(all.of(piece)) {
    dtype = l.dtype[t];
    const int size = dtype == SIM_FP32 ? 4 : 2, most = kClipPieceBytes / size;
    byte = (int64_t)(piece - l.first[t]) * kClipPieceBytes;
    const int64_t left = l.count[t] - byte / size;
    n = (int)(left < most ? left : most);
  }
};

// A vector's squares, in fp32 where that is exact enough: a sum from 2^-90 on
// has lost nothing to underflow that it could see.  (In 64 bits throughout the
// conversions bound the kernel.)
template <int DT>
__device__ __forceinline__ void add_squares(u32x4 v, double& sum) {
  constexpr int V = epv<DT>();
  float f[V], s = 0.0f;
  unpack<DT>(v, f);
#pragma unroll
  for (int t = 0; t < V; t++) s = __builtin_fmaf(f[t], f[t], s);
  if (DT == SIM_FP16 || (s >= 0x1p-90f && s < __builtin_inff())) {
    sum += (double)s;
  } else {
#pragma unroll
    for (int t = 0; t < V; t++) sum = __builtin_fma((double)f[t], (double)f[t], sum);
  }
}
template <int DT>
__device__ __forceinline__ void squares_of(const char* in, int n, double& sum) {
  constexpr int V = epv<DT>();
  if (n == kVectors * V) {
    u32x4 v[kEach];
#pragma unroll
    for (int i = 0; i < kEach; i++) v[i] = ld_row_lane<DT, false>(in, 0, (i * kBlock + threadIdx.x) * V);
#pragma unroll
    for (int i = 0; i < kEach; i++) add_squares<DT>(v[i], sum);
  } else {
    for (int i = threadIdx.x; i < n / V; i += kBlock) add_squares<DT>(ld_row<DT>(in, (int64_t)i * V), sum);
    const int i = n / V * V + threadIdx.x;
    if (i < n) {
      const double f = (double)load_elem<DT>(in, i);
      sum = __builtin_fma(f, f, sum);
    }
  }
}

// max_norm / norm as a float c and a power of two, which is 1 unless the quotient is
// below fp32's normal numbers, where c alone would have lost bits (1e30 clipped to
// 1e-13: c = 5e-44, of 5 bits) that the product has: then c lies in [1/2, 1).
struct Factor {
  float power, c;
  __device__ __forceinline__ Factor(double norm, float max_norm) : power(1.0f) {
    // (a NaN norm makes everything NaN)
    const double q = norm <= (double)max_norm ? 1.0 : (double)max_norm / norm;
    c = (float)q;
    if (q > 0.0 && q < 0x1p-126) {
      const int e = __builtin_amdgcn_frexp_exp(q), k = e < -149 ? -149 : e;
      power = (float)__builtin_amdgcn_ldexp(1.0, k);
      c = (float)__builtin_amdgcn_ldexp(q, -k);
    }
  }
  __device__ __forceinline__ float operator()(float g) const { return g * power * c; }
};
template <int DT>
__device__ __forceinline__ u32x4 scaled(u32x4 v, const Factor& by) {
  constexpr int V = epv<DT>();
  float f[V];
  unpack<DT>(v, f);
#pragma unroll
  for (int t = 0; t < V; t++) f[t] = by(f[t]);
  return pack_rounded<DT>(f);
}
// A whole piece's vectors are given, the others' read.
template <int DT>
__device__ __forceinline__ void scale_to(const char* in, char* out, int n, const Factor& by, const u32x4 (&v)[kEach]) {
  constexpr int V = epv<DT>();
  if (n == kVectors * V) {
#pragma unroll
    for (int i = 0; i < kEach; i++) st_row_lane<DT, true>(out, 0, (i * kBlock + threadIdx.x) * V, scaled<DT>(v[i], by));
  } else {
    for (int i = threadIdx.x; i < n / V; i += kBlock)
      st_row<DT>(out, (int64_t)i * V, scaled<DT>(ld_row<DT>(in, (int64_t)i * V), by));
    const int i = n / V * V + threadIdx.x;
    if (i < n) store_elem<DT>(out, i, by(load_elem<DT>(in, i)));
  }
}

// Four waves per SIMD, in both passes: with eight the reads and writes of more
// pieces interleave in memory (809 M bf16 748 us a call, 772).
#define SIMAR_CLIP_WAVES __attribute__((amdgpu_waves_per_eu(4, 4)))
__global__ void __launch_bounds__(kBlock) SIMAR_CLIP_WAVES k_clip_squares(ClipList l, double* squares) {
  const Tensors all(l);
  double sum = 0.0;
  for (uint32_t piece = blockIdx.x; piece < l.pieces; piece += gridDim.x) {
    const Piece p(l, all, piece);
    const char* in = (const char*)l.in[p.t] + p.byte;
    if (p.dtype == SIM_FP32) squares_of<SIM_FP32>(in, p.n, sum);
    else if (p.dtype == SIM_FP16) squares_of<SIM_FP16>(in, p.n, sum);
    else squares_of<SIM_BF16>(in, p.n, sum);
  }
  sum = block_sum64(sum);
  if (threadIdx.x == 0) squares[blockIdx.x] = sum;
}

// The sum of all squares, in every thread.
__device__ __forceinline__ double sum_of(const ClipNorm& n) {
  double sum = 0.0;
  if (n.parts) {
    for (int i = threadIdx.x; i < n.nparts; i += kBlock) {
      const double p = (double)n.parts[i];
      sum = __builtin_fma(p, p, sum);
    }
  } else {
    for (int i = threadIdx.x; i < n.nsquares; i += kBlock) sum += n.squares[i];
  }
  return block_sum64(sum);
}
// The norm that the factor is formed of: a list's own in 64 bits, rounded only as
// norm[0] (2^-24 of the factor, the same for every element); the ranks' as norm[0]
// holds it, so that all ranks have the same factor whatever launches their own lists
// take.  Past fp32's range it is infinite, as norm[0] is.
__device__ __forceinline__ double norm_of(const ClipNorm& n) {
  if (n.known) return n.known[0];
  if (n.parts && n.nparts == 1) return (double)fabsf(n.parts[0]);
  const double norm = sqrt(sum_of(n));
  const float rounded = (float)norm;
  return n.parts || rounded == __builtin_inff() ? (double)rounded : norm;
}

__global__ void __launch_bounds__(kBlock) k_clip_join(ClipNorm n) {
  const double norm = norm_of(n);
  if (threadIdx.x == 0) {
    n.norm[0] = (float)norm;
    // (every thread has read its squares before the norm is there)
    if (n.keep) n.keep[0] = norm;
  }
}

// A workgroup scales one piece, whose vectors are on their way while the norm is
// found.  The last pieces come first: they are what the squares' pass, which reads
// without the streaming hint, left in the caches (235 MB of bf16 111 us, 115 with
// the hint and from the front).
__global__ void __launch_bounds__(kBlock) SIMAR_CLIP_WAVES k_clip_scale(ClipList l, ClipNorm n) {
  const Piece p(l, Tensors(l), gridDim.x - 1 - blockIdx.x);
  const char* in = (const char*)l.in[p.t] + p.byte;
  char* out = (char*)l.out[p.t] + p.byte;
  u32x4 v[kEach] = {};
  if (p.n * (p.dtype == SIM_FP32 ? 4 : 2) == kClipPieceBytes) {
#pragma unroll
    for (int i = 0; i < kEach; i++) v[i] = ld_row_lane<SIM_BF16, true>(in, 0, (i * kBlock + threadIdx.x) * 8);
  }
  const double norm = norm_of(n);
  if (n.norm && blockIdx.x == 0 && threadIdx.x == 0) n.norm[0] = (float)norm;
  const Factor by(norm, n.max_norm);
  if (n.in_place && by.power == 1.0f && by.c == 1.0f) return;
  if (p.dtype == SIM_FP32) scale_to<SIM_FP32>(in, out, p.n, by, v);
  else if (p.dtype == SIM_FP16) scale_to<SIM_FP16>(in, out, p.n, by, v);
  else scale_to<SIM_BF16>(in, out, p.n, by, v);
}

}  // namespace

hipError_t launch_clip_squares(const ClipList& l, double* squares, hipStream_t s) {
  return launch<k_clip_squares>(dim3(clip_workgroups(l.pieces)), dim3(kBlock), s, l, squares);
}
hipError_t launch_clip_join(const ClipNorm& n, hipStream_t s) { return launch<k_clip_join>(dim3(1), dim3(kBlock), s, n); }
hipError_t launch_clip_scale(const ClipList& l, const ClipNorm& n, hipStream_t s) {
  return launch<k_clip_scale>(dim3(l.pieces), dim3(kBlock), s, l, n);
}

}  // namespace simar
