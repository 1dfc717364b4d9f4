// k_clip.hip -- the norm over many tensors, and the tensors scaled down to a
// largest norm (gfx950).
//
// norm = sqrt(sum g^2) over all elements of all tensors, rounded to fp32;
// g' = g * min(1, max_norm / norm).  Squares are summed in 64 bits: fp32 and bf16 gradients of
// 1e-25 or 1e25 are within their types' range, their squares are not within
// fp32's.  Tensors are cut into pieces of kClipPiece elements; a workgroup takes a
// run of pieces, and the workgroups' sums are added up in their order, so that
// the same list gives the same bits.
#include <algorithm>

#include "launch.h"
#include "layer.h"
#include "loss_device.h"

namespace simar {
namespace {

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

// this workgroup's run of pieces
struct Run {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Run(const ClipList& l)
      : lo((uint32_t)((uint64_t)l.pieces * blockIdx.x / gridDim.x)),
        hi((uint32_t)((uint64_t)l.pieces * (blockIdx.x + 1) / gridDim.x)) {}
};
// the last tensor whose first piece is not after `piece` (tensors without
// elements have no piece: they share their first with the next one)
__device__ __forceinline__ int tensor_of(const ClipList& l, uint32_t piece) {
  int lo = 0, hi = l.tensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= piece) lo = mid;
    else hi = mid;
  }
  return lo;
}

// f(vector) for the whole vectors and f1(element) for what is left, of the
// elements [lo, hi); U vectors of a thread are under way at once
constexpr int kFlight = 8;

template <int DT>
__device__ __forceinline__ double squares_of(const char* in, int n) {
  constexpr int V = epv<DT>();
  double sum = 0.0;
  const int nv = n / V;
  for (int v0 = threadIdx.x; v0 < nv; v0 += kBlock * kFlight) {
    u32x4 v[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; i++) {
      v[i] = u32x4{0, 0, 0, 0};
      if (v0 + i * kBlock < nv) v[i] = ld_row<DT>(in, (int64_t)(v0 + i * kBlock) * V);
    }
#pragma unroll
    for (int i = 0; i < kFlight; i++) {
      float f[V];
      unpack<DT>(v[i], f);
      if constexpr (DT == SIM_FP16) {
        // (the squares of eight halves are within fp32's range)
        float s = 0.0f;
#pragma unroll
        for (int t = 0; t < V; t++) s = __builtin_fmaf(f[t], f[t], s);
        sum += (double)s;
      } else {
#pragma unroll
        for (int t = 0; t < V; t++) sum = __builtin_fma((double)f[t], (double)f[t], sum);
      }
    }
  }
  const int i = nv * V + threadIdx.x;
  if (i < n) {
    const double f = (double)load_elem<DT>(in, i);
    sum = __builtin_fma(f, f, sum);
  }
  return sum;
}

template <int DT>
__device__ __forceinline__ void scale_to(const char* in, char* out, int n, float c) {
  constexpr int V = epv<DT>();
  const int nv = n / V;
  for (int v0 = threadIdx.x; v0 < nv; v0 += kBlock * kFlight) {
    u32x4 v[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; i++)
      if (v0 + i * kBlock < nv) v[i] = ld_row<DT>(in, (int64_t)(v0 + i * kBlock) * V);
#pragma unroll
    for (int i = 0; i < kFlight; i++) {
      if (v0 + i * kBlock >= nv) continue;
      float f[V];
      unpack<DT>(v[i], f);
#pragma unroll
      for (int t = 0; t < V; t++) f[t] *= c;
      st_row<DT>(out, (int64_t)(v0 + i * kBlock) * V, pack_rounded<DT>(f));
    }
  }
  const int i = nv * V + threadIdx.x;
  if (i < n) store_elem<DT>(out, i, load_elem<DT>(in, i) * c);
}

__global__ void __launch_bounds__(kBlock) k_clip_squares(ClipList l, double* squares) {
  const Run run(l);
  double sum = 0.0;
  int t = tensor_of(l, run.lo);
  for (uint32_t piece = run.lo; piece < run.hi; piece++) {
    while (t + 1 < l.tensors && l.first[t + 1] <= piece) t++;
    const int64_t at = (int64_t)(piece - l.first[t]) * kClipPiece;
    const int n = (int)(l.count[t] - at < kClipPiece ? l.count[t] - at : kClipPiece);
    const int dt = l.dtype[t];
    if (dt == SIM_FP32) sum += squares_of<SIM_FP32>((const char*)l.in[t] + at * 4, n);
    else if (dt == SIM_FP16) sum += squares_of<SIM_FP16>((const char*)l.in[t] + at * 2, n);
    else sum += squares_of<SIM_BF16>((const char*)l.in[t] + at * 2, n);
  }
  sum = block_sum64(sum);
  if (threadIdx.x == 0) squares[blockIdx.x] = sum;
}

// the norm of all, in every thread
__device__ __forceinline__ double norm_of(const ClipNorm& n) {
  double sum = 0.0;
  if (n.parts) {
    for (int i = threadIdx.x; i < n.nparts; i += kBlock) {
      const double p = (double)n.parts[i];
      sum = __builtin_fma(p, p, sum);
    }
  } else {
    for (int i = threadIdx.x; i < n.nsquares; i += kBlock) sum += n.squares[i];
  }
  return sqrt(block_sum64(sum));
}

__global__ void __launch_bounds__(kBlock) k_clip_join(ClipNorm n) {
  const double norm = norm_of(n);
  if (threadIdx.x == 0) n.norm[0] = (float)norm;
}

__global__ void __launch_bounds__(kBlock) k_clip_scale(ClipList l, ClipNorm n) {
  const float norm = (float)norm_of(n);
  if (n.norm && blockIdx.x == 0 && threadIdx.x == 0) n.norm[0] = norm;
  // (a NaN norm makes everything NaN)
  const float c = norm <= n.max_norm ? 1.0f : (float)((double)n.max_norm / (double)norm);
  if (n.in_place && c == 1.0f) return;
  const Run run(l);
  int t = tensor_of(l, run.lo);
  for (uint32_t piece = run.lo; piece < run.hi; piece++) {
    while (t + 1 < l.tensors && l.first[t + 1] <= piece) t++;
    const int64_t at = (int64_t)(piece - l.first[t]) * kClipPiece;
    const int m = (int)(l.count[t] - at < kClipPiece ? l.count[t] - at : kClipPiece);
    const int dt = l.dtype[t];
    const char* in = (const char*)l.in[t];
    char* out = (char*)l.out[t];
    if (dt == SIM_FP32) scale_to<SIM_FP32>(in + at * 4, out + at * 4, m, c);
    else if (dt == SIM_FP16) scale_to<SIM_FP16>(in + at * 2, out + at * 2, m, c);
    else scale_to<SIM_BF16>(in + at * 2, out + at * 2, m, c);
  }
}

}  // namespace

hipError_t launch_clip_squares(const ClipList& l, double* squares, hipStream_t s) {
  return launch<k_clip_squares>(dim3(clip_workgroups(l.pieces)), dim3(kBlock), s, l, squares);
}
hipError_t launch_clip_join(const ClipNorm& n, hipStream_t s) { return launch<k_clip_join>(dim3(1), dim3(kBlock), s, n); }
hipError_t launch_clip_scale(const ClipList& l, const ClipNorm& n, hipStream_t s) {
  return launch<k_clip_scale>(dim3(std::max(1, clip_workgroups(l.pieces))), dim3(kBlock), s, l, n);
}

}  // namespace simar
