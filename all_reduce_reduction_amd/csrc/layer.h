// layer.h -- argument blocks and launchers of the norm, expert and clipping
// kernels (k_norm.hip, k_norm_grad.hip, k_experts.hip, k_clip.hip), shared with
// their entry points (api_layer.cpp).
//
// Row t of a matrix starts at element t * stride of its base (byte t * pitch
// where rows are only moved); only the alignment of single elements is assumed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "simar.h"

namespace simar {

// api.cpp: whether sim_init has run; making the library's device current; its
// number of compute units
bool library_ready();
int library_device();
int library_cus();

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;  // NULL: none
  int64_t residual_stride;
  int64_t rows;
  int cols;
  const void* gain;      // NULL: all 1
  int gain_dtype;
  float eps;
  void* sum;             // NULL: not written
  int64_t sum_stride;
  void* out;
  int64_t out_stride;
  float* scales;         // NULL: out has x's type; else it is e4m3
  int group;             // columns of a scale; 0: a row's
  int64_t groups;        // scales of a row
};

struct NormGradArgs {
  const void* h;
  int64_t h_stride;
  int64_t rows;
  int cols;
  const void* gain;
  int gain_dtype;
  float eps;
  const void* dy;
  int64_t dy_stride;
  const void* dsum;      // NULL: none
  int64_t dsum_stride;
  void* dx;
  int64_t dx_stride;
  float* dgain;          // NULL: not wanted
  float* partial;        // [workgroups][cols]
  int workgroups;
};

struct DispatchArgs {
  const void* x;
  int64_t x_pitch;       // bytes
  int64_t row_bytes;
  const float* scales;   // NULL: none
  int64_t scale_bytes;   // of a row
  const int32_t* chosen;
  int64_t tokens;
  int topk, experts;
  void* rows;
  int64_t rows_pitch;
  float* row_scales;
  int32_t* place;
  int32_t* offsets;
  uint32_t* counts;      // [chunks][experts]; NULL: every chunk counts all slots
  int chunks;            // 0: one launch
  int64_t chunk;         // slots per chunk
};

struct CombineArgs {
  const void* rows;
  int64_t rows_stride;
  int64_t nrows;
  int64_t cols;
  const int32_t* place;
  const float* weights;  // NULL: all 1
  int64_t tokens;
  int topk;
  void* out;
  int64_t out_stride;
};

struct CombineGradArgs {
  const void* dy;
  int64_t dy_stride;
  const void* rows;
  int64_t rows_stride;
  int64_t nrows;
  int64_t cols;
  const int32_t* place;
  const float* weights;  // NULL: all 1
  int64_t tokens;
  int topk;
  void* drows;           // NULL: not wanted
  int64_t drows_stride;
  float* dweights;       // NULL: not wanted
};

// Tensors are cut into pieces.
constexpr int kClipPieceBytes = 16384;
// Tensors of one launch: the kernel's argument block stays below 4 KiB.
constexpr int kClipTensors = 120;
struct ClipList {
  int tensors;
  uint32_t pieces;                  // of all tensors
  uint32_t first[kClipTensors];     // a tensor's first piece
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t count[kClipTensors];
  uint8_t dtype[kClipTensors];
};
// What the squares' sums became.
struct ClipNorm {
  const double* squares;  // [nsquares]: a list's own
  int nsquares;
  const float* parts;     // [nparts]: every rank's norm; NULL: the list's own squares are all
  int nparts;
  float max_norm;
  float* norm;            // NULL: another launch writes it
  int in_place;
  const double* known;    // NULL, or the norm itself, as another launch left it
  double* keep;           // NULL, or where launch_clip_join leaves the norm (over the squares, say)
};

// layer_sizes.cpp
// Threads of a row, and 16-byte vectors of each.  The least threads, in whole
// waves, that hold a row: only the last vector of a thread may then lie past the
// row's end.
inline int row_threads(int64_t vectors, int per_thread) {
  return (int)((vectors + 64 * per_thread - 1) / (64 * per_thread)) * 64;
}
inline bool row_vectors_fit(int64_t cols, int per_vector, int threads, int per_thread) {
  return (int64_t)threads * per_thread * per_vector >= cols &&
         (int64_t)threads * (per_thread - 1) * per_vector <= cols;
}
// A gradient's rows: `lanes` lanes of a workgroup of kNormShortThreads (0: a whole
// workgroup of `threads`) take a row, per_thread vectors each.
constexpr int kNormShortThreads = 512;
struct NormGradShape {
  int lanes, per_thread, threads;
};
NormGradShape norm_grad_shape(int64_t cols, int per_vector);
int norm_grad_workgroups(int64_t rows, int64_t cols, int dtype, bool dgain);
int dispatch_chunks(int64_t slots, int experts, int64_t* chunk);  // 0: one launch for all slots
bool dispatch_counts(int64_t slots, int experts);     // whether a launch of its own counts the chunks' slots
int64_t clip_pieces(int64_t count, int dtype);
int clip_workgroups(uint32_t pieces);

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);
hipError_t launch_combine(const CombineArgs& a, int dtype, hipStream_t s);
hipError_t launch_combine_grad(const CombineGradArgs& a, int dtype, hipStream_t s);
hipError_t launch_clip_squares(const ClipList& l, double* squares, hipStream_t s);
hipError_t launch_clip_join(const ClipNorm& n, hipStream_t s);
hipError_t launch_clip_scale(const ClipList& l, const ClipNorm& n, hipStream_t s);

}  // namespace simar
