// layer_sizes.cpp -- how the norm, expert and clipping operators cut their work
// into workgroups, chunks and pieces: what their entry points need to know to
// say how much scratch a call takes.
#include <algorithm>

#include "layer.h"

namespace simar {

NormGradShape norm_grad_shape(int64_t cols, int per_vector) {
  const int64_t nv = (cols + per_vector - 1) / per_vector;
  if (nv <= 128) return {nv <= 8 ? 8 : nv <= 16 ? 16 : nv <= 32 ? 32 : 64, nv <= 64 ? 1 : 2, kNormShortThreads};
  // (eight elements where a workgroup has the threads for it)
  const int r = nv <= 1024 && per_vector == 8 ? 1 : nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
  return {0, r, row_threads(nv, r)};
}
int norm_grad_workgroups(int64_t rows, int64_t cols, int dtype) {
  const NormGradShape f = norm_grad_shape(cols, dtype == SIM_FP32 ? 4 : 8);
  // 16 waves on each compute unit (32, without the next row's loads ahead, read and
  // write more rows at once, which costs memory more than it hides: 16,384 x 8,192
  // bf16 181 us, 185; 4,096 x 5,120 38 us, 45.5); each takes the same number of
  // rows, or one less.
  const int64_t most = library_cus() * std::max<int64_t>(1, 16 / (f.threads / 64));
  const int64_t turns = f.lanes ? (rows + f.threads / f.lanes - 1) / (f.threads / f.lanes) : rows;
  const int64_t each = std::max<int64_t>(1, (turns + most - 1) / most);
  return (int)std::max<int64_t>(1, (turns + each - 1) / each);
}

// Up to so many slots each token's workgroup may read all of them (512 tokens of 4
// KiB, 8 slots: 8.8 us, 10.3 in two launches; 1,000 tokens, 6 slots: 15.0, 14.6 in
// three).
constexpr int64_t kFewSlots = 4096;
int dispatch_chunks(int64_t slots, int64_t* chunk) {
  *chunk = 0;
  if (slots <= kFewSlots) return 0;
  *chunk = std::max<int64_t>(1024, ((slots + 511) / 512 + 1023) / 1024 * 1024);
  return (int)((slots + *chunk - 1) / *chunk);
}

// Up to so many slots every chunk's workgroup counts all of them.  5,120 slots of 64
// experts: 11.0 us a call, 12.9 with a launch that counts; 8,192 of 4: 10.2, 12.9;
// 16,384 of 256: 10.1, 12.9, but of 4, whose counters are in each other's way, 14.8,
// 12.9; 32,768 of 256: 13.6, 13.1.
bool dispatch_counts(int64_t slots, int experts) { return slots > (experts >= 32 ? 16384 : 8192); }

int64_t clip_pieces(int64_t count, int dtype) {
  const int64_t each = kClipPieceBytes / (dtype == SIM_FP32 ? 4 : 2);
  return (count + each - 1) / each;
}
int clip_workgroups(uint32_t pieces) { return (int)std::min<int64_t>(pieces, 8 * (int64_t)library_cus()); }

}  // namespace simar
