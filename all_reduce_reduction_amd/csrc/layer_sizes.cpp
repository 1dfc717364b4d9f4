// layer_sizes.cpp -- how the norm, expert and clipping operators cut their work
// into workgroups, chunks and pieces: what their entry points need to know to
// say how much scratch a call takes.
#include <algorithm>

#include "layer.h"

namespace simar {

int norm_grad_workgroups(int64_t rows, int64_t cols, int dtype) {
  const int64_t nv = (cols * (dtype == SIM_FP32 ? 4 : 2) + 15) / 16;
  const int64_t threads = nv <= 64 ? 64 : nv <= 512 ? 256 : 1024;
  // as many as run at once
  const int64_t most = library_cus() * (threads == 1024 ? 2 : threads == 256 ? 6 : 16);
  return (int)std::max<int64_t>(1, std::min(rows, most));
}

// Up to so many slots each token's workgroup reads all of them.
constexpr int64_t kFewSlots = 4096;
int dispatch_chunks(int64_t slots, int64_t* chunk) {
  *chunk = 0;
  if (slots <= kFewSlots) return 0;
  *chunk = std::max<int64_t>(2048, ((slots + 511) / 512 + 1023) / 1024 * 1024);
  return (int)((slots + *chunk - 1) / *chunk);
}

int64_t clip_pieces(int64_t count) { return (count + kClipPiece - 1) / kClipPiece; }
int clip_workgroups(uint32_t pieces) { return (int)std::min<int64_t>(pieces, 8 * (int64_t)library_cus()); }

}  // namespace simar
