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
int norm_grad_workgroups(int64_t rows, int64_t cols, int dtype, bool dgain) {
  const int per_vector = dtype == SIM_FP32 ? 4 : 8;
  const NormGradShape f = norm_grad_shape(cols, per_vector);
  const bool ahead = f.per_thread * per_vector <= 8;  // (the next row's loads under way)
  const int64_t turns = f.lanes ? (rows + f.threads / f.lanes - 1) / (f.threads / f.lanes) : rows;
  // One workgroup where its turns cost less than a second launch: 2 rows x 4,096 bf16
  // 4.1 us, 8.6 with a workgroup each, 4 rows 6.0, 8.7, 8 rows 10.0, 8.7; 60 x 320,
  // 8 turns, 7.2, 8.7; without loads ahead 2 x 10,933 7.1, 8.7, 8 x 12,000 18.2, 8.7.
  // Without dgain there is no second launch, and there are no partial sums below: 512
  // rows x 64 bf16 4.6 us, 7.2 in one workgroup; 249 x 10,216 5.3, 7.1 with two rows each.
  if (turns <= (!dgain ? 1 : f.lanes ? 8 : ahead ? 4 : f.per_thread == 2 ? 2 : 1)) return 1;
  // 16 waves on each compute unit (32, without the next row's loads ahead, read and
  // write more rows at once, which costs memory more than it hides: 16,384 x 8,192
  // bf16 183 us, 186.5; 16,384 x 4,096 92, 108; 4,096 x 5,120 36.7, 42.0); each takes the
  // same number of rows, or one less.
  const int64_t most = library_cus() * std::max<int64_t>(1, 16 / (f.threads / 64));
  int64_t each = std::max<int64_t>(1, (turns + most - 1) / most);
  // Where a row each would make 4 MB of partial sums, two rows each, or up to four
  // while that leaves no compute unit idle: 400 x 4,096 bf16 9.0 us, 11.3 with one
  // each, four 10.5; 249 x 10,216 15.6, 18.4, four 18.3; 1,003 x 2,261 fp32 11.0, 12.5
  // with two; 200 x 4,096, 3 MB, 8.9, 8.7 with one.  Four vectors per thread, whose
  // rows follow each other without loads ahead, lose by it (152 x 16,010 fp32 26.9,
  // 23.0 with one).
  if (dgain && !f.lanes && f.per_thread <= 2 && rows * cols >= 1 << 20)
    each = std::max(each, ahead ? std::min<int64_t>(4, std::max<int64_t>(2, (turns + library_cus() - 1) / library_cus())) : 2);
  return (int)std::max<int64_t>(1, (turns + each - 1) / each);
}

// Up to so many slots each token's workgroup may read all of them (tokens of 4 KiB: 512
// with 8 slots 9.2 us, 11.2 in two launches; 640 with 8 slots 12.1, 12.2; 1,000 with 6
// slots 14.9, 12.8).
constexpr int64_t kFewSlots = 4096;
// More slots are cut into chunks of 1,024, or so many more that there are at most 512.
// Each chunk's workgroup reads the counts of all chunks, kCountsPerSlot at most for each
// of its own slots (what all of them read would else grow with the square of the slots):
// chunks are made longer until that holds.  Places alone, with that many counts per slot
// or less, and with chunks of half the length: 16,384 tokens, 32 slots, 1,024 experts
// 23.1 us, 30.8 (75.4 with a quarter); 65,536, 32 slots, 1,024 experts 41.5, 83; 65,536,
// 8 slots, 256 experts 13.8, 25.7; 16,384, 16 slots, 512 experts 14.3, 18.3.  Longer ones
// than that: 65,536, 32 slots, 1,024 experts 60.9; 16,384, 8 slots, 256 experts 10.5
// with twice the length, 9.5.
constexpr int64_t kCountsPerSlot = 64;
int dispatch_chunks(int64_t slots, int experts, int64_t* chunk) {
  *chunk = 0;
  if (slots <= kFewSlots) return 0;
  *chunk = std::max<int64_t>(1024, ((slots + 511) / 512 + 1023) / 1024 * 1024);
  const auto chunks = [&] { return (slots + *chunk - 1) / *chunk; };
  while (chunks() * experts > kCountsPerSlot * *chunk) *chunk *= 2;
  return (int)chunks();
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
