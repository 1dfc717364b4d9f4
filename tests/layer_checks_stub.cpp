// Stand-ins for the library and the kernels, so that the entry points of
// api_layer.cpp run on a machine without a GPU: their checks are the real ones,
// a launch only counts, and looks at what the kernels rely on.
#include "layer.h"

static int launches, bad;
extern "C" int stub_launches(void) { return launches; }
extern "C" int stub_bad(void) { return bad; }

namespace simar {
bool library_ready() { return true; }
int library_device() { return SIM_OK; }
int library_cus() { return 256; }

static hipError_t made(bool fine) {
  launches++;
  bad += !fine;
  return hipSuccess;
}
hipError_t launch_norm(const NormArgs& a, int, hipStream_t) { return made(a.x && a.out && a.rows > 0); }
hipError_t launch_norm_grad(const NormGradArgs& a, int, hipStream_t) {
  return made(a.workgroups >= 1 && (a.workgroups == 1 || !a.dgain || a.partial));
}
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t) {
  return made(a.chunks == 0 ? a.tokens * a.topk <= 4096
                            : (a.counts || !dispatch_counts(a.tokens * a.topk, a.experts)) && a.chunk % 1024 == 0 &&
                                  a.chunks * a.chunk >= a.tokens * a.topk);
}
hipError_t launch_combine(const CombineArgs& a, int, hipStream_t) { return made(a.rows || a.nrows == 0); }
hipError_t launch_combine_grad(const CombineGradArgs& a, int, hipStream_t) { return made(a.drows || a.dweights); }
static bool whole(const ClipList& l) {
  int64_t pieces = 0;
  for (int t = 0; t < l.tensors; t++) {
    if (l.first[t] != pieces || l.count[t] <= 0) return false;
    pieces += clip_pieces(l.count[t], l.dtype[t]);
  }
  return l.tensors >= 1 && l.tensors <= kClipTensors && pieces == l.pieces;
}
hipError_t launch_clip_squares(const ClipList& l, double* squares, hipStream_t) { return made(whole(l) && squares); }
hipError_t launch_clip_join(const ClipNorm& n, hipStream_t) { return made(n.norm != nullptr); }
hipError_t launch_clip_scale(const ClipList& l, const ClipNorm& n, hipStream_t) {
  return made(whole(l) && (n.parts || n.squares));
}
}  // namespace simar
