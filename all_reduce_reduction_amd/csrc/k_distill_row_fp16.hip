// k_distill_row_fp16.hip -- the one-workgroup-per-row distillation step for fp16.
#include "distill_row.h"

namespace simar {
hipError_t launch_distill_row_fp16(const DistillArgs& a, hipStream_t s) { return launch_row<SIM_FP16>(a, s); }
}  // namespace simar
