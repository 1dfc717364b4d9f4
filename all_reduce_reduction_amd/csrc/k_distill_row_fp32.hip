// k_distill_row_fp32.hip -- the one-workgroup-per-row distillation step for fp32.
#include "distill_row.h"

namespace simar {
hipError_t launch_distill_row_fp32(const DistillArgs& a, hipStream_t s) { return launch_row<SIM_FP32>(a, s); }
}  // namespace simar
