// The float32 instances of the linear-attention sweep for rows of any alignment and width.
#include "ss_la_sweep.h"

namespace ss {
hipError_t launch_la_sweep_f32_any(const LaSweeps& p, hipStream_t s) {
    return la::launch_sweep_type<float, false>(p, s);
}
}  // namespace ss
