// The float32 instances of the linear-attention sweep.
#include "ss_la_sweep.h"

namespace ss {
hipError_t launch_la_sweep_f32(const LaSweep& p, hipStream_t s) {
    return la::launch_sweep_type<float>(p, s);
}
}  // namespace ss
