// The bf16 instances of the linear-attention sweep for rows of aligned 16-byte pieces.
#include "ss_la_sweep.h"

namespace ss {
hipError_t launch_la_sweep_bf16(const LaSweeps& p, hipStream_t s) {
    return la::launch_sweep_type<bf16_t, true>(p, s);
}
}  // namespace ss
