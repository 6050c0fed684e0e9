// pa_attend_cap.cu -- pa_extend_scored with capped scores.
#include "pa_attend_scored.cuh"

namespace pa {
template pa_status run_attend_scored<kCap>(const ScoredCall &x);
}  // namespace pa
