// pa_attend_cap_bias.cu -- pa_extend_scored with capped scores that fall with distance.
#include "pa_attend_scored.cuh"

namespace pa {
template pa_status run_attend_scored<kCap | kBias>(const ScoredCall &x);
}  // namespace pa
