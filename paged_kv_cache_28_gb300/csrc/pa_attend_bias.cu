// pa_attend_bias.cu -- pa_extend_scored with scores that fall with distance.
#include "pa_attend_scored.cuh"

namespace pa {
template pa_status run_attend_scored<kBias>(const ScoredCall &x);
}  // namespace pa
