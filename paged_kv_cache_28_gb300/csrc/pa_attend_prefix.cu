// pa_attend_prefix.cu -- pa_extend_scored with a prefix alone.
#include "pa_attend_scored.cuh"

namespace pa {
template pa_status run_attend_scored<0>(const ScoredCall &x);
}  // namespace pa
