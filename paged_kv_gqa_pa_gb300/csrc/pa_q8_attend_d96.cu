// head_dim 96 instances of the attention over the 8-bit cache (1 to 4 tiles of 8 query rows).
#include "pa_q8_attend.cuh"

namespace pa {
extern const Q8Instance kQ8D96[4] = {q8_instance<96, 1>(), q8_instance<96, 2>(), q8_instance<96, 3>(), q8_instance<96, 4>()};
}  // namespace pa
