// head_dim 256 instances of the attention over the 8-bit cache (1 to 2 tiles of 8 query rows).
#include "pa_q8_attend.cuh"

namespace pa {
extern const Q8Instance kQ8D256[2] = {q8_instance<256, 1>(), q8_instance<256, 2>()};
}  // namespace pa
