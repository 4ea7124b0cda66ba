// head_dim 128 instances of the attention over the 8-bit cache (3 to 4 tiles of 8 query rows).
#include "pa_q8_attend.cuh"

namespace pa {
extern const Q8Instance kQ8D128b[2] = {q8_instance<128, 3>(), q8_instance<128, 4>()};
}  // namespace pa
