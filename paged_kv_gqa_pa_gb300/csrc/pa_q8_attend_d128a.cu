// head_dim 128 instances of the attention over the 8-bit cache (1 to 2 tiles of 8 query rows).
#include "pa_q8_attend.cuh"

namespace pa {
extern const Q8Instance kQ8D128a[2] = {q8_instance<128, 1>(), q8_instance<128, 2>()};
}  // namespace pa
