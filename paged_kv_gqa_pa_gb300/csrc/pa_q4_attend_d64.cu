// head_dim 64 instances of the attention over the 4-bit cache.
#include "pa_q4_attend.cuh"

namespace pa {
template cudaError_t launch_q4_attend_d<64, __half>(const Q4AttendParams&, dim3, cudaStream_t);
template cudaError_t launch_q4_attend_d<64, __nv_bfloat16>(const Q4AttendParams&, dim3,
                                                           cudaStream_t);
template cudaError_t q4_attend_clusters<64, __half>(int, int, int*);
template cudaError_t q4_attend_clusters<64, __nv_bfloat16>(int, int, int*);
}  // namespace pa
