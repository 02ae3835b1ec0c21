// fa_paged_decode_d256.cu -- instantiation of the decode over the 16-bit paged cache for head dim 256.
#include "fa_paged_decode.cuh"

namespace fa {

fa_status launch_paged_decode_d256(const PagedDecodeArgs& a, cudaStream_t s) { return launch_paged_decode_d<256>(a, s); }

}  // namespace fa
