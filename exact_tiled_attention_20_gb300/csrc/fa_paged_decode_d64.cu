// fa_paged_decode_d64.cu -- instantiation of the decode over the 16-bit paged cache for head dim 64.
#include "fa_paged_decode.cuh"

namespace fa {

fa_status launch_paged_decode_d64(const PagedDecodeArgs& a, cudaStream_t s) { return launch_paged_decode_d<64>(a, s); }

}  // namespace fa
