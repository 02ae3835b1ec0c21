// fa_kv8_decode_d256.cu -- decode over the 8-bit paged cache, head dim 256.
#include "fa_kv8_decode.cuh"

namespace fa {

fa_status launch_kv8_decode_d256(const Kv8DecodeArgs& a, cudaStream_t s) { return launch_kv8_decode_d<256>(a, s); }

}  // namespace fa
