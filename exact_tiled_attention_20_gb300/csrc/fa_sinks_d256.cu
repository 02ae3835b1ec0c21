// fa_sinks_d256.cu -- forward kernel instantiations with sinks for head dim 256; tiles as without.
#include "fa_fwd.cuh"

namespace fa {

fa_status launch_sinks_d256(const FwdArgs& a, cudaStream_t s) {
    return launch_fwd_cfg<FwdConfig<256, 64, 1, 2>, true>(a, s);
}

}  // namespace fa
