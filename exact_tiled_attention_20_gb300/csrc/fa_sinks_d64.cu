// fa_sinks_d64.cu -- forward kernel instantiations with sinks for head dim 64; tiles as without.
#include "fa_fwd.cuh"

namespace fa {

fa_status launch_sinks_d64(const FwdArgs& a, cudaStream_t s) {
    return launch_fwd_cfg<FwdConfig<64, 128, 2, 3>, true>(a, s);
}

}  // namespace fa
