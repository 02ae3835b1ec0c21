// fa_sinks_d96.cu -- forward kernel instantiations with sinks for head dim 96; tiles as without.
#include "fa_fwd.cuh"

namespace fa {

fa_status launch_sinks_few_d96(const FwdArgs& a, cudaStream_t s);

fa_status launch_sinks_d96(const FwdArgs& a, cudaStream_t s) {
    if (a.sinks <= 32) return launch_sinks_few_d96(a, s);
    return launch_fwd_cfg<FwdConfig<96, 128, 2, 2>, true>(a, s);
}

}  // namespace fa
