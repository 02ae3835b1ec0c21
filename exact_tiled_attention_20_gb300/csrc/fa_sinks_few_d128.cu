// fa_sinks_few_d128.cu -- the same for at most 32 sinks.
#include "fa_fwd.cuh"

namespace fa {

fa_status launch_sinks_few_d128(const FwdArgs& a, cudaStream_t s) {
    return launch_fwd_cfg<FwdConfig<128, 128, 2, 2>, true, 2>(a, s);
}

}  // namespace fa
