// moe_choose_bf16.cu -- choices by BF16 logits (in a translation unit of their own, for the build's time).
#include "moe_choose.cuh"

namespace tkg {
tkg_status launch_choose_bf16(RouteParams& p, cudaStream_t stream) { return launch_choose<LogitBF16>(p, stream); }
}  // namespace tkg
