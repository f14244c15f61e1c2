// moe_choose_f32.cu -- choices by F32 logits (in a translation unit of their own, for the build's time).
#include "moe_choose.cuh"

namespace tkg {
tkg_status launch_choose_f32(RouteParams& p, cudaStream_t stream) { return launch_choose<LogitF32>(p, stream); }
}  // namespace tkg
