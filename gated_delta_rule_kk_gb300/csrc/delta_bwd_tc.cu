#include "delta_bwd.h"
namespace gdn {
bool delta_bwd_tc_supported(const DeltaBwdParams &, bool) { return false; }
int64_t delta_bwd_tc_block(const DeltaBwdParams &) { return 0; }
cudaError_t launch_delta_bwd_tc(const DeltaBwdParams &, cudaStream_t) { return cudaErrorNotSupported; }
}
