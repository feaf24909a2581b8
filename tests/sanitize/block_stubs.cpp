// Host-only stand-ins for the launchers of the operators around the experts, next to
// launch_stubs.cpp, for the sanitizer build of the C ABI.  The workspace sizes, which the
// argument checks use, are some positive number of bytes per row.
#include "block.hpp"

namespace w4a8 {

int64_t mlp_i8_workspace_bytes(int64_t M, int64_t, int64_t I) { return 5 * M * I; }
hipError_t launch_dense_i8(const DenseArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_mlp_i8(const MlpArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_norm(const NormArgs&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace w4a8
