#include "ssm.hpp"
namespace ttt {
bool ssm_mfma_supported(const SsmArgs &) { return false; }
hipError_t launch_ssm_mfma(const SsmArgs &, hipStream_t) { return hipErrorNotSupported; }
}  // namespace ttt
