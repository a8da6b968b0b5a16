// extend_direct_64.cu - extend under score rules with few query blocks, straight
// from the pool: the kernel of direct_tc.cuh at head_dim 64.
#include "extend_direct.cuh"

namespace pkv {
namespace direct {

cudaError_t launch_rules_64(const DirectArgs &a, bool tma,
                            const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm,
                            cudaStream_t stream) {
  return launch_rules<64>(a, tma, km, vm, qm, stream);
}

}  // namespace direct
}  // namespace pkv
