// qk_moe_down.cu -- the down product of an expert layer (qk_moe.cuh).
#include "qk_moe.cuh"

namespace qk {
namespace moe {

cudaError_t launch_down(int type, Args& a, int sms, cudaStream_t s, bool launch) {
    return launch_product<true>(type, a, sms, s, launch);
}

}  // namespace moe
}  // namespace qk
