// qk_moe_up.cu -- the gate and up products of an expert layer (qk_moe.cuh).
#include "qk_moe.cuh"

namespace qk {
namespace moe {

cudaError_t launch_up(int type, Args& a, int sms, cudaStream_t s, bool launch) {
    return launch_product<false>(type, a, sms, s, launch);
}

}  // namespace moe
}  // namespace qk
