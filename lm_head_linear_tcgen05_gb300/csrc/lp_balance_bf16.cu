// lp_balance_bf16.cu - the balance loss of bf16 logits.
#include "lp_balance.cuh"

namespace lp {

cudaError_t launch_balance_loss_bf16(const BalanceParams& p, cudaStream_t s) { return launch_types<false>(p, s); }

}  // namespace lp
