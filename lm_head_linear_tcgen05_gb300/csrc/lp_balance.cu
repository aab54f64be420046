// lp_balance.cu - the balance loss of fp32 logits, and its workspace (the kernels are in lp_balance.cuh; bf16 logits
// have a file of their own so that the two are compiled side by side).
#include "lp_balance.cuh"

namespace lp {

size_t balance_ws_bytes(int64_t T, int64_t E, int64_t K, int64_t n_seqs) {
  if (one_launch(T, E, K, n_seqs)) return 0;
  size_t bytes;
  carve(nullptr, E, n_seqs, &bytes);
  return bytes;
}

cudaError_t launch_balance_loss(const BalanceParams& p, bool logits_f32, cudaStream_t s) {
  return logits_f32 ? launch_types<true>(p, s) : launch_balance_loss_bf16(p, s);
}

}  // namespace lp
