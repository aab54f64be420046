"""A policy update of a small language model whose embedding is tied to its head.

    python examples/tied_policy_step.py [--steps 20] [--objective policy|preference]

The model is one table W [V, H] and one matrix M [H, H]: a token's hidden state is
x = e + tanh(e M) with e = sqrt(H) W[id], and the next token's logits are x W^T. Each step runs

    lp_embedding            e from the token ids
    lp_forward              logp and entropy of the sampled tokens, without the logits
    lp_policy_loss          (or lp_preference_loss) the loss with grad_logp and grad_entropy
    lp_backward_ex          dX, and the head's gradient into a fp32 dW
    lp_embedding_backward   the embedding's gradient, added to that same dW

and takes a gradient step on an fp32 copy of W. The batch is made up: random tokens, of which those
from the lower half of the vocabulary are rewarded (preferred); the loss falls as they become likelier.
Needs a GB300 and the built library.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_linear_tcgen05_gb300 as lp  # noqa: E402


def make_batch(sequences, tokens, vocab, gen):
    """Packed sequences: ids, next ids, offsets, the mask of the answers (prompts do not count) and one
    reward per sequence, whether its answer came from the lower half of the vocabulary."""
    good = torch.arange(sequences, device="cuda") % 2 == 0
    ids = torch.randint(0, vocab // 2, (sequences, tokens + 1), generator=gen, device="cuda")
    ids += torch.where(good, 0, vocab // 2)[:, None]
    prompt = tokens // 4
    ids[:, :prompt] = torch.randint(0, vocab, (sequences, prompt), generator=gen, device="cuda")
    mask = (torch.arange(tokens, device="cuda") >= prompt).repeat(sequences)
    cu = torch.arange(0, sequences * tokens + 1, tokens, dtype=torch.int32, device="cuda")
    return (ids[:, :-1].reshape(-1).to(torch.int32), ids[:, 1:].reshape(-1).to(torch.int32), cu, mask,
            torch.where(good, 1.0, -1.0))


def train(steps=20, objective="policy", sequences=16, tokens=128, hidden=256, vocab=1000, lr=0.05, seed=0):
    """Runs `steps` updates; returns the loss of each."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    part = lp.VocabPartition(vocab_real=vocab, vocab_padded=vocab, ranges=((0, vocab),))
    master = torch.empty((vocab, hidden), device="cuda").normal_(0.0, 0.02, generator=gen)
    M = torch.empty((hidden, hidden), device="cuda").normal_(0.0, hidden ** -0.5, generator=gen)
    ids, y, cu, mask, reward = make_batch(sequences, tokens, vocab, gen)
    scale, dW, first, losses = math.sqrt(hidden), torch.zeros_like(master), None, []
    for _ in range(steps):
        W = master.to(torch.bfloat16)
        e = lp.lp_embedding(ids, [W], part, scale=scale, out_dtype=torch.float32)
        h = torch.tanh(e @ M)
        X = (e + h).to(torch.bfloat16)
        out = lp.lp_forward(X, [W], None, part, y, 1.0)
        first = out["logp"].clone() if first is None else first      # the policy the tokens came from
        if objective == "policy":
            loss = lp.lp_policy_loss(out["logp"], first, reward, ref_logp=first, entropy=out["entropy"], mask=mask,
                                     cu_seqlens=cu, clip_high=0.28, kl_coef=0.01, entropy_coef=1e-3,
                                     aggregation="seq_mean_token_mean")
        else:
            loss = lp.lp_preference_loss(out["logp"], cu, ref_logp=first, mask=mask, beta=0.1,
                                         length_normalised=True)
        grad_entropy = loss.get("grad_entropy")
        g = lp.lp_backward_ex(X, [W], None, part, y, 1.0, out["lse"], loss["grad_logp"], bias_grad=False,
                              entropy=None if grad_entropy is None else out["entropy"], grad_entropy=grad_entropy,
                              dW=[dW])
        dE = g["dX"] + ((1 - h * h) * g["dX"]) @ M.T
        lp.lp_embedding_backward(ids, dE, part, scale=scale, accumulate=True, dW=[dW])
        master -= lr * dW / (dW.norm() + 1e-12)
        losses.append(float(loss["loss"]))
        if lp.lp_get_device_error() != 0:
            raise RuntimeError("the library recorded a device error")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--objective", choices=("policy", "preference"), default="policy")
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.objective)):
        print(f"step {i}: loss {loss:.6f}")


if __name__ == "__main__":
    main()
