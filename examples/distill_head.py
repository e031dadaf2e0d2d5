"""A language-model head learns from a teacher, then from rewards.

Shows the log-probability and distillation calls as they are used together, on a linear
head over given hidden states (random ones here):

  1. the teacher's logits go through ``foak_logprobs_forward``, which keeps each token's top
     K probabilities at the distillation temperature -- all that has to be stored of them;
  2. the student's logits go through ``foak_distill_fwd_bwd``, which mixes the distance to
     those probabilities with the labels' cross-entropy and leaves the gradient in place of
     the logits; the head's gradient is one product of that with the hidden states;
  3. the student samples tokens from its own top list, ``foak_logprobs_forward`` scores them,
     and ``foak_logprobs_backward`` gives the gradient of a policy loss with an entropy bonus.

Run:  python examples/distill_head.py [--tokens N] [--vocab V] [--hidden D] [--top-k K] [--steps S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import cross_entropy_loss_gb300 as ce  # noqa: E402


def logits_of(hidden, weight):
    out = torch.empty(hidden.shape[0], weight.shape[0], dtype=torch.bfloat16, device=hidden.device)
    return ce.foak_gemm_bf16(hidden, weight, out)


def head_gradient(dlogits, hidden, vocab):
    """dW = dlogits^T hidden in float32."""
    dw = torch.empty(vocab, hidden.shape[1], dtype=torch.float32, device=hidden.device)
    return ce.foak_gemm_bf16(dlogits, hidden, dw, a_mn_major=True, b_mn_major=True, mode=ce.FOAK_GEMM_F32)


def run(tokens=1024, vocab=32000, hidden=512, top_k=32, steps=20, temperature=2.0, ce_weight=0.3, lr=1.0,
        seed=0, device="cuda"):
    """Returns the losses of the distillation steps, and of the policy steps the mean log
    probability of the rewarded tokens.

    The softmax's curvature is at most 1/2 and that of the hidden states about
    (1 + sqrt(hidden / tokens))^2, so plain gradient steps of 1 descend for hidden <= tokens.
    """
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, scale):
        return scale * torch.randn(*shape, generator=gen, device=device)

    h = normal(tokens, hidden, scale=1.0).bfloat16()
    teacher = normal(vocab, hidden, scale=2.0 * hidden ** -0.5).bfloat16()
    master = normal(vocab, hidden, scale=0.5 * hidden ** -0.5)  # the student's weights in float32

    # 1. the teacher's targets; its likeliest token is the label, except for some padding
    z = logits_of(h, teacher)
    top = ce.foak_logprobs_forward(z, top_k=top_k, temperature=temperature, want_entropy=False, want_lse=False,
                                   want_stats=False)
    labels = top["top_ids"][:, 0].long()
    labels[::17] = -100
    del z

    # 2. distillation
    losses = []
    for _ in range(steps):
        logits = logits_of(h, master.bfloat16())
        r = ce.foak_distill_fwd_bwd(logits, labels, top["top_ids"], top["top_logprobs"], ce_weight=ce_weight,
                                    kd_weight=(1.0 - ce_weight) * temperature ** 2, temperature=temperature)
        master -= lr * head_gradient(r["dlogits"], h, vocab)
        losses.append(r["loss"])
    losses = torch.cat(losses).tolist()

    # 3. rewards: of two of the student's own likely tokens, the second is the better one
    own = ce.foak_logprobs_forward(logits_of(h, master.bfloat16()), top_k=2, want_stats=False)["top_ids"].long()
    own[labels < 0] = -100
    reward = torch.tensor([-1.0, 1.0], device=device)
    scores = []
    for _ in range(steps):
        logits = logits_of(h, master.bfloat16())
        grad = torch.zeros_like(master)
        for i in range(2):
            y = own[:, i].contiguous()
            f = ce.foak_logprobs_forward(logits, y)
            n = (y >= 0).sum()
            # loss = -(reward * logp + 0.001 * entropy) / n
            dl, _ = ce.foak_logprobs_backward(logits, y, f["stats"], (-reward[i] / n).expand(tokens).contiguous(),
                                              f["entropy"], (-0.001 / n).expand(tokens).contiguous())
            grad += head_gradient(dl, h, vocab)
            if i == 1:
                scores.append(f["logp"].sum() / n)
        master -= lr * grad
    return losses, torch.stack(scores).tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=1024)
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--hidden", type=int, default=512)
    p.add_argument("--top-k", type=int, default=32)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    losses, scores = run(a.tokens, a.vocab, a.hidden, a.top_k, a.steps)
    print("distillation loss      ", " ".join(f"{x:.4f}" for x in losses))
    print("rewarded tokens' logp  ", " ".join(f"{x:.4f}" for x in scores))


if __name__ == "__main__":
    main()
