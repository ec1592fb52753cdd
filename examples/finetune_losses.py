"""Fine-tuning with the losses of this package and its Adafactor step.

A small model (an embedding, a mixing layer and an output layer) is trained in
three stages, each a few steps on a batch of synthetic token sequences:

  distill      toward the top entries of a fixed teacher of the same kind
  preference   to prefer the sequences that follow a rule to ones that do not
  policy       with rewards for sampled tokens, clipped against the policy that
               sampled them, and a KL term that holds it near the model of the
               stage before (its loss begins at 0 with each new set of samples)

Reference and old log-probabilities come from ``token_logprobs``.  The gradient
of the logits is written over them (``grad=logits``), so a step keeps one
[tokens, vocab] tensor.

    python examples/finetune_losses.py [--vocab 32000] [--steps 10]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_efficient_optimizer_gb300 as meo  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab, width, seed):
        super().__init__()
        torch.manual_seed(seed)
        self.embed = torch.nn.Embedding(vocab, width)
        self.mix = torch.nn.Linear(width, width)
        self.out = torch.nn.Linear(width, vocab, bias=False)

    def forward(self, tokens):
        x = self.embed(tokens)
        return torch.nn.functional.linear((x + torch.tanh(self.mix(x))).bfloat16(), self.out.weight.bfloat16())


def step(model, opt, tokens, loss):
    """One step: logits, loss and gradient over them, the weights' gradients, the optimizer."""
    logits = model(tokens)
    out = loss(logits.detach())
    logits.backward(out.grad)
    opt.step()
    opt.zero_grad(set_to_none=True)
    return out.loss


def shifted(tokens, prompt):
    """Inputs and targets of next-token prediction; the prompt is not trained on."""
    targets = tokens[:, 1:].clone()
    targets[:, : prompt - 1] = -100
    return tokens[:, :-1], targets


def follow_rule(first, length, vocab):
    """Sequences in which every token is the one before times five plus one."""
    out = [first]
    for _ in range(length - 1):
        out.append((out[-1] * 5 + 1) % vocab)
    return torch.stack(out, 1)


def distill(model, teacher, opt, steps, batch, length, vocab, top=16, tau=2.0):
    tokens = torch.randint(0, vocab, (batch, length), device="cuda")
    with torch.no_grad():
        t = 8 * teacher(tokens).float()  # an untrained teacher is nearly uniform: sharpened
        values, ids = t.topk(top)
        lse = torch.logsumexp(t / tau, -1)
    for _ in range(steps):
        yield step(model, opt, tokens, lambda x: meo.distill_loss(x, ids, values, lse, temperature=tau, grad=x))


def preference(model, reference, opt, steps, pairs, length, vocab):
    good = follow_rule(torch.randint(0, vocab, (pairs,), device="cuda"), length, vocab)
    bad = torch.cat([good[:, :1], torch.randint(0, vocab, (pairs, length - 1), device="cuda")], 1)
    inputs, targets = shifted(torch.cat([good, bad]), prompt=2)
    with torch.no_grad():
        ref = meo.token_logprobs(reference(inputs), targets).logp
    for _ in range(steps):
        yield step(model, opt, inputs, lambda x: meo.preference_loss(x, targets, ref, beta=0.2, grad=x))


def policy(model, reference, opt, steps, batch, length, vocab):
    for k in range(steps):
        if k % 4 == 0:  # new samples every four steps
            inputs = torch.randint(0, vocab, (batch, length), device="cuda")
            with torch.no_grad():
                logits = model(inputs)
                # a quarter of the samples follow the rule, the others the model
                drawn = torch.multinomial(torch.softmax(logits.float().flatten(0, 1), -1), 1).view(batch, length)
                right = (inputs * 5 + 1) % vocab
                targets = torch.where(torch.rand(batch, length, device="cuda") < 0.25, right, drawn)
                old = meo.token_logprobs(logits, targets).logp
                ref = meo.token_logprobs(reference(inputs), targets).logp
                reward = (targets == right).float()
                advantages = reward - reward.mean(1, keepdim=True)
        yield step(model, opt, inputs, lambda x: meo.policy_loss(x, targets, advantages, old, ref, clip_high=0.28,
                                                                 kl_coef=0.01, grad=x))


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--length", type=int, default=64)
    ap.add_argument("--steps", type=int, default=10)
    args = ap.parse_args(argv)
    model, teacher = Model(args.vocab, args.width, 0).cuda(), Model(args.vocab, args.width, 1).cuda()
    opt = meo.Adafactor(model.parameters(), lr=3e-3, relative_step=False, scale_parameter=False)
    size = (args.batch, args.length, args.vocab)
    frozen = Model(args.vocab, args.width, 0).cuda()
    torch.manual_seed(2)
    results = {}
    # a preference adds up a sequence's tokens: at the first stage's rate one step goes past its minimum
    for name, lr, stage in (("distill", 3e-3, lambda: distill(model, teacher, opt, args.steps, *size)),
                            ("preference", 1e-4, lambda: preference(model, frozen, opt, args.steps, *size)),
                            ("policy", 1e-4, lambda: policy(model, frozen, opt, args.steps, *size))):
        frozen.load_state_dict(model.state_dict())
        for group in opt.param_groups:
            group["lr"] = lr
        losses = torch.stack(list(stage())).tolist()
        results[name] = losses
        print(f"{name:11s} " + " ".join(f"{v:8.4f}" for v in losses))
    return results


if __name__ == "__main__":
    main()
