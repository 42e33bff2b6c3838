"""Preference tuning, then policy tuning, of a small language model in fp16.

Every step: the model's forward in torch, the loss and its gradient to the
logits through the library (multiplied by the loss scale that the library
keeps on the device), torch's backward through the model, then the gradient
norm with the overflow test and AdamW with 8-bit moments over all tensors,
gated, clipped and loss-scaled on the device.  Nothing waits for the host
between steps.

    python examples/preference_tuning.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_partitioned_mixed_plan_amd as z  # noqa: E402

DEV, DTYPE = "cuda:0", torch.float16
VOCAB, WIDTH, PAIRS, LENGTH, PROMPT = 1000, 128, 16, 24, 8


class Model:
    """Embedding, one hidden layer over the last two tokens, and a head."""

    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(0)
        new = lambda *s, std: (torch.randn(*s, generator=g, device=DEV) * std)
        self.master = [new(VOCAB, WIDTH, std=0.5), new(2 * WIDTH, 4 * WIDTH, std=0.06),
                       torch.zeros(4 * WIDTH, device=DEV), new(4 * WIDTH, VOCAB, std=0.04)]
        self.param = [m.to(DTYPE).requires_grad_() for m in self.master]
        for p in self.param:
            p.grad = torch.zeros_like(p)

    def logits(self, tokens):
        """[sequences, length] tokens -> the scores of each next token, a row per position."""
        emb, w1, b1, w2 = self.param
        x = emb[tokens]
        x = torch.cat([x[:, :-1], torch.nn.functional.pad(x, (0, 0, 1, 0))[:, :-2]], -1)
        return torch.relu(x.flatten(0, 1) @ w1 + b1) @ w2


class Optimizer:
    """AdamW over the model's tensors: 8-bit moments, biases without decay."""

    def __init__(self, model, lr, scale):
        sizes = [m.numel() for m in model.master]
        decay = [int(m.dim() > 1) for m in model.master]
        self.many = z.zero_many_create(sizes, state_bits=8, groups=decay, n_groups=2)
        codes = lambda ns: [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in ns]
        z.zero_many_bind(self.many, [p.grad for p in model.param], model.master, codes(sizes),
                         codes(sizes), codes(self.many.blocks()), codes(self.many.blocks()),
                         [p.detach() for p in model.param])
        z.zero_many_state_upload(self.many, 0, z.LossScaler(scale, window=50), seed=1)
        self.hparams = [z.AdamHParams(lr=lr, weight_decay=wd) for wd in (0.0, 0.01)]
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
        self.flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.grads = [p.grad for p in model.param]

    def scale(self):
        return z.zero_many_device_scale(self.many)

    def step(self):
        z.zero_many_grad_norm(self.many, self.sumsq, self.flag)
        z.zero_many_adam_step(self.many, self.hparams, flag=self.flag, sumsq=self.sumsq,
                              max_norm=1.0)
        for g in self.grads:
            g.zero_()


def make_pairs(seed):
    """Chosen answers count upwards from the prompt's last word, rejected ones are noise."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    seqs = torch.randint(0, VOCAB, (2 * PAIRS, LENGTH + 1), generator=g, device=DEV)
    seqs[1::2, :PROMPT] = seqs[0::2, :PROMPT]  # a pair shares its prompt
    run = torch.arange(1, LENGTH + 2 - PROMPT, device=DEV)
    seqs[0::2, PROMPT:] = (seqs[0::2, PROMPT - 1:PROMPT] + run) % VOCAB
    labels = seqs[:, 1:].clone()
    labels[:, :PROMPT - 1] = -100  # the prompt itself is not scored
    return seqs, labels.reshape(-1)


def new(*shape):
    return torch.empty(*shape, device=DEV)


def preference_steps(model, opt, steps):
    rows = 2 * PAIRS * LENGTH
    offsets = torch.arange(0, rows + 1, LENGTH, device=DEV)
    seqs, labels = make_pairs(1)
    ref, logp, lse, dlogp = (new(rows) for _ in range(4))
    loss, pair_loss, rewards = new(steps), new(PAIRS), new(PAIRS, 2)
    with torch.no_grad():  # the frozen reference is the model as it starts
        z.zero_token_logp(model.logits(seqs), labels, ref)
    for i in range(steps):
        logits = model.logits(seqs)
        raw = logits.detach()
        z.zero_token_logp(raw, labels, logp, lse)
        z.zero_preference_loss(logp, ref, offsets, loss[i:], pair_loss, rewards, dlogp,
                               labels=labels, beta=0.2, loss_scale_dev=opt.scale())
        grad = torch.empty_like(raw)
        z.zero_token_logp_grad(raw, labels, lse, dlogp, grad)
        logits.backward(grad)
        opt.step()
    return loss, rewards


def policy_steps(model, opt, steps):
    rows = 2 * PAIRS * LENGTH
    seqs, labels = make_pairs(2)
    # the reward: counting answers are good, noise is not
    advantage = torch.tensor([1.0, -1.0], device=DEV).repeat(PAIRS).repeat_interleave(LENGTH)
    answered = LENGTH - PROMPT + 1
    old, logp, terms, loss = new(rows), new(rows), new(rows, 4), new(steps, 4)
    with torch.no_grad():
        z.zero_token_logp(model.logits(seqs), labels, old)
    ref = old.clone()
    for i in range(steps):
        logits = model.logits(seqs)
        raw = logits.detach()
        grad = torch.empty_like(raw)
        z.zero_policy_loss(raw, labels, old, advantage, grad, logp, terms, loss[i], ref_logp=ref,
                           kl_coef=0.02, norm=1.0 / (2 * PAIRS * answered),
                           loss_scale_dev=opt.scale())
        logits.backward(grad)
        opt.step()
    return loss


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    steps = ap.parse_args(argv).steps
    model = Model()
    opt = Optimizer(model, lr=2e-3, scale=2.0 ** 16)
    loss, rewards = preference_steps(model, opt, steps)
    first, last = loss[0].item(), loss[-1].item()
    margin = (rewards[:, 0] - rewards[:, 1]).mean().item()
    print(f"preference loss {first:.4f} -> {last:.4f}, reward margin {margin:.2f}")
    policy = policy_steps(model, opt, steps)
    print(f"policy loss {policy[0, 0].item():.4f} -> {policy[-1, 0].item():.4f}, "
          f"KL {policy[-1, 2].item():.4f}, clipped {policy[-1, 3].item():.2f}")
    state = z.zero_many_state_download(opt.many)
    print(f"{state.applied_steps} steps applied, {state.skipped_steps} skipped, loss scale "
          f"{state.scale:g}, {opt.many.state_bytes} bytes of moments for "
          f"{opt.many.total_numel} parameters")
    return first, last, margin, policy.cpu(), state


if __name__ == "__main__":
    main()
    z.release_all()
