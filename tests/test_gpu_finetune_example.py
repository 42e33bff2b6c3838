"""The fine-tuning example end to end, and one of its steps against the same
step in plain torch."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import finetune_reference as R
import zero_partitioned_mixed_plan_amd as z

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "preference_tuning.py")


def _example():
    spec = importlib.util.spec_from_file_location("preference_tuning", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns():
    first, last, margin, policy, state = _example().main(["--steps", "40"])
    assert abs(first - math.log(2)) < 1e-5  # the model starts as its own reference
    assert last < 0.5 * first and margin > 0
    assert torch.isfinite(policy).all() and policy[-1, 0] < policy[0, 0]
    assert state.applied_steps + state.skipped_steps == 80 and state.skipped_steps < 20


def test_first_step_against_plain_torch():
    """The example's first preference step: the loss's gradient to every parameter through
    torch's autograd of the plain loss, in fp32 on the CPU from the same fp16 weights."""
    ex = _example()
    model = ex.Model()
    seqs, labels = ex.make_pairs(1)
    rows = labels.numel()
    logits = model.logits(seqs)
    raw = logits.detach()
    f = lambda *s: torch.empty(*s, device=ex.DEV)
    logp, lse, dlogp, grad = f(rows), f(rows), f(rows), torch.empty_like(raw)
    ref = torch.zeros(rows, device=ex.DEV)
    cu = torch.arange(0, rows + 1, ex.LENGTH, device=ex.DEV)
    scale = 4096.0
    z.zero_token_logp(raw, labels, logp, lse)
    loss, pair, rew = f(1), f(ex.PAIRS), f(ex.PAIRS, 2)
    z.zero_preference_loss(logp, ref, cu, loss, pair, rew, dlogp, labels=labels, beta=0.2,
                           loss_scale=scale)
    z.zero_token_logp_grad(raw, labels, lse, dlogp, grad)
    # plain: the same loss from the same logits, by autograd in 64 bits
    x = raw.double().cpu().requires_grad_()
    lab = labels.cpu()
    lp = torch.log_softmax(x, 1).gather(1, lab.clamp(min=0)[:, None])[:, 0]
    lp = torch.where(lab >= 0, lp, 0.0).view(2 * ex.PAIRS, ex.LENGTH).sum(1)
    beta = R.f32(0.2)
    want = -torch.nn.functional.logsigmoid(beta * (lp[0::2] - lp[1::2])).mean()
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-5 * want.item()
    got = grad.double().cpu() / scale
    size = x.grad.abs()
    # half a step of fp16 (and of its subnormals at this scale), the coefficient's 1e-5
    tol = size * (2.0 ** -11 + 2e-5) + 2.0 ** -25 / scale
    assert ((got - x.grad).abs() <= tol).all()
    assert np.isfinite(got.numpy()).all()
