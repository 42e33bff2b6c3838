"""Random configurations of the losses and the many-tensor step, against their
plain statements with the tolerances of test_gpu_losses and bit for bit as in
test_gpu_many."""
import math

import numpy as np
import pytest
import torch

import finetune_reference as R
import test_gpu_losses as L
import test_gpu_many as M
import zero_partitioned_mixed_plan_amd as z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(24))
def test_random_losses(seed):
    rng = np.random.default_rng(1000 + seed)
    vocab = int(np.exp(rng.uniform(0, math.log(150000))))
    rows = int(np.exp(rng.uniform(0, math.log(max(2, min(3000, 3000000 // vocab))))))
    dt = rng.choice(["bf16", "f16", "f32"])
    pad, shift, oshift = (int(x) for x in rng.integers(0, 20, 3))
    inv_t = float(rng.choice([1.0, 0.5, 1.7]))
    m = L.Matrix(rows, vocab, dt, pad, shift, seed=seed, sigma=float(rng.uniform(0.5, 8)))
    m.labels[torch.from_numpy(rng.random(rows) < 0.3)] = -1
    if rng.random() < 0.3:  # a masked vocabulary
        m.host[:, torch.from_numpy(rng.random(vocab) < 0.5)] = -math.inf
        keep = m.labels >= 0
        m.host[torch.nonzero(keep)[:, 0], m.labels[keep]] = 1.0
    print(f"[random] rows={rows} vocab={vocab} {dt} pad={pad} shift={shift},{oshift} T={inv_t}",
          flush=True)
    logits, lab, logp, lse = L._logp(m, inv_t)
    x, wlse = L._check_logp(m, logp, lse, inv_t)
    dlogp = torch.randn(rows, generator=m.g)
    out = L.Matrix(rows, vocab, dt, pad, oshift)
    obuf, dl = out.device()
    z.zero_token_logp_grad(logits, lab, lse, dlogp.to(L.DEV), dl, inv_temperature=inv_t)
    want = R.logits_grad(x, m.labels, wlse, dlogp, inv_t)
    L._close(dl, want, L._grad_tol(want, x, wlse, dlogp, inv_t, dt), "dlogits")
    out.guards_untouched(obuf)
    _, wlogp, _ = R.token_logp(m.host, m.labels, inv_t)
    _, _, _, old, ref, adv, weight = L._policy_inputs(m, inv_t)
    kl = float(rng.choice([0.0, 0.1]))
    got = L._policy(m, logits, lab, old, ref, adv, weight, inv_t, kl, dl)
    L._check_policy(m, x, wlogp, wlse, old, ref, adv, weight, inv_t, kl, 1.0, *got, dl, dt)
    out.guards_untouched(obuf)


@pytest.mark.parametrize("seed", range(24))
def test_random_many(seed):
    rng = np.random.default_rng(2000 + seed)
    n = int(np.exp(rng.uniform(0, math.log(300))))
    sizes = [int(s) for s in np.exp(rng.uniform(0, math.log(rng.integers(2, 20000)), n))]
    if rng.random() < 0.3:
        sizes[int(rng.integers(n))] = 0
    gdt = rng.choice(["bf16", "f16", "f32"])
    pdt = rng.choice(["bf16", "f16", None])
    bits = int(rng.choice([8, 8, 32]))
    shift, groups = int(rng.integers(0, 40)), int(rng.integers(1, 3))
    none = [i for i in range(n) if rng.random() < 0.05]
    print(f"[random] {n} tensors, {sum(sizes)} elements, {gdt} {pdt} {bits} bits shift={shift} "
          f"groups={groups} none={none}", flush=True)
    m = M.Model(sizes, gdt, pdt, bits, shift, seed=seed, groups=groups, none=none, scale=16.0)
    first = int(rng.integers(0, 1000))
    z.zero_many_state_upload(m.many, first, z.LossScaler(16.0, dynamic=False), seed=seed)
    for t in range(first + 1, first + 4):
        m.new_grads()
        sumsq, flag, want = M._norm(m)
        assert abs(sumsq.item() - want) <= (sum(sizes) + 1) * 2.0 ** -53 * want
        assert flag.item() == 0
        clip = float(rng.choice([0.0, 0.01, 1e9]))
        z.zero_many_adam_step(m.many, m.hp, flag=flag, sumsq=sumsq, max_norm=clip)
        m.plain_step(t, 16.0, R.clip_coef(sumsq.item(), 16.0, clip), seed)
        m.check()
