"""The plain statements the operator tests compare with, against closed forms,
torch's own functions and differences (CPU)."""
import math

import numpy as np
import pytest
import torch

import finetune_reference as R


def _problem(seed=0, rows=9, vocab=23):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(rows, vocab, generator=g, dtype=torch.float64) * 2
    labels = torch.randint(0, vocab, (rows,), generator=g)
    labels[::4] = -100
    return logits, labels, g


def test_logp_is_log_softmax():
    logits, labels, _ = _problem()
    _, logp, lse = R.token_logp(logits, labels, 0.5)
    want = torch.log_softmax(logits * 0.5, 1)
    for r in range(len(labels)):
        if labels[r] < 0:
            assert logp[r] == 0 and lse[r] == 0
        else:
            assert abs(logp[r] - want[r, labels[r]]) < 1e-14
            assert abs(lse[r] - torch.logsumexp(logits[r] * 0.5, 0)) < 1e-14


def _directional(loss, grad, x, g, h=1e-5, tol=1e-8):
    u = torch.randn(x.shape, generator=g, dtype=torch.float64)
    slope = (loss(x + h * u) - loss(x - h * u)) / (2 * h)
    assert abs(slope - float((grad * u).sum())) < tol * (1 + abs(slope))


@pytest.mark.parametrize("kind,average,smoothing", [("sigmoid", False, 0.0), ("sigmoid", True, 0.1),
                                                    ("squared", True, 0.0), ("squared", False, 0.0)])
def test_preference_gradient_against_differences(kind, average, smoothing):
    logits, labels, g = _problem(3)
    cu = [0, 3, 5, 5, 9]
    ref = torch.randn(9, generator=g, dtype=torch.float64).numpy()

    def run(x):
        _, logp, lse = R.token_logp(x, labels)
        return R.preference(logp.numpy(), ref, labels.numpy(), cu, kind, 0.7, smoothing, average,
                            0.5), lse
    (loss, _, _, dlogp), lse = run(logits)
    grad = R.logits_grad(logits, labels, lse, torch.from_numpy(dlogp))
    _directional(lambda x: run(x)[0][0], grad, logits, g)
    # equal log ratios: the sigmoid loss is log 2
    zero = R.preference(ref, ref, None, cu, "sigmoid", 0.7)
    assert np.allclose(zero[1], math.log(2.0), atol=1e-15)


def test_policy_gradient_against_differences():
    logits, labels, g = _problem(5)
    logits.requires_grad_(False)
    _, logp, _ = R.token_logp(logits, labels)
    old = logp + torch.tensor([-0.5, -0.1, 0.05, 0.1, 0.5, -0.3, 0.3, 0.01, -0.01])
    ref = logp + 0.3 * torch.randn(9, generator=g, dtype=torch.float64)
    adv = torch.randn(9, generator=g, dtype=torch.float64)
    weight = torch.rand(9, generator=g, dtype=torch.float64)
    weight[2] = 0

    def run(x):
        _, lp, lse = R.token_logp(x, labels, 0.8)
        return R.policy(lp, labels, old, ref, adv, weight, 0.2, 0.3, 0.1, 0.25), lse
    (loss, terms, dlogp), lse = run(logits)
    x = logits * R.f32(0.8)
    grad = R.logits_grad(x, labels, lse, dlogp, 0.8)
    _directional(lambda y: run(y)[0][0][0], grad, logits, g)
    assert set(terms[:, 2].tolist()) == {0.0, 1.0}  # the clip acts on some tokens


def test_8_bit_first_moment_is_nearest():
    rng = np.random.default_rng(0)
    m = (rng.normal(size=2000) * np.exp(rng.uniform(-9, 3, 2000))).astype(np.float32)
    codes, scale = R.pack_m(m)
    back = R.unpack_m(codes, scale)
    grid = R.e4m3_values()
    grid = np.sort(grid[np.isfinite(grid)])
    e = R.per_element(scale, 2000)
    y = np.ldexp(m.astype(np.float64), 134 - e)
    nearest = np.abs(y[:, None] - grid[None]).min(1)
    assert np.array_equal(np.abs(np.ldexp(back.astype(np.float64), 134 - e) - y), nearest)
    # packing what was unpacked changes nothing
    again, scale2 = R.pack_m(back)
    assert np.array_equal(R.unpack_m(again, scale2), back)


def test_8_bit_second_moment_is_unbiased_and_never_zero():
    rng = np.random.default_rng(1)
    v = (np.exp(rng.uniform(-14, 0, 512)) * 1e-8).astype(np.float32)
    v[7], v[300] = 0.0, 1e-25
    total = np.zeros(512)
    n = 2000
    for t in range(n):
        codes, scale = R.pack_v(v, 512 * 3, R.key_of(11, t))
        assert codes[7] == 0 and (np.delete(codes, 7) > 0).all()
        total += R.unpack_v(codes, scale)
    e = R.per_element(scale, 512)
    step = np.ldexp(1.0, np.maximum(np.floor(np.log2(np.maximum(v, 1e-30))), e - 127 - 30).astype(
        int) - 3)
    # the mean of n roundings, each uniform within a step: 6 standard errors (0.5 step / sqrt n)
    near = np.abs(total / n - v) < 6 * 0.5 * step / math.sqrt(n) + 1e-12 * v
    assert near[v > 1e-15].all()
    assert near.mean() > 0.99


def test_random_bits_are_balanced():
    n = 1 << 16
    a = R.random16(0, n, R.key_of(1, 1)) / 65536.0
    b = R.random16(0, n, R.key_of(1, 2)) / 65536.0
    se = 1 / math.sqrt(n)
    assert abs(a.mean() - 0.5) < 5 * 0.29 * se
    for x, y in ((a[:-1], a[1:]), (a[:-2], a[2:]), (a, b), (a[:-256], a[256:])):
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 * se
    far = R.random16((1 << 34) + 6, 512, 77)
    assert not np.array_equal(far, R.random16(6, 512, 77))
