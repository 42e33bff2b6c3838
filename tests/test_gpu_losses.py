"""Log-probabilities, preference loss and policy loss on the GPU against their
plain 64-bit statements.

Tolerances.  u = 2^-24 is half a step of fp32 at 1.  A row's x = logits * T
carries u |x|; an exponential's argument x - base two more roundings of at
most 2 u max|x| each and 1.5 u for the product with log2 e, its result 4 u;
a thread adds at most `terms` of them in fp32 (terms u), everything beyond is
fp64.  So lse is off by at most
    E = u (6 max|x| + terms + 8) + u |lse|,  terms <= ceil(vocab / 64) + 8
and logp by 2 E.  A gradient entry g ([j = label] - p) is off by |g| p (2 E +
4 u) + 3 u |g|, and half a step of its type (eps / 2 of the value, or half
the smallest subnormal).
"""
import math

import numpy as np
import pytest
import torch

import finetune_reference as R
import zero_partitioned_mixed_plan_amd as z

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133, "f32": 2.0 ** -149}


def _lse_tol(x, lse):
    fin = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(1)
    return U * (6 * fin + math.ceil(x.shape[1] / 64) + 16) + U * lse.abs()


def _close(got, want, tol, what=""):
    got, want = got.double().cpu(), want.double().cpu()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(),
                           got[bad][:3].tolist(), want[bad][:3].tolist())


def _grad_tol(want, x, lse, dlogp, inv_t, dt):
    g = (dlogp.double() * inv_t).abs()[:, None]
    p = (x - lse[:, None]).exp()
    e = _lse_tol(x, lse)[:, None]
    out = g * (p * (2 * e + 4 * U) + 3 * U)
    half = torch.finfo(DT[dt]).eps / 2
    return torch.nan_to_num(out * (1 + half) + half * want.abs() + TINY[dt] / 2, nan=math.inf)


class Matrix:
    """Logits in a buffer of their own: row stride, offset from alignment, guard elements."""

    def __init__(self, rows, vocab, dt, pad=0, shift=0, seed=0, sigma=3.0):
        g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + vocab)
        self.rows, self.vocab, self.dt, self.stride, self.shift = rows, vocab, dt, vocab + pad, shift
        self.host = (torch.randn(rows, vocab, generator=g) * sigma).to(DT[dt])
        self.labels = torch.randint(0, vocab, (rows,), generator=g)
        if rows > 2:
            self.labels[1::3] = -100
            self.labels[0], self.labels[2] = 0, vocab - 1
        self.g = g

    def device(self):
        n = self.rows * self.stride + self.shift + 8
        buf = torch.full((n,), 7.0, dtype=DT[self.dt], device=DEV)
        m = buf[self.shift:self.shift + self.rows * self.stride].view(self.rows, self.stride)
        m = m[:, :self.vocab]
        m.copy_(self.host.to(DEV))
        return buf, m

    def guards_untouched(self, buf):
        keep = torch.ones(buf.numel(), dtype=torch.bool)
        at = torch.arange(self.rows)[:, None] * self.stride + torch.arange(self.vocab) + self.shift
        keep[at.reshape(-1)] = False
        assert (buf.cpu()[keep] == 7.0).all()


def _new(*n):
    return torch.full(n, 123.0, device=DEV)


def _logp(m, inv_t=1.0, **kw):
    buf, logits = m.device()
    lab = m.labels.to(DEV)
    logp, lse = _new(m.rows), _new(m.rows)
    z.zero_token_logp(logits, lab, logp, lse, inv_temperature=inv_t, **kw)
    return logits, lab, logp, lse


def _check_logp(m, logp, lse, inv_t=1.0):
    x, wlogp, wlse = R.token_logp(m.host, m.labels, inv_t)
    e = _lse_tol(x, wlse)
    _close(lse, wlse, e, "lse")
    _close(logp, wlogp, 2 * e, "logp")
    return x, wlse


SHAPES = [(1, 1), (3, 2), (5, 7), (4, 63), (4, 64), (4, 65), (3, 255), (6, 257), (7, 511),
          (5, 513), (5, 1000), (3, 2047), (3, 4096), (5, 4099), (4, 8192), (4, 8200), (3, 16385),
          (3, 32000), (3, 32771), (4, 50257), (3, 65536), (2, 65541), (3, 128256), (2, 131072),
          (2, 131079), (1, 262147)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logp_and_gradient(rows, vocab, dt):
    for i, (pad, shift, oshift, inv_t) in enumerate([(0, 0, 0, 1.0), (3, 1, 1, 0.7),
                                                     (8, 0, 5, 1.25)]):
        m = Matrix(rows, vocab, dt, pad, shift, seed=i)
        logits, lab, logp, lse = _logp(m, inv_t)
        x, wlse = _check_logp(m, logp, lse, inv_t)
        dlogp = torch.randn(rows, generator=m.g)
        if rows > 3:
            dlogp[3] = 0.0
        out = Matrix(rows, vocab, dt, pad, oshift)
        obuf, dl = out.device()
        z.zero_token_logp_grad(logits, lab, lse, dlogp.to(DEV), dl, inv_temperature=inv_t)
        # against the formula with the kernel's own lse, then with the exact one
        want = R.logits_grad(x, m.labels, wlse, dlogp, inv_t)
        _close(dl, want, _grad_tol(want, x, wlse, dlogp, inv_t, dt), "dlogits")
        out.guards_untouched(obuf)
        # in place
        z.zero_token_logp_grad(logits, lab, lse, dlogp.to(DEV), logits, inv_temperature=inv_t)
        assert torch.equal(logits, dl)


def test_no_rows():
    e = torch.empty(0, 5, device=DEV, dtype=torch.bfloat16)
    lab = torch.empty(0, dtype=torch.int64, device=DEV)
    f = torch.empty(0, device=DEV)
    z.zero_token_logp(e, lab, f, f)
    z.zero_token_logp_grad(e, lab, f, f, e)
    loss = _new(4)
    z.zero_policy_loss(e, lab, f, f, e, f, torch.empty(0, 4, device=DEV), loss)
    assert loss.tolist() == [0, 0, 0, 0]


def _special(dt, vocab):
    """Rows with masked words, nothing left, infinities and NaN; labels outside."""
    m = Matrix(12, vocab, dt, pad=1, shift=1, seed=5)
    low = torch.finfo(DT[dt]).min
    m.labels[:] = torch.arange(12) % vocab
    h = m.host
    h[0, :] = -math.inf                       # nothing left
    h[1, :] = low                             # the type's lowest value everywhere
    h[2, 1:] = -math.inf                      # one word left, the label
    m.labels[2] = 0
    h[3, :] = -math.inf                       # one word left, not the label
    h[3, 4] = 2.0
    m.labels[3] = 5
    h[4, ::2] = -math.inf
    h[5, ::2] = low
    h[6, 3] = math.nan
    h[7, 3] = math.inf
    m.labels[8] = vocab                       # outside
    m.labels[9] = 1 << 40
    m.labels[10] = -1                         # masked, with NaN in its logits
    h[10, :] = math.nan
    h[11, :] = 0.0
    return m


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [7, 300, 9001, 50257, 140001])
def test_rows_with_masks_infinities_and_nan(vocab, dt):
    m = _special(dt, vocab)
    logits, lab, logp, lse = _logp(m)
    x, wlogp, wlse = R.token_logp(m.host, m.labels)
    # a row of the lowest value: lse = low + log vocab, its tolerance is a step of the type
    e = _lse_tol(x, torch.nan_to_num(wlse, posinf=0, neginf=0))
    for r in range(12):
        if r in (7,):  # an infinite logit: no distribution
            assert math.isnan(logp[r].item())
            continue
        _close(lse[r:r + 1], wlse[r:r + 1], e[r:r + 1], f"lse {r}")
        _close(logp[r:r + 1], wlogp[r:r + 1], 2 * e[r:r + 1], f"logp {r}")
    assert logp[0].item() == -math.inf and logp[3].item() == -math.inf
    assert logp[2].item() == 0.0 and logp[10].item() == 0.0
    assert math.isnan(logp[6].item()) and math.isnan(logp[8].item()) and math.isnan(logp[9].item())
    dlogp = torch.ones(12)
    out = torch.full_like(logits, 9.0)
    z.zero_token_logp_grad(logits, lab, lse, dlogp.to(DEV), out)
    want = R.logits_grad(x, m.labels, wlse, dlogp)
    tol = _grad_tol(want, x, wlse, dlogp, 1.0, dt)
    rows = [0, 2, 3, 4, 5, 10, 11]
    _close(out[rows], want[rows], tol[rows], "dlogits")
    assert (out[0] == 0).all() and (out[10] == 0).all()
    assert torch.isnan(out[6]).all()
    assert (out[3, [0, 1, 2, 3]] == 0).all()


# ------------------------------------------------------------ preference
def _pref_case(lens, seed, labels=True):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    n = int(cu[-1])
    logp = (-3 + rng.normal(size=n)).astype(np.float32)
    ref = (logp + 0.3 * rng.normal(size=n)).astype(np.float32)
    lab = rng.integers(-1, 4, n) if labels else None
    return cu, logp, ref, lab


PREF = [dict(lens=[5, 3], labels=True), dict(lens=[1, 1], labels=False),
        dict(lens=[0, 0], labels=False), dict(lens=[0, 7], labels=True),
        dict(lens=[255, 257, 256, 1, 0, 3], labels=True), dict(lens=[5000, 20000], labels=True),
        dict(lens=[(37 * i) % 90 for i in range(2 * 700)], labels=True)]


@pytest.mark.parametrize("case", PREF)
@pytest.mark.parametrize("kind,average,smoothing", [("sigmoid", False, 0.0), ("sigmoid", True, 0.1),
                                                    ("squared", True, 0.0), ("squared", False, 0.0)])
def test_preference(case, kind, average, smoothing):
    cu, logp, ref, lab = _pref_case(case["lens"], 3, case["labels"])
    if lab is not None and len(case["lens"]) == 6:
        lab[:255] = -1  # a sequence with every token masked
    pairs = len(cu) // 2
    n = len(logp)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    for use_ref, scale in ((True, 1.0), (False, 1024.0)):
        loss, pair, rew, dlogp = _new(1), _new(pairs), _new(pairs, 2), _new(max(n, 1))[:n]
        z.zero_preference_loss(d(logp), d(ref) if use_ref else None, d(cu), loss, pair, rew, dlogp,
                               labels=None if lab is None else d(lab), kind=kind, beta=0.3,
                               label_smoothing=smoothing, average=average, norm=0.25,
                               loss_scale=scale)
        want = R.preference(logp, ref if use_ref else None, lab, cu, kind, 0.3, smoothing, average,
                            0.25, scale)
        # fp64 inside: one rounding to fp32 each (the sums' order is worth 1e-9 of them)
        t = lambda a: torch.from_numpy(np.atleast_1d(np.asarray(a, np.float64)))
        for got, w, what in zip((loss, pair, rew, dlogp), want, ("loss", "pair", "rewards",
                                                                 "dlogp")):
            w = t(w)
            # the mean adds the fp32 pair losses: half a step each
            k = 2 if what == "loss" else 1
            _close(got, w, k * U * w.abs() * (1 + 1e-6) + 1e-9 * w.abs() + 1e-12, what)


def test_preference_no_pairs():
    loss = _new(1)
    f = torch.empty(0, device=DEV)
    cu = torch.zeros(1, dtype=torch.int64, device=DEV)
    z.zero_preference_loss(f, None, cu, loss, f, f, f)
    assert loss.item() == 0.0


def test_preference_extremes():
    """Margins far past what exp holds, and forbidden tokens (-inf)."""
    cu = np.array([0, 1, 2, 3, 4, 5, 6], np.int64)
    logp = np.array([2e4, -2e4, -2e4, 2e4, -np.inf, 0.0], np.float32)
    d = lambda a: torch.from_numpy(a).to(DEV)
    loss, pair, rew, dlogp = _new(1), _new(3), _new(3, 2), _new(6)
    z.zero_preference_loss(d(logp), None, d(cu), loss, pair, rew, dlogp, beta=1.0, norm=1.0)
    assert pair.tolist() == [0.0, 4e4, math.inf]
    assert dlogp.tolist() == [0.0, 0.0, -1.0, 1.0, -1.0, 1.0]


def test_device_loss_scale():
    cu, logp, ref, lab = _pref_case([5, 3, 2, 8], 1)
    d = lambda a: torch.from_numpy(a).to(DEV)
    scale = torch.tensor([512.0], dtype=torch.float64, device=DEV)
    out = []
    for kw in (dict(loss_scale=512.0), dict(loss_scale=3.0, loss_scale_dev=scale.data_ptr())):
        o = [_new(1), _new(2), _new(2, 2), _new(18)]
        z.zero_preference_loss(d(logp), d(ref), d(cu), *o, labels=d(lab), **kw)
        out.append(o)
    assert all(torch.equal(a, b) for a, b in zip(*out))


# ------------------------------------------------------------ policy
def _policy_inputs(m, inv_t):
    x, logp, lse = R.token_logp(m.host, m.labels, inv_t)
    g = torch.Generator().manual_seed(9)
    n = m.rows
    # old scores keep the ratio away from where the clip begins (0.8 and 1.3)
    shift = torch.tensor([-0.6, -0.1, 0.0, 0.1, 0.15, 0.5])[torch.randint(0, 6, (n,), generator=g)]
    old = (torch.nan_to_num(logp, neginf=-50.0) + shift).float()
    ref = (torch.nan_to_num(logp, neginf=-50.0) + 0.4 * torch.randn(n, generator=g)).float()
    adv = torch.randn(n, generator=g)
    weight = torch.rand(n, generator=g) + 0.1
    if n > 4:
        weight[4] = 0.0
        adv[3] = 0.0
    return x, logp, lse, old, ref, adv, weight


def _policy(m, logits, lab, old, ref, adv, weight, inv_t, kl, dl, scale=1.0, **kw):
    d = lambda a: None if a is None else a.to(DEV)
    logp, terms, loss = _new(m.rows), _new(m.rows, 4), _new(4)
    z.zero_policy_loss(logits, lab, d(old), d(adv), dl, logp, terms, loss, ref_logp=d(ref),
                       weight=d(weight), clip_low=0.2, clip_high=0.3, kl_coef=kl, norm=1 / 64,
                       inv_temperature=inv_t, loss_scale=scale, **kw)
    return logp, terms, loss


def _check_policy(m, x, wlogp, wlse, old, ref, adv, weight, inv_t, kl, scale, logp, terms, loss,
                  dl, dt):
    e = 2 * _lse_tol(x, wlse)
    _close(logp, wlogp, e, "logp")
    wloss, wterms, wd = R.policy(wlogp, m.labels, old, ref, adv, weight, 0.2, 0.3, kl, 1 / 64,
                                 scale)
    a = adv.double().abs()
    r = (wlogp - old.double()).exp()
    eq = torch.zeros_like(r) if ref is None else (ref.double() - wlogp).exp()
    tol = torch.zeros_like(wterms)
    tol[:, 0] = a * r * (2 * e) + U * wterms[:, 0].abs()
    tol[:, 1] = (eq + 1) * 2 * e + U * wterms[:, 1].abs() if ref is not None else 0.0
    tol = torch.where(wterms[:, 3:] != 0, tol, 0.0)
    _close(terms, wterms, tol, "terms")
    w = wterms[:, 3]
    per = (w * (tol[:, 0] + U * wterms[:, 0].abs())).sum() / 64
    perk = (w * (tol[:, 1] + U * wterms[:, 1].abs())).sum() / 64
    ltol = torch.stack([per + kl * perk, per, perk, torch.zeros_like(per)])
    wl = torch.from_numpy(wloss)
    _close(loss, wl, ltol + 2 * U * wl.abs() + 1e-12, "loss")
    # the coefficient's own error, then the row's
    dtol = (a * r * 2 * e + kl * eq * 2 * e) * w * scale / 64 + 2 * U * wd.abs()
    want = R.logits_grad(x, m.labels, wlse, wd, inv_t)
    one = R.logits_grad(x, m.labels, wlse, torch.where(wd != 0, 1.0, 0.0), inv_t).abs()
    _close(dl, want, _grad_tol(want, x, wlse, wd, inv_t, dt) + 1.01 * one * dtol[:, None],
           "dlogits")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_policy(rows, vocab, dt):
    for i, (pad, shift, oshift, inv_t, kl, plain) in enumerate([
            (0, 0, 0, 1.0, 0.1, False), (3, 1, 1, 0.7, 0.05, False), (8, 0, 5, 1.25, 0.0, True)]):
        m = Matrix(rows, vocab, dt, pad, shift, seed=20 + i)
        x, wlogp, wlse, old, ref, adv, weight = _policy_inputs(m, inv_t)
        if plain:
            ref, weight = None, None
        scale = 4096.0 if dt == "f16" else 1.0
        buf, logits = m.device()
        lab = m.labels.to(DEV)
        out = Matrix(rows, vocab, dt, pad, oshift)
        obuf, dl = out.device()
        got = _policy(m, logits, lab, old, ref, adv, weight, inv_t, kl, dl, scale)
        _check_policy(m, x, wlogp, wlse, old, ref, adv, weight, inv_t, kl, scale, *got, dl, dt)
        out.guards_untouched(obuf)
        got2 = _policy(m, logits, lab, old, ref, adv, weight, inv_t, kl, logits, scale)  # in place
        assert all(torch.equal(a, b) for a, b in zip(got, got2))
        assert torch.equal(logits, dl)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [300, 50257, 140001])
def test_policy_rows_with_masks_and_nan(vocab, dt):
    m = _special(dt, vocab)
    n = m.rows
    _, logits = m.device()
    lab = m.labels.to(DEV)
    f = lambda v: torch.full((n,), v, device=DEV)
    dl = torch.full_like(logits, 9.0)
    logp, terms, loss = _new(n), _new(n, 4), _new(4)
    weight = f(1.0)
    weight[[6, 7, 8, 9]] = 0.0  # tokens whose scores are NaN, left out by their weight
    z.zero_policy_loss(logits, lab, f(-2.0), f(1.0), dl, logp, terms, loss, weight=weight)
    assert torch.isfinite(loss).all()
    assert (dl[[0, 6, 7, 8, 9, 10]] == 0).all()  # nothing left, weight 0, masked
    assert torch.isnan(logp[[6, 7, 8, 9]]).all() and logp[10] == 0
    assert (terms[[6, 7, 8, 9, 10]] == 0).all()
    # a NaN with a weight reaches the loss and its own row, and no other
    weight[6] = 1.0
    before = dl.clone()
    z.zero_policy_loss(logits, lab, f(-2.0), f(1.0), dl, logp, terms, loss, weight=weight)
    assert torch.isnan(loss[0]) and torch.isnan(dl[6]).all()
    keep = [r for r in range(n) if r != 6]
    assert torch.equal(dl[keep], before[keep])


def test_policy_infinite_kl_without_a_coefficient():
    """A reference score far above the policy's: the KL is infinite, and stays out of the loss
    and the gradient while its coefficient is 0."""
    m = Matrix(4, 300, "f32", seed=3)
    m.labels[:] = 5
    m.host[0, 5] = -900.0
    _, logits = m.device()
    f = lambda v: torch.full((4,), v, device=DEV)
    dl, logp, terms, loss = torch.empty_like(logits), _new(4), _new(4, 4), _new(4)
    z.zero_policy_loss(logits, m.labels.to(DEV), f(-3.0), f(1.0), dl, logp, terms, loss,
                       ref_logp=f(0.0), kl_coef=0.0)
    assert math.isinf(terms[0, 1].item()) and math.isinf(loss[2].item())
    assert torch.isfinite(loss[:2]).all() and torch.isfinite(dl).all()


# ------------------------------------------------------- streams and graphs
def _whole_pass(bufs, stream=None):
    logits, lab, ref, cu, logp, lse, dlogp, loss, pair, rew, dl = bufs
    z.zero_token_logp(logits, lab, logp, lse, stream=stream)
    z.zero_preference_loss(logp, ref, cu, loss, pair, rew, dlogp, labels=lab, stream=stream)
    z.zero_token_logp_grad(logits, lab, lse, dlogp, dl, stream=stream)


def _pass_bufs(dt="bf16", vocab=5003):
    m = Matrix(40, vocab, dt, seed=2)
    _, logits = m.device()
    cu = torch.tensor([0, 9, 15, 30, 40], device=DEV)
    ref = torch.full((40,), -8.0, device=DEV)
    return [logits, m.labels.to(DEV), ref, cu, _new(40), _new(40), _new(40), _new(1), _new(2),
            _new(2, 2), torch.empty_like(logits)]


def test_other_stream_and_repeatability():
    a, b = _pass_bufs(), _pass_bufs()
    _whole_pass(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _whole_pass(b, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a[4:], b[4:]))


def test_graph_replays():
    a, b = _pass_bufs(), _pass_bufs()
    old, adv = torch.full((40,), -8.0, device=DEV), torch.ones(40, device=DEV)
    pol = [[torch.empty_like(a[0]), _new(40), _new(40, 4), _new(4)] for _ in range(2)]

    def both(x, p):
        _whole_pass(x)
        z.zero_policy_loss(x[0], x[1], old, adv, p[0], p[1], p[2], p[3], ref_logp=x[2],
                           kl_coef=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        both(a, pol[0])
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            both(a, pol[0])
    torch.cuda.synchronize()
    for i in range(4):
        fresh = torch.randn(40, a[0].shape[1], device=DEV).to(a[0].dtype) * (1 + i)
        a[0].copy_(fresh)
        b[0].copy_(fresh)
        graph.replay()
        both(b, pol[1])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a[4:] + pol[0], b[4:] + pol[1]))


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^32 elements."""
    vocab, rows = 131072, 32780
    buf = torch.zeros(rows * vocab, dtype=torch.bfloat16, device=DEV)
    logits = buf.view(rows, vocab)
    m = Matrix(6, vocab, "bf16", seed=8)
    m.labels[:] = torch.tensor([0, 5, -1, 7, vocab - 1, 3])
    logits[-6:] = m.host.to(DEV)
    lab = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
    lab[-6:] = m.labels.to(DEV)
    logp, lse = _new(rows), _new(rows)
    z.zero_token_logp(logits, lab, logp, lse)
    x, wlse = _check_logp(m, logp[-6:], lse[-6:])
    assert (logp[:-6] == 0).all()
    dlogp = torch.ones(6)
    full = torch.zeros(rows, device=DEV)
    full[-6:] = 1.0
    z.zero_token_logp_grad(logits, lab, lse, full, logits)
    want = R.logits_grad(x, m.labels, wlse, dlogp)
    _close(logits[-6:], want, _grad_tol(want, x, wlse, dlogp, 1.0, "bf16"), "dlogits")
    assert int(torch.count_nonzero(logits[:-6])) == 0


# --------------------------------------------------------------- differences
def test_gradients_against_differences():
    """Slopes of the 64-bit losses along random directions, against the fp32 gradients."""
    m = Matrix(40, 97, "f32", seed=4)
    x0 = m.host.double()
    g = torch.Generator().manual_seed(1)
    cu = [0, 9, 15, 30, 40]
    ref = (-4 + torch.randn(40, generator=g)).float()
    adv, h = torch.randn(40, generator=g), 1e-5
    _, lp0, _ = R.token_logp(x0, m.labels)
    old = (lp0 + torch.tensor([-0.6, 0.05, 0.1, 0.5] * 10)).float()

    def pref(x):
        return R.preference(R.token_logp(x, m.labels)[1].numpy(), ref.numpy(), m.labels.numpy(),
                            cu, norm=0.5)[0]

    def policy(x):
        return R.policy(R.token_logp(x, m.labels)[1], m.labels, old, ref, adv, None, 0.2, 0.2, 0.1,
                        1 / 40)[0][0]

    _, logits = m.device()
    lab = m.labels.to(DEV)
    logp, lse, dlogp, dl = _new(40), _new(40), _new(40), torch.empty_like(logits)
    z.zero_token_logp(logits, lab, logp, lse)
    z.zero_preference_loss(logp, ref.to(DEV), torch.tensor(cu, device=DEV), _new(1), _new(2),
                           _new(2, 2), dlogp, labels=lab, norm=0.5)
    z.zero_token_logp_grad(logits, lab, lse, dlogp, dl)
    dl2 = torch.empty_like(logits)
    z.zero_policy_loss(logits, lab, old.to(DEV), adv.to(DEV), dl2, logp, _new(40, 4), _new(4),
                       ref_logp=ref.to(DEV), kl_coef=0.1, norm=1 / 40)
    for f, grad in ((pref, dl), (policy, dl2)):
        grad = grad.double().cpu()
        for k in range(3):
            u = torch.randn(x0.shape, generator=g, dtype=torch.float64)
            slope = (f(x0 + h * u) - f(x0 - h * u)) / (2 * h)
            # the difference is good to h^2 and 1e-16 / h; the gradient's entries to 1e-5 of g
            size = float((grad * u).abs().sum())
            assert abs(slope - float((grad * u).sum())) < 1e-8 + 2e-5 * size
