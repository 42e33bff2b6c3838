"""Refusals of the loss and many-tensor entry points, through the C ABI: every
one is decided on the host, before any device work (no GPU is needed)."""
import ctypes

import pytest

from zero_partitioned_mixed_plan_amd import _abi
from zero_partitioned_mixed_plan_amd._abi import (ZERO_BF16, ZERO_EALIGN, ZERO_EINVAL, ZERO_ENULL,
                                                  ZERO_ESTATE, ZERO_F16, ZERO_F32, lib)

P = 0x10000  # an address that is never read: each call below ends before a launch
NAN, INF = float("nan"), float("inf")


def _message():
    return lib.zero_last_error().decode()


def _logp(logits=P, dtype=ZERO_BF16, rows=4, vocab=10, stride=10, labels=P, inv_t=1.0, logp=P,
          lse=P):
    return lib.zero_token_logp(logits, dtype, rows, vocab, stride, labels, inv_t, logp, lse, None)


def _grad(logits=P, dtype=ZERO_BF16, rows=4, vocab=10, stride=10, labels=P, inv_t=1.0, lse=P,
          dlogp=P, dlogits=2 * P, dstride=10):
    return lib.zero_token_logp_grad(logits, dtype, rows, vocab, stride, labels, inv_t, lse, dlogp,
                                    dlogits, dstride, None)


MATRIX = [(dict(rows=(1 << 31) + 1), ZERO_EINVAL), (dict(dtype=0), ZERO_EINVAL), (dict(dtype=4), ZERO_EINVAL), (dict(rows=-1), ZERO_EINVAL),
          (dict(vocab=0), ZERO_EINVAL), (dict(vocab=(1 << 30) + 1, stride=1 << 40), ZERO_EINVAL),
          (dict(stride=9), ZERO_EINVAL), (dict(rows=1 << 40, stride=1 << 40), ZERO_EINVAL),
          (dict(inv_t=0.0), ZERO_EINVAL), (dict(inv_t=-1.0), ZERO_EINVAL),
          (dict(inv_t=NAN), ZERO_EINVAL), (dict(inv_t=INF), ZERO_EINVAL),
          (dict(logits=None), ZERO_ENULL), (dict(labels=None), ZERO_ENULL),
          (dict(logits=P + 1), ZERO_EALIGN), (dict(logits=P + 2, dtype=ZERO_F32), ZERO_EALIGN),
          (dict(labels=P + 4), ZERO_EALIGN)]


@pytest.mark.parametrize("kw,code", MATRIX + [(dict(logp=None), ZERO_ENULL),
                                              (dict(logp=P + 2), ZERO_EALIGN),
                                              (dict(lse=P + 1), ZERO_EALIGN)])
def test_token_logp_refusals(kw, code):
    assert _logp(**kw) == code and _message()


@pytest.mark.parametrize("kw,code", MATRIX + [
    (dict(lse=None), ZERO_ENULL), (dict(dlogp=None), ZERO_ENULL), (dict(dlogits=None), ZERO_ENULL),
    (dict(dstride=9), ZERO_EINVAL), (dict(dlogits=P + 1), ZERO_EALIGN),
    (dict(rows=1 << 21, dstride=1 << 40), ZERO_EINVAL),
    (dict(dlogits=P, dstride=12), ZERO_EINVAL)])  # in place with another stride
def test_token_logp_grad_refusals(kw, code):
    assert _grad(**kw) == code and _message()


def test_no_rows_is_no_work():
    assert _logp(rows=0, logits=None, labels=None, logp=None, lse=None) == 0
    assert _grad(rows=0, logits=None, labels=None, lse=None, dlogp=None, dlogits=None) == 0


def _pref(logp=P, ref=P, labels=P, rows=4, seq=P, pairs=1, norm=1.0, beta=0.1, smoothing=0.0,
          kind=0, average=0, scale=1.0, scale_dev=None, loss=P, pair=P, rewards=P, dlogp=P,
          cfg=True):
    c = _abi.zero_preference_t(norm, beta, smoothing, kind, average)
    return lib.zero_preference_loss(logp, ref, labels, rows, seq, pairs,
                                    ctypes.byref(c) if cfg else None, scale, scale_dev, loss, pair,
                                    rewards, dlogp, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=False), ZERO_ENULL), (dict(loss=None), ZERO_ENULL), (dict(rows=-1), ZERO_EINVAL),
    (dict(pairs=-1), ZERO_EINVAL), (dict(pairs=1 << 33), ZERO_EINVAL), (dict(beta=0.0), ZERO_EINVAL),
    (dict(beta=NAN), ZERO_EINVAL), (dict(beta=INF), ZERO_EINVAL), (dict(smoothing=1.0), ZERO_EINVAL),
    (dict(smoothing=-0.1), ZERO_EINVAL), (dict(kind=2), ZERO_EINVAL),
    (dict(kind=1, smoothing=0.1), ZERO_EINVAL), (dict(norm=NAN), ZERO_EINVAL),
    (dict(scale=0.0), ZERO_EINVAL), (dict(scale=INF), ZERO_EINVAL), (dict(scale_dev=P + 4), ZERO_EALIGN),
    (dict(logp=None), ZERO_ENULL), (dict(dlogp=None), ZERO_ENULL), (dict(pair=None), ZERO_ENULL),
    (dict(rewards=None), ZERO_ENULL), (dict(seq=None), ZERO_ENULL), (dict(seq=P + 4), ZERO_EALIGN),
    (dict(labels=P + 4), ZERO_EALIGN), (dict(ref=P + 1), ZERO_EALIGN)])
def test_preference_refusals(kw, code):
    assert _pref(**kw) == code and _message()


def _policy(norm=1.0, lo=0.2, hi=0.2, kl=0.0, inv_t=1.0, scale=1.0, scale_dev=None, old=P, ref=P,
            adv=P, weight=P, logp=P, terms=P, loss=P, dlogits=2 * P, dstride=10, cfg=True, logits=P,
            dtype=ZERO_F16, rows=4, vocab=10, stride=10, labels=P):
    c = _abi.zero_policy_t(norm, lo, hi, kl, inv_t)
    return lib.zero_policy_loss(logits, dtype, rows, vocab, stride, labels, old, ref, adv, weight,
                                ctypes.byref(c) if cfg else None, scale, scale_dev, logp, terms,
                                loss, dlogits, dstride, None)


@pytest.mark.parametrize("kw,code", MATRIX + [
    (dict(cfg=False), ZERO_ENULL), (dict(loss=None), ZERO_ENULL), (dict(lo=1.0), ZERO_EINVAL),
    (dict(lo=-0.1), ZERO_EINVAL), (dict(hi=-0.1), ZERO_EINVAL), (dict(hi=INF), ZERO_EINVAL),
    (dict(kl=-1.0), ZERO_EINVAL), (dict(kl=NAN), ZERO_EINVAL), (dict(kl=0.1, ref=None), ZERO_EINVAL),
    (dict(scale=-1.0), ZERO_EINVAL), (dict(norm=INF), ZERO_EINVAL), (dict(old=None), ZERO_ENULL),
    (dict(adv=None), ZERO_ENULL), (dict(logp=None), ZERO_ENULL), (dict(terms=None), ZERO_ENULL),
    (dict(dlogits=None), ZERO_ENULL), (dict(terms=P + 8), ZERO_EALIGN),
    (dict(weight=P + 2), ZERO_EALIGN), (dict(dstride=9), ZERO_EINVAL),
    (dict(dlogits=P, dstride=11), ZERO_EINVAL)])
def test_policy_refusals(kw, code):
    assert _policy(**kw) == code and _message()


# ------------------------------------------------------------ many tensors
def _create(numels, groups=None, n_groups=1, bits=8):
    h = ctypes.c_void_p()
    arr = (ctypes.c_int64 * max(len(numels), 1))(*numels)
    grp = None if groups is None else (ctypes.c_int32 * len(groups))(*groups)
    return lib.zero_many_create(arr, grp, len(numels), n_groups, bits, ctypes.byref(h)), h


@pytest.mark.parametrize("kw", [dict(numels=[1, -1]), dict(numels=[1 << 60]),
                                dict(numels=[1 << 47, 1 << 47]),
                                dict(numels=[4], bits=16), dict(numels=[4], n_groups=0),
                                dict(numels=[4], n_groups=17), dict(numels=[4], groups=[1]),
                                dict(numels=[4], groups=[-1], n_groups=2)])
def test_create_refusals(kw):
    rc, h = _create(**kw)
    assert rc == ZERO_EINVAL and not h.value and _message()


def test_create_null():
    assert lib.zero_many_create(None, None, 1, 1, 8, ctypes.byref(ctypes.c_void_p())) == ZERO_ENULL
    assert lib.zero_many_create(None, None, 0, 1, 8, None) == ZERO_ENULL
    assert lib.zero_many_info(None, ctypes.byref(_abi.zero_many_info_t())) == ZERO_ENULL
    lib.zero_many_destroy(None)


def test_info_and_offsets():
    numels = [0, 1, 256, 257, 1000]
    rc, h = _create(numels, groups=[0, 1, 0, 1, 0], n_groups=2)
    assert rc == 0
    info = _abi.zero_many_info_t()
    assert lib.zero_many_info(h, ctypes.byref(info)) == 0
    assert (info.total_numel, info.padded_numel) == (1514, 256 + 256 + 512 + 1024)
    assert info.state_bytes == 2 * (1514 + 8)
    out = (ctypes.c_int64 * 5)()
    assert lib.zero_many_offsets(h, out, 5) == 5
    assert list(out) == [0, 0, 256, 512, 1024]
    assert lib.zero_many_offsets(h, None, 0) == 5
    assert lib.zero_many_offsets(h, None, 1) == ZERO_ENULL
    assert lib.zero_many_offsets(h, out, -1) == ZERO_EINVAL
    lib.zero_many_destroy(h)
    rc, h = _create(numels, bits=32)
    assert lib.zero_many_info(h, ctypes.byref(info)) == 0 and info.state_bytes == 8 * 1514
    lib.zero_many_destroy(h)


def _bind(h, n, gdt=ZERO_BF16, pdt=ZERO_BF16, **over):
    b = _abi.zero_many_buffers_t()
    keep = []
    for k in ("grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
              "param"):
        v = over.get(k, [P] * n)
        if v is not None:
            arr = (ctypes.c_void_p * n)(*v)
            keep.append(arr)
            setattr(b, k, ctypes.cast(arr, ctypes.c_void_p))
    b.grad_dtype, b.param_dtype = gdt, pdt
    return lib.zero_many_bind(h, ctypes.byref(b), None)


@pytest.mark.parametrize("over,code", [
    (dict(grad=None), ZERO_ENULL), (dict(gdt=0), ZERO_EINVAL), (dict(pdt=ZERO_F32), ZERO_EINVAL),
    (dict(master=None), ZERO_ENULL), (dict(exp_avg=None), ZERO_ENULL),
    (dict(exp_avg_sq=None), ZERO_ENULL), (dict(exp_avg_scale=None), ZERO_EINVAL),
    (dict(exp_avg_sq_scale=None, exp_avg_scale=None), ZERO_EINVAL),
    (dict(master=[P, None]), ZERO_ENULL), (dict(exp_avg=[P, None]), ZERO_ENULL),
    (dict(exp_avg_scale=[None, P]), ZERO_ENULL), (dict(param=[P, None]), ZERO_ENULL),
    (dict(grad=[P, P + 1]), ZERO_EALIGN), (dict(grad=[P + 2, P], gdt=ZERO_F32), ZERO_EALIGN),
    (dict(master=[P + 2, P]), ZERO_EALIGN), (dict(param=[P + 1, P]), ZERO_EALIGN)])
def test_bind_refusals(over, code):
    rc, h = _create([300, 5])
    assert rc == 0
    assert _bind(h, 2, **over) == code and _message()
    # nothing was bound
    assert lib.zero_many_grad_norm(h, P, P, None) == ZERO_ESTATE
    lib.zero_many_destroy(h)


def test_bind_32_bits_refuses_scales_and_odd_moments():
    rc, h = _create([300], bits=32)
    assert _bind(h, 1) == ZERO_EINVAL
    none = dict(exp_avg_scale=None, exp_avg_sq_scale=None)
    assert _bind(h, 1, exp_avg=[P + 2], **none) == ZERO_EALIGN
    assert lib.zero_many_bind(None, None, None) == ZERO_ENULL
    lib.zero_many_destroy(h)


def test_calls_before_bind_and_upload():
    rc, h = _create([300])
    hp = (_abi.zero_adam_hparams_t * 1)(_abi.zero_adam_hparams_t(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 0))
    step = lambda hp=hp, n=1, flag=P, sumsq=P, mx=1.0, norm=P: lib.zero_many_adam_step(
        h, hp, n, flag, sumsq, mx, norm, None)
    assert step() == ZERO_ESTATE
    assert step(hp=None) == ZERO_ENULL
    assert step(n=2) == ZERO_EINVAL
    assert step(mx=-1.0) == ZERO_EINVAL and step(mx=NAN) == ZERO_EINVAL
    assert step(sumsq=None) == ZERO_ENULL and step(sumsq=None, mx=0.0) == ZERO_ENULL
    assert step(sumsq=P + 4) == ZERO_EALIGN and step(flag=P + 2) == ZERO_EALIGN
    bad = (_abi.zero_adam_hparams_t * 1)(_abi.zero_adam_hparams_t(1e-3, 1.0, 0.999, 1e-8, 0.0, 1, 0))
    assert step(hp=bad) == ZERO_EINVAL
    assert lib.zero_many_grad_norm(h, P, P, None) == ZERO_ESTATE
    assert lib.zero_many_grad_norm(h, None, P, None) == ZERO_ENULL
    assert lib.zero_many_grad_norm(h, P + 4, P, None) == ZERO_EALIGN
    assert lib.zero_many_state_values(h, P, P, None) == ZERO_ESTATE
    assert lib.zero_many_state_values(h, P + 4, P, None) == ZERO_EALIGN
    sc = _abi.zero_scaler_t()
    assert lib.zero_many_state_download(h, None, None, None, None, None) == ZERO_ESTATE
    assert lib.zero_many_device_scale(h, ctypes.byref(ctypes.c_void_p())) == ZERO_ESTATE
    good = _abi.zero_scaler_t(1.0, 1.0, 0.5, 2.0, 1000, 0, 1, 0)
    assert lib.zero_many_state_upload(h, -1, ctypes.byref(good), 0, None) == ZERO_EINVAL
    assert lib.zero_many_state_upload(h, 0, ctypes.byref(sc), 0, None) == ZERO_EINVAL
    assert lib.zero_many_state_upload(h, 0, None, 0, None) == ZERO_ENULL
    lib.zero_many_destroy(h)


def test_binding_checks_its_arguments():
    torch = pytest.importorskip("torch")
    import zero_partitioned_mixed_plan_amd as z
    many = z.zero_many_create([10, 20], groups=[0, 1], n_groups=2)
    assert (many.total_numel, many.padded_numel, many.blocks()) == (30, 512, [1, 1])
    with pytest.raises(ValueError, match="2 entries"):
        z.zero_many_bind(many, [None])
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_many_bind(many, [torch.zeros(10), None])
    with pytest.raises(ValueError, match="need 2 groups"):
        z.zero_many_create([10, 20], groups=[0])
    host = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_token_logp(host, torch.zeros(4, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(ValueError, match="kind"):
        z.zero_preference_loss(None, None, None, None, None, None, None, kind="hinge")
    many.close()
    with pytest.raises(z.ZeroError, match="ZERO_ENULL"):
        many.offsets()
