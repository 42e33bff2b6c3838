"""The many-tensor AdamW step on the GPU.  The update's operations each round
once to fp32 in a pinned order and the 8-bit codes are exact functions of the
result, so every comparison is bit for bit; the norm adds exact squares in
fp64, n of them to within n 2^-53 of their sum."""
import math

import numpy as np
import pytest
import torch

import finetune_reference as R
import zero_partitioned_mixed_plan_amd as z

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [1, 0, 3, 255, 256, 257, 1023, 1024, 1025, 5000, 4, 2048, 100003]


def _bits(t):
    t = t.detach().cpu()
    if t.dtype == torch.float32:
        return t.view(torch.int32).numpy()
    if t.dtype in (torch.float16, torch.bfloat16):
        return t.view(torch.int16).numpy()
    return t.numpy()


def _place(host, shift):
    """A device copy that starts `shift` elements behind an aligned address, with guards."""
    buf = torch.full((host.numel() + shift + 16,), 77, dtype=host.dtype, device=DEV)
    view = buf[shift:shift + host.numel()]
    view.copy_(host.to(DEV))
    return buf, view


class Model:
    """Tensors on the host (numpy, the plain step) and on the device."""

    def __init__(self, sizes, gdt, pdt, bits, shift=0, seed=0, groups=2, none=(), scale=1.0,
                 sigma=1e-2):
        rng = np.random.default_rng(seed)
        self.sizes, self.gdt, self.pdt, self.bits, self.none = sizes, gdt, pdt, bits, set(none)
        self.rng, self.scale, self.sigma = rng, scale, sigma
        self.group = [i % groups for i in range(len(sizes))]
        self.hp = [z.AdamHParams(lr=2e-3, weight_decay=0.0), z.AdamHParams(
            lr=1e-3, beta1=0.8, beta2=0.99, weight_decay=0.1, adamw=False)][:groups]
        self.off, at = [], 0
        for n in sizes:
            self.off.append(at)
            at += -(-n // 256) * 256
        self.padded = at
        self.p = [rng.normal(0, 0.02, n).astype(np.float32) for n in sizes]
        self.m = [np.zeros(n, np.float32) for n in sizes]
        self.v = [np.zeros(n, np.float32) for n in sizes]
        nb = [-(-n // 256) for n in sizes]
        self.code = [[np.zeros(n, np.uint8) for n in sizes] for _ in range(2)]
        self.sc = [[np.zeros(b, np.uint8) for b in nb] for _ in range(2)]
        self.bufs = []

        def put(arrays, dtype=None):
            out = []
            for a in arrays:
                t = torch.from_numpy(a)
                buf, view = _place(t if dtype is None else t.to(dtype), shift)
                self.bufs.append((buf, shift, t.numel()))
                out.append(view)
            return out
        self.d_p = put(self.p)
        if bits == 8:
            self.d_m, self.d_v = put(self.code[0]), put(self.code[1])
            self.d_ms, self.d_vs = put(self.sc[0]), put(self.sc[1])
        else:
            self.d_m, self.d_v = put(self.m), put(self.v)
            self.d_ms = self.d_vs = None
        self.d_half = None if pdt is None else put(self.p, DT[pdt])
        self.d_g = put([np.zeros(n, np.float32) for n in sizes], DT[gdt])
        self.many = z.zero_many_create(sizes, state_bits=bits, groups=self.group, n_groups=groups)
        self.bind()

    def bind(self):
        grads = [None if i in self.none else g for i, g in enumerate(self.d_g)]
        z.zero_many_bind(self.many, grads, self.d_p, self.d_m, self.d_v, self.d_ms, self.d_vs,
                         self.d_half)

    def new_grads(self, edit=None):
        self.g = []
        for i, n in enumerate(self.sizes):
            g = torch.from_numpy((self.rng.normal(0, self.sigma, n) * self.scale).astype(np.float32))
            g = g.to(DT[self.gdt])
            if edit is not None:
                edit(i, g)
            self.d_g[i].copy_(g.to(DEV))
            self.g.append(g.float().numpy())

    def plain_step(self, t, scale, coef, seed):
        key = R.key_of(seed, t)
        for i, n in enumerate(self.sizes):
            if i in self.none or n == 0:
                continue
            hp = self.hp[self.group[i]]
            c = R.scalars(hp, t, scale, coef)
            if self.bits == 8:
                self.m[i] = R.unpack_m(self.code[0][i], self.sc[0][i])
                self.v[i] = R.unpack_v(self.code[1][i], self.sc[1][i])
            self.p[i], self.m[i], self.v[i] = R.adam(self.g[i], self.p[i], self.m[i], self.v[i], c,
                                                     hp.adamw)
            if self.bits == 8:
                self.code[0][i], self.sc[0][i] = R.pack_m(self.m[i])
                self.code[1][i], self.sc[1][i] = R.pack_v(self.v[i], self.off[i], key)

    def check(self):
        for i, n in enumerate(self.sizes):
            assert np.array_equal(_bits(self.d_p[i]), self.p[i].view(np.int32)), ("master", i)
            if self.pdt is not None:
                want = torch.from_numpy(self.p[i]).to(DT[self.pdt])
                if i not in self.none:
                    assert np.array_equal(_bits(self.d_half[i]), _bits(want)), ("param", i)
            pairs = ((self.d_m, self.m, 0), (self.d_v, self.v, 1))
            for dev, host, k in pairs:
                if self.bits == 32:
                    assert np.array_equal(_bits(dev[i]), host[i].view(np.int32)), (k, i)
                else:
                    scale = (self.d_ms, self.d_vs)[k][i]
                    assert np.array_equal(_bits(scale), self.sc[k][i]), ("scale", k, i)
                    assert np.array_equal(_bits(dev[i]), self.code[k][i]), ("codes", k, i)
        for buf, shift, n in self.bufs:
            b = buf.cpu()
            assert (b[:shift] == 77).all() and (b[shift + n:] == 77).all()


def _norm(model):
    sumsq = torch.full((1,), -1.0, dtype=torch.float64, device=DEV)
    flag = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    z.zero_many_grad_norm(model.many, sumsq, flag)
    want = math.fsum((model.g[i].astype(np.float64) ** 2).sum() for i in range(len(model.sizes))
                     if i not in model.none)
    return sumsq, flag, want


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("gdt,pdt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"),
                                     ("bf16", None), ("f32", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_steps(bits, gdt, pdt, shift):
    scale = 1024.0 if gdt == "f16" else 1.0
    m = Model(SIZES, gdt, pdt, bits, shift, seed=bits + shift, none=(6,), scale=scale)
    sc = z.LossScaler(scale, dynamic=False)
    z.zero_many_state_upload(m.many, 0, sc, seed=99)
    norm_out = torch.zeros(2, device=DEV)
    n = sum(SIZES)
    for t in range(1, 5):
        m.new_grads()
        sumsq, flag, want = _norm(m)
        assert abs(sumsq.item() - want) <= n * 2.0 ** -53 * want and flag.item() == 0
        clip = 0.5 if t % 2 else 0.0
        z.zero_many_adam_step(m.many, m.hp, flag=flag, sumsq=sumsq, max_norm=clip,
                              norm_out=norm_out)
        coef = R.clip_coef(sumsq.item(), scale, clip)
        assert (coef < 1) == bool(clip)
        m.plain_step(t, scale, coef, 99)
        m.check()
        got = norm_out.tolist()
        assert got[0] == pytest.approx(math.sqrt(sumsq.item()) / scale, rel=2.0 ** -23)
        assert got[1] == pytest.approx(coef, rel=2.0 ** -23)
    st = z.zero_many_state_download(m.many)
    assert (st.applied_steps, st.skipped_steps, st.last_flag) == (4, 0, 0)
    vals = [torch.full((m.padded,), 5.0, device=DEV) for _ in range(2)]
    z.zero_many_state_values(m.many, *vals)
    for k, v in enumerate(vals):
        want = np.zeros(m.padded, np.float32)
        for i, nn in enumerate(SIZES):
            src = (m.m, m.v)[k][i]
            if bits == 8:
                src = (R.unpack_m, R.unpack_v)[k](m.code[k][i], m.sc[k][i])
            want[m.off[i]:m.off[i] + nn] = src
        assert np.array_equal(_bits(v), want.view(np.int32))
    one = torch.full((m.padded,), 5.0, device=DEV)
    z.zero_many_state_values(m.many, exp_avg_sq=one)
    assert torch.equal(one, vals[1])


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("shift", [5, 31, 33])
def test_steps_at_odd_addresses(bits, shift):
    """Tensors that start anywhere in a cache line, sizes about its and a chunk's end."""
    sizes = [1, 31, 32, 33, 480, 481, 482, 511, 512, 513, 991, 2047, 2048, 2049, 4097]
    m = Model(sizes, "bf16", "bf16", bits, shift, seed=shift)
    z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False), seed=8)
    for t in range(1, 4):
        m.new_grads()
        sumsq, flag, want = _norm(m)
        assert abs(sumsq.item() - want) <= sum(sizes) * 2.0 ** -53 * want and flag.item() == 0
        z.zero_many_adam_step(m.many, m.hp, flag=flag)
        m.plain_step(t, 1.0, 1.0, 8)
        m.check()


def _wide(bits):
    """Moments over forty orders of magnitude, subnormals and huge values."""
    m = Model([3000, 777], "f32", "bf16", bits, seed=4, groups=1)

    def spread(i, g):
        k = torch.from_numpy(m.rng.uniform(-45, 15, g.numel()).astype(np.float32))
        g.copy_(torch.sign(g) * torch.pow(10.0, k.double()).float())
        g[::7] = 0.0
        g[256:512] = 0.0           # a block of zeros
        g[512:700] = 1e-30         # squares below every normal number
        if g.numel() > 2000:
            g[1500] = 1e18
    return m, spread


@pytest.mark.parametrize("bits", [8, 32])
def test_extreme_magnitudes(bits):
    m, spread = _wide(bits)
    z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False), seed=5)
    for t in range(1, 4):
        m.new_grads(spread)
        z.zero_many_adam_step(m.many, m.hp)
        m.plain_step(t, 1.0, 1.0, 5)
        m.check()


def test_nonfinite_first_moments_become_nan():
    """No flag is given, so the step goes ahead: the NaN and inf stay in their own elements."""
    m = Model([600], "f32", None, 8, seed=6, groups=1)

    def edit(i, g):
        g[3], g[5], g[400] = math.nan, math.inf, -math.inf
    z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False))
    m.new_grads(edit)
    z.zero_many_adam_step(m.many, m.hp)
    codes = m.d_m[0].cpu().numpy()
    assert [int(codes[k]) & 0x7F for k in (3, 5, 400)] == [0x7F] * 3
    rest = np.delete(np.arange(600), [3, 5, 400])
    assert not ((codes[rest] & 0x7F) == 0x7F).any()
    assert np.isfinite(m.d_p[0].cpu().numpy()[rest]).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("gdt", ["f16", "bf16", "f32"])
def test_overflow_skips_and_scales(bits, gdt):
    """Infinities and NaN at edges: state untouched, t kept, scale halved."""
    m = Model([5, 300, 4099], gdt, "bf16", bits, shift=1, seed=8, scale=256.0, sigma=1e-3)
    sc = z.LossScaler(256.0, dynamic=True, window=2)
    z.zero_many_state_upload(m.many, 0, sc, seed=3)
    scale, t, good = 256.0, 0, 0
    places = {2: (0, 4, math.inf), 4: (1, 256, math.nan), 5: (2, 4098, -math.inf), 8: (2, 0, math.nan)}
    for it in range(1, 10):
        bad = places.get(it)

        def edit(i, g):
            if bad is not None and bad[0] == i:
                g[bad[1]] = bad[2]
        m.new_grads(edit)
        sumsq, flag, _ = _norm(m)
        assert flag.item() == (bad is not None)
        z.zero_many_adam_step(m.many, m.hp, flag=flag, sumsq=sumsq if it % 2 else None,
                              max_norm=1.0 if it % 2 else 0.0)
        if bad is not None:
            scale, good = max(scale * 0.5, 1.0), 0
        else:
            t += 1
            m.plain_step(t, scale, R.clip_coef(sumsq.item(), scale, 1.0 if it % 2 else 0.0), 3)
            good += 1
            if good >= 2:
                scale, good = scale * 2, 0
        m.check()
        st = z.zero_many_state_download(m.many, scaler=sc)
        assert (st.applied_steps, st.skipped_steps, st.scale, st.last_flag) == (
            t, it - t, scale, int(bad is not None))
        assert sc.scale == scale
    # a norm that is not finite skips without a flag, too
    sumsq.fill_(math.nan)
    z.zero_many_adam_step(m.many, m.hp, sumsq=sumsq)
    m.check()
    assert z.zero_many_state_download(m.many).last_flag == 1


@pytest.mark.parametrize("gdt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("where", ["first", "last", "block", "chunk"])
def test_norm_flag_positions(gdt, where):
    m = Model([1, 1024, 70001], gdt, None, 32, seed=2, groups=1)
    big = torch.finfo(DT[gdt]).max

    def clean(i, g):
        g[-1] = big if gdt != "f32" else 1e19  # the largest finite value is no overflow
    m.new_grads(clean)
    sumsq, flag, want = _norm(m)
    assert flag.item() == 0 and abs(sumsq.item() - want) <= 71026 * 2.0 ** -53 * want
    i, k = {"first": (0, 0), "last": (2, 70000), "block": (1, 255), "chunk": (1, 1023)}[where]
    for value in (math.inf, -math.inf, math.nan):
        m.d_g[i][k] = value
        z.zero_many_grad_norm(m.many, sumsq, flag)
        assert flag.item() == 1


def test_grads_alone_and_nothing_at_all():
    sumsq = torch.full((1,), 7.0, dtype=torch.float64, device=DEV)
    flag = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    many = z.zero_many_create([5, 9], state_bits=32)
    g = [torch.full((5,), 2.0, device=DEV), torch.full((9,), 1.0, device=DEV)]
    z.zero_many_bind(many, g)
    z.zero_many_grad_norm(many, sumsq, flag)
    assert sumsq.item() == 29.0 and flag.item() == 0
    with pytest.raises(z.ZeroError, match="ZERO_ESTATE"):
        z.zero_many_adam_step(many, z.AdamHParams())
    many.close()
    for sizes in ([], [0, 0]):
        many = z.zero_many_create(sizes, state_bits=32)
        e = [torch.empty(0, device=DEV) for _ in sizes]
        z.zero_many_bind(many, e, e, e, e)
        z.zero_many_state_upload(many, 0, z.LossScaler(1.0, dynamic=False))
        z.zero_many_grad_norm(many, sumsq, flag)
        z.zero_many_adam_step(many, z.AdamHParams(), flag=flag, sumsq=sumsq, max_norm=1.0)
        assert sumsq.item() == 0.0 and flag.item() == 0
        assert z.zero_many_state_download(many).applied_steps == 1
        many.close()


def test_32_bit_step_equals_the_flat_shard():
    """The same AdamW as zero_adam_step, tensor by tensor instead of one flat shard."""
    sizes = [700, 64, 4096]
    m = Model(sizes, "bf16", "bf16", 32, seed=12, groups=1)
    m.hp = [z.AdamHParams()]
    z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False))
    plan = z.zero_partition_plan(sizes, 1, 0, 1)
    master = torch.cat(m.d_p).clone()
    mom, var = torch.zeros_like(master), torch.zeros_like(master)
    flat = torch.empty(sum(sizes), dtype=torch.bfloat16, device=DEV)
    half = torch.empty_like(flat)
    for t in range(1, 4):
        m.new_grads()
        z.zero_flatten_grads(plan, -1, m.d_g, flat)
        assert z.zero_adam_step(plan, m.hp[0], t, 1.0, flat, master, mom, var, half) == 0
        z.zero_many_adam_step(m.many, m.hp)
        for got, want in ((m.d_p, master), (m.d_m, mom), (m.d_v, var), (m.d_half, half)):
            assert torch.equal(torch.cat(got), want)


def test_other_stream_repeats_and_resume():
    """Two runs on two streams, one of them stopped and resumed half way: the same bits."""
    runs = []
    for resume in (False, True):
        m = Model([513, 2000], "bf16", "bf16", 8, seed=3)
        s = torch.cuda.Stream()
        z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False), seed=21, stream=s)
        for t in range(6):
            m.new_grads()
            s.wait_stream(torch.cuda.current_stream())
            if resume and t == 3:
                sc = z.LossScaler(1.0, dynamic=False)
                st = z.zero_many_state_download(m.many, stream=s, scaler=sc)
                m.many.close()
                m.many = z.zero_many_create(m.sizes, state_bits=8, groups=m.group, n_groups=2)
                m.bind()
                z.zero_many_state_upload(m.many, st.applied_steps, sc, seed=21, stream=s)
            z.zero_many_adam_step(m.many, m.hp, stream=s)
            s.synchronize()
        runs.append(m)
    a, b = runs
    for x, y in ((a.d_p, b.d_p), (a.d_m, b.d_m), (a.d_v, b.d_v), (a.d_vs, b.d_vs), (a.d_half, b.d_half)):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("bits", [8, 32])
def test_graph_replays(bits):
    sizes = [300, 5000, 1 << 16]
    a = Model(sizes, "f16", "f16", bits, seed=31, scale=64.0)
    b = Model(sizes, "f16", "f16", bits, seed=31, scale=64.0)
    sums = [torch.zeros(1, dtype=torch.float64, device=DEV) for _ in range(2)]
    flags = [torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2)]

    def step(m, k):
        z.zero_many_grad_norm(m.many, sums[k], flags[k])
        z.zero_many_adam_step(m.many, m.hp, flag=flags[k], sumsq=sums[k], max_norm=0.3)
    for m in (a, b):
        z.zero_many_state_upload(m.many, 0, z.LossScaler(64.0, window=3), seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(a, 0)
        # what waits is refused, and the capture goes on
        with pytest.raises(z.ZeroError, match="ZERO_ESTATE"):
            z.zero_many_state_download(a.many)
        with pytest.raises(z.ZeroError, match="ZERO_ESTATE"):
            a.bind()
    for it in range(6):
        def edit(i, g):
            if it == 3 and i == 1:
                g[77] = math.inf
        a.new_grads(edit)
        b.new_grads(edit)
        graph.replay()
        step(b, 1)
        torch.cuda.synchronize()
        for x, y in ((a.d_p, b.d_p), (a.d_m, b.d_m), (a.d_v, b.d_v), (a.d_half, b.d_half)):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
        assert torch.equal(sums[0], sums[1]) or (it == 3)
    sa, sb = (z.zero_many_state_download(m.many) for m in (a, b))
    assert sa == sb and (sa.applied_steps, sa.skipped_steps) == (5, 1)


@pytest.mark.parametrize("bits", [8, 32])
def test_bind_keeps_what_a_graph_was_captured_with(bits):
    sizes = [300, 5000]
    m = Model(sizes, "bf16", "bf16", bits, seed=41)
    z.zero_many_state_upload(m.many, 0, z.LossScaler(1.0, dynamic=False), seed=3)
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        z.zero_many_grad_norm(m.many, sumsq, flag)
        z.zero_many_adam_step(m.many, m.hp, flag=flag, sumsq=sumsq)
    args = [m.d_g, m.d_p, m.d_m, m.d_v, m.d_ms, m.d_vs, m.d_half]
    for change in ({0: [g.half() for g in m.d_g]}, {0: [g.float() for g in m.d_g]}, {6: None},
                   {6: [h.half() for h in m.d_half]}, {k: None for k in range(1, 7)}):
        with pytest.raises(z.ZeroError, match="captured"):
            z.zero_many_bind(m.many, *[change.get(i, a) for i, a in enumerate(args)])
    # tensors without a gradient have no type, and moved ones are seen
    z.zero_many_bind(m.many, [None, None], *args[1:])
    graph.replay()
    torch.cuda.synchronize()
    assert (sumsq.item(), flag.item()) == (0, 0)
    m.d_g = [g.clone() for g in m.d_g]
    m.bind()
    for t in range(2, 5):
        m.new_grads()
        graph.replay()
        torch.cuda.synchronize()
        m.plain_step(t, 1.0, 1.0, 3)
        m.check()


def test_a_graph_of_the_norm_keeps_the_gradients_type_alone():
    g = [torch.ones(1000, device=DEV).bfloat16()]
    many = z.zero_many_create([1000], state_bits=32)
    z.zero_many_bind(many, g)
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        z.zero_many_grad_norm(many, sumsq, flag)
    with pytest.raises(z.ZeroError, match="captured"):
        z.zero_many_bind(many, [g[0].float()])
    state = [[torch.zeros(1000, device=DEV)] for _ in range(3)]
    z.zero_many_bind(many, [2 * g[0]], *state)
    graph.replay()
    torch.cuda.synchronize()
    assert (sumsq.item(), flag.item()) == (4000, 0)


def test_offsets_past_32_bits():
    """The end of a tensor of more than 2^32 elements, moments in 8 bits."""
    n = (1 << 32) + 1300
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(n, device=DEV)
    m8, v8 = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), dtype=torch.uint8, device=DEV) for _ in range(2))
    tail = 1300 + 256
    rng = np.random.default_rng(0)
    g[-tail:] = torch.from_numpy(rng.normal(0, 1e-2, tail).astype(np.float32)).to(DEV).bfloat16()
    host = g[-tail:].float().cpu().numpy()
    many = z.zero_many_create([n], state_bits=8)
    z.zero_many_bind(many, [g], [p], [m8], [v8], [ms], [vs])
    z.zero_many_state_upload(many, 0, z.LossScaler(1.0, dynamic=False), seed=17)
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    z.zero_many_grad_norm(many, sumsq, flag)
    want = math.fsum(host.astype(np.float64) ** 2)
    assert abs(sumsq.item() - want) <= 1e-12 * want
    hp = z.AdamHParams()
    z.zero_many_adam_step(many, hp)
    wp, wm, wv = R.adam(host, np.zeros(tail, np.float32), np.zeros(tail, np.float32),
                        np.zeros(tail, np.float32), R.scalars(hp, 1, 1.0), True)
    wc, wms = R.pack_m(wm)
    wvc, wvs = R.pack_v(wv, n - tail, R.key_of(17, 1))
    assert (n - tail) % 256 == 0
    assert np.array_equal(_bits(p[-tail:]), wp.view(np.int32))
    assert np.array_equal(_bits(m8[-tail:]), wc) and np.array_equal(_bits(v8[-tail:]), wvc)
    assert np.array_equal(_bits(ms[-len(wms):]), wms) and np.array_equal(_bits(vs[-len(wvs):]), wvs)
    assert int(torch.count_nonzero(p[:-tail])) == 0
