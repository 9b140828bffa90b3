"""GPU parity of gq_adamw_step against its definition (include/gq.h).

The reference performs the stated binary32 operations one by one in numpy
(IEEE single precision on the host: add, multiply, divide and square root are
correctly rounded there as well), so weights, states, codes and scales must be
equal bit for bit.  Against the formula in binary64 the weights are off by a few
roundings: 2^-22 (|p| + |update|) in fp32.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F = np.float32
BLOCK = 256


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


def _hash(index, key):
    M = np.uint64(0xFFFFFFFF)
    z = ((index & M) * np.uint64(0x9E3779B9) + (index >> np.uint64(32)) * np.uint64(0x7FEB3529) + np.uint64(key)) & M
    z = ((z ^ (z >> np.uint64(16))) * np.uint64(0x21F0AAAD)) & M
    z = ((z ^ (z >> np.uint64(15))) * np.uint64(0x735A2D97)) & M
    return z ^ (z >> np.uint64(15))


def _blocks(a):
    return np.pad(a, (0, -len(a) % BLOCK)).reshape(-1, BLOCK)


def _f4(q):
    t = q * q
    return t * t


def reference(p, g, m, v, ms, vs, step, seed, tensor, wd, lr, b1, b2, eps, grad_scale=None, first=0):
    """One tensor's step in binary32 (numpy arrays in, new ones out; p fp32, rounded by the caller for bf16);
    `first`: the index of their first element, a multiple of 256."""
    n = len(p)
    if grad_scale is not None:
        g = g * F(grad_scale)
    if ms is not None:
        m = (_blocks(m).astype(F) * ms[:, None]).reshape(-1)[:n]
        v = (_f4(_blocks(v).astype(F)) * vs[:, None]).reshape(-1)[:n]
    m = m * F(b1) + g * F(1 - b1)
    v = v * F(b2) + (g * g) * F(1 - b2)
    d = np.sqrt(v) * F(1 / np.sqrt(1 - b2 ** step)) + F(eps)
    p = p * F(1 - lr * wd) - (m / d) * F(lr / (1 - b1 ** step))
    if ms is None:
        return p, m, v, None, None
    key = (seed + step * 0x632BE5AB + tensor * 0x2C1B3C6D) & 0xFFFFFFFF
    z = _blocks(_hash(np.arange(first, first + n, dtype=np.uint64), key))
    um, uv = (z >> np.uint64(16)).astype(F) * F(2.0 ** -16), (z & np.uint64(0xFFFF)).astype(F) * F(2.0 ** -16)
    mb, vb = _blocks(m), _blocks(v)
    am, av = np.abs(mb).max(1), vb.max(1)
    km, kv = am >= F(2.0 ** -80), av >= F(2.0 ** -80)
    one = F(1)
    im = np.where(km, F(127) / np.where(km, am, one), F(0))[:, None]
    iv = np.where(kv, F(255.0 ** 4) / np.where(kv, av, one), F(0))[:, None]
    qm = np.clip(np.floor(mb * im + um), -127, 127)
    x = vb * iv
    f = _f4(np.arange(256).astype(F))                          # q0 by search in the table, not by roots
    q0 = np.clip(np.searchsorted(f, x, side="right") - 1, 0, 254)
    lo, hi = f[q0], f[q0 + 1]
    qv = q0 + (uv * (hi - lo) < x - lo)
    qv = np.where((x > 0) & (qv == 0), 1, qv)
    return (p, qm.astype(np.int8).reshape(-1)[:n], qv.astype(np.uint8).reshape(-1)[:n],
            np.where(km, am * F(1 / 127), F(0)).astype(F), np.where(kv, av * F(1 / 255.0 ** 4), F(0)).astype(F))


def _bf16(a):
    return torch.from_numpy(a).to(torch.bfloat16)


class Tensors:
    """A list of tensors with states; `odd`: not 16-byte aligned."""

    def __init__(self, sizes, p="f32", g="f32", bits=32, odd=False, seed=0, zero=False):
        rng = np.random.default_rng(seed)
        self.bits, self.sizes = bits, sizes
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}

        def dev(a, dtype):
            t = torch.zeros(len(a) + 1, dtype=dtype, device="cuda")
            t = t[1:] if odd else t[:-1]
            t.copy_(torch.from_numpy(a))
            return t

        mk = lambda f, dtype: [dev(f(n), dtype) for n in sizes]  # noqa: E731
        nb = lambda n: -(-n // BLOCK)  # noqa: E731
        self.p = mk(lambda n: (rng.standard_normal(n) * 0.1).astype(F), dt[p])
        self.g = mk(lambda n: (rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n)) * 1e-3).astype(F), dt[g])
        k = 0 if zero else 1
        if bits == 32:
            self.m = mk(lambda n: k * (rng.standard_normal(n) * 1e-3).astype(F), torch.float32)
            self.v = mk(lambda n: k * (rng.random(n) * 1e-6).astype(F), torch.float32)
            self.scales = None
        else:
            self.m = mk(lambda n: k * rng.integers(-127, 128, n).astype(np.int8), torch.int8)
            self.v = mk(lambda n: k * rng.integers(0, 256, n).astype(np.uint8), torch.uint8)
            self.scales = (mk(lambda n: k * (rng.random(nb(n)) * 1e-5).astype(F), torch.float32) if not odd else
                           [dev(k * (rng.random(nb(n)) * 1e-5).astype(F), torch.float32) for n in sizes],
                           [dev(k * (rng.random(nb(n)) * 1e-15).astype(F), torch.float32) for n in sizes])

    def host(self):
        h = lambda ts: [t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy().copy() for t in ts]  # noqa: E731
        none = [None] * len(self.p)
        ms, vs = (none, none) if self.scales is None else (h(self.scales[0]), h(self.scales[1]))
        return list(zip(h(self.p), h(self.g), h(self.m), h(self.v), ms, vs))

    def step(self, gq, **kw):
        gq.adamw_step(self.p, self.g, self.m, self.v, scales=self.scales, **kw)


HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


def _expect(T, before, step, seed=0, wd=0.01, hyper=HYPER, grad_scale=None):
    wds = wd if isinstance(wd, list) else [wd] * len(T.p)
    for i, (b, w) in enumerate(zip(before, wds)):
        with np.errstate(all="ignore"):
            p, m, v, ms, vs = reference(*b, step, seed, i, w, hyper["lr"], *hyper["betas"], hyper["eps"], grad_scale)
        want = torch.from_numpy(p).to(T.p[i].dtype)
        assert torch.equal(T.p[i].cpu(), want), (i, "p", int((T.p[i].cpu() != want).sum()))
        for name, got, ref in (("m", T.m[i], m), ("v", T.v[i], v)) + (
                () if ms is None else (("ms", T.scales[0][i], ms), ("vs", T.scales[1][i], vs))):
            got = got.cpu().numpy()
            assert np.array_equal(got, ref), (i, name, int((got != ref).sum()), len(ref))


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_step_is_bit_exact(gq, p, g, bits, odd):
    T = Tensors([1, 7, 8, 255, 256, 257, 2048, 2049, 70001], p, g, bits, odd)
    before = T.host()
    T.step(gq, step=5, seed=77, weight_decay=0.01, **HYPER)
    _expect(T, before, 5, 77)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_nothing_and_on(gq, bits):
    """First step from zero states, then three more, each against the reference on the states at hand."""
    T = Tensors([3000, 100], bits=bits, zero=True)
    for step in (1, 2, 3, 4):
        before = T.host()
        T.step(gq, step=step, seed=3, weight_decay=[0.1, 0.0], **HYPER)
        _expect(T, before, step, 3, [0.1, 0.0])


def test_many_tensors_and_empty_ones(gq):
    """More tensors than one launch takes, empty ones among them, one decay each."""
    sizes = [(37 * i) % 700 for i in range(450)]
    T = Tensors(sizes, bits=8)
    wd = [0.001 * (i % 3) for i in range(450)]
    before = T.host()
    T.step(gq, step=9, seed=1 << 31, weight_decay=wd, **HYPER)
    _expect(T, before, 9, 1 << 31, wd)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_and_tiny_gradients(gq, bits):
    """Blocks of zeros store zero states and move nothing but by decay; tiny and huge values stay in the definition."""
    T = Tensors([256 * 6], bits=bits, zero=True)
    g = T.g[0].view(6, 256)
    g[0] = 0
    g[1] = 1e-30
    g[2] *= 1e18
    g[3, 1:] = 0
    g[4] = 1e-42                                               # subnormal
    before = T.host()
    T.step(gq, step=1, weight_decay=0.0, **HYPER)
    _expect(T, before, 1, 0, 0.0)
    assert torch.equal(T.p[0][:256].cpu(), torch.from_numpy(before[0][0][:256]))


def test_against_the_formula(gq):
    T = Tensors([5000])
    (p, g, m, v, _, _), = T.host()
    T.step(gq, step=12, weight_decay=0.1, **HYPER)
    p, g, m, v = (a.astype(np.float64) for a in (p, g, m, v))
    m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
    u = 3e-3 * (m / (1 - 0.9 ** 12)) / (np.sqrt(v / (1 - 0.95 ** 12)) + 1e-8)
    want = p * (1 - 3e-4) - u
    # roundings: two of p, about eight of u (with its sums' cancellation in m at most |0.9 m| + |0.1 g|)
    big = 3e-3 * ((np.abs(0.9 * T_m(m, g)) + np.abs(0.1 * g)) / (1 - 0.9 ** 12)) / (np.sqrt(v / (1 - 0.95 ** 12)) + 1e-8)
    assert (np.abs(T.p[0].cpu().numpy() - want) <= 2.0 ** -23 * np.abs(p) + 10 * 2.0 ** -24 * (big + np.abs(u))).all()


def T_m(m, g):
    """The old first moment from the new one."""
    return (m - 0.1 * g) / 0.9


def test_copies_grad_scale_and_no_state_change_elsewhere(gq):
    T = Tensors([600, 300], bits=8)
    copies = [torch.zeros(600, dtype=torch.bfloat16, device="cuda"), None]
    scale = torch.tensor([0.25], device="cuda")
    before = T.host()
    T.step(gq, step=2, copies=copies, grad_scale=scale, weight_decay=0.01, **HYPER)
    _expect(T, before, 2, grad_scale=0.25)
    assert torch.equal(copies[0], T.p[0].to(torch.bfloat16))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_follows_device_step_and_lr(gq, bits):
    """One captured step, replayed with the step and the rate moving on in device memory, is the eager sequence."""
    T, U = Tensors([5000, 77], bits=bits), Tensors([5000, 77], bits=bits)
    step, lr = torch.ones((), dtype=torch.int64, device="cuda"), torch.full((), 1e-3, device="cuda")
    keep = [t.clone() for t in T.p + T.m + T.v + (T.scales[0] + T.scales[1] if bits == 8 else [])]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.step(gq, step=step, lr=lr, betas=(0.9, 0.95), seed=5)
        step += 1
        lr *= 0.5
    for t, k in zip(T.p + T.m + T.v + (T.scales[0] + T.scales[1] if bits == 8 else []), keep):
        assert torch.equal(t, k)                               # a capture runs nothing
    rate = torch.full((), 1e-3)
    for k in range(1, 5):
        g.replay()
        U.step(gq, step=k, lr=float(rate), betas=(0.9, 0.95), seed=5)
        rate *= 0.5
    torch.cuda.synchronize()
    for a, b in zip(T.p + T.m + T.v, U.p + U.m + U.v):
        assert torch.equal(a, b)


def test_rounding_of_states_is_unbiased(gq):
    """What the codes stand for has the states' mean: 4096 blocks of one value beside the block's maximum.

    The mean of N = 4096 independent roundings is off by at most 5 step / (2 sqrt N) with probability above 0.9999."""
    n = 4096 * BLOCK
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g.view(-1, BLOCK)[:, 0] = 1.0                              # the block's maximum
    g.view(-1, BLOCK)[:, 5] = 0.0703
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = ([torch.zeros(n // BLOCK, device="cuda")], [torch.zeros(n // BLOCK, device="cuda")])
    gq.adamw_step([p], [g], [m], [v], step=1, lr=0.0, betas=(0.9, 0.95), scales=sc, seed=123)
    got_m = (m.view(-1, BLOCK)[:, 5].double() * sc[0][0].double()).mean().item()
    codes = v.view(-1, BLOCK)[:, 5].double()
    got_v = (codes ** 4 * sc[1][0].double()).mean().item()
    m_true, v_true = 0.1 * 0.0703, 0.05 * 0.0703 ** 2
    k = int(codes.min().item())
    step_m, step_v = 0.1 / 127, ((k + 1) ** 4 - k ** 4) * 0.05 / 255 ** 4
    assert codes.max().item() == k + 1
    assert abs(got_m - m_true) <= 5 * step_m / (2 * 64) + 1e-6 * m_true
    assert abs(got_v - v_true) <= 5 * step_v / (2 * 64) + 1e-6 * v_true


def test_more_elements_than_32_bits_count(gq):
    """2^32 + 700 elements: the last blocks, whose index needs the hash's high word, against the reference."""
    n, tail = (1 << 32) + 700, 700 + 512
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    sc = [torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(4)
    g[-tail:] = torch.from_numpy(rng.standard_normal(tail).astype(F)).cuda()
    gq.adamw_step([p], [g], [m], [v], step=1, scales=([sc[0]], [sc[1]]), seed=9, weight_decay=0.0, **HYPER)
    zero = np.zeros(-(-tail // BLOCK), F)
    w, qm, qv, ms, vs = reference(np.zeros(tail, F), g[-tail:].float().cpu().numpy(), np.zeros(tail, np.int8),
                                  np.zeros(tail, np.uint8), zero, zero, 1, 9, 0, 0.0, HYPER["lr"], 0.9, 0.95, 1e-8,
                                  first=n - tail)
    assert torch.equal(p[-tail:].cpu(), _bf16(w))
    assert np.array_equal(m[-tail:].cpu().numpy(), qm) and np.array_equal(v[-tail:].cpu().numpy(), qv)
    assert np.array_equal(sc[0][-len(ms):].cpu().numpy(), ms) and np.array_equal(sc[1][-len(vs):].cpu().numpy(), vs)
    assert not m[:1 << 20].any() and not sc[0][:1000].any()


def test_mixed_state_sizes_in_one_call(gq):
    """The C entry takes 8-bit and 32-bit states in one batch; a tensor's place in it keeps its random bits."""
    A, B = Tensors([300, 5000], bits=8, seed=1), Tensors([700], bits=32, seed=2)
    before = A.host()[:1] + B.host() + A.host()[1:]
    order = [(A, 0), (B, 0), (A, 1)]
    arr = (gq.GQAdamWTensor * 3)()
    for d, (T, i) in zip(arr, order):
        d.p, d.g, d.m, d.v, d.numel = (T.p[i].data_ptr(), T.g[i].data_ptr(), T.m[i].data_ptr(), T.v[i].data_ptr(),
                                       T.p[i].numel())
        d.state_bits, d.weight_decay = T.bits, 0.01
        if T.bits == 8:
            d.m_scale, d.v_scale = T.scales[0][i].data_ptr(), T.scales[1][i].data_ptr()
    h = gq.GQAdamWHyper(lr=HYPER["lr"], beta1=0.9, beta2=0.95, eps=1e-8, step=7, seed=11)
    assert gq.LIB.gq_adamw_step(arr, 3, h, torch.cuda.current_stream().cuda_stream) == 0
    for k, ((T, i), b) in enumerate(zip(order, before)):
        p, m, v, ms, vs = reference(*b, 7, 11, k, 0.01, HYPER["lr"], 0.9, 0.95, 1e-8)
        assert np.array_equal(T.p[i].cpu().numpy(), p) and np.array_equal(T.m[i].cpu().numpy(), m)
        assert np.array_equal(T.v[i].cpu().numpy(), v)


def test_refusals(gq):
    T = Tensors([10], bits=8)
    with pytest.raises(TypeError):
        gq.adamw_step(T.p, T.g, T.m, T.v, step=1, lr=1e-3)
    with pytest.raises(ValueError):
        gq.adamw_step(T.p, T.g, T.m, T.v[:0], step=1, lr=1e-3, scales=T.scales)
    with pytest.raises(ValueError):
        gq.adamw_step(T.p, [T.g[0][:5]], T.m, T.v, step=1, lr=1e-3, scales=T.scales)
    with pytest.raises(ValueError):
        gq.adamw_step(T.p, T.g, T.m, T.v, step=1, lr=1e-3, scales=([T.scales[0][0][:0]], T.scales[1]))
    with pytest.raises(ValueError):
        gq.adamw_step(T.p, [T.g[0].cpu()], T.m, T.v, step=1, lr=1e-3, scales=T.scales)
    for bad in (dict(step=0, lr=1e-3), dict(step=1, lr=float("nan")), dict(step=1, lr=1e-3, betas=(1.0, 0.9)),
                dict(step=1, lr=1e-3, eps=-1.0)):
        with pytest.raises(gq.GQError):
            T.step(gq, **bad)
    gq.adamw_step([], [], [], [], step=1, lr=1e-3)
