"""gq_adamw_step with 8-bit states whose first moment is held in square codes (GQ_ADAMW_8_SQUARE, codes="square"): bit for
bit against the definition in include/gq.h, and both kinds of codes over many steps against 32-bit states.

The reference is that of test_gpu_adamw.py for everything but the first moment's codes, which it performs one binary32
operation at a time in numpy, with the square root found by search.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_adamw import BLOCK, HYPER, Tensors, _blocks, _hash, reference

F = np.float32
SQUARES = np.arange(128, dtype=F) ** 2


def reference_square(p, g, m, v, ms, vs, step, seed, tensor, wd, lr, b1, b2, eps, grad_scale=None):
    """One tensor's step, m in square codes: the weights, v and the scales' blocks as in `reference`."""
    n = len(p)
    g2 = g if grad_scale is None else g * F(grad_scale)
    q = _blocks(m).astype(F)
    m32 = ((q * np.abs(q)) * ms[:, None]).reshape(-1)[:n]
    # `reference` on a first moment given as it is (one code of value 1, each element's own scale), to share the rest
    p, _, qv, _, nvs = reference_of(p, g2, m32, v, vs, step, seed, tensor, wd, lr, b1, b2, eps)
    m32 = m32 * F(b1) + g2 * F(1 - b1)
    key = (seed + step * 0x632BE5AB + tensor * 0x2C1B3C6D) & 0xFFFFFFFF
    um = _blocks((_hash(np.arange(n, dtype=np.uint64), key) >> np.uint64(16)).astype(F) * F(2.0 ** -16))
    mb = _blocks(m32)
    am = np.abs(mb).max(1)
    keep = am >= F(2.0 ** -80)
    im = np.where(keep, F(16129) / np.where(keep, am, F(1)), F(0))[:, None]
    x = np.abs(mb) * im
    q0 = np.clip(np.searchsorted(SQUARES, x, side="right") - 1, 0, 126)
    lo = SQUARES[q0]
    q = q0 + (um * (SQUARES[q0 + 1] - lo) < x - lo)
    q = np.where(mb < 0, -q, q)
    return p, q.astype(np.int8).reshape(-1)[:n], qv, np.where(keep, am * F(1 / 127 ** 2), F(0)).astype(F), nvs


def reference_of(p, g, m32, v, vs, step, seed, tensor, wd, lr, b1, b2, eps):
    """`reference` with the first moment in binary32 and the second in codes."""
    n = len(p)
    v32 = ((_blocks(v).astype(F) ** 2) ** 2 * vs[:, None]).reshape(-1)[:n]
    w, _, _, _, _ = reference(p, g, m32, v32, None, None, step, seed, tensor, wd, lr, b1, b2, eps)
    zero = np.zeros(len(vs), F)
    _, _, qv, _, nvs = reference(p, g, np.zeros(n, np.int8), v, zero, vs, step, seed, tensor, wd, lr, b1, b2, eps)
    return w, None, qv, None, nvs


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


def _same(T, i, p, m, v, ms, vs, what):
    for name, got, want in (("p", T.p[i], torch.from_numpy(p).to(T.p[i].dtype)), ("m", T.m[i], torch.from_numpy(m)),
                            ("v", T.v[i], torch.from_numpy(v)), ("ms", T.scales[0][i], torch.from_numpy(ms)),
                            ("vs", T.scales[1][i], torch.from_numpy(vs))):
        assert torch.equal(got.cpu(), want), (what, i, name, int((got.cpu() != want).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("p,g", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_square_codes_are_bit_exact(gq, p, g, odd):
    T = Tensors([1, 7, 8, 255, 256, 257, 2048, 2049, 70001], p, g, 8, odd)
    before = T.host()
    scale = torch.tensor([0.5], device="cuda")
    T.step(gq, step=5, seed=77, weight_decay=0.01, codes="square", grad_scale=scale, **HYPER)
    for i, b in enumerate(before):
        with np.errstate(all="ignore"):
            _same(T, i, *reference_square(*b, 5, 77, i, 0.01, HYPER["lr"], 0.9, 0.95, 1e-8, 0.5), (p, g, odd))


@pytest.mark.gpu
def test_square_codes_from_nothing_and_at_the_ends(gq):
    """From zero states; blocks of zeros, of one value, of tiny and huge values, of one value beside zeros."""
    T = Tensors([256 * 7 + 5], bits=8, zero=True)
    g = T.g[0][:256 * 7].view(7, 256)
    g[0], g[1], g[5] = 0, 1e-30, -0.25
    g[2] *= 1e18
    g[3, 1:] = 0
    g[4] = 1e-42
    for step in (1, 2, 3):
        before = T.host()
        T.step(gq, step=step, seed=3, weight_decay=0.1, codes="square", **HYPER)
        with np.errstate(all="ignore"):
            _same(T, 0, *reference_square(*before[0], step, 3, 0, 0.1, HYPER["lr"], 0.9, 0.95, 1e-8), step)
    assert (T.m[0][256 * 5:256 * 6].cpu() == -127).all() and not T.m[0][:256].any()


@pytest.mark.gpu
def test_all_kinds_of_states_in_one_batch(gq):
    """The C entry takes the three kinds side by side, in any order, more of them than one launch takes."""
    sizes = [(91 * i) % 600 for i in range(230)]
    kinds = [Tensors(sizes, bits=b, seed=s) for s, b in enumerate((8, 32, 8))]
    before = [T.host() for T in kinds]
    arr = (gq.GQAdamWTensor * (3 * len(sizes)))()
    for j, d in enumerate(arr):
        k, i = j % 3, j // 3
        T = kinds[k]
        d.p, d.g, d.m, d.v, d.numel = (T.p[i].data_ptr(), T.g[i].data_ptr(), T.m[i].data_ptr(), T.v[i].data_ptr(), sizes[i])
        d.state_bits, d.weight_decay = (8, 32, gq.ADAMW_CODES["square"])[k], 0.01
        if k != 1:
            d.m_scale, d.v_scale = T.scales[0][i].data_ptr(), T.scales[1][i].data_ptr()
    h = gq.GQAdamWHyper(lr=HYPER["lr"], beta1=0.9, beta2=0.95, eps=1e-8, step=7, seed=11)
    assert gq.LIB.gq_adamw_step(arr, len(arr), h, torch.cuda.current_stream().cuda_stream) == 0
    for j in range(len(arr)):
        k, i = j % 3, j // 3
        T, args = kinds[k], (7, 11, j, 0.01, HYPER["lr"], 0.9, 0.95, 1e-8)
        if k == 1:
            p, m, v, _, _ = reference(*before[k][i], *args)
            assert np.array_equal(T.p[i].cpu().numpy(), p) and np.array_equal(T.m[i].cpu().numpy(), m)
            assert np.array_equal(T.v[i].cpu().numpy(), v)
        else:
            _same(T, i, *(reference_square if k else reference)(*before[k][i], *args), j)


@pytest.mark.gpu
def test_square_codes_have_the_mean_of_what_they_stand_for(gq):
    """4096 blocks of one value beside the block's maximum: the mean of N = 4096 independent roundings within a step of w
    is off by at most 5 w / (2 sqrt N) with probability above 0.9999, and by 2^-16 w for the random numbers' 16 bits."""
    n = 4096 * BLOCK
    for value in (0.0703, -0.0003, 1e-5):
        p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        g.view(-1, BLOCK)[:, 0], g.view(-1, BLOCK)[:, 5] = 1.0, value
        m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
        sc = ([torch.zeros(n // BLOCK, device="cuda")], [torch.zeros(n // BLOCK, device="cuda")])
        gq.adamw_step([p], [g], [m], [v], step=1, lr=0.0, betas=(0.9, 0.95), scales=sc, seed=123, codes="square")
        q = m.view(-1, BLOCK)[:, 5].double()
        assert q.abs().max() - q.abs().min() == 1 and (q * value >= 0).all()
        got = (q * q.abs() * sc[0][0].double()).mean().item()
        w = (2 * q.abs().min().item() + 1) * 0.1 / 127 ** 2
        assert abs(got - 0.1 * value) <= w * (5 / (2 * 64) + 2.0 ** -16) + 1e-6 * abs(0.1 * value)


# The largest |update| / lr and its root mean square over 200 steps, b = (0.9, 0.95), 16 blocks, no decay: 32-bit states,
# linear codes, square codes.  Computed with the references on the host, of which the kernel is a copy bit for bit: what
# the tests below allow is the figures' own rounding to three digits.
FIGURES = {0.0: ((1.00, 0.255), (1.25, 0.255), (1.02, 0.255)), 1.0: ((1.00, 0.255), (4.54, 0.270), (1.23, 0.257)),
           2.0: ((1.00, 0.255), (279, 1.995), (26.6, 0.341)), "outlier": ((1.00, 0.255), (32.3, 1.141), (2.69, 0.293))}


def _gradients(kind, n):
    """200 steps' gradients: N(0, 1) times a scale of each element's own, exp(kind * N(0, 1)) or one in a block 1000
    times the rest."""
    rng = np.random.default_rng(0)
    if kind == "outlier":
        s = np.ones(n)
        s[::BLOCK] = 1000
    else:
        s = np.exp(kind * rng.standard_normal(n))
    for _ in range(200):
        yield (s * 1e-3 * rng.standard_normal(n)).astype(F)


def _figures(kind, step, n=16 * BLOCK):
    """`step`(gradient, number) -> the weights after it, from 0."""
    old, largest, squares = np.zeros(n, F), 0.0, 0.0
    for t, g in enumerate(_gradients(kind, n), 1):
        p = step(g, t)
        u = (p - old).astype(np.float64) / 1e-3
        old, largest, squares = p, max(largest, np.abs(u).max()), squares + (u * u).mean()
    return largest, (squares / 200) ** 0.5


def _agree(got, want):
    assert all(abs(a - b) <= 0.005 * max(b, 1) for a, b in zip(got, want)), (got, want)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("kind", list(FIGURES))
def test_many_steps_by_the_definition(kind, which):
    """What the definition itself does to the updates (no GPU): square codes keep them near those of 32-bit states."""
    n = 16 * BLOCK
    state = [np.zeros(n, F)] + ([np.zeros(n, F), np.zeros(n, F), None, None] if which == 0 else
                                [np.zeros(n, np.int8), np.zeros(n, np.uint8), np.zeros(16, F), np.zeros(16, F)])

    def step(g, t):
        state[:] = (reference_square if which == 2 else reference)(state[0], g, *state[1:], t, 1, 0, 0.0, 1e-3, 0.9, 0.95,
                                                                   1e-8)
        return state[0]

    _agree(_figures(kind, step), FIGURES[kind][which])


@pytest.mark.gpu
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("kind", list(FIGURES))
def test_many_steps(gq, kind, which):
    n = 16 * BLOCK
    z = lambda dt, k=n: [torch.zeros(k, dtype=dt, device="cuda")]  # noqa: E731
    p, m, v = z(torch.float32), z(torch.int8 if which else torch.float32), z(torch.uint8 if which else torch.float32)
    scales = (z(torch.float32, 16), z(torch.float32, 16)) if which else None

    def step(g, t):
        gq.adamw_step(p, [torch.from_numpy(g).cuda()], m, v, step=t, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0,
                      scales=scales, seed=1, codes=("linear", "linear", "square")[which])
        return p[0].cpu().numpy().copy()

    _agree(_figures(kind, step), FIGURES[kind][which])


@pytest.mark.gpu
def test_refusals(gq):
    T, U = Tensors([10], bits=8), Tensors([10], bits=32)
    for bad in (dict(codes="cubic"), dict(codes=None)):
        with pytest.raises(ValueError):
            T.step(gq, step=1, lr=1e-3, **bad)
    with pytest.raises(ValueError):                            # codes of 32-bit states
        U.step(gq, step=1, lr=1e-3, codes="square")
