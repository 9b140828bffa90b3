"""GPU parity of gq_tile_weight, gq_gemm_epilogue and gq_gemm_grouped.

The reference is the definition in binary64: W = q * s exactly (the codes come
from the oracle's own unpacking of random packed rows), Z = X W^T + b, the
activation, the residual.  X is bf16, so the products are exact in binary32.

Tolerances, element by element, before the last rounding:
  |Z - exact| <= A := (K/8 + 32) * 2^-24 * sum_k |x w| + 2^-23 * (|z| + |b|)
(binary32 sums in the tensor cores' order, truncation allowed; one rounding
each for the scale and the bias).  An activation multiplies an error by its
slope, at most S on the values in question (1 for none and relu, 2 |z| + A for
the squares, 1.13 for silu and the two gelus), and its own binary32 steps err
by at most 16 * 2^-24 of max(|z|, 1): a factor of at most 1 from the special
function unit's exponential (2^-22 relative) and reciprocal (2^-23), the exponent's
own rounding through z^2 s (1 - s) < 2, the normal distribution's approximation
(1e-7, 2 * 2^-24), and a handful of roundings.  The residual adds one rounding 2^-24 |y|.  Y in bf16 adds half
a step, 2^-8 |y| (2^-9 of the next power of two).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import synth

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "relu2", "leaky_relu2", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


def _act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "relu2":
        return z.clamp(min=0) ** 2
    if act == "leaky_relu2":
        return torch.where(z > 0, z, z / 2) ** 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z


class Weight:
    """Random packed codes and scales of E experts, as an export holds them, and W in binary64."""

    def __init__(self, gq, rng, E, N, K, qbits):
        prb = gq.gq_packed_row_bytes(K, qbits)
        top = 31 if qbits == 6 else 127
        q = rng.integers(-top, top + 1, (E, N, K)).astype(np.int8)
        q[..., -1] = rng.choice([-top, top], (E, N))          # the extreme codes at the ragged end
        self.packed = torch.from_numpy(pack(q, qbits).reshape(E, N, prb)).cuda()
        s = (rng.uniform(0.5, 1.5, (E, N)) * 4 / top / np.sqrt(K)).astype(np.float16)
        self.scale = torch.from_numpy(s).cuda()
        self.w = torch.from_numpy(q).cuda().double() * self.scale.double()[..., None]


def pack(q, qbits):
    """The export's packed rows of codes [.., K]: int8 as they are, int6 four in three bytes."""
    if qbits == 8:
        return q.view(np.uint8)
    K = q.shape[-1]
    u = np.zeros(q.shape[:-1] + (-(-K // 4) * 4,), np.uint32)
    u[..., :K] = q.astype(np.int32) & 63
    u = u.reshape(*q.shape[:-1], -1, 4)
    v = u[..., 0] | u[..., 1] << 6 | u[..., 2] << 12 | u[..., 3] << 18
    return np.stack((v & 255, v >> 8 & 255, v >> 16), -1).astype(np.uint8).reshape(*q.shape[:-1], -1)


def _x(rng, M, K, ldx=None):
    """bf16 [M, K] in rows of ldx elements (a multiple of 8); NaN behind each row's K elements."""
    ldx = ldx or -(-K // 8) * 8
    x = np.full((M, ldx), np.nan, np.float32)
    x[:, :K] = rng.standard_normal((M, K))
    return torch.from_numpy(x).cuda().to(torch.bfloat16)[:, :K]


def _check(y, x, w, bias, residual, act, what):
    K = x.shape[1]
    x64 = x.double()
    z = x64 @ w.t()
    b = torch.zeros((), dtype=torch.float64, device="cuda") if bias is None else bias.double()
    z = z + b
    err = (K / 8 + 32) * 2.0 ** -24 * (x64.abs() @ w.abs().t()) + 2.0 ** -23 * (z.abs() + b.abs())
    slope = {"none": 1, "relu": 1, "relu2": 2 * z.abs() + err, "leaky_relu2": 2 * z.abs() + err}.get(act, 1.13)
    out = _act64(z, act)
    err = err * slope + 16 * 2.0 ** -24 * z.abs().clamp(min=1)
    if act in ("relu2", "leaky_relu2"):
        err = err + 2.0 ** -24 * out
    if residual is not None:
        out = out + residual.double()
        err = err + 2.0 ** -24 * out.abs()
    if y.dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (out.abs() + err)
    bad = (y.double() - out).abs() > err
    assert not bad.any() and torch.isfinite(y).all(), (
        what, int(bad.sum()), bad.nonzero()[:3].tolist(), float(((y.double() - out).abs() / err).max()))


def _extra(rng, kind, *shape):
    if kind == "none":
        return None
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    return t if kind == "f32" else t.to(torch.bfloat16)


def _run(gq, M, N, K, qbits, act="none", bias="none", residual="none", out=torch.bfloat16, seed=0):
    rng = np.random.default_rng(seed + M + 3 * N + 7 * K)
    W = Weight(gq, rng, 1, N, K, qbits)
    tiles = gq.tile_weight(W.packed[0], K, qbits)
    x, b, r = _x(rng, M, K), _extra(rng, bias, N), _extra(rng, residual, M, N)
    pad = torch.full((M + 1, N + 5), 7.0, dtype=out, device="cuda")
    y = gq.gemm_epilogue(x, tiles, W.scale[0], qbits, bias=b, act=act, residual=r, y=pad[:M, :N], check_status=True)
    assert (pad[:, N:] == 7).all() and (pad[M] == 7).all()
    _check(y, x, W.w[0], b, r, act, (M, N, K, qbits, act, bias, residual, out))


# ------------------------------------------------------------------- tiles --

@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 64), (3, 130, 70), (2, 5, 513), (1, 300, 1584)])
def test_tiles_hold_the_codes(gq, E, N, K, qbits):
    """Every code where the layout says, read bit by bit; code 0 in the padding."""
    rng = np.random.default_rng(N + K)
    top = 31 if qbits == 6 else 127
    q = rng.integers(-top, top + 1, (E, N, K)).astype(np.int8)
    tiles = gq.tile_weight(torch.from_numpy(pack(q, qbits)).cuda(), K, qbits).cpu().numpy()
    rts, kbs, chunks = -(-N // 128), -(-K // 64), 3 if qbits == 6 else 4
    t = tiles.reshape(E, rts, kbs, chunks, 128, 16).transpose(0, 1, 4, 2, 3, 5).reshape(E, rts * 128, kbs, chunks * 16)
    full = np.zeros((E, rts * 128, kbs * 64), np.int64)
    full[:, :N, :K] = q
    full = full.reshape(E, rts * 128, kbs, 64)
    for k in range(64):
        if qbits == 8:
            got = t[..., k // 4 * 4 + (0, 2, 1, 3)[k % 4]].view(np.int8).astype(np.int64)
        else:
            g, j, half = k // 16, k % 16 // 2, k % 2
            got = np.full(full.shape[:-1], -32, np.int64)
            for bit in range(6):
                if j < 6:
                    word, at = j % 3, bit + (0 if j < 3 else 6)
                elif bit < 4:
                    word, at = j - 6, 12 + bit
                else:
                    word, at = 2, 12 + 2 * (j - 6) + bit - 4
                place = (3 * g + word) * 32 + 16 * half + at
                got += ((t[..., place // 8] >> (place % 8)) & 1).astype(np.int64) << bit
        assert np.array_equal(got, full[..., k]), k


def test_export_to_tiles_to_layer(gq):
    """The path a user takes: export a weight, lay it out, run the layer; W is gq.dequant's fp32 w_hat."""
    rng = np.random.default_rng(5)
    w = torch.from_numpy(synth.random_matrix(rng, 200, 333, "t3")).cuda()
    x = _x(rng, 9, 333)
    for qbits in (6, 8):
        (o,) = gq.export_pack([gq.Request(w, qbits, 0.999)])
        y = gq.gemm_epilogue(x, gq.tile_weight(o.packed, 333, qbits), o.scale_f16, qbits, out_dtype=torch.float32)
        _check(y, x, gq.dequant(o.packed, o.scale_f16, qbits, 200, 333).double(), None, None, "none", qbits)


# ---------------------------------------------------------------- products --

@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 64), (1, 1536, 512), (1, 100, 8192), (2, 130, 65), (16, 256, 128), (17, 300, 1000),
    (31, 384, 4096), (33, 528, 1584), (64, 1000, 192), (65, 129, 2048), (127, 1584, 528), (128, 512, 1024),
    (129, 256, 64), (200, 2048, 320), (257, 1000, 777), (1000, 1792, 512), (2049, 300, 136), (513, 4100, 264),
])
def test_product(gq, M, N, K, qbits):
    _run(gq, M, N, K, qbits, out=torch.float32)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,bias,residual,out", [
    (3, "f32", "bf16", torch.bfloat16), (40, "bf16", "f32", torch.float32), (300, "none", "bf16", torch.bfloat16),
    (600, "f32", "none", torch.bfloat16),
])
def test_epilogue(gq, M, act, bias, residual, out):
    _run(gq, M, 272, 384, 6, act, bias, residual, out)


# Many rows and enough columns that the tiles go over pairs of SMs: odd and ragged sizes, odd counts of column blocks,
# more units than pairs.
@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("M,N,K,act,bias,residual,out", [
    (500, 5700, 1544, "none", "none", "none", torch.float32), (257, 8191, 1601, "silu", "bf16", "bf16", torch.bfloat16),
    (1100, 8192, 1536, "gelu", "f32", "f32", torch.bfloat16), (300, 8200, 2048, "gelu_tanh", "f32", "bf16", torch.float32),
    (97, 12000, 1600, "relu2", "none", "f32", torch.float32), (2500, 2050, 1664, "leaky_relu2", "bf16", "bf16", torch.bfloat16),
    (101, 12000, 2072, "relu", "f32", "f32", torch.bfloat16),
])
def test_many_rows(gq, M, N, K, qbits, act, bias, residual, out):
    _run(gq, M, N, K, qbits, act, bias, residual, out)


@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("M,N,K", [
    (2050, 4100, 8), (2300, 4096, 64), (2048, 4100, 72), (3000, 3000, 200), (2050, 4000, 320), (4100, 2050, 528),
])
def test_many_rows_of_few_columns(gq, M, N, K, qbits):
    """Over pairs of SMs with fewer stages to a unit than there are slots for them: a unit's sums are drained while the
    next units' stages are under way."""
    _run(gq, M, N, K, qbits, "silu", "f32", "bf16")


@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("K", [40, 136, 264])
def test_grouped_many_rows_of_few_columns(gq, K, qbits):
    _grouped(gq, [70, 0, 300, 5, 64, 200, 31, 90, 128, 1, 255, 40, 77, 33, 96, 120], 2500, K, qbits, "gelu_tanh", "f32",
             "f32", torch.bfloat16, first=1, behind=20)


def test_more_rows_than_one_wave(gq):
    """Enough tiles that every block takes several."""
    _run(gq, 3000, 4096, 128, 6, "silu", "bf16", "bf16")


def test_no_columns_and_no_rows(gq):
    """K = 0: Y = act(bias) + residual; M = 0 and N = 0: nothing."""
    b = torch.tensor([1.0, -2.0, 3.0], device="cuda")
    r = torch.ones(2, 3, device="cuda")
    x = torch.empty((2, 0), dtype=torch.bfloat16, device="cuda")
    y = gq.gemm_epilogue(x, torch.empty(0, dtype=torch.uint8, device="cuda"),
                         torch.ones(3, dtype=torch.float16, device="cuda"), 6, bias=b, act="relu2", residual=r,
                         out_dtype=torch.float32)
    assert y.tolist() == [[2.0, 1.0, 10.0]] * 2
    W = Weight(gq, np.random.default_rng(1), 1, 40, 64, 6)
    t = gq.tile_weight(W.packed[0], 64, 6)
    assert gq.gemm_epilogue(x.new_empty((0, 64)), t, W.scale[0], 6).shape == (0, 40)


def test_residual_in_place(gq):
    rng = np.random.default_rng(8)
    for M in (5, 140):
        W = Weight(gq, rng, 1, 200, 256, 8)
        x = _x(rng, M, 256)
        y = _extra(rng, "bf16", M, 200)
        r = y.clone()
        t = gq.tile_weight(W.packed[0], 256, 8)
        out = gq.gemm_epilogue(x, t, W.scale[0], 8, act="silu", residual=y, y=y)
        assert out.data_ptr() == y.data_ptr()
        _check(y, x, W.w[0], None, r, "silu", M)


def test_special_values_propagate(gq):
    """NaN and infinities in a row of X reach that row's outputs and no other's."""
    rng = np.random.default_rng(9)
    for M, N, K in ((4, 300, 200), (70, 300, 200), (300, 300, 200), (300, 5700, 1540)):
        W = Weight(gq, rng, 1, N, K, 6)
        t = gq.tile_weight(W.packed[0], K, 6)
        x = _x(rng, M, K)
        clean = gq.gemm_epilogue(x, t, W.scale[0], 6, act="relu")
        x2 = _x(rng, M, K).copy_(x)                            # (a clone's rows would not start on 16 bytes)
        x2[1, 7], x2[2, 5] = float("nan"), float("inf")
        y = gq.gemm_epilogue(x2, t, W.scale[0], 6, act="relu")
        q0 = W.w[0][:, 5] == 0
        assert y[1].isnan().all()
        assert torch.equal(y[2].isnan(), q0) and (y[2][W.w[0][:, 5] > 0] == float("inf")).all()
        keep = torch.ones(M, dtype=torch.bool)
        keep[1] = keep[2] = False
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("act,at", [("silu", -np.inf), ("gelu", np.inf), ("gelu_tanh", np.inf), ("relu", np.inf),
                                    ("silu", 1e30), ("gelu", -1e30), ("gelu_tanh", -1e30), ("gelu", 40.0),
                                    ("silu", -80.0), ("gelu_tanh", -30.0), ("relu2", -np.inf), ("leaky_relu2", -np.inf)])
def test_activations_far_out(gq, act, at):
    """Where the exponential over- or underflows: the formula's value."""
    W = Weight(gq, np.random.default_rng(3), 1, 40, 64, 8)
    x = torch.zeros((5, 64), dtype=torch.bfloat16, device="cuda")
    b = torch.full((40,), at, device="cuda")
    y = gq.gemm_epilogue(x, gq.tile_weight(W.packed[0], 64, 8), W.scale[0], 8, bias=b, act=act, out_dtype=torch.float32)
    z = torch.tensor(at, dtype=torch.float64)
    if act == "silu":
        want = z / (1 + torch.exp(-z))
    elif act == "gelu":
        want = 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    elif act == "gelu_tanh":
        want = 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    else:
        want = _act64(z, act)
    want = float(want)
    if np.isnan(want):
        assert y.isnan().all()
    elif np.isinf(want):
        assert (y == want).all()
    else:
        assert (y.double() - want).abs().max() <= 16 * 2.0 ** -24 * max(abs(want), 1.0)


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (24, 700, 2048), (300, 512, 640), (300, 8192, 1600)])
def test_same_bits_every_time(gq, M, N, K):
    """No atomics: the same call gives the same bits, eager, on another stream and replayed from a graph."""
    rng = np.random.default_rng(10)
    W = Weight(gq, rng, 1, N, K, 6)
    t, x = gq.tile_weight(W.packed[0], K, 6), _x(rng, M, K)
    call = lambda y=None: gq.gemm_epilogue(x, t, W.scale[0], 6, act="gelu", y=y, out_dtype=torch.float32)  # noqa: E731
    want = call()
    for _ in range(20):
        assert torch.equal(call(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two = [call() for _ in range(5)]
    also = gq.gemm_epilogue(x, t, W.scale[0], 6, act="gelu", out_dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in two + [also])
    y1, y2 = torch.empty_like(want), torch.empty_like(want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        call(y1)
    with torch.cuda.graph(g2):
        call(y2)
    for _ in range(3):
        y1.zero_(), y2.zero_()
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1, want) and torch.equal(y2, want)


def test_two_streams_at_once(gq):
    """Calls of both kernels that run side by side do not disturb each other."""
    rng = np.random.default_rng(14)
    jobs = []
    for M, N, K in ((3, 640, 4096), (200, 1000, 1024), (300, 6000, 1536)):
        W = Weight(gq, rng, 1, N, K, 6)
        t, x = gq.tile_weight(W.packed[0], K, 6), _x(rng, M, K)
        jobs.append((x, t, W.scale[0], gq.gemm_epilogue(x, t, W.scale[0], 6, act="silu")))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    for _ in range(20):
        for (x, t, s, _), st, g in zip(jobs, streams, got):
            with torch.cuda.stream(st):
                g.append(gq.gemm_epilogue(x, t, s, 6, act="silu"))
    torch.cuda.synchronize()
    for (_, _, _, want), g in zip(jobs, got):
        assert all(torch.equal(y, want) for y in g)


def test_a_row_of_dependent_calls(gq):
    """Each call reads what the one before wrote (their blocks may overlap in time), eager and captured."""
    rng = np.random.default_rng(15)
    Ws = [Weight(gq, rng, 1, 512, 512, 6) for _ in range(3)]
    ts = [gq.tile_weight(W.packed[0], 512, 6) for W in Ws]
    for M in (1, 40, 130):
        x0 = _x(rng, M, 512)

        def chain(x):
            for _ in range(10):
                for W, t in zip(Ws, ts):
                    x = gq.gemm_epilogue(x, t, W.scale[0], 6, act="silu", residual=x)
            return x

        x = x0
        for _ in range(10):
            for W, t in zip(Ws, ts):
                x = gq.gemm_epilogue(x, t, W.scale[0], 6, act="silu", residual=x)
                torch.cuda.synchronize()
        assert torch.equal(chain(x0), x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = chain(x0)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, x)


def test_offsets_past_32_bits(gq):
    """Y of more than 2^31 elements, and experts' codes past 2^31 bytes."""
    rng = np.random.default_rng(16)
    W = Weight(gq, rng, 1, 16400, 64, 6)
    x = _x(rng, 131200, 64)
    y = gq.gemm_epilogue(x, gq.tile_weight(W.packed[0], 64, 6), W.scale[0], 6, act="relu")
    for s in (slice(0, 100), slice(131100, 131200)):
        _check(y[s], x[s], W.w[0], None, None, "relu", s)
    del y, x
    E, N, K = 34, 8192, 8192
    nbytes = gq.LIB.gq_tile_bytes(N, K, 8)
    assert E * nbytes > 1 << 31
    W = Weight(gq, rng, 1, N, K, 8)
    tiles = torch.zeros((E, nbytes), dtype=torch.uint8, device="cuda")
    tiles[E - 1] = gq.tile_weight(W.packed[0], K, 8)
    scale = torch.zeros((E, N), dtype=torch.float16, device="cuda")
    scale[E - 1] = W.scale[0]
    for M in (6, 3500):
        x = _x(rng, M, K)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = M
        y = gq.gemm_grouped(x, off, tiles, scale, 8)
        _check(y[-50:], x[-50:], W.w[0], None, None, "none", M)


# ----------------------------------------------------------------- grouped --

def _grouped(gq, counts, N, K, qbits, act="none", bias="none", residual="none", out=torch.float32, first=0, behind=0):
    rng = np.random.default_rng(sum(counts) + 3 * N + 7 * K)
    E, M = len(counts), first + sum(counts) + behind
    W = Weight(gq, rng, E, N, K, qbits)
    tiles = gq.tile_weight(W.packed, K, qbits)
    x, b, r = _x(rng, M, K), _extra(rng, bias, E, N), _extra(rng, residual, M, N)
    off = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    pad = torch.full((M, N + 3), 7.0, dtype=out, device="cuda")
    y = gq.gemm_grouped(x, torch.from_numpy(off).cuda(), tiles, W.scale, qbits, bias=b, act=act, residual=r,
                        y=pad[:, :N], check_status=True)
    assert (pad[:, N:] == 7).all() and (pad[:first] == 7).all() and (pad[M - behind:] == 7).all()
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start < s.stop:
            _check(y[s], x[s], W.w[e], None if b is None else b[e], None if r is None else r[s], act, (e, counts))


@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 64), ([0, 1, 0], 130, 100), ([1] * 8, 256, 512), ([5, 0, 0, 17, 1], 300, 1000),
    ([0] * 20 + [3] + [0] * 40 + [2], 200, 320), ([16, 15, 17, 33], 528, 1584), ([100, 0, 250, 7], 384, 200),
    ([1, 700, 2], 1584, 528), ([128, 256, 129, 64, 0, 511], 300, 136), ([40] * 30, 264, 72), ([0, 0], 64, 64),
])
def test_grouped(gq, counts, N, K, qbits):
    _grouped(gq, counts, N, K, qbits)


@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("counts", [[200, 0, 257, 31, 600, 1], [128] * 9, [0, 0, 900, 0]])
def test_grouped_many_rows(gq, counts, qbits):
    """Over pairs of SMs: ragged, empty and lone experts, a padded batch."""
    _grouped(gq, counts, 2500, 1600, qbits, "gelu", "f32", "bf16", torch.bfloat16, first=2, behind=40)


@pytest.mark.parametrize("act", ["silu", "leaky_relu2"])
@pytest.mark.parametrize("counts", [[1, 0, 2], [30, 200, 0, 3]])
def test_grouped_epilogue_and_padding(gq, counts, act):
    _grouped(gq, counts, 260, 192, 6, act, "bf16", "f32", torch.bfloat16, first=3, behind=70)


def test_grouped_bad_offsets_are_reported(gq):
    """Offsets outside the batch or descending: a status, no write outside Y."""
    rng = np.random.default_rng(11)
    for N, K, M in ((140, 128, 50), (4100, 1600, 650)):        # the second over pairs of SMs
        W = Weight(gq, rng, 3, N, K, 6)
        tiles, x = gq.tile_weight(W.packed, K, 6), _x(rng, M, K)
        for off in ([0, 10, 5, M], [-4, 10, 20, M], [0, 20, M + 1, M + 1], [0, 1 << 30, 1 << 30, 1 << 30],
                    [-(1 << 31), -5, -1, 2], [0, M, 0, M]):
            pad = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
            with pytest.raises(gq.GQError, match="0x8"):
                gq.gemm_grouped(x, torch.tensor(off, dtype=torch.int32, device="cuda"), tiles, W.scale, 6,
                                y=pad[1:M + 1], check_status=True)
            assert (pad[0] == 7).all() and (pad[M + 1] == 7).all()
    W = Weight(gq, rng, 70, 64, 64, 6)                         # a bad offset behind every row's expert
    off = torch.tensor([0] + [5] * 69 + [4], dtype=torch.int32, device="cuda")
    with pytest.raises(gq.GQError, match="0x8"):
        gq.gemm_grouped(_x(rng, 5, 64), off, gq.tile_weight(W.packed, 64, 6), W.scale, 6, check_status=True)


@pytest.mark.parametrize("E,active,rows,N,K", [
    (33, 33, 3, 130, 64), (100, 7, 40, 200, 72), (300, 300, 2, 130, 40), (1100, 25, 30, 70, 64), (2500, 3, 1, 64, 24),
    (40, 40, 120, 2500, 1600), (700, 90, 90, 1000, 24),
])
def test_grouped_many_experts(gq, E, active, rows, N, K):
    """More experts than lanes of a warp, most of them without a row."""
    counts = np.zeros(E, np.int64)
    rng = np.random.default_rng(E)
    counts[rng.permutation(E)[:active]] = rng.integers(1, 2 * rows, active)
    counts[E - 1] = max(counts[E - 1], 1)
    _grouped(gq, counts.tolist(), N, K, 6, "silu", "f32", "bf16", torch.bfloat16, first=2, behind=3)


def test_grouped_bad_offsets_of_many_experts(gq):
    rng = np.random.default_rng(13)
    W = Weight(gq, rng, 300, 64, 64, 8)
    x, tiles = _x(rng, 90, 64), gq.tile_weight(W.packed, 64, 8)
    for at, value in ((0, -1), (1, 91), (150, 3), (299, 91), (300, 60), (300, 1 << 30)):
        off = np.minimum(np.arange(301), 90).astype(np.int32)
        off[at] = value
        pad = torch.full((92, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(gq.GQError, match="0x8"):
            gq.gemm_grouped(x, torch.from_numpy(off).cuda(), tiles, W.scale, 8, y=pad[1:91], check_status=True)
        assert (pad[0] == 7).all() and (pad[91] == 7).all()


def test_grouped_bad_offsets_overlapping(gq):
    """Expert ranges that overlap, each in order by itself: reported, and none of their tiles worked on by the pairs of
    SMs (65535 experts of the whole batch would be as many products).  With no columns too."""
    rng = np.random.default_rng(12)
    E, M, N, K = 8, 1024, 2048, 1600
    W = Weight(gq, rng, E, N, K, 8)
    x, tiles = _x(rng, M, K), gq.tile_weight(W.packed, K, 8)
    off = torch.tensor([0, M] * 4 + [0], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gq.GQError, match="0x8"):
        gq.gemm_grouped(x, off, tiles, W.scale, 8, y=y, check_status=True)
    assert (y == 7).all()
    b = _extra(rng, "f32", E, N)
    for o in (off, torch.tensor([0] * 8 + [M + 1], dtype=torch.int32, device="cuda")):
        with pytest.raises(gq.GQError, match="0x8"):
            gq.gemm_grouped(x[:, :0], o, tiles[:, :0], W.scale, 8, bias=b, check_status=True)


def test_grouped_equals_single_weights(gq):
    """An expert's rows get the same bits as gemm_epilogue on that weight where one schedule serves both."""
    rng = np.random.default_rng(12)
    W = Weight(gq, rng, 2, 256, 256, 8)
    tiles, x = gq.tile_weight(W.packed, 256, 8), _x(rng, 24, 256)
    off = torch.tensor([0, 10, 24], dtype=torch.int32, device="cuda")
    y = gq.gemm_grouped(x, off, tiles, W.scale, 8, act="silu")
    for e, s in ((0, slice(0, 10)), (1, slice(10, 24))):
        _check(y[s], x[s], W.w[e], None, None, "silu", e)


# ---------------------------------------------------------------- refusals --

def test_helper_refusals(gq):
    rng = np.random.default_rng(13)
    W = Weight(gq, rng, 2, 64, 128, 6)
    t, x = gq.tile_weight(W.packed, 128, 6), _x(rng, 4, 128)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    ok = dict(x=x, tiles=t[0], scale_f16=W.scale[0], qbits=6)
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x.t()), dict(tiles=t), dict(tiles=t[0][:-16]),
                dict(qbits=8), dict(scale_f16=W.scale[0].float()), dict(act="swish"), dict(bias=W.scale[0][:3]),
                dict(residual=x), dict(y=x), dict(tiles=t[0].cpu()), dict(out_dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            gq.gemm_epilogue(**{**ok, **bad})
    for bad in (off.long(), off[:-1], off.cpu()):
        with pytest.raises(ValueError):
            gq.gemm_grouped(x, bad, t, W.scale, 6)
    with pytest.raises(gq.GQError):                            # rows that do not start on 16 bytes
        gq.gemm_epilogue(_x(rng, 4, 136)[:, 1:129], t[0], W.scale[0], 6)
