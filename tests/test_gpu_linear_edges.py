"""GPU parity of the layer products where a kernel's own structure has an edge: the last column tile ends inside a warp
and the epilogue makes several trips, alone and with the K range shared by a cluster; and the binding's edges: calls on a
stream other than the current one.

Reference, tolerances and inputs are those of test_gpu_linear.py.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_linear import Weight, _check, _extra, _grouped, _run, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


@pytest.mark.parametrize("N", [1, 31, 33, 97, 130, 2079])
@pytest.mark.parametrize("M,K", [(9, 64), (9, 2048), (32, 192), (32, 4096), (63, 128), (63, 1024), (128, 64), (128, 1600)])
def test_last_columns_end_inside_a_warp(gq, M, N, K):
    """Lanes without a column leave the epilogue's branches early; the loads from tensor memory and the cluster's barriers
    that follow are executed by whole warps.  One K range a tile (few column blocks) and a split one."""
    _run(gq, M, N, K, 6, "silu", "f32", "bf16")


def test_last_columns_of_experts_end_inside_a_warp(gq):
    for counts, K in (([20, 0, 32, 11], 64), ([20, 0, 32, 11], 2048), ([100, 70, 0, 120], 128), ([100, 70, 0, 120], 1536)):
        _grouped(gq, counts, 161, K, 8, "relu2", "bf16", "f32", torch.bfloat16, first=1, behind=2)


def _busy(stream, ms=100):
    """`stream` behind what is queued already, and busy for about `ms`."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 1.9e6))


@pytest.mark.parametrize("raw", [False, True])
def test_status_of_a_call_on_another_stream(gq, raw):
    """check_status waits for the call on the stream that it runs on: a bad offset is reported, a good call is not taken
    for a bad one by what the status word's memory held before."""
    rng = np.random.default_rng(21)
    W = Weight(gq, rng, 2, 130, 192, 6)
    tiles, x = gq.tile_weight(W.packed, 192, 6), _x(rng, 20, 192)
    good, bad = (torch.tensor(o, dtype=torch.int32, device="cuda") for o in ([0, 7, 20], [0, 7, 21]))
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for s in (torch.cuda.current_stream(), side):              # memory that the status word may come from
        with torch.cuda.stream(s):
            keep = [torch.full((1,), 8, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del keep
    _busy(side)
    y = gq.gemm_grouped(x, good, tiles, W.scale, 6, stream=stream, check_status=True)
    assert side.query()                                        # the call was waited for
    _check(y[:7], x[:7], W.w[0], None, None, "none", raw)
    _check(y[7:], x[7:], W.w[1], None, None, "none", raw)
    _busy(side)
    with pytest.raises(gq.GQError, match="0x8"):
        gq.gemm_grouped(x, bad, tiles, W.scale, 6, stream=stream, check_status=True)


def test_results_on_another_stream_keep_their_memory(gq):
    """A result dropped while its call is still queued on another stream is not handed out to the current one."""
    rng = np.random.default_rng(22)
    W = Weight(gq, rng, 1, 200, 320, 8)
    tiles, x = gq.tile_weight(W.packed[0], 320, 8), _x(rng, 9, 320)
    want = gq.gemm_epilogue(x, tiles, W.scale[0], 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: gq.gemm_epilogue(x, tiles, W.scale[0], 8, stream=side),
                 lambda: gq.tile_weight(W.packed[0], 320, 8, stream=side)):
        _busy(side)
        out = call()
        shape, dtype, at = out.shape, out.dtype, out.data_ptr()
        del out
        others = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(16)]
        assert all(t.data_ptr() != at for t in others) and not side.query()
        torch.cuda.synchronize()
    _busy(side, 20)
    y = gq.gemm_epilogue(x, gq.tile_weight(W.packed[0], 320, 8, stream=side), W.scale[0], 8, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_every_way_to_name_a_stream(gq):
    """The current stream, the default one by its handle 0, a torch stream, its handle, an object that holds one; the
    current one a side stream too."""
    class Holder:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    rng = np.random.default_rng(29)
    W = Weight(gq, rng, 1, 130, 192, 6)
    x = _x(rng, 5, 192)
    want = gq.gemm_epilogue(x, gq.tile_weight(W.packed[0], 192, 6), W.scale[0], 6)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for cur in (torch.cuda.default_stream(), other):
        with torch.cuda.stream(cur):
            for s in (None, 0, torch.cuda.current_stream(), side, side.cuda_stream, Holder(side), torch.cuda.default_stream()):
                y = gq.gemm_epilogue(x, gq.tile_weight(W.packed[0], 192, 6, stream=s), W.scale[0], 6, stream=s,
                                     check_status=True)
                torch.cuda.synchronize()
                assert torch.equal(y, want)


def test_stream_refusals(gq):
    W = Weight(gq, np.random.default_rng(23), 1, 64, 64, 6)
    x = _x(np.random.default_rng(23), 3, 64)
    with pytest.raises(ValueError):
        gq.gemm_epilogue(x.cpu(), W.packed[0], W.scale[0], 6, stream=torch.cuda.Stream())
    with pytest.raises(ValueError):
        gq.tile_weight(W.packed[0].cpu(), 64, 6, stream=torch.cuda.Stream())


@pytest.mark.parametrize("first,counts,behind,K", [(3, [4, 0, 9], 20, 192), (0, [0, 0, 0], 7, 64), (1, [5, 1, 1], 2, 0),
                                                   (2, [300, 260, 0], 60, 1600)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_rows_of_no_expert_are_zero_in_a_new_result(gq, first, counts, behind, K, out):
    """A padded batch without a given y: memory that other tensors have left behind does not show."""
    rng = np.random.default_rng(24)
    M, N = first + sum(counts) + behind, 2500
    W = Weight(gq, rng, 3, N, max(K, 1), 6)
    tiles = gq.tile_weight(W.packed, K, 6) if K else torch.empty((3, 0), dtype=torch.uint8, device="cuda")
    off = torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    x, bias = _x(rng, M, max(K, 1))[:, :K], torch.ones((3, N), device="cuda")
    junk = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    del junk
    y = gq.gemm_grouped(x, off, tiles, W.scale, 6, bias=bias, out_dtype=out)
    assert not y[:first].any() and not y[M - behind:].any()
    for e in range(3):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start < s.stop and K:
            _check(y[s], x[s], W.w[e], bias[e], None, "none", e)
        elif s.start < s.stop:
            assert (y[s] == 1).all()


@pytest.mark.parametrize("M,N", [(0, 130), (9, 0), (0, 0)])
@pytest.mark.parametrize("K", [64, 0])
def test_offsets_of_an_empty_product_are_looked_at(gq, M, N, K):
    """No rows or no columns: offsets that leave the batch or descend are reported as anywhere else."""
    W = Weight(gq, np.random.default_rng(25), 3, max(N, 1), 64, 6)
    tiles = gq.tile_weight(W.packed[:, :N].contiguous(), K, 6) if K else torch.empty((3, 0), dtype=torch.uint8, device="cuda")
    scale, x = W.scale[:, :N].contiguous(), torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    call = lambda *off: gq.gemm_grouped(x, torch.tensor(off, dtype=torch.int32, device="cuda"), tiles, scale, 6,  # noqa: E731
                                        check_status=True)
    assert call(0, M // 2, M // 2, M).shape == (M, N)
    for off in ((0, 0, 0, M + 1), (-1, 0, 0, M), (0, M + 1, 0, M), (0, M, M - 1, M), (M + 1, M + 1, M + 1, M + 1)):
        with pytest.raises(gq.GQError, match="0x8"):
            call(*off)


# ------------------------------------------------------ over pairs of SMs --

def _over_pairs(fn):
    """fn() with the kernel of 256 x 256 tiles over pairs of SMs: the sizes are there to reach it, so that a change of the
    rule that picks it does not leave it untested.  (Where the profiler sees no kernel at all this is not looked at.)"""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        fn()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if "linear" in e.name and "kernel" in e.name]
    assert not names or any("linear_pair_kernel" in n for n in names), names


@pytest.mark.parametrize("qbits", [6, 8])
@pytest.mark.parametrize("M,N,K", [
    (24001, 4865, 40), (16401, 4097, 72),                      # one stage a unit, of one and of two column blocks
    (8193, 4225, 136), (6401, 4097, 200),                      # two
    (6201, 4101, 320), (4101, 4097, 328),                      # three
    (4101, 4100, 393), (3300, 4300, 505),                      # four
    (3301, 4301, 520),                                         # five: more than there are slots
])
def test_pairs_with_few_stages_a_unit(gq, M, N, K, qbits):
    """Several units a pair, with as many or fewer stages to a unit than there are slots for them: a unit's sums are
    drained while the next units' stages are under way."""
    _over_pairs(lambda: _run(gq, M, N, K, qbits, "silu", "f32", "bf16"))


@pytest.mark.parametrize("N,K", [(28001, 40), (14201, 104), (8201, 136), (8201, 264), (5001, 440)])
def test_pairs_of_experts_with_few_stages_a_unit(gq, N, K):
    counts = [70, 0, 300, 5, 64, 200, 31, 90, 128, 1, 255, 40, 77, 33, 96, 120]
    _over_pairs(lambda: _grouped(gq, counts, N, K, 6, "gelu_tanh", "f32", "f32", torch.bfloat16, first=1, behind=25))


@pytest.mark.parametrize("qbits", [6, 8])
def test_pairs_of_one_expert_among_empty_ones(gq, qbits):
    _over_pairs(lambda: _grouped(gq, [0, 0, 900, 0], 4601, 1600, qbits, "gelu", "f32", "bf16", torch.bfloat16, first=2,
                                 behind=40))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_pairs_with_the_residual_in_place(gq, kind):
    rng = np.random.default_rng(26)
    for M, N, K in ((515, 5001, 1600), (3301, 4301, 520)):
        W = Weight(gq, rng, 1, N, K, 8)
        x, t = _x(rng, M, K), gq.tile_weight(W.packed[0], K, 8)
        y = _extra(rng, kind, M, N)
        r = y.clone()
        _over_pairs(lambda: gq.gemm_epilogue(x, t, W.scale[0], 8, act="relu2", residual=y, y=y))
        _check(y, x, W.w[0], None, r, "relu2", (M, N, K))


def test_an_expert_has_the_bits_of_its_own_product(gq):
    """Same tile width and an unsplit K range in the grouped call and in each expert's own: the same bits."""
    rng = np.random.default_rng(27)
    for counts, N, K in (([10, 14], 19300, 200), ([16, 1, 9, 3], 19300, 136), ([100, 80], 19300, 200)):
        W = Weight(gq, rng, len(counts), N, K, 8)
        tiles, x = gq.tile_weight(W.packed, K, 8), _x(rng, sum(counts), K)
        off = np.concatenate([[0], np.cumsum(counts)]).tolist()
        y = gq.gemm_grouped(x, torch.tensor(off, dtype=torch.int32, device="cuda"), tiles, W.scale, 8, act="silu",
                            out_dtype=torch.float32)
        for e, (a, b) in enumerate(zip(off, off[1:])):
            own = _x(rng, b - a, K).copy_(x[a:b])              # (a slice of x need not start on 16 bytes)
            assert torch.equal(y[a:b], gq.gemm_epilogue(own, tiles[e], W.scale[e], 8, act="silu",
                                                        out_dtype=torch.float32)), (counts, e)


# ------------------------------------------------------ captured neighbours --

def test_captured_between_memsets_and_joined_streams(gq):
    """In one graph: a buffer cleared by a memset and written just before, products on two streams that join, the status
    word of a C call, a copy behind; replayed on new inputs."""
    rng = np.random.default_rng(28)
    W = [Weight(gq, rng, 1, 512, 512, 6) for _ in range(3)]
    t = [gq.tile_weight(w.packed[0], 512, 6) for w in W]
    for M in (1, 20, 200):
        x = torch.zeros((M, 512), dtype=torch.bfloat16, device="cuda")
        part = torch.zeros((M, 512), dtype=torch.bfloat16, device="cuda")
        status = torch.full((1,), 15, dtype=torch.int32, device="cuda")
        last = torch.zeros((M, 512), dtype=torch.bfloat16, device="cuda")

        def step():
            part.zero_()
            part[: M // 2 + 1].copy_(x[: M // 2 + 1])
            h = gq.gemm_epilogue(part, t[0], W[0].scale[0], 6, act="silu")
            cur = torch.cuda.current_stream()
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                b = gq.gemm_epilogue(h, t[1], W[1].scale[0], 6, act="gelu")
                b.zero_() if M == 20 else b.mul_(0.5)
                b = gq.gemm_epilogue(x, t[1], W[1].scale[0], 6, residual=b, y=b)
            a = gq.gemm_epilogue(h, t[2], W[2].scale[0], 6, act="relu")
            cur.wait_stream(side)
            b.record_stream(cur)
            e = gq.GQEpilogue(residual=b.data_ptr(), ldr=512, residual_dtype=1, y_dtype=1)
            y = torch.zeros_like(x)
            assert gq.LIB.gq_gemm_epilogue(a.data_ptr(), M, 512, 512, t[0].data_ptr(), W[0].scale.data_ptr(), 6, 512,
                                           gq.C.byref(e), y.data_ptr(), 512, status.data_ptr(), cur.cuda_stream) == 0
            last.copy_(y)
            return a, b, y

        side = torch.cuda.Stream()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for seed in range(3):
            x.copy_(_x(np.random.default_rng(seed), M, 512))
            step()
            torch.cuda.synchronize()
            want = last.clone()
            last.zero_(), status.fill_(15)
            for _ in range(2):
                graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(last, want) and status.item() == 0 and last.any()
