"""Status words of the quantizing calls on a stream other than the current one."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


@pytest.mark.parametrize("raw", [False, True])
def test_status_is_that_of_the_call(gq, raw):
    """The status is read after the call has run on its stream, not before: a busy side stream, a weight with a NaN and
    one without in turn."""
    good = torch.randn(40, 96, device="cuda")
    bad = good.clone()
    bad[7, 5] = float("nan")
    H = gq.gptq_hessian(torch.randn(200, 96, device="cuda"))
    calls = [lambda w, s: gq.fakequant([gq.Request(w, 6, 0.99)], stream=s)[0],
             lambda w, s: gq.export_pack([gq.Request(w, 8, 0.99)], stream=s)[0],
             lambda w, s: gq.row_clip_select([gq.Request(w, 6, 0.99)], stream=s)[0],
             lambda w, s: gq.gptq_quantize(gq.Request(w, 6, 0.99), H, stream=s),
             lambda w, s: gq.gptq_quantize_batch([gq.Request(w, 6, 0.99)], [H], stream=s)[0]]
    side = torch.cuda.Stream()
    for call in calls:
        for w, want in ((bad, 1), (good, 0), (bad, 1)):
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                torch.cuda._sleep(int(40 * 1.9e6))
            assert call(w, side.cuda_stream if raw else side).status == want
            assert side.query()
