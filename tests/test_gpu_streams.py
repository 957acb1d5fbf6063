"""Outputs made by calls on another stream than the current one: their memory is not what the current stream's
work has yet to write."""
import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_append as tp
import test_gpu_attention as ta
import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def calls():
    a = tp.make(3, 50, 8, 2, 64, 64, torch.bfloat16, seed=1)
    yield lambda stream=None: [tp.call(a, stream=stream)]
    s = ta.make([300, 7], 50, 8, 2, 64, torch.bfloat16, seed=2)
    yield lambda stream=None: list(ta.call(s, stream=stream))
    x, tok = tl.rows(60, 60, 301, torch.bfloat16, seed=3)
    yield lambda stream=None: list(sv.spec_verify_logprobs(x, tok, top_n=4, stream=stream))


def test_outputs_on_another_stream():
    side = torch.cuda.Stream()
    for call in calls():
        want = call()
        call(stream=side)  # the workspace of this stream
        for t in want:
            torch.empty_like(t).fill_(7)  # (a kernel's first launch may wait for the device)
        torch.cuda._sleep(1000)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # the current stream is behind ...
        late = [torch.empty_like(t) for t in want]
        for t in late:
            t.fill_(7)  # ... and writes memory that the allocator has back already
        del t, late
        got = call(stream=side)
        side.synchronize()
        assert not torch.cuda.current_stream().query()  # (or the sleep was too short to show anything)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
