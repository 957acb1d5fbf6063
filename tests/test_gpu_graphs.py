"""Graphs captured from calls without a workspace: replayed in any order, beside calls outside them that need
larger ones, every replay gives what a call gives."""
import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_attention as ta
import test_gpu_logprobs as tl
from speculative_decoding_verification_verify_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def calls():
    """(name, call into given outputs, the outputs), each with work that is joined across CTAs."""
    for N in (1, 16):
        s = ta.make([40000, 300], N, 4, 1, 128, seed=N, tree=N > 1)
        out = torch.zeros_like(s["q"])
        yield f"attention {N}", lambda s=s, out=out: ta.call(s, out=out), [out]
    x, tok = tl.rows(1, 3, 128256, torch.bfloat16, seed=41)
    lp, ent = torch.zeros((2, 1, 3), device=DEV)
    yield "logprobs", lambda: sv.spec_verify_logprobs(x, tok, logprobs=lp, entropy=ent, top_n=4), [lp, ent]
    c = wl.chain_b64k7(DEV, B=4, k=3, V=40009, seed=3)
    o, n = torch.zeros((4, 4), dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    yield "rejection", lambda: sv.spec_verify_rejection(c.logits, c.drafts, None, temperature=1.0, seed=3, offset=1,
                                                        out_tokens=o, accept_len=n), [o, n]
    conf = torch.rand((40, 7), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    cost = 1e-3 + torch.arange(40 * 7 + 1, device=DEV, dtype=torch.float64) * 1e-5
    a = torch.zeros(40, dtype=torch.int32, device=DEV)
    yield "budget", lambda: sv.spec_verify_plan_budget(conf, cost, admitted=a), [a]


def test_replays_in_any_order():
    made = []
    for name, f, outs in calls():
        f()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        graphs = []
        for twice in (1, 2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(twice):
                    f()
            graphs.append(g)
        made.append((name, graphs, outs, want, f))  # f: a graph's inputs have to live

    def replay(order, when):
        for name, graphs, outs, want, _ in order:
            for g in reversed(graphs):  # the later captured first
                for _ in range(2):
                    for t in outs:
                        t.zero_()
                    g.replay()
                    torch.cuda.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(outs, want)), (name, when)

    replay(made[::-1], "first")
    replay(made, "again")
    # Calls outside that need more, on the default stream and on the one that was captured from; then what
    # was given back is written.
    big = ta.make([3000], 64, 4, 1, 128, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ta.call(big)
    ta.call(big, stream=side)
    torch.cuda.synchronize()
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
    replay(made, "beside other calls")
    assert all(bool((t == 255).all()) for t in junk)
    replay(made[::-1], "last")


def test_capture_ids():
    side = torch.cuda.Stream()
    assert sv.binding._capture_id(0, side, side.cuda_stream) == 0 and sv.binding._capture_id(0, None, 0) == 0
    x, seen = torch.zeros(4, device=DEV), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cur = torch.cuda.current_stream()
            x.add_(1)
            seen.append(sv.binding._capture_id(0, None, cur.cuda_stream))
            assert sv.binding._capture_id(0, cur, cur.cuda_stream) == seen[-1]
            assert sv.binding._capture_id(0, side, side.cuda_stream) == 0
    assert 0 not in seen and seen[0] != seen[1]
