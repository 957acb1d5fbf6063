"""Waits inside the kernels that run out: with a limit of a few clocks, which debug builds take, ordinary waits
do.  The call then ends by itself, says so, reads and writes nothing out of range, and the next call is right."""
import contextlib

import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_attention as ta
import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
USUAL = 1000000000


@pytest.fixture(scope="module")
def lib():
    torch.cuda.set_device(DEV)
    sv.load_library()
    return sv.load_debug_library()


@contextlib.contextmanager
def limit(lib, clocks):
    with sv.using_library(lib):
        sv.spec_verify_debug_wait_clocks(clocks, lib)
        try:
            yield
        finally:
            torch.cuda.synchronize()
            sv.spec_verify_debug_wait_clocks(USUAL, lib)


def run_out(lib, call, nbytes):
    """call(workspace, status) -> outputs, under limits from none to ample."""
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_verify_wait_timeouts(lib)
    with limit(lib, USUAL):
        want = [t.clone() for t in call(ws, status)]
        torch.cuda.synchronize()
        assert int(status) == 0 and sv.spec_verify_wait_timeouts(lib) == 0
    for clocks in (-1, 0, 100, 1000, 3000, 10000, 100000, -1):
        for _ in range(3):
            ws.zero_()
            status.zero_()
            with limit(lib, clocks):
                got = call(ws, status)
                torch.cuda.synchronize()
            said, count = int(status), sv.spec_verify_wait_timeouts(lib)
            assert (said, count > 0) in ((0, False), (7, True))
            assert clocks >= 0 or said == 7
            assert sv.spec_verify_debug_fault(lib) == 0
            assert said == 7 or all(torch.equal(a, b) for a, b in zip(got, want))
        ws.zero_()
        status.zero_()
        with limit(lib, USUAL):
            got = call(ws, status)
            torch.cuda.synchronize()
        assert int(status) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B,T,V", [(1, 3, 40009), (3, 7, 9001), (40, 8, 20011), (700, 64, 41)])
def test_logprobs(lib, B, T, V):
    x, tok = tl.rows(B, T, V, torch.bfloat16, seed=V)

    def call(ws, status):
        return sv.spec_verify_logprobs(x, tok, top_n=5, workspace=ws, dev_status=status)

    run_out(lib, call, sv.spec_verify_logprobs_workspace_bytes(B, T, V, 5))


@pytest.mark.parametrize("committed,N,Hq,Hkv,D,dtype", [
    ([700], 1, 4, 1, 128, torch.bfloat16), ([40000, 3], 8, 8, 2, 128, torch.bfloat16), ([30000], 16, 4, 1, 64, torch.float16),
    ([0, 130, 700, 3, 128] * 40, 3, 8, 8, 80, torch.bfloat16), ([3000] * 64, 20, 4, 1, 128, torch.float16)])
def test_attention(lib, committed, N, Hq, Hkv, D, dtype):
    s = ta.make(committed, N, Hq, Hkv, D, dtype, seed=N, tree=N > 1)

    def call(ws, status):
        return ta.call(s, workspace=ws, dev_status=status)

    run_out(lib, call, sv.spec_verify_attention_workspace_bytes(len(committed), N, Hq, Hkv, D, s["slot_table"].shape[1]))


def test_after_a_reset_calls_without_a_workspace_are_right(lib):
    s = ta.make([40000, 700], 8, 4, 1, 128, torch.bfloat16, seed=5, tree=True)
    x, tok = tl.rows(1, 3, 40009, torch.bfloat16, seed=5)
    with limit(lib, USUAL):
        want, said = ta.call(s), sv.spec_verify_logprobs(x, tok, top_n=3)
    for clocks in (-1, 2000, -1):
        with limit(lib, clocks):
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            ta.call(s, dev_status=status)
            sv.spec_verify_logprobs(x, tok, top_n=3, dev_status=status)
            torch.cuda.synchronize()
        assert clocks >= 0 or int(status) == 7
        sv.spec_verify_reset_workspaces()
        with limit(lib, USUAL):
            got, again = ta.call(s), sv.spec_verify_logprobs(x, tok, top_n=3)
            torch.cuda.synchronize()
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
        assert all(torch.equal(a, b) for a, b in zip(again, said))
