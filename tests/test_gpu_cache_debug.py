"""The operators over a cache of 8-bit rows and the prompt's chunks: the range-checked build's small cases, waits that run
out, the example that runs them together."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_attention_e4m3 as te
import test_gpu_cache as tc
import test_gpu_chunk as th
from test_gpu_timeouts import run_out

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lib():
    torch.cuda.set_device(0)
    sv.load_library()
    return sv.load_debug_library()


def _cases():
    for D, rot, dt, tree, e4m3 in ((64, 64, BF, True, True), (128, 96, FP, False, True), (80, 0, BF, False, False)):
        s = tc.setup(3, 7, 6, 2, D, rot, dt, e4m3, seed=D, tree=tree)
        nn = torch.tensor([7, 0, 3], dtype=torch.int32, device="cuda")
        yield f"append {D}", lambda s=s, nn=nn: (tc.call(s, num_nodes=nn, interleaved=s["k"].shape[-1] == 128), s["k_cache"],
                                                 s["v_cache"])
    for e4m3 in (True, False):
        k, v, _, _, table = tc.pool_of(3, 50, 3, 80, BF, e4m3)
        first, num = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3, 20], [30, 0, 17]))
        yield f"read {e4m3}", lambda k=k, v=v, table=table, first=first, num=num: tuple(sv.spec_verify_kv_read(
            k, v, table, first, 30, num_rows=num, kv_heads=3, head_dim=80, dtype=BF))
    for N, Hq, Hkv, D, dt in ((1, 4, 4, 64, BF), (8, 8, 2, 128, FP), (20, 8, 2, 96, BF), (64, 4, 1, 128, BF)):
        s = te.make([0, 130, 700, 3, 128], N, Hq, Hkv, D, dt, seed=N, tree=N > 1)
        nn = torch.tensor([N, 0, N, (N + 1) // 2, N], dtype=torch.int32, device="cuda")
        yield f"nodes {N}", lambda s=s, nn=nn: tuple(te.call(s, num_nodes=nn))
    for N, Hq, Hkv, D, dt, e4m3 in ((1, 4, 4, 64, BF, False), (70, 8, 2, 128, FP, True), (300, 6, 2, 80, BF, True),
                                    (131, 4, 1, 128, BF, False)):
        s = th.make([0, 130, 2700, 3], N, Hq, Hkv, D, dt, e4m3, seed=N)
        nn = torch.tensor([N, 0, N, (N + 1) // 2], dtype=torch.int32, device="cuda")
        yield f"chunk {N}", lambda s=s, nn=nn: tuple(th.call(s, num_nodes=nn))


def test_debug_build_checks_and_matches(lib):
    for name, f in _cases():
        want = [t.clone() for t in f()]
        with sv.using_library(lib):
            sv.spec_verify_debug_fault(lib)
            got = f()
            torch.cuda.synchronize()
            assert sv.spec_verify_debug_fault(lib) == 0, name
        for a, b in zip(got, want):
            assert torch.equal(a, b) or torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())), name


@pytest.mark.parametrize("committed,N,Hq,Hkv,D,dtype", [
    ([700], 1, 4, 1, 128, BF), ([40000, 3], 8, 8, 2, 128, BF), ([30000], 16, 4, 1, 64, FP),
    ([0, 130, 700, 3, 128] * 40, 3, 8, 8, 80, BF), ([3000] * 64, 20, 4, 1, 128, FP)])
def test_waits_of_nodes_run_out(lib, committed, N, Hq, Hkv, D, dtype):
    s = te.make(committed, N, Hq, Hkv, D, dtype, seed=N, tree=N > 1)
    run_out(lib, lambda ws, status: te.call(s, workspace=ws, dev_status=status),
            sv.spec_verify_attention_e4m3_workspace_bytes(len(committed), N, Hq, Hkv, D, s["slot_table"].shape[1]))


@pytest.mark.parametrize("committed,N,Hq,Hkv,D,dtype,e4m3", [
    ([700], 1, 4, 1, 128, BF, False), ([40000, 3], 100, 8, 2, 128, BF, True), ([0], 900, 4, 1, 64, FP, False),
    ([0, 130, 700, 3, 128] * 20, 33, 8, 8, 80, BF, False), ([3000] * 8, 200, 4, 1, 128, FP, True)])
def test_waits_of_chunks_run_out(lib, committed, N, Hq, Hkv, D, dtype, e4m3):
    s = th.make(committed, N, Hq, Hkv, D, dtype, e4m3, seed=N)
    run_out(lib, lambda ws, status: th.call(s, workspace=ws, dev_status=status),
            sv.spec_verify_attention_chunk_workspace_bytes(len(committed), N, Hq, Hkv, D, s["slot_table"].shape[1]))


def test_the_example():
    """From prompt to verification over one cache of 8-bit rows: the text is that of decoding token by token."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    import cache8_step

    text, got, keys, committed, rate = cache8_step.run(steps=24)
    assert torch.equal(text, got) and rate >= 1.0
    for b, c in enumerate(committed.tolist()):
        assert torch.isfinite(keys[b].float()).all() and keys[b, :c].float().abs().amax((1, 2)).min() > 0
        assert not keys[b, c:].any()
