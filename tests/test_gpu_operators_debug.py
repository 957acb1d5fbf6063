"""The range-checked build of the operators around verification: small cases of each record no index out of
range and give the release build's bits."""
import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_append as ta
import test_gpu_attention as tt
import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def debug_lib():
    torch.cuda.set_device(0)
    sv.load_library()
    return sv.load_debug_library()


def _cases():
    for D, rot, dt, tree in ((64, 64, BF, True), (128, 96, FP, False), (80, 0, BF, False)):
        s = ta.make(3, 7, 6, 2, D, rot, dt, seed=D, tree=tree)
        nn = torch.tensor([7, 0, 3], dtype=torch.int32, device="cuda")
        yield f"append {D}", lambda s=s, nn=nn: (ta.call(s, num_nodes=nn, interleaved=s["k"].shape[-1] == 128), s["k_cache"],
                                                 s["v_cache"])
    for N, Hq, Hkv, D, dt in ((1, 4, 4, 64, BF), (8, 8, 2, 128, FP), (20, 8, 2, 96, BF), (64, 4, 1, 128, BF)):
        s = tt.make([0, 130, 700, 3, 128], N, Hq, Hkv, D, dt, seed=N, tree=N > 1)
        nn = torch.tensor([N, 0, N, (N + 1) // 2, N], dtype=torch.int32, device="cuda")
        yield f"attention {N}", lambda s=s, nn=nn: tuple(tt.call(s, num_nodes=nn))
    s = tt.make([40000], 4, 4, 1, 128, BF, seed=9)
    yield "attention split", lambda: tuple(tt.call(s))
    for V, dt, top in ((1, BF, 2), (4099, BF, 20), (20011, torch.float32, 5), (40000, BF, 0)):
        x, tok = tl.rows(3, 4, V, dt, seed=V)
        tok[1, 2:] = -1
        index = torch.tensor([[0, 2, 3, 1]] * 3, dtype=torch.int32, device="cuda")
        yield f"logprobs {V}", lambda x=x, tok=tok, index=index, top=top: tuple(
            t for t in sv.spec_verify_logprobs(x, tok, row_index=index, top_n=top) if t is not None)
    flat = torch.zeros((1, 2, 30011), device="cuda")
    yield "logprobs flat", lambda: tuple(sv.spec_verify_logprobs(flat, torch.ones((1, 2), dtype=torch.int32, device="cuda"),
                                                                 top_n=32))


def test_debug_build_checks_and_matches(debug_lib):
    for name, f in _cases():
        want = [t.clone() for t in f()]
        with sv.using_library(debug_lib):
            sv.spec_verify_debug_fault(debug_lib)
            got = f()
            torch.cuda.synchronize()
            assert sv.spec_verify_debug_fault(debug_lib) == 0, name
        for a, b in zip(got, want):
            assert torch.equal(a, b) or torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())), name
