"""spec_verify_kv_append with fewer nodes than rows: the rows past num_nodes are not read (the range-checked
build looks at every row that is), and nothing of them is written."""
import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_append as ta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (3, 1, 64), (64, 16, 128)])  # one pass of a thread's loads, few, several
@pytest.mark.parametrize("tree", [False, True])
def test_rows_past_num_nodes_are_not_read(Hq, Hkv, D, tree):
    torch.cuda.set_device(0)
    lib = sv.load_debug_library()
    s = ta.make(4, 6, Hq, Hkv, D, D, torch.bfloat16, seed=Hq, tree=tree)
    nodes = [6, 0, 1, 4]
    nn = torch.tensor(nodes, dtype=torch.int32, device="cuda")
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    want = ta.call(s)
    full = s["k_cache"].clone(), s["v_cache"].clone()
    s["k_cache"].copy_(k), s["v_cache"].copy_(v)
    with sv.using_library(lib):
        sv.spec_verify_debug_fault(lib)
        got = ta.call(s, num_nodes=nn)
        torch.cuda.synchronize()
        assert sv.spec_verify_debug_fault(lib) == 0
    for b in range(4):
        n = nodes[b]
        assert torch.equal(got[b, :n], want[b, :n]) and not got[b, n:].any()
        c = int(s["committed"][b])
        slot = s["slot_table"][b, c:c + 6].long()
        assert torch.equal(s["k_cache"][slot[:n]], full[0][slot[:n]]) and torch.equal(s["v_cache"][slot[:n]], full[1][slot[:n]])
        assert torch.equal(s["k_cache"][slot[n:]], k[slot[n:]]) and torch.equal(s["v_cache"][slot[n:]], v[slot[n:]])
