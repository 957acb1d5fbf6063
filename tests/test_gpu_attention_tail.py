"""spec_verify_attention where one position outweighs each of very many others: what these add up to is
part of the answer in both 16-bit types."""
import pytest
import torch

import plain64
import speculative_decoding_verification_verify_gb300 as sv
from test_gpu_attention import BF, DEV, FP, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("below", [14.5, 18.0, 22.0, 24.5, 25.2, 26.0])
@pytest.mark.parametrize("B", [1, 304])
def test_one_weight_over_a_long_tail(dtype, below, B):
    """One position 2^below above 131071 others, whose values have another mean: 1 against -1.  One request is
    split over the GPU; of as many as the GPU takes side by side, none is, and the tail is one sum.  (All
    requests' tables name the same slots.)"""
    c, D = 131071, 64
    score = torch.full((c + 1,), -below * 0.6931471805599453, device=DEV)
    score[4321] = 0.0
    k = (score / 8).to(dtype)[:, None, None].expand(-1, 1, D).contiguous()  # ones . k / sqrt(64) = 8 k
    v = torch.where(score == 0, 1.0, -1.0).to(dtype)[:, None, None].expand(-1, 1, D).contiguous()
    s = dict(q=torch.ones((B, 1, 1, D), dtype=dtype, device=DEV), k_cache=k, v_cache=v,
             slot_table=torch.arange(c + 1, dtype=torch.int32, device=DEV).repeat(B, 1),
             committed=torch.full((B,), c, dtype=torch.int32, device=DEV))
    got = sv.spec_verify_attention(**s, want_lse=True)
    one = {n: s[n][:1] for n in ("q", "slot_table", "committed")}
    out, lse, tol, lse_tol = plain64.attention(one["q"], k, v, one["slot_table"], one["committed"])
    for b in range(B):
        same(got.out[b:b + 1].double(), out, tol)
        same(got.lse[b:b + 1].double(), lse, lse_tol)
