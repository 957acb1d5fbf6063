"""spec_verify_attention with scores of any size that fp32 holds."""
import math

import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
from test_gpu_attention import BF, DEV, FP, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


@pytest.mark.parametrize("order", ["random", "rising", "falling", "below zero"])
@pytest.mark.parametrize("N,Hq", [(1, 2), (8, 4), (16, 4)])
@pytest.mark.parametrize("dtype,size", [(BF, 17), (BF, 24), (BF, 28), (BF, 35), (BF, 57), (BF, 110), (FP, 17), (FP, 24), (FP, 27)])
def test_the_largest_score_takes_all(dtype, size, N, Hq, order):
    """Scores are whole multiples of 2^(size - 7) and exact in fp32; the next to the largest is at least 2^10
    below it and has no weight.  The row is then one value, unrounded, and lse the score itself (a few
    roundings of 2^-24 relative)."""
    lengths = [1, 130, 700]
    s = make(lengths, N, Hq, 1, 64, dtype, seed=size)
    up = (size + 3) // 2
    s["q"].zero_()
    s["q"][..., 0] = 2.0 ** up
    g = torch.Generator(device=DEV)
    g.manual_seed(size)
    for b, c in enumerate(lengths):
        n = c + N
        grid = torch.randint(-100, 100, (n,), generator=g, device=DEV).float() / 128
        grid[int(torch.randint(0, c, (1,), generator=g, device=DEV))] = 101 / 128  # one, seen by all nodes
        if order == "below zero":
            grid -= 1.0  # (102 / 128 below zero and more: the same steps)
        elif order != "random":
            grid = grid.sort(descending=order == "falling").values
            if order == "rising":
                grid[c - 1], grid[c:] = 101 / 128, -1.0  # the largest is the last that all nodes see
        slot = s["slot_table"][b, :n].long()
        s["k_cache"][slot, 0, 0] = (grid * 2.0 ** (size + 3 - up)).to(dtype)
        score = s["k_cache"][slot, 0, 0].double() * 2.0 ** up / 8
        at = int(score[:c].argmax())
        assert int((score == score[at]).sum()) == 1
        got = call({**s, **{k: s[k][b:b + 1] for k in ("q", "slot_table", "committed")}})
        assert torch.equal(got.out[0], s["v_cache"][slot[at], 0].expand(N, Hq, 64))
        assert float((got.lse.double() - score[at]).abs().max()) <= 2.0 ** -21 * float(score[at].abs())


@pytest.mark.parametrize("dtype,size", [(BF, 17), (BF, 24), (BF, 35), (BF, 57), (BF, 110), (FP, 24), (FP, 27)])
@pytest.mark.parametrize("N,Hq", [(1, 2), (16, 4)])
def test_parts_of_a_request(dtype, size, N, Hq):
    """The same over a request that many CTAs share: parts whose references lie whole exponents apart, and one
    score that two parts hold alike, whose values then count half each."""
    c = 40000
    s = make([c], N, Hq, 1, 64, dtype, seed=size)
    up = (size + 3) // 2
    s["q"].zero_()
    s["q"][..., 0] = 2.0 ** up
    g = torch.Generator(device=DEV)
    g.manual_seed(size)
    grid = torch.randint(-100, 100, (c + N,), generator=g, device=DEV).float() / 128
    grid[1234], grid[38000] = 101 / 128, 101 / 128
    slot = s["slot_table"][0, : c + N].long()
    s["k_cache"][slot, 0, 0] = (grid * 2.0 ** (size + 3 - up)).to(dtype)
    got = call(s)
    a, b = s["v_cache"][slot[1234], 0].double(), s["v_cache"][slot[38000], 0].double()
    # The weights are alike and exact, so is their sum; a product with its reciprocal and the rounding of the row.
    tol = (2.0 ** -8 if dtype is BF else 2.0 ** -11) * ((a + b) / 2).abs() + 2.0 ** -21 * (a.abs() + b.abs()) + 2.0 ** -24
    assert bool(((got.out[0].double() - (a + b) / 2).abs() <= tol).all())
    lse = float(s["k_cache"][slot[1234], 0, 0].double() * 2.0 ** up / 8) + math.log(2.0)
    assert float((got.lse.double() - lse).abs().max()) <= 2.0 ** -21 * abs(lse)
