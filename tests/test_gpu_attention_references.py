"""Every attention over scores so large that a reference times the scale keeps no digits behind the point, or passes fp32;
and infinite values among positions of next to no weight."""
import math

import pytest
import torch

import test_gpu_attention as ta
import test_gpu_attention_e4m3 as te
import test_gpu_chunk as th

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}
FORMS = ["nodes", "nodes e4m3", "chunk", "chunk e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def call(form, s, scale):
    if form == "nodes":
        return ta.call(s, scale=scale)
    if form == "nodes e4m3":
        return te.call(te.pack(s, *s["k_cache"].shape[1:]), scale=scale)
    return th.call(th.pack(s, form == "chunk e4m3"), scale=scale)


def by_class(form, dtype, c, N, Hq, scale, big, step, order, seed):
    """Positions' scores are big + step * m for m in -15 .. 15, exact in fp32; a value's dimension 15 + m is 1, the others
    0, so that a row's element is the weight of all positions of one m.  Returns what the kernel gives and that."""
    s = ta.make([c], N, Hq, 1, 64, dtype, seed=seed)
    L = c + N
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    # Few positions of each of the larger scores: each class has its share of the weight.
    m = (-15 + 30 * torch.rand(L, generator=g, device=DEV) ** 4).round().long()
    if order != "random":
        m = m.sort(descending=order == "falling").values
    at = s["slot_table"][0, :L].long()
    up = 2.0 ** (math.frexp(abs(big))[1] // 2)
    s["q"].zero_()
    s["q"][..., 0], s["q"][..., 1] = up, step / 4 if step < 64 else step / 64
    s["k_cache"][at], s["v_cache"][at] = 0, 0
    s["k_cache"][at, 0, 0] = big / up
    s["k_cache"][at, 0, 1] = (m * (4 if step < 64 else 64)).to(dtype)
    s["v_cache"][at, 0, 15 + m] = 1
    got = call(form, s, scale)
    score = big + step * m.double()
    seen = torch.arange(L, device=DEV) <= c + torch.arange(N, device=DEV)[:, None]
    w = torch.where(seen, score, -math.inf) * scale
    top = w.amax(1, keepdim=True)
    e = (w - top).exp()
    z = e.sum(1, keepdim=True)
    share = torch.zeros((N, 64), dtype=torch.float64, device=DEV)
    share.index_add_(1, 15 + m, e / z)
    return got, share, (top + z.log())[:, 0]


def compare(got, share, lse, dtype, L):
    # A weight, the sum of rounded ones and the result are rounded to the type, half a step each; the exponent's
    # product with log2(e) and 2^x are 2^-17 relative at exponents to 100, the sums (L / 16 + 96) 2^-24.  Weights in fp16 have
    # digits down to 2^-32 of the reference's, which may be 2^8 below the largest.
    u = HALF[dtype]
    tol = share * (3 * u + 2.0 ** -17 + (L / 16 + 96) * 2.0 ** -24) + (L * 2.0 ** -32 + 2.0 ** -24 if dtype is FP else 2.0 ** -80)
    off = float(((got.out[0].double() - share[:, None]).abs() / tol[:, None]).max())
    assert off <= 1.0, f"{off:.2f} of the tolerance"
    assert ((got.lse[0].double() - lse[:, None]).abs() <= 2.0 ** -21 * lse.abs()[:, None] + 2.0 ** -17).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("c,N,Hq", [(700, 8, 2), (700, 20, 4), (40000, 8, 2)])
@pytest.mark.parametrize("order", ["rising", "random", "falling"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_around_2_24(form, c, N, Hq, order, sign):
    """Differences of 4 times the scale, between tiles and between the parts of a request that many CTAs share.  With a
    scale of ln 2 the references times it lie on both sides of 2^24."""
    for dtype, scale in ((BF, 1.0), (FP, math.log(2.0)), (BF, math.log(2.0)), (BF, 0.125)):
        got, share, lse = by_class(form, dtype, c, N, Hq, scale, sign * 2.0 ** 24, 4, order, seed=c + N)
        compare(got, share, lse, dtype, c + N)


@pytest.mark.parametrize("form", ["nodes", "chunk"])
@pytest.mark.parametrize("c", [700, 40000])
@pytest.mark.parametrize("order", ["rising", "random", "falling"])
@pytest.mark.parametrize("sign", [1, -1])
def test_references_beyond_fp32(form, c, order, sign):
    """Scores are numbers of fp32, their products with the scale are not: the largest takes all."""
    got, share, _ = by_class(form, BF, c, 8, 2, 2.0 ** 60, sign * 2.0 ** 100, 2.0 ** 90, order, seed=c)
    assert ((share == 0) | (share == share.amax(1, keepdim=True))).all()
    compare(got._replace(lse=torch.zeros_like(got.lse)), share, torch.zeros_like(share[:, 0]), BF, c + 8)
    assert (got.lse == sign * math.inf).all()


@pytest.mark.parametrize("form", ["nodes", "chunk"])
@pytest.mark.parametrize("c", [300, 40000])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinite_values_of_little_weight(form, c, bad):
    """A value that is not finite shows in each row that sees it, though its weight is below fp32's numbers; the other
    elements are the others'."""
    s = ta.make([c], 4, 2, 1, 64, BF, seed=c)
    at = s["slot_table"][0, : c + 4].long()
    s["q"].zero_()
    s["q"][..., 0] = 1
    s["k_cache"][at] = 0
    s["k_cache"][at[c - 30], 0, 0] = 256  # (the others' weights: e^-256)
    s["v_cache"][at[5], 0, 7] = bad
    got = call(form, s, 1.0)
    assert not torch.isfinite(got.out[..., 7].float()).any()
    want = s["v_cache"][at[c - 30], 0].expand_as(got.out)
    rest = torch.arange(64, device=DEV) != 7
    assert torch.equal(got.out[..., rest], want[..., rest])
