"""The 8-bit cache at the ends of the types' ranges."""
import math

import pytest
import torch

import plain64_cache as pc
import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_cache as tc
from plain64 import rotate

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 32])
def test_infinite_keys_saturate(dtype, interleaved, rot):
    """An infinity in either place of a pair, in both, and where nothing is rotated: what is infinite after the rotation
    is 57344 with its sign, and only an infinity less another is NaN."""
    s = tc.setup(1, 1, 2, 6, 64, rot, dtype, True, seed=rot, norm=False, committed=[3])
    i = torch.arange(rot // 2, device=DEV)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    k = s["k"][0, 0]
    k[0, a[3]], k[1, b[5]], k[2, a[0]], k[2, b[0]] = math.inf, -math.inf, math.inf, math.inf
    k[3, a[1]], k[3, b[2]], k[3, 63] = -math.inf, math.inf, math.nan
    k[4, 62] = -math.inf
    tc.call(s, interleaved=interleaved)
    cs = s["cos_sin"][3].double()
    assert (cs != 0).all()
    y, size = rotate(k.double(), cs[: rot // 2], cs[rot // 2:], rot, interleaved)
    row = s["k_cache"][int(s["slot_table"][0, 3])]
    got = pc.decode(row, 6, 64)
    infinite, fine = torch.isinf(y), torch.isfinite(y)
    assert int(infinite[:4].sum()) >= 6
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    assert torch.equal(got[infinite], pc.LARGEST * 2.0 ** pc.HI * y[infinite].sign())
    e = row[6 * 64: 6 * 65].int() - 127
    assert torch.equal(e[infinite.any(1)], torch.full_like(e[infinite.any(1)], pc.HI))
    # Half a step of four digits, the smallest step 2^(e - 9); three roundings of fp32 before.
    half = torch.maximum(y.abs() * 2.0 ** -4, 2.0 ** (e.double()[:, None] - 10)) + 2.0 ** -22 * size
    assert ((got - y).abs() <= half)[fine].all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_norms_whose_factors_pass_fp32(e4m3):
    """The root's reciprocal times the weight is beyond fp32; the values are not."""
    for seed, up in ((1, 100), (2, 66)):
        s = tc.setup(2, 2, 4, 2, 64, 64, BF, e4m3, seed=seed)
        for x in ("q", "k"):
            s[x].mul_(2.0 ** -60)
            s[x][..., 5::16] *= 2.0 ** -60
            s[x + "_norm"].mul_(2.0 ** up)
        got = tc.check(s, eps=0.0)
        assert torch.isfinite(got.float()).all() and got.float().abs().max() > 2.0 ** (up - 2)


def test_the_smallest_values_are_the_same_for_all_who_read_them():
    """Keys whose finest digits lie below bf16's smallest subnormal: each kernel sees the same 16 bits.  An attention's
    lse over one position is the scaled product with its key: with a query of one dimension, an element of the key."""
    D = 64
    s = tc.setup(1, 1, D, 1, D, D, BF, True, seed=3, norm=False, committed=[0])
    s["cos_sin"] = tc.make(1, 1, 1, 1, D, D, BF, committed=[40])["cos_sin"][7:8].contiguous()
    s["k"].mul_(2.0 ** -129)
    tc.call(s)
    back = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["slot_table"], s["committed"], 1, kv_heads=1, head_dim=D,
                                  dtype=BF).k[0, 0, 0].double()
    row = s["k_cache"][int(s["slot_table"][0, 0])]
    stored = pc.decode(row, 1, D)[0]
    assert int(((stored * 2.0 ** 133) % 1 != 0).sum()) > 4
    assert ((back - stored).abs() < 2.0 ** -133).all()
    q = torch.eye(D, device=DEV).mul(2.0 ** 100).to(BF).view(1, 1, D, D)
    for f in (sv.spec_verify_attention_e4m3, sv.spec_verify_attention_chunk):
        lse = f(q, s["k_cache"], s["v_cache"], s["slot_table"], s["committed"], kv_heads=1, scale=2.0 ** 40, want_lse=True).lse
        seen = lse[0, 0].double() / 2.0 ** 140
        # The product is exact; the scale's and the logarithm's base's roundings are a few of 2^-24 of scores from 2^7 on.
        assert ((seen - back).abs() <= 2.0 ** -21 * back.abs()).all()
