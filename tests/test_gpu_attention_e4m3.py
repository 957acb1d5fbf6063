"""spec_verify_attention_e4m3 against attention's definition in 64 bits over the values that the rows stand for."""
import math

import numpy as np
import pytest
import torch

import plain64
import plain64_cache as pc
import speculative_decoding_verification_verify_gb300 as sv
import test_gpu_attention as ta

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def make(committed, N, Hq, Hkv, D, dtype=BF, spread=True, **kw):
    """As the 16-bit test's, heads of different magnitudes; unheld slots are NaN rows with all bits set."""
    s = ta.make(committed, N, Hq, Hkv, D, dtype, **kw)
    if spread:
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        shape = s["v_cache"].shape[:2]
        s["v_cache"] *= 2.0 ** torch.randint(-6, 7, shape, generator=g, device=DEV)[..., None].to(dtype)
        s["k_cache"] *= 2.0 ** torch.randint(-2, 1, shape, generator=g, device=DEV)[..., None].to(dtype)
    return pack(s, Hkv, D)


def pack(s, Hkv, D):
    dt = s["q"].dtype
    held = ~torch.isnan(s["k_cache"]).all(-1).all(-1)
    for x in ("k", "v"):
        rows = pc.encode(s[x + "_cache"], dt)
        rows[~held] = 0xFF
        s[x + "_rows"] = rows
        s[x + "_val"] = torch.where(held[:, None, None], pc.decode(rows, Hkv, D), math.nan)
    return s


def call(s, **more):
    return sv.spec_verify_attention_e4m3(s["q"], s["k_rows"], s["v_rows"], s["slot_table"], s["committed"],
                                         kv_heads=s["k_val"].shape[1], parents=s["parents"], want_lse=True, **more)


def check(s, num_nodes=None, scale=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn = None if num_nodes is None else torch.tensor(num_nodes, dtype=torch.int32, device=DEV)
    got = call(s, num_nodes=nn, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    out, lse, tol, lse_tol = plain64.attention(s["q"], s["k_val"], s["v_val"], s["slot_table"], s["committed"],
                                               s["parents"], num_nodes, scale)
    ta.same(got.out.double(), out, tol)
    ta.same(got.lse.double(), lse, lse_tol)
    return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 32, 8, 128), (8, 32, 8, 128), (1, 4, 4, 64), (5, 7, 1, 64), (3, 6, 2, 80),
                                        (4, 5, 1, 96), (2, 16, 1, 112), (16, 8, 1, 128), (64, 2, 1, 128)])
def test_chain_lengths(dtype, N, Hq, Hkv, D):
    check(make([0, 1, 31, 127, 128, 129, 400], N, Hq, Hkv, D, dtype, seed=N + D))


@pytest.mark.parametrize("N,G", [(2, 1), (7, 3), (8, 4), (17, 2), (33, 8), (64, 4), (64, 8)])
def test_trees(N, G):
    check(make([0, 60, 125, 256], N, 2 * G, 2, 64 if N % 2 else 128, BF if N % 3 else FP, seed=N, tree=True))


@pytest.mark.parametrize("L", [126, 127, 128, 254, 255, 256, 383, 511, 640])
def test_lengths_around_tiles(L):
    check(make([L, L + 1], 1, 4, 1, 128, BF, seed=L))
    check(make([L - 3, L - 1], 6, 2, 2, 64, FP, seed=L, tree=True))


def test_ragged_nodes_many_requests_and_long_ones():
    got = check(make([100, 0, 37, 300, 0], 6, 8, 2, 128, BF, seed=1, tree=True), num_nodes=[6, 0, 1, 4, 3])
    assert not got.out[1].any() and (got.lse[1] == -math.inf).all()
    check(make([int(x) for x in np.random.default_rng(0).integers(0, 90, 200)], 1, 2, 1, 64, BF, seed=3))
    check(make([20000, 3, 5000], 4, 4, 1, 128, FP, seed=4))
    check(make([131072 - 5], 5, 8, 2, 128, BF, seed=5, tree=True))


@pytest.mark.parametrize("Hkv", [5, 76, 77, 160])
def test_more_heads_than_runs(Hkv):
    """A key head has CTAs of its own while there are enough of them."""
    check(make([100, 0, 300], 1, Hkv, Hkv, 64, BF, seed=Hkv))
    check(make([9000, 700], 3, 2 * Hkv, Hkv, 64, FP, seed=Hkv))


def test_magnitudes_of_the_whole_range():
    """Values of heads from 2^-60 to beyond the largest that a row holds."""
    for dtype, lo, hi in ((BF, -60, 14), (FP, -14, 13)):
        s = ta.make([300, 40], 3, 8, 8, 64, dtype, seed=6)
        p = torch.linspace(lo, hi, 8, device=DEV).round()
        s["v_cache"] = (s["v_cache"].double() * 2.0 ** p[:, None].double()).to(dtype)
        check(pack(s, 8, 64))


def test_what_a_node_does_not_see_has_no_part():
    for c in (0, 5, 124, 250):
        s = make([c], 8, 4, 2, 128, BF, seed=8, spread=False)
        s["parents"] = torch.tensor([[-1, 0, 0, 1, 1, 2, 2, 5]], dtype=torch.int32, device=DEV)
        clean = call(s)
        slot = s["slot_table"][0].long()
        s["v_rows"][slot[c + 4], :] = 0x7F                 # NaN, all of it
        s["v_rows"][slot[c + 6], 128 + 100] = 0xFF         # NaN in head 1
        s["k_rows"][slot[c + 6], 3] = 0x7F                 # and in head 0's key
        got = call(s)
        for n in (0, 1, 2, 3, 5, 7):  # nodes whose paths avoid 4 and 6
            assert torch.equal(got.out[0, n], clean.out[0, n]) and torch.equal(got.lse[0, n], clean.lse[0, n])
        assert torch.isnan(got.out[0, 4].float()).all()
        assert torch.isnan(got.out[0, 6, :2].float()).all() and torch.isnan(got.lse[0, 6, :2]).all()
        assert torch.isnan(got.out[0, 6, 2:, 100].float()).all()
        assert int(torch.isnan(got.out[0, 6, 2:].float()).sum()) == 2


def test_strides_and_far_slots():
    s = make([90, 17], 4, 8, 8, 128, BF, seed=10, tree=True)
    want = call(s)
    n, row = s["k_rows"].shape
    slots = 2_100_000
    pool = torch.full((slots, 2, row), 0xFF, dtype=torch.uint8, device=DEV)
    pool[slots - n:, 0], pool[slots - n:, 1] = s["k_rows"], s["v_rows"]
    got = call(dict(s, k_rows=pool[:, 0], v_rows=pool[:, 1], slot_table=s["slot_table"] + (slots - n)))
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


def test_faults_are_the_requests_own():
    def run(edit, code, bad):
        s = make([140, 20, 300, 64], 4, 4, 2, 64, BF, seed=11, tree=True)
        want = call(s)
        more = edit(s) or {}
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = call(s, dev_status=status, **more)
        torch.cuda.synchronize()
        assert int(status) == code
        for b in range(4):
            if b in bad:
                assert torch.isnan(got.out[b].float()).all() and torch.isnan(got.lse[b]).all()
            else:
                assert torch.equal(got.out[b], want.out[b]) and torch.equal(got.lse[b], want.lse[b])

    def slots(s):
        s["slot_table"][0, 3] = -1
        s["slot_table"][2, 302] = s["k_rows"].shape[0]

    run(slots, 6, (0, 2))

    def tree(s):
        s["parents"][1, 3] = 3
        s["parents"][3, 0] = 0

    run(tree, 3, (1, 3))

    def length(s):
        s["committed"][2] = s["slot_table"].shape[1] - 3
        s["committed"][0] = -1

    run(length, 5, (0, 2))


def test_same_bits_streams_and_graphs():
    s = make([5000, 3, 900], 8, 8, 2, 128, BF, seed=13, tree=True)
    want = call(s)
    for _ in range(3):
        got = call(s)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(s, stream=side)
    side.synchronize()
    assert torch.equal(got.out, want.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s)
    for _ in range(3):
        got.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
