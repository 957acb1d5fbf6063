"""spec_verify_attention_chunk against its definition in 64 bits, over caches of 16-bit and of 8-bit rows."""
import math

import numpy as np
import pytest
import torch

import plain64_cache as pc
import plain64_chunk
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


def make(committed, N, Hq, Hkv, D, dtype=BF, e4m3=False, **kw):
    return pack(ta.make(committed, N, Hq, Hkv, D, dtype, **kw), e4m3)


def pack(s, e4m3):
    """The cache as the kernel takes it and as what it stands for; slots that nobody holds are NaN."""
    Hkv, D = s["k_cache"].shape[1:]
    held = ~torch.isnan(s["k_cache"]).all(-1).all(-1)
    for x in ("k", "v"):
        if e4m3:
            rows = pc.encode(s[x + "_cache"], s["q"].dtype)
            rows[~held] = 0xFF
            s[x + "_rows"], s[x + "_val"] = rows, pc.decode(rows, Hkv, D)
        else:
            s[x + "_rows"] = s[x + "_val"] = s[x + "_cache"]
    return s


def call(s, **more):
    return sv.spec_verify_attention_chunk(s["q"], s["k_rows"], s["v_rows"], s["slot_table"], s["committed"],
                                          kv_heads=s["k_val"].shape[1], want_lse=True, **more)


def check(s, num_nodes=None, scale=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn = None if num_nodes is None else torch.tensor(num_nodes, dtype=torch.int32, device=DEV)
    got = call(s, num_nodes=nn, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    out, lse, tol, lse_tol = plain64_chunk.chunk(s["q"], s["k_val"], s["v_val"], s["slot_table"], s["committed"], num_nodes,
                                                 scale)
    ta.same(got.out.double(), out, tol)
    ta.same(got.lse.double(), lse, lse_tol)
    return got


FORMS = [(BF, False), (FP, False), (BF, True), (FP, True)]


@pytest.mark.parametrize("dtype,e4m3", FORMS)
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 4, 1, 128), (1, 2, 2, 64), (3, 32, 8, 128), (65, 8, 2, 128), (130, 3, 1, 64),
                                        (300, 4, 4, 128), (257, 7, 1, 80), (150, 10, 2, 96), (70, 16, 1, 112)])
def test_lengths_and_heads(dtype, e4m3, N, Hq, Hkv, D):
    check(make([0, 1, 100, 127, 128, 500], N, Hq, Hkv, D, dtype, e4m3, seed=N + D))


@pytest.mark.parametrize("dtype,e4m3", FORMS)
def test_whole_prompts(dtype, e4m3):
    check(make([0], 1500, 4, 2, 128, dtype, e4m3, seed=1))
    check(make([0], 1111, 2, 1, 64, dtype, e4m3, seed=2))


@pytest.mark.parametrize("N", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257])
def test_rows_around_blocks(N):
    for G in (1, 2, 4):
        check(make([7, 121], N, G, 1, 64, FP if N % 2 else BF, seed=N))


@pytest.mark.parametrize("c", [0, 1, 62, 63, 64, 65, 126, 127, 128, 129, 254, 255, 256])
def test_positions_around_tiles(c):
    check(make([c], 66, 4, 2, 128, BF, seed=c))
    check(make([c], 5, 3, 1, 64, BF, True, seed=c))


@pytest.mark.parametrize("e4m3", [False, True])
def test_ragged_batches(e4m3):
    s = make([100, 0, 37, 3000, 0, 0], 333, 8, 2, 128, BF, e4m3, seed=3)
    got = check(s, num_nodes=[333, 0, 1, 200, 333, 64])
    assert not got.out[1].any() and (got.lse[1] == -math.inf).all()
    check(make([0, 0], 40, 2, 1, 64, FP, e4m3, seed=4), num_nodes=[0, 0])


def test_many_requests():
    rng = np.random.default_rng(5)
    check(make([int(x) for x in rng.integers(0, 90, 700)], 3, 2, 1, 64, BF, seed=5), num_nodes=[int(x) for x in rng.integers(0, 4, 700)])


@pytest.mark.parametrize("N,Hq,Hkv,e4m3", [(1, 1, 1, False), (40, 8, 2, True), (300, 8, 2, False), (90, 4, 1, False)])
def test_long_prefixes_are_split(N, Hq, Hkv, e4m3):
    check(make([60000], N, Hq, Hkv, 128, BF, e4m3, seed=N))
    check(make([30000, 5, 9000], N, Hq, Hkv, 64, FP, e4m3, seed=N))


@pytest.mark.parametrize("order", ["rising", "falling", "spike", "steep"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_far_apart(order, dtype):
    s = ta.make([1500, 700], 90, 4, 2, 64, dtype, seed=6)
    s["q"] = torch.ones_like(s["q"])
    for b, c in enumerate([1500, 700]):
        j = torch.arange(c + 90, device=DEV).float()
        x = {"rising": j / 8, "falling": -j / 8, "steep": j * 16, "spike": torch.where(j == c // 2, 60.0, 0.0)}[order]
        s["k_cache"][s["slot_table"][b, : c + 90].long()] = (x / 8)[:, None, None].expand(-1, 2, 64).to(dtype)
    check(pack(s, False))
    check(make([900], 70, 4, 1, 128, dtype, seed=7, q_scale=40.0))


def test_scores_beyond_the_references_digits():
    """Scores whose product with the scale has no digits left behind the point."""
    s = ta.make([300], 40, 2, 1, 64, BF, seed=8)
    s["q"], s["k_cache"] = torch.ones_like(s["q"]), torch.zeros_like(s["k_cache"])
    at = s["slot_table"][0].long()
    s["k_cache"][at[:340], 0, 0] = 2.0 ** 26
    s["k_cache"][at[5], 0, 1] = 1.0
    s["k_cache"][at[200], 0, 1] = 2.0
    got = call(pack(s, False), scale=1.0)
    v = s["v_cache"][at[:340], 0].double()
    # fp32 holds 2^26 + 1 and + 2 as 2^26: the weights are then equal; every row's mean.
    for n in (0, 39):
        want = v[: 300 + n + 1].mean(0)
        assert (got.out[0, n, 0].double() - want).abs().max() <= 2.0 ** -7 * v.abs().max()
    assert torch.isfinite(got.out.float()).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("c,N,G", [(0, 150, 2), (61, 130, 4), (120, 300, 1), (5000, 40, 4)])
def test_what_a_node_does_not_see_has_no_part(c, N, G, e4m3):
    s = make([c], N, 2 * G, 2, 128, BF, e4m3, seed=9)
    clean = call(s)
    slot = s["slot_table"][0].long()
    at = [N // 3, N // 3 + 1, N - 1]
    if e4m3:
        s["v_rows"][slot[c + at[0]], 7] = 0x7F
        s["v_rows"][slot[c + at[1]], 128 + 100] = 0xFF
        s["k_rows"][slot[c + at[2]], 3] = 0x7F
        bad = math.nan
    else:
        s["v_rows"][slot[c + at[0]], 0, 7] = math.inf
        s["v_rows"][slot[c + at[1]], 1, 100] = math.nan
        s["k_rows"][slot[c + at[2]], 0, 3] = math.nan
        bad = math.inf
    got = call(s)
    for n in range(N):
        o, w = got.out[0, n].clone(), clean.out[0, n].clone()
        if n == at[2]:
            assert torch.isnan(o[:G].float()).all() and torch.isnan(got.lse[0, n, :G]).all()
            o[:G], w[:G] = 0, 0
        else:
            assert torch.equal(got.lse[0, n], clean.lse[0, n])
        if n >= at[0]:
            x = o[:G, 7].float()
            assert n == at[2] or (torch.isnan(x).all() if math.isnan(bad) else (x == bad).all())
            o[:G, 7], w[:G, 7] = 0, 0
        if n >= at[1]:
            assert torch.isnan(o[G:, 100].float()).all()
            o[G:, 100], w[G:, 100] = 0, 0
        assert torch.equal(o, w), n


def test_infinities_that_are_seen():
    s = make([300, 40], 3, 2, 1, 64, BF, seed=9)
    slot = s["slot_table"].long()
    s["v_rows"][slot[0, 17], 0, 3] = math.inf
    s["v_rows"][slot[0, 200], 0, 4] = -math.inf
    s["v_rows"][slot[1, 5], 0, 9] = math.nan
    got = call(s).out.float()
    assert (got[0, :, :, 3] == math.inf).all() and (got[0, :, :, 4] == -math.inf).all()
    assert torch.isnan(got[1, :, :, 9]).all()
    assert int((~torch.isfinite(got)).sum()) == 3 * 2 * 3


@pytest.mark.parametrize("e4m3", [False, True])
def test_strides_and_far_slots(e4m3):
    s = make([90, 17], 70, 8, 8, 128, BF, e4m3, seed=10)
    want = call(s)
    qkv = torch.randn((2, 70, 24 * 128 + 8), device=DEV).to(BF)
    q = qkv[..., : 8 * 128].unflatten(2, (8, 128))
    q.copy_(s["q"])
    n, row = s["k_rows"].shape[0], s["k_rows"].shape[1:]
    slots = 2_100_000 if e4m3 else 1_100_000
    pool = torch.empty((slots, 2, *row), dtype=s["k_rows"].dtype, device=DEV)
    pool[slots - n:, 0], pool[slots - n:, 1] = s["k_rows"], s["v_rows"]
    got = call(dict(s, q=q, k_rows=pool[:, 0], v_rows=pool[:, 1], slot_table=s["slot_table"] + (slots - n)))
    assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_faults(e4m3):
    def run(edit, code, bad):
        s = make([140, 20, 300, 64], 80, 4, 2, 64, BF, e4m3, seed=11)
        want = plain64_chunk.chunk(s["q"], s["k_val"], s["v_val"], s["slot_table"], s["committed"])
        more = edit(s) or {}
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = call(s, dev_status=status, **more)
        torch.cuda.synchronize()
        assert int(status) == code
        for b in range(4):
            for n in range(80):
                if (b, n) in bad:
                    assert torch.isnan(got.out[b, n].float()).all() and torch.isnan(got.lse[b, n]).all()
                else:  # (the cuts of the batch's work are others without a request, so the bits may be)
                    ta.same(got.out[b, n].double(), want[0][b, n], want[2][b, n])
                    ta.same(got.lse[b, n].double(), want[1][b, n], want[3][b, n])

    def slots(s):
        s["slot_table"][0, 3] = -1
        s["slot_table"][2, 300 + 55] = s["k_rows"].shape[0]

    run(slots, 6, {(0, n) for n in range(80)} | {(2, n) for n in range(55, 80)})

    def length(s):
        s["committed"][2] = s["slot_table"].shape[1] - 79
        s["committed"][0] = -1

    run(length, 5, {(b, n) for b in (0, 2) for n in range(80)})

    def nodes(s):
        return dict(num_nodes=torch.tensor([80, -1, 80, 81], dtype=torch.int32, device=DEV))

    run(nodes, 5, {(b, n) for b in (1, 3) for n in range(80)})


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_heads_and_two_calls_at_once(e4m3):
    s, t = make([0, 400], 90, 160, 160, 64, BF, e4m3, seed=14), make([2000], 70, 8, 1, 128, BF, e4m3, seed=15)
    one, two = check(s), check(t)
    side = [torch.cuda.Stream() for _ in range(2)]
    for x in side:
        x.wait_stream(torch.cuda.current_stream())
    got = [(call(s, stream=side[0]), call(t, stream=side[1])) for _ in range(5)]
    torch.cuda.synchronize()
    for a, c in got:
        assert torch.equal(a.out, one.out) and torch.equal(c.out, two.out) and torch.equal(c.lse, two.lse)


def test_slots_past_a_request_are_not_followed():
    s = make([33, 129], 70, 4, 1, 128, BF, seed=12)
    want = call(s)
    st = s["slot_table"].clone()
    for b, c in enumerate([33, 129]):
        st[b, c + 70:] = 2 ** 30
    assert torch.equal(call(dict(s, slot_table=st)).out, want.out)


def test_chunks_of_a_prompt_are_the_prompt():
    """A prompt at once and in chunks behind what was written before: within two tolerances of each other."""
    s = make([0], 700, 8, 2, 64, BF, seed=13)
    whole = check(s)
    at = 0
    for n in (1, 255, 300, 144):
        c = torch.tensor([at], dtype=torch.int32, device=DEV)
        part = dict(s, q=s["q"][:, at: at + n].contiguous(), committed=c)
        check(part)
        got = call(part)
        assert (got.out.float() - whole.out[:, at: at + n].float()).abs().max() <= 2.0 ** -5
        at += n


def test_same_bits_streams_graphs_and_a_shared_workspace():
    s = make([5000, 3, 900], 100, 8, 2, 128, BF, seed=13)
    want = call(s)
    for _ in range(3):
        got = call(s)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(s, stream=side)
    side.synchronize()
    assert torch.equal(got.out, want.out)
    out = torch.zeros_like(want.out)
    ws = torch.zeros(sv.spec_verify_attention_chunk_workspace_bytes(3, 100, 8, 2, 128, s["slot_table"].shape[1]),
                     dtype=torch.uint8, device=DEV)
    t = ta.make([700, 0, 50], 8, 8, 2, 128, BF, seed=14, tree=True)
    nodes = ta.call(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, out=out, workspace=ws)
        again = ta.call(t, workspace=ws)  # one workspace serves both, its counters are left alone
        call(s, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.out) and torch.equal(again.out, nodes.out)
