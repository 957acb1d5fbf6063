"""spec_verify_attention against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import plain64
import speculative_decoding_verification_verify_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def make(committed, N, Hq, Hkv, D, dtype=BF, seed=0, tree=False, q_scale=2.0, extra=5, max_pos=None):
    """Random nodes over a cache whose slots are in random order; slots that nobody holds are NaN."""
    rng = np.random.default_rng(seed)
    B = len(committed)
    max_pos = max(committed) + N + 3 if max_pos is None else max_pos
    slots = B * max_pos + extra
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    table = torch.randperm(slots, generator=g, device=DEV)[: B * max_pos].view(B, max_pos).int()
    k = torch.randn((slots, Hkv, D), generator=g, device=DEV).to(dtype)
    v = torch.randn((slots, Hkv, D), generator=g, device=DEV).to(dtype)
    held = torch.zeros(slots, dtype=torch.bool, device=DEV)
    for b, c in enumerate(committed):
        held[table[b, : c + N].long()] = True
    k[~held], v[~held] = math.nan, math.nan
    parents = None
    if tree:
        p = np.full((B, N), -1, np.int32)
        for j in range(1, N):
            p[:, j] = rng.integers(max(0, j - 4), j, B)
        parents = torch.from_numpy(p).to(DEV)
    q = (torch.randn((B, N, Hq, D), generator=g, device=DEV) * q_scale).to(dtype)
    return dict(q=q, k_cache=k, v_cache=v, slot_table=table,
                committed=torch.tensor(committed, dtype=torch.int32, device=DEV), parents=parents)


def call(s, **more):
    return sv.spec_verify_attention(s["q"], s["k_cache"], s["v_cache"], s["slot_table"], s["committed"],
                                    parents=s["parents"], want_lse=True, **more)


def check(s, num_nodes=None, scale=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn = None if num_nodes is None else torch.tensor(num_nodes, dtype=torch.int32, device=DEV)
    got = call(s, num_nodes=nn, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    out, lse, tol, lse_tol = plain64.attention(s["q"], s["k_cache"], s["v_cache"], s["slot_table"], s["committed"],
                                               s["parents"], num_nodes, scale)
    same(got.out.double(), out, tol)
    same(got.lse.double(), lse, lse_tol)
    return got


def same(got, want, tol):
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    off = ((got - want).abs() / tol.clamp(min=1e-300))[fine]
    if off.numel():
        assert off.max() <= 1.0, f"{float(off.max()):.3f} of the tolerance"


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 32, 8, 128), (8, 32, 8, 128), (1, 4, 4, 64), (5, 7, 1, 64), (3, 6, 2, 80),
                                        (4, 5, 1, 96), (2, 16, 1, 112), (16, 8, 1, 128), (64, 2, 1, 128)])
def test_chain_lengths(dtype, N, Hq, Hkv, D):
    check(make([0, 1, 31, 127, 128, 129, 400], N, Hq, Hkv, D, dtype, seed=N + D))


@pytest.mark.parametrize("N,G", [(2, 1), (7, 3), (8, 4), (17, 2), (33, 8), (64, 4), (64, 8)])
def test_trees(N, G):
    check(make([0, 60, 125, 256], N, 2 * G, 2, 64 if N % 2 else 128, BF, seed=N, tree=True))


@pytest.mark.parametrize("L", [126, 127, 128, 254, 255, 256, 383, 511, 640])
def test_lengths_around_tiles(L):
    check(make([L, L + 1], 1, 4, 1, 128, BF, seed=L))
    check(make([L - 3, L - 1], 6, 2, 2, 64, FP, seed=L, tree=True))


def test_ragged_nodes_leave_empty_rows():
    s = make([100, 0, 37, 300, 0], 6, 8, 2, 128, BF, seed=1, tree=True)
    got = check(s, num_nodes=[6, 0, 1, 4, 3])
    assert not got.out[1].any() and (got.lse[1] == -math.inf).all()
    s = make([0, 0], 4, 2, 1, 64, FP, seed=2)
    check(s, num_nodes=[0, 0])


def test_many_requests_and_one_long_one():
    check(make([int(x) for x in np.random.default_rng(0).integers(0, 90, 200)], 1, 2, 1, 64, BF, seed=3))
    check(make([20000, 3, 5000], 4, 4, 1, 128, BF, seed=4))


def test_one_request_split_over_the_whole_gpu():
    check(make([131072 - 5], 5, 8, 2, 128, BF, seed=5, tree=True))


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_scores_far_apart(order):
    """Scores that rise along the cache raise the running maximum at every step; a spike leaves the rest
    nothing.  Weights span the whole of fp32's range."""
    s = make([1500, 700], 3, 4, 2, 64, BF, seed=6)
    s["q"] = torch.ones_like(s["q"])
    for b, c in enumerate([1500, 700]):
        j = torch.arange(c + 3, device=DEV).float()
        x = {"rising": j / 8, "falling": -j / 8, "spike": torch.where(j == c // 2, 60.0, 0.0)}[order]
        s["k_cache"][s["slot_table"][b, : c + 3].long()] = (x / 8)[:, None, None].expand(-1, 2, 64).to(BF)
    check(s)
    check(make([900], 4, 4, 1, 128, BF, seed=7, q_scale=40.0))


def test_what_a_node_does_not_see_has_no_part():
    """NaN and infinities in siblings' keys and values, in every kind of place of a tile."""
    for c in (0, 5, 124, 250):
        s = make([c], 8, 4, 2, 128, BF, seed=8)
        s["parents"] = torch.tensor([[-1, 0, 0, 1, 1, 2, 2, 5]], dtype=torch.int32, device=DEV)
        clean = call(s)
        slot = s["slot_table"][0].long()
        s["v_cache"][slot[c + 3], 0, 7] = math.inf
        s["v_cache"][slot[c + 4], 1] = math.nan
        s["v_cache"][slot[c + 6], 1, 100] = -math.inf
        s["k_cache"][slot[c + 6], 0, 3] = math.nan
        s["k_cache"][slot[c + 3], 1, 9] = math.inf
        got = call(s)
        for n in (0, 1, 2, 5, 7):  # nodes whose paths avoid 3, 4 and 6
            assert torch.equal(got.out[0, n], clean.out[0, n]) and torch.equal(got.lse[0, n], clean.lse[0, n])
        assert (got.out[0, 3, :2, 7] == math.inf).all()
        assert torch.isfinite(got.out[0, 3, :2].float()).sum() == 2 * 127
        assert torch.isnan(got.out[0, 4, 2:].float()).all() and torch.isfinite(got.out[0, 4, :2].float()).all()
        assert torch.isnan(got.out[0, 6, :2].float()).all() and torch.isnan(got.lse[0, 6, :2]).all()
        assert (got.out[0, 6, 2:, 100] == -math.inf).all()


def test_infinities_that_are_seen():
    s = make([300, 40], 2, 2, 1, 64, BF, seed=9)
    slot = s["slot_table"].long()
    s["v_cache"][slot[0, 17], 0, 3] = math.inf
    s["v_cache"][slot[0, 200], 0, 4] = -math.inf
    s["v_cache"][slot[1, 5], 0, 9] = math.nan
    got = call(s).out.float()
    assert (got[0, :, :, 3] == math.inf).all() and (got[0, :, :, 4] == -math.inf).all()
    assert torch.isnan(got[1, :, :, 9]).all()
    assert int((~torch.isfinite(got)).sum()) == 2 * 2 * 3


def test_strides_and_far_slots():
    """Queries inside a projection's rows, K and V interleaved in one pool beyond 2^32 bytes."""
    s = make([90, 17], 4, 8, 8, 128, BF, seed=10, tree=True)
    want = call(s)
    qkv = torch.randn((2, 4, 24 * 128 + 8), device=DEV).to(BF)
    q = qkv[..., : 8 * 128].unflatten(2, (8, 128))
    q.copy_(s["q"])
    n = s["k_cache"].shape[0]
    slots = 1_100_000
    pool = torch.full((slots, 2, 8, 128), math.nan, dtype=BF, device=DEV)
    pool[slots - n:, 0], pool[slots - n:, 1] = s["k_cache"], s["v_cache"]
    got = call(dict(s, q=q, k_cache=pool[:, 0], v_cache=pool[:, 1], slot_table=s["slot_table"] + (slots - n)))
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
        s["slot_table"][2, 302] = s["k_cache"].shape[0]

    run(slots, 6, (0, 2))

    def tree(s):
        s["parents"][1, 3] = 3
        s["parents"][3, 0] = 0

    run(tree, 3, (1, 3))

    def length(s):
        s["committed"][2] = s["slot_table"].shape[1] - 3
        s["committed"][0] = -1

    run(length, 5, (0, 2))

    def nodes(s):
        return dict(num_nodes=torch.tensor([4, -1, 4, 5], dtype=torch.int32, device=DEV))

    run(nodes, 5, (1, 3))


def test_slots_past_a_request_are_not_followed():
    s = make([33, 129], 3, 4, 1, 128, BF, seed=12)
    want = call(s)
    st = s["slot_table"].clone()
    for b, c in enumerate([33, 129]):
        st[b, c + 3:] = 2 ** 30
    got = call(dict(s, slot_table=st))
    assert torch.equal(got.out, want.out)


def test_same_bits_streams_graphs_and_a_shared_workspace():
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
    out = torch.zeros_like(want.out)
    ws = torch.zeros(sv.spec_verify_attention_workspace_bytes(3, 8, 8, 2, 128, s["slot_table"].shape[1]),
                     dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.out)
    # The workspace's counters are zero again: a verifier takes the same one.
    from speculative_decoding_verification_verify_gb300 import workloads as wl

    inp = wl.chain_tiny(DEV)
    a = sv.spec_verify_greedy(inp.logits, inp.drafts)
    need = sv.spec_verify_workspace_bytes(sv.MODE_GREEDY, *inp.shape)
    big = torch.zeros(max(need, ws.numel()), dtype=torch.uint8, device=DEV)
    call(s, workspace=big)
    b = sv.spec_verify_greedy(inp.logits, inp.drafts, workspace=big)
    assert torch.equal(a.out_tokens, b.out_tokens)
    assert not big[: 256 * 1024].any()


def test_after_an_append():
    """The pair as used: appended rows are what attention reads."""
    import test_gpu_append as ta

    a = ta.make(2, 5, 4, 2, 64, 64, BF, seed=14, committed=[130, 9], tree=True)
    s = make([130, 9], 5, 4, 2, 64, BF, seed=14, max_pos=a["slot_table"].shape[1])
    s["parents"] = a["parents"]
    s["q"] = sv.spec_verify_kv_append(a["q"], a["k"], a["v"], s["k_cache"], s["v_cache"], s["slot_table"], s["committed"],
                                      a["cos_sin"], parents=a["parents"])
    check(s)


def test_refusals():
    s = make([5], 2, 4, 2, 64, BF)
    with pytest.raises(TypeError):
        call(dict(s, q=s["q"].float()))
    with pytest.raises(TypeError):
        call(dict(s, k_cache=s["k_cache"].half()))
    with pytest.raises(ValueError):
        call(dict(s, v_cache=s["v_cache"][:, :1]))
    with pytest.raises(ValueError):
        call(dict(s, k_cache=s["k_cache"].transpose(1, 2)))
    with pytest.raises(ValueError):
        call(s, out=s["q"][:, :1])
    with pytest.raises(TypeError):
        call(dict(s, committed=s["committed"].long()))
    with pytest.raises(sv.SpecVerifyError):
        call(s, scale=-1.0)
    with pytest.raises(sv.SpecVerifyError):
        call(s, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)[:100])
    with pytest.raises(sv.SpecVerifyError):
        call(make([5], 65, 1, 1, 64, BF))
    with pytest.raises(sv.SpecVerifyError):
        call(make([5], 2, 4, 3, 64, BF))  # heads do not divide
    with pytest.raises(sv.SpecVerifyError):
        call(make([5], 2, 4, 2, 72, BF))


def test_long_rows_of_empty_requests_between_others():
    """Runs of requests without nodes (and with wrong lengths) before, between and after live ones: more
    segments without work than any part of the kernel lists ahead."""
    committed = [0] * 7 + [300] + [5] * 60 + [130, 1000] + [0] * 40 + [64]
    s = make(committed, 2, 8, 8, 64, BF, seed=15)
    nn = [2 if c in (300, 130, 1000, 64) else 0 for c in committed]
    check(s, num_nodes=nn)
    want = call(s, num_nodes=torch.tensor(nn, dtype=torch.int32, device=DEV))
    nn[20] = -1
    nn[-3] = 3
    got = call(s, num_nodes=torch.tensor(nn, dtype=torch.int32, device=DEV))
    bad = [20, len(nn) - 3]
    assert torch.isnan(got.out[bad].float()).all()
    keep = [b for b in range(len(nn)) if b not in bad]
    assert torch.equal(got.out[keep], want.out[keep])


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 2, 128), (1, 3, 3, 64), (8, 8, 2, 80), (16, 8, 2, 128)])
def test_many_parts_of_a_request(N, Hq, Hkv, D):
    """Requests cut into more parts than one join takes: every width of rows; the same bits from call to call;
    counters left at zero; a wrong slot in one part reaches all the rows, and only this request's."""
    s = make([30011, 17], N, Hq, Hkv, D, BF, seed=21, tree=N > 1)
    want = check(s)
    nbytes = sv.spec_verify_attention_workspace_bytes(2, N, Hq, Hkv, D, s["slot_table"].shape[1])
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    for _ in range(20):
        got = call(s, workspace=ws)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)
    torch.cuda.synchronize()
    assert not ws[: 256 * 1024].any()
    s["slot_table"][0, 20001] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = call(s, workspace=ws, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 6
    assert torch.isnan(got.out[0].float()).all() and torch.isnan(got.lse[0]).all()
    assert torch.equal(got.out[1], want.out[1]) and torch.equal(got.lse[1], want.lse[1])
    assert not ws[: 256 * 1024].any()


@pytest.mark.parametrize("N,G", [(16, 4), (8, 4), (3, 4)])
def test_infinities_beside_a_path(N, G):
    """Values that are not finite in one node's slot reach the nodes that see it, for every width of rows."""
    s = make([129, 250], N, 2 * G, 2, 128, BF, seed=22, tree=True)
    for b, c in enumerate([129, 250]):
        s["v_cache"][int(s["slot_table"][b, c + 1]), 1, 5] = math.inf
        s["v_cache"][int(s["slot_table"][b, c + N - 1]), 0, 100] = math.nan
    check(s)


@pytest.mark.parametrize("N", [1, 16])
def test_more_requests_than_threads(N):
    """Each thread of the prologue then counts several requests."""
    rng = np.random.default_rng(23)
    check(make([int(x) for x in rng.integers(0, 200, 1601)], N, 4, 1, 64, FP, seed=23, tree=N > 1),
          num_nodes=[int(x) for x in rng.integers(0, N + 1, 1601)])
