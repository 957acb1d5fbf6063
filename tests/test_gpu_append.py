"""spec_verify_kv_append against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
from plain64 import HALF_STEP, SMALLEST, path_of, rotate

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def random_parents(B, N, rng):
    p = np.full((B, N), -1, np.int32)
    for j in range(1, N):
        p[:, j] = rng.integers(max(0, j - 5), j, B)
    return p


def table_of(positions, rot, base=10000.0):
    freq = base ** (-np.arange(0, rot, 2) / rot)
    angle = np.arange(positions)[:, None] * freq
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(DEV)


def make(B, N, Hq, Hkv, D, rot, dtype, seed=0, committed=None, tree=False, max_pos=None, fused=True):
    rng = np.random.default_rng(seed)
    committed = rng.integers(0, 50, B) if committed is None else np.asarray(committed)
    max_pos = int(committed.max()) + N + 3 if max_pos is None else max_pos
    slots = B * N + 9
    table = np.full((B, max_pos), -7, np.int32)  # entries that the operator must not follow
    perm = rng.permutation(slots)[: B * N].reshape(B, N)
    for b in range(B):
        table[b, committed[b]:committed[b] + N] = perm[b]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    qkv = torch.randn((B, N, W + (24 if fused else 0)), generator=g, device=DEV).to(dtype)
    q, k, v = (t.unflatten(2, (-1, D)) for t in qkv[..., :W].split([Hq * D, Hkv * D, Hkv * D], 2))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().to(DEV)  # noqa: E731
    return dict(q=q, k=k, v=v, k_cache=torch.randn((slots, Hkv, D), generator=g, device=DEV).to(dtype),
                v_cache=torch.randn((slots, Hkv, D), generator=g, device=DEV).to(dtype), slot_table=t(table),
                committed=t(committed), cos_sin=table_of(max_pos + 2, rot) if rot else None,
                parents=t(random_parents(B, N, rng)) if tree else None)


def call(s, **more):
    kw = {k: s[k] for k in ("parents",) if s.get(k) is not None}
    return sv.spec_verify_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_table"], s["committed"],
                                    s["cos_sin"], **kw, **more)


def check(s, interleaved=False, num_nodes=None):
    """Run it and compare the queries and the whole of both caches."""
    B, N, Hq, D = s["q"].shape
    dt = s["q"].dtype
    u, tiny = HALF_STEP[dt], SMALLEST[dt]
    rot = 0 if s["cos_sin"] is None else s["cos_sin"].shape[1]
    k0, v0 = s["k_cache"].clone(), s["v_cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn = None if num_nodes is None else torch.tensor(num_nodes, dtype=torch.int32, device=DEV)
    got = call(s, interleaved=interleaved, num_nodes=nn, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    want_k, want_v = k0.double(), v0.double()
    tol_k = torch.zeros_like(want_k)
    for b in range(B):
        c = int(s["committed"][b])
        up = None if s["parents"] is None else s["parents"][b].tolist()
        nodes = N if num_nodes is None else num_nodes[b]
        for n in range(N):
            if n >= nodes:
                assert not got[b, n].any()
                continue
            pos = c + len(path_of(up, n)) - 1
            slot = int(s["slot_table"][b, c + n])
            for x, is_q in ((s["q"][b, n].double(), True), (s["k"][b, n].double(), False)):
                if rot:
                    cs = s["cos_sin"][pos].double()
                    y, size = rotate(x, cs[: rot // 2], cs[rot // 2:], rot, interleaved)
                    # two products and their sum in fp32 (three roundings at most), one rounding to the type
                    tol = u * y.abs() + 3 * 2.0 ** -24 * size + tiny
                    tol[..., rot:] = 0
                else:
                    y, tol = x, torch.zeros_like(x)
                if is_q:
                    assert ((got[b, n].double() - y).abs() <= tol).all()
                else:
                    want_k[slot], tol_k[slot] = y, tol
            want_v[slot] = s["v"][b, n].double()
    assert ((s["k_cache"].double() - want_k).abs() <= tol_k).all()
    assert torch.equal(s["v_cache"].double(), want_v)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot", [(1, 1, 32, 8, 128, 128), (3, 5, 6, 2, 64, 64), (2, 9, 7, 1, 80, 32),
                                              (5, 2, 3, 3, 96, 96), (1, 130, 4, 2, 128, 64), (2, 3, 1, 1, 16, 16),
                                              (2, 3, 2, 1, 256, 256), (2, 4, 4, 2, 128, 0)])
def test_chain(dtype, B, N, Hq, Hkv, D, rot):
    for interleaved in (False, True):
        check(make(B, N, Hq, Hkv, D, rot, dtype, seed=N), interleaved)


@pytest.mark.parametrize("N", [1, 2, 8, 33, 64])
def test_tree_positions_go_by_depth_and_slots_by_node(N):
    check(make(4, N, 4, 2, 64, 64, BF, seed=N, tree=True))


def test_ragged_nodes_and_contiguous_rows():
    check(make(4, 6, 8, 4, 64, 32, BF, seed=1, tree=True, fused=False), num_nodes=[6, 0, 1, 4])
    check(make(3, 70, 2, 1, 64, 64, FP, seed=2, fused=False), True, num_nodes=[70, 69, 0])


def test_far_positions():
    """Positions around 2^17: the table holds what fp32 angles could not."""
    check(make(2, 3, 2, 2, 128, 128, BF, seed=3, committed=[131072, 0]))


def test_a_prompt_of_odd_length_from_position_zero():
    check(make(2, 257, 2, 1, 64, 64, FP, seed=4, committed=[0, 0], max_pos=257))


def test_strided_caches_and_far_slots():
    """K and V interleaved in one pool of more than 2^32 bytes: slot strides, and offsets beyond 32 bits."""
    s = make(2, 4, 4, 8, 128, 128, BF, seed=5)
    slots = 1_100_000
    pool = torch.zeros((slots, 2, 8, 128), dtype=BF, device=DEV)
    st = s["slot_table"].clone()
    for b in range(2):
        c = int(s["committed"][b])
        st[b, c:c + 4] = torch.tensor([slots - 1 - 4 * b - i for i in range(4)], dtype=torch.int32)
    q = call(dict(s, k_cache=pool[:, 0], v_cache=pool[:, 1], slot_table=st))
    small = call(s)
    assert torch.equal(q, small)
    for b in range(2):
        c = int(s["committed"][b])
        a, z = st[b, c:c + 4].long(), s["slot_table"][b, c:c + 4].long()
        assert torch.equal(pool[a, 0], s["k_cache"][z]) and torch.equal(pool[a, 1], s["v_cache"][z])
    assert not pool[: slots - 8].any()


def test_faults_leave_slots_alone():
    def run(edit, codes, bad_rows):
        s = make(4, 4, 2, 1, 64, 64, BF, seed=6, committed=[5, 6, 7, 8], tree=True)
        more = edit(s) or {}
        k0, v0 = s["k_cache"].clone(), s["v_cache"].clone()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = call(s, dev_status=status, **more)
        assert int(status) == codes
        nan = torch.isnan(got.float()).all(-1).all(-1).cpu()
        want = torch.zeros((4, 4), dtype=torch.bool)
        for b, n in bad_rows:
            want[b, n] = True
        assert torch.equal(nan, want)
        good = s["slot_table"].clone()
        changed = (s["k_cache"] != k0).any(-1).any(-1)
        for b in range(4):
            for n in range(4):
                slot = int(good[b, int(s["committed"][b]) + n]) if 0 <= int(s["committed"][b]) + n < good.shape[1] else -1
                if 0 <= slot < changed.numel():
                    assert bool(changed[slot]) != bool(want[b, n])
        assert int(changed.sum()) == 16 - len(bad_rows)
        assert int((s["v_cache"] != v0).any(-1).any(-1).sum()) == 16 - len(bad_rows)

    def bad_slot(s):
        s["slot_table"][1, 6 + 2] = s["k_cache"].shape[0]
        s["slot_table"][2, 7] = -1

    run(bad_slot, 6, [(1, 2), (2, 0)])

    def bad_tree(s):
        s["parents"][3, 2] = 2

    run(bad_tree, 3, [(3, n) for n in range(4)])

    def bad_length(s):
        s["committed"][0] = s["slot_table"].shape[1] - 3

    run(bad_length, 5, [(0, n) for n in range(4)])

    def bad_nodes(s):
        return dict(num_nodes=torch.tensor([4, 5, 4, 4], dtype=torch.int32, device=DEV))

    run(bad_nodes, 5, [(1, n) for n in range(4)])


def test_nan_and_infinity_pass_through():
    s = make(1, 3, 2, 1, 64, 32, BF, seed=7)
    s["v"][0, 1, 0, 5] = math.inf
    s["k"][0, 2, 0, 40] = math.nan  # past the rotated part
    call(s)
    c = int(s["committed"][0])
    slot = s["slot_table"][0, c:c + 3].long()
    assert torch.isinf(s["v_cache"][slot[1], 0, 5]) and torch.isnan(s["k_cache"][slot[2], 0, 40])
    assert torch.isnan(s["k_cache"][slot].float()).sum() == 1


def test_streams_graphs_and_refusals():
    s = make(2, 3, 4, 2, 64, 64, BF, seed=8)
    want, k = call(s), s["k_cache"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    s["k_cache"].zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    written = s["k_cache"].any(-1).any(-1)
    assert torch.equal(out, want) and torch.equal(s["k_cache"][written], k[written]) and int(written.sum()) == 6
    with pytest.raises(TypeError):
        call(dict(s, k=s["k"].half()))
    with pytest.raises(TypeError):
        call(dict(s, q=s["q"].float(), k=s["k"].float(), v=s["v"].float()))
    with pytest.raises(ValueError):
        call(dict(s, q=s["q"].transpose(1, 2)))
    with pytest.raises(ValueError):
        call(dict(s, v_cache=s["v_cache"][:-1]))
    with pytest.raises(ValueError):
        call(dict(s, committed=s["committed"][:1]))
    with pytest.raises(ValueError):
        call(s, q_out=out[:1])
    with pytest.raises(sv.SpecVerifyError):
        call(dict(s, cos_sin=torch.zeros((9, 24), device=DEV)))  # rotary_dim not a multiple of 16
    with pytest.raises(sv.SpecVerifyError):  # a base that is not 16-byte aligned
        shifted = torch.zeros(s["q"].numel() + 1, dtype=BF, device=DEV)[1:].view(s["q"].shape)
        call(dict(s, q=shifted))
