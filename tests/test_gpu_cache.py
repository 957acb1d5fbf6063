"""spec_verify_kv_append_ex and spec_verify_kv_read against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import plain64_cache as pc
import speculative_decoding_verification_verify_gb300 as sv
from plain64 import HALF_STEP, SMALLEST, path_of, rotate
from test_gpu_append import make

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def setup(B, N, Hq, Hkv, D, rot, dtype, e4m3, seed=0, norm=True, pad=0, **kw):
    s = make(B, N, Hq, Hkv, D, rot, dtype, seed=seed, **kw)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1)
    w = (1 + 0.2 * torch.randn((2, D), generator=g, device=DEV)).to(dtype)
    s["q_norm"], s["k_norm"] = (w[0].clone(), w[1].clone()) if norm else (None, None)
    if e4m3:
        slots, row = s["k_cache"].shape[0], pc.row_bytes(Hkv, D)
        pool = torch.randint(0, 256, (2, slots, row + pad), generator=g, device=DEV, dtype=torch.uint8)
        s["k_cache"], s["v_cache"] = pool[0, :, :row], pool[1, :, :row]
    return s


def call(s, **more):
    return sv.spec_verify_kv_append_ex(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_table"], s["committed"],
                                       s["cos_sin"], q_norm=s["q_norm"], k_norm=s["k_norm"], parents=s["parents"], **more)


def definition(s, x, weight, b, n, interleaved, eps):
    """A node's head vectors in 64 bits and, per element, how far 32 bits may be off.

    A head's sum of squares is at most 40 roundings off (16 terms a lane, two each, five exchanges), half of that in its
    root; the quotient, eps, the root (2 units) and the two products add 8: below 32 * 2^-24 = 2^-19 of a value.
    The rotation's products and sum are 2 roundings of their terms' magnitudes more."""
    x = x[b, n].double()
    d = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
        d = 2.0 ** -19
    rot = 0 if s["cos_sin"] is None else s["cos_sin"].shape[1]
    if rot:
        up = None if s["parents"] is None else s["parents"][b].tolist()
        cs = s["cos_sin"][int(s["committed"][b]) + len(path_of(up, n)) - 1].double()
        x, size = rotate(x, cs[: rot // 2], cs[rot // 2:], rot, interleaved)
    else:
        size = x.abs()
    return x, size * (d + 2.0 ** -22)


def check(s, interleaved=False, num_nodes=None, eps=1e-6):
    B, N, Hq, D = s["q"].shape
    Hkv, dt = s["k"].shape[2], s["q"].dtype
    u, tiny = HALF_STEP[dt], SMALLEST[dt]
    e4m3 = s["k_cache"].dtype is torch.uint8
    before = [s[x].clone() for x in ("k_cache", "v_cache")]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn = None if num_nodes is None else torch.tensor(num_nodes, dtype=torch.int32, device=DEV)
    got = call(s, interleaved=interleaved, num_nodes=nn, dev_status=status, eps=eps)
    torch.cuda.synchronize()
    assert int(status) == 0
    touched = torch.zeros(before[0].shape[0], dtype=torch.bool, device=DEV)
    for b in range(B):
        nodes = N if num_nodes is None else num_nodes[b]
        assert not got[b, nodes:].any()
        for n in range(nodes):
            y, d = definition(s, s["q"], s["q_norm"], b, n, interleaved, eps)
            assert ((got[b, n].double() - y).abs() <= d + u * (y.abs() + d) + tiny).all()
            slot = int(s["slot_table"][b, int(s["committed"][b]) + n])
            touched[slot] = True
            y, d = definition(s, s["k"], s["k_norm"], b, n, interleaved, eps)
            v = s["v"][b, n].double()
            if not e4m3:
                assert ((s["k_cache"][slot].double() - y).abs() <= d + u * (y.abs() + d) + tiny).all()
                assert torch.equal(s["v_cache"][slot], s["v"][b, n])
                continue
            row = s["k_cache"][slot]
            e = row[Hkv * D: Hkv * (D + 1)].int() - 127
            close = 1 + 2.0 ** -18
            assert ((e == pc.exponents(y, dt)) | (e == pc.exponents(y * close, dt)) | (e == pc.exponents(y / close, dt))).all()
            largest = pc.LARGEST * pc.two_to(e)[:, None]
            want = torch.minimum(y.abs(), largest) * y.sign()
            half = torch.maximum(2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=1e-300))) - 4), 2.0 ** (e.double()[:, None] - 10))
            off = (pc.decode(row, Hkv, D) - want).abs()
            assert (off <= half * (1 + 1e-6) + 2 * d).all()
            assert not row[Hkv * (D + 1):].any()
            assert torch.equal(s["v_cache"][slot], pc.encode(v, dt))
    for x, old in zip(("k_cache", "v_cache"), before):
        assert torch.equal(s[x][~touched].view(torch.uint8), old[~touched].view(torch.uint8))
    return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(32, 8, 128, 128), (4, 2, 64, 32), (3, 1, 80, 80), (6, 3, 96, 64), (2, 2, 16, 16),
                                          (5, 1, 256, 64), (2, 1, 512, 512), (7, 7, 112, 0)])
def test_sizes(dtype, e4m3, Hq, Hkv, D, rot):
    check(setup(2, 3, Hq, Hkv, D, rot, dtype, e4m3, seed=D))
    check(setup(2, 2, Hq, Hkv, D, rot, dtype, e4m3, seed=D, pad=48), interleaved=True)


@pytest.mark.parametrize("e4m3", [False, True])
def test_trees_and_ragged_nodes(e4m3):
    s = setup(4, 9, 8, 2, 128, 128, BF, e4m3, seed=3, tree=True)
    check(s, num_nodes=[9, 0, 1, 5])
    check(setup(1, 64, 2, 1, 64, 64, FP, e4m3, seed=4, tree=True))


def test_norms_apart():
    for q, k in ((True, False), (False, True), (False, False)):
        s = setup(2, 2, 4, 2, 64, 64, BF, True, seed=5)
        s["q_norm"], s["k_norm"] = s["q_norm"] if q else None, s["k_norm"] if k else None
        check(s)


def test_without_norms_the_bits_are_those_of_append():
    s = setup(3, 5, 8, 2, 128, 64, BF, False, seed=6, norm=False, tree=True)
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    want = sv.spec_verify_kv_append(s["q"], s["k"], s["v"], k, v, s["slot_table"], s["committed"], s["cos_sin"],
                                    parents=s["parents"])
    got = call(s)
    assert torch.equal(got, want)
    assert torch.equal(s["k_cache"].view(torch.int16), k.view(torch.int16))
    assert torch.equal(s["v_cache"].view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_every_value_of_16_bits(dtype):
    """All values of the type through the 8-bit rows: those of one magnitude, then each next to 1 and to the largest."""
    x = torch.arange(-32768, 32768, device=DEV, dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[torch.isfinite(x)]
    for other in (0.0, 1.0, float(torch.finfo(dtype).max)):
        rows = x.view(-1, 1).expand(-1, 16).clone()
        rows[:, 1::2] = other
        n = rows.shape[0] // 8 * 8
        v = rows[:n].view(1, n // 8, 8, 16)
        s = dict(q=v, k=v, v=v, slot_table=torch.randperm(n // 8, device=DEV)[None].int(),
                 committed=torch.zeros(1, dtype=torch.int32, device=DEV), cos_sin=None, parents=None, q_norm=None, k_norm=None,
                 k_cache=torch.zeros((n // 8, pc.row_bytes(8, 16)), dtype=torch.uint8, device=DEV),
                 v_cache=torch.zeros((n // 8, pc.row_bytes(8, 16)), dtype=torch.uint8, device=DEV))
        call(s)
        want = pc.encode(v[0], dtype)
        slots = s["slot_table"][0].long()
        assert torch.equal(s["k_cache"][slots], want) and torch.equal(s["v_cache"][slots], want)
        got = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["slot_table"], s["committed"], n // 8, kv_heads=8,
                                     head_dim=16, dtype=dtype)
        # Exact: four digits and an exponent of the type's own range (the smallest bf16 values are rounded once more).
        want = pc.decode(want, 8, 16)
        assert torch.equal(got.k[0].double(), want.to(dtype).double()) and torch.equal(got.v, got.k)
        if dtype is FP:
            assert torch.equal(got.k[0].double(), want)


def test_values_that_are_not_finite():
    s = setup(1, 1, 2, 3, 64, 0, BF, True, seed=7, norm=False)
    s["v"][0, 0, 0, 5], s["v"][0, 0, 1, 3], s["v"][0, 0, 1, 4] = math.nan, math.inf, -math.inf
    s["v"][0, 0, 2, :] = math.nan
    call(s)
    got = pc.decode(s["v_cache"][int(s["slot_table"][0, int(s["committed"][0])])], 3, 64)
    want = pc.decode(pc.encode(s["v"][0, 0], BF), 3, 64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got[2]).all()
    assert float(got[1, 3]) == 57344 and float(got[1, 4]) == -57344
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def test_zero_rows_and_eps():
    s = setup(1, 2, 2, 1, 64, 64, BF, True, seed=8)
    s["q"][:], s["k"][:], s["v"][:] = 0, 0, 0
    assert not check(s).any()
    check(setup(1, 2, 2, 1, 64, 64, BF, True, seed=8), eps=0.5)


def test_faults_are_the_nodes_own():
    def run(edit, code, bad):
        s = setup(3, 4, 4, 2, 64, 64, BF, True, seed=9, tree=True)
        old = s["k_cache"].clone()
        want = call(s)
        full = s["k_cache"].clone()
        s["k_cache"].copy_(old)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        nodes = s["slot_table"].gather(1, s["committed"].long()[:, None] + torch.arange(4, device=DEV))
        got = call(s, dev_status=status, **(edit(s) or {}))
        torch.cuda.synchronize()
        assert int(status) == code
        for b in range(3):
            for n in range(4):
                slot = int(nodes[b, n])
                if (b, n) in bad:
                    assert torch.isnan(got[b, n].float()).all() and torch.equal(s["k_cache"][slot], old[slot])
                else:
                    assert torch.equal(got[b, n], want[b, n]) and torch.equal(s["k_cache"][slot], full[slot])

    def slots(s):
        s["slot_table"][0, int(s["committed"][0]) + 2] = s["k_cache"].shape[0]
        s["slot_table"][1, int(s["committed"][1])] = -1

    run(slots, 6, {(0, 2), (1, 0)})

    def tree(s):
        s["parents"][2, 3] = 3

    run(tree, 3, {(2, n) for n in range(4)})

    def nodes(s):
        return dict(num_nodes=torch.tensor([4, 5, -1], dtype=torch.int32, device=DEV))

    run(nodes, 5, {(b, n) for b in (1, 2) for n in range(4)})

    def position(s):
        s["committed"][1] = s["slot_table"].shape[1] - 3

    run(position, 5, {(1, n) for n in range(4)})


# ---- reading back ---------------------------------------------------------------------------------
def pool_of(B, positions, Hkv, D, dtype, e4m3, seed=0, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    slots = B * positions + 7
    table = torch.randperm(slots, generator=g, device=DEV)[: B * positions].view(B, positions).int()
    x = torch.randn((2, slots, Hkv, D), generator=g, device=DEV).to(dtype)
    if not e4m3:
        return x[0], x[1], x[0].double(), x[1].double(), table
    rows = torch.full((2, slots, pc.row_bytes(Hkv, D) + pad), 0xFF, dtype=torch.uint8, device=DEV)
    rows = rows[:, :, : pc.row_bytes(Hkv, D)]
    rows.copy_(pc.encode(x, dtype))
    val = pc.decode(rows, Hkv, D)
    return rows[0], rows[1], val[0], val[1], table


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,N,Hkv,D", [(1, 1, 1, 16), (3, 37, 8, 128), (2, 130, 3, 80), (5, 9, 1, 512), (70, 3, 2, 64)])
def test_read(dtype, e4m3, B, N, Hkv, D):
    k, v, kv, vv, table = pool_of(B, N + 40, Hkv, D, dtype, e4m3, seed=N, pad=16)
    rng = np.random.default_rng(N)
    first, num = rng.integers(0, 40, B), rng.integers(0, N + 1, B)
    num[0] = N
    dev = lambda a: torch.from_numpy(a).int().to(DEV)  # noqa: E731
    for count in (None, num):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = sv.spec_verify_kv_read(k, v, table, dev(first), N, num_rows=None if count is None else dev(count),
                                     kv_heads=Hkv, head_dim=D, dtype=dtype, dev_status=status)
        assert int(status) == 0
        for b in range(B):
            n = N if count is None else int(count[b])
            slot = table[b, first[b]: first[b] + n].long()
            assert torch.equal(got.k[b, :n].double(), kv[slot]) and torch.equal(got.v[b, :n].double(), vv[slot])
            assert not got.k[b, n:].any() and not got.v[b, n:].any()


def test_read_faults():
    k, v, kv, vv, table = pool_of(4, 20, 2, 64, BF, True)
    first = torch.tensor([3, -1, 15, 0], dtype=torch.int32, device=DEV)
    num = torch.tensor([6, 6, 6, 2], dtype=torch.int32, device=DEV)
    table[0, 5] = k.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.spec_verify_kv_read(k, v, table, first, 6, num_rows=num, kv_heads=2, head_dim=64, dtype=BF, dev_status=status)
    assert int(status) == 6
    assert torch.isnan(got.k[1:3].float()).all() and torch.isnan(got.v[1:3].float()).all()
    assert torch.isnan(got.k[0, 2].float()).all()
    for b, n in ((0, 0), (0, 1), (0, 3), (0, 5), (3, 0), (3, 1)):
        assert torch.equal(got.v[b, n].double(), vv[int(table[b, int(first[b]) + n])])
    assert not got.k[3, 2:].any()


def test_far_slots():
    """Rows beyond 2^32 bytes of the pool, from a stride that is not the row's."""
    Hkv, D = 8, 128
    row, slots, n = pc.row_bytes(Hkv, D), 2_100_000, 5
    pool = torch.zeros((slots, 2, row + 16), dtype=torch.uint8, device=DEV)
    k, v = pool[:, 0, :row], pool[:, 1, :row]
    table = torch.arange(slots - n, slots, device=DEV)[None].int()
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = setup(1, n, 8, Hkv, D, 128, BF, False, seed=11, committed=[0], max_pos=n)
    s.update(k_cache=k, v_cache=v, slot_table=table)
    check(s)
    got = sv.spec_verify_kv_read(k, v, table, zero, n, kv_heads=Hkv, head_dim=D, dtype=BF)
    assert torch.equal(got.v[0].double(), pc.decode(pc.encode(s["v"][0], BF), Hkv, D))
    assert torch.equal(got.k[0].double(), pc.decode(k[slots - n:], Hkv, D))


def test_streams_and_graphs():
    s = setup(2, 3, 8, 2, 128, 128, BF, True, seed=12)
    old = s["k_cache"].clone()
    want, rows = call(s), None
    rows = s["k_cache"].clone()
    zero = s["committed"]
    back = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["slot_table"], zero, 3, kv_heads=2, head_dim=128, dtype=BF)
    side = torch.cuda.Stream()
    s["k_cache"].copy_(old)
    side.wait_stream(torch.cuda.current_stream())
    got = call(s, stream=side)
    again = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["slot_table"], zero, 3, kv_heads=2, head_dim=128, dtype=BF,
                                   stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(s["k_cache"], rows) and torch.equal(again.k, back.k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(s)
        again = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["slot_table"], zero, 3, kv_heads=2, head_dim=128,
                                       dtype=BF)
    for _ in range(2):
        s["k_cache"].copy_(old)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(s["k_cache"], rows) and torch.equal(again.k, back.k)


def test_compaction_moves_8_bit_rows():
    """An accepted path's rows with their powers of two, by spec_verify_kv_compact as it is."""
    B, N, Hkv, D = 3, 6, 2, 64
    s = setup(B, N, 4, Hkv, D, 64, BF, False, seed=13, tree=True)
    row, slots = pc.row_bytes(Hkv, D), s["k_cache"].shape[0]
    pool = torch.zeros((2, slots, row), dtype=torch.uint8, device=DEV)
    s.update(k_cache=pool[0], v_cache=pool[1])
    table = torch.arange(slots, device=DEV)[torch.randperm(slots, device=DEV)].int()
    P = slots // B
    s["slot_table"] = table[: B * P].view(B, P).contiguous()
    s["committed"] = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    s["cos_sin"] = None
    call(s)
    nodes = [pool[:, s["slot_table"][b, int(s["committed"][b]):][:N].long()].clone() for b in range(B)]
    index = torch.tensor([[0, 2, 5, -1, -1, -1], [0, 1, -1, -1, -1, -1], [0, 3, 4, 5, -1, -1]], dtype=torch.int32, device=DEV)
    length = torch.tensor([2, 1, 3], dtype=torch.int32, device=DEV)
    out, status = sv.spec_verify_kv_compact(pool, s["slot_table"], s["committed"], index, length, stacked=True)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b in range(B):
        n = int(length[b]) + 1
        c = int(s["committed"][b])
        assert int(out[b]) == c + n
        got = pool[:, s["slot_table"][b, c: c + n].long()]
        assert torch.equal(got, nodes[b][:, index[b, :n].long()])
