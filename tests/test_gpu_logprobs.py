"""spec_verify_logprobs against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import plain64
import speculative_decoding_verification_verify_gb300 as sv
from speculative_decoding_verification_verify_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    torch.cuda.set_device(DEV)


def check(logits, tokens, top_n=0, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.spec_verify_logprobs(logits, tokens, top_n=top_n, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    want = plain64.logprobs(logits, tokens, top_n=top_n, **kw)
    near(got.logprobs, want["logprobs"], want["tol"])
    near(got.entropy, want["entropy"], want["entropy_tol"])
    assert torch.equal(got.ranks, want["ranks"])
    if top_n:
        assert torch.equal(got.top_ids, want["top_ids"])
        near(got.top_logprobs, want["top_logprobs"], want["top_tol"])
    else:
        assert got.top_ids is None and got.top_logprobs is None
    return got


def near(got, want, tol):
    got = got.double()
    want = want.masked_fill(want < -torch.finfo(torch.float32).max, -math.inf)  # beyond fp32
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine])
    off = ((got - want).abs() - tol)[fine]
    assert not off.numel() or off.max() <= 0, f"{float(off.max())} over the tolerance"


def rows(B, R, V, dtype, seed=0, scale=3.0, peak=8.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((B, R, V), generator=g, device=DEV) * scale
    x[..., 0] += peak
    tok = torch.randint(0, V, (B, R), generator=g, device=DEV).int()
    tok[:, 0] = 0
    return x[..., torch.randperm(V, generator=g, device=DEV)].to(dtype).contiguous(), tok


@pytest.mark.parametrize("dtype", [BF, FP32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 127, 1000, 2049, 4099, 8191, 8193, 32003, 128256, 151936])
def test_vocabularies(dtype, V):
    x, tok = rows(2, 3, V, dtype, seed=V)
    for top in (0, 1, 20):
        check(x, tok, top, temperature=0.8)


@pytest.mark.parametrize("B,R", [(1, 1), (1, 4), (3, 64), (64, 8), (300, 2)])
def test_batches(B, R):
    x, tok = rows(B, R, 5003, BF, seed=B)
    check(x, tok, 5)


@pytest.mark.parametrize("top", [1, 2, 3, 31, 32])
def test_alternatives(top):
    x, tok = rows(2, 2, 20011, BF, seed=top)
    check(x, tok, top)
    x, tok = rows(2, 2, 17, FP32, seed=top)  # more wanted than there are
    check(x, tok, top)


@pytest.mark.parametrize("dtype", [BF, FP32])
def test_orders_and_ties(dtype):
    """Rows in rising and falling order, all equal, and of few values: ties go to the lower token."""
    V = 30011
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    up = torch.linspace(-20, 20, V, device=DEV)
    few = torch.randint(0, 4, (V,), generator=g, device=DEV).float()
    last = torch.zeros(V, device=DEV)
    last[-25:] = 1.0
    x = torch.stack([up, up.flip(0), torch.zeros(V, device=DEV), few, last])[None].to(dtype).contiguous()
    check(x, torch.tensor([[V - 1, 5, 77, 1234, 12]], dtype=torch.int32, device=DEV), 32)


@pytest.mark.parametrize("dtype", [BF, FP32])
@pytest.mark.parametrize("T", [0.3, 1.0])
def test_masked_tokens(dtype, T):
    """Grammar masks of -inf and of the type's lowest value; rows with one or few tokens left, and one of
    nothing but lowest values."""
    low = torch.finfo(dtype).min
    x, tok = rows(1, 8, 9001, dtype, seed=2)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    hide = torch.rand((9001,), generator=g, device=DEV) < 0.95
    x[0, 0, hide], x[0, 1, hide] = -math.inf, low
    x[0, 2], x[0, 3] = -math.inf, low
    x[0, 2, 4000], x[0, 3, 4000] = 1.5, 1.5
    x[0, 4] = low
    x[0, 5] = -math.inf
    x[0, 5, 8990:] = 2.0
    x[0, 6, ::2] = -math.inf
    x[0, 7] = -math.inf
    x[0, 7, 3], x[0, 7, 4] = low, low / 2
    tok[0] = torch.tensor([int((~hide).nonzero()[3]), int((~hide).nonzero()[5]), 4000, 4000, 11, 8995, 7, 4])
    check(x, tok, 20, temperature=T)
    tok[0] = int(hide.nonzero()[0])  # masked tokens have probability 0 where the mask is -inf
    tok[0, 4:6] = 0
    tok[0, 3] = 4000
    tok[0, 1] = int((~hide).nonzero()[0])
    tok[0, 7] = 4
    check(x, tok, 3, temperature=T)


def test_peaked_and_flat():
    """Entropies near 0 and near ln V; logits of large size."""
    x, tok = rows(2, 2, 50021, FP32, seed=4, peak=60.0)
    check(x, tok, 4)
    x, tok = rows(2, 2, 50021, FP32, seed=5, scale=1e-3, peak=0.0)
    check(x, tok, 4)
    x, tok = rows(2, 2, 50021, FP32, seed=6)
    check(x + 3000.0, tok, 4)
    check(x * 100, tok, 4, temperature=2.0)


def test_absent_tokens_and_row_indices():
    x, tok = rows(5, 6, 3001, BF, seed=7)
    x[1, 2] = math.nan  # a row that nothing asks for
    g = torch.Generator().manual_seed(7)
    index = torch.stack([torch.randperm(6, generator=g) for _ in range(5)]).int().to(DEV)
    index[1] = torch.tensor([0, 2, 1, 4, 3, 5])  # the row of NaN stays with an entry whose token is absent
    tok[0, 3:], tok[1], tok[4, 0] = -1, -1, -1
    check(x, tok, 3)
    index[2, 4:] = -1
    tok[1, 0], index[1, 0] = 17, 5
    check(x, tok, 3, row_index=index)
    few = tok[:, :2].contiguous()
    check(x, few, 3)
    check(x, few, 3, row_index=index[:, 2:4].contiguous())


def test_temperatures_per_request():
    x, tok = rows(6, 3, 7001, BF, seed=8)
    t = torch.tensor([0.0, 0.25, 1.0, 3.0, 0.0, 0.7], device=DEV)
    check(x, tok, 2, temperatures=t)


def test_unaligned_logits():
    x, tok = rows(3, 3, 10007, BF, seed=9)
    for off in (1, 3, 7):
        buf = torch.empty(x.numel() + 8, dtype=BF, device=DEV)
        view = buf[off:off + x.numel()].view(x.shape)
        view.copy_(x)
        check(view, tok, 8)


def test_faults_are_the_entrys_own():
    x, tok = rows(2, 8, 5003, BF, seed=10)
    want = sv.spec_verify_logprobs(x, tok, top_n=3)
    x[0, 1, 70], x[0, 2, 5000], x[0, 3] = math.nan, math.inf, -math.inf
    tok[0, 4], tok[0, 5] = -2, 5003
    index = torch.arange(8, device=DEV).repeat(2, 1).int()
    index[0, 6], index[0, 7] = 8, -2
    bad = [1, 2, 3, 4, 5, 6, 7]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.spec_verify_logprobs(x, tok, row_index=index, top_n=3, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 2
    for b in range(2):
        for t in range(8):
            if b == 0 and t in bad:
                assert torch.isnan(got.logprobs[b, t]) and torch.isnan(got.entropy[b, t]) and int(got.ranks[b, t]) == -1
                assert (got.top_ids[b, t] == -1).all() and torch.isnan(got.top_logprobs[b, t]).all()
            else:
                for g, w in zip(got, want):
                    assert torch.equal(g[b, t], w[b, t])
    status.zero_()
    tok[0, 6:] = -1
    sv.spec_verify_logprobs(x[:, 6:].contiguous(), tok[:, 4:6].contiguous(), dev_status=status)
    assert int(status) == 1
    status.zero_()
    sv.spec_verify_logprobs(x[1:], tok[1:], temperatures=torch.tensor([-1.0], device=DEV), dev_status=status)
    assert int(status) == 2


def test_of_what_a_verification_emitted():
    """Chain and tree: the tokens and rows as the verifiers return them."""
    c = wl.chain_b64k7(DEV, B=16, k=5, V=5003)
    r = sv.spec_verify_rejection(c.logits, c.drafts, None, temperature=1.0, seed=3, offset=0)
    got = check(c.logits, r.out_tokens, 4)
    n = r.accept_len.cpu().numpy()
    assert np.array_equal((got.ranks > 0).sum(1).cpu().numpy(), n + 1)
    t = wl.tree_b48(DEV, B=9, N=8, V=4001)
    r = sv.spec_verify_tree(t.logits, t.node_tokens, t.parents, mode=0)
    got = check(t.logits, r.out_tokens, 4, row_index=r.accept_index)
    said = r.out_tokens >= 0
    assert (got.ranks[said] == 1).all() and torch.equal(got.top_ids[said][:, 0], r.out_tokens[said])


def test_same_bits_streams_graphs_and_a_shared_workspace():
    x, tok = rows(4, 4, 60013, BF, seed=11)
    want = sv.spec_verify_logprobs(x, tok, top_n=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (sv.spec_verify_logprobs(x, tok, top_n=20), sv.spec_verify_logprobs(x, tok, top_n=20, stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.zeros(sv.spec_verify_logprobs_workspace_bytes(4, 4, 60013, 20) + 512 * 1024, dtype=torch.uint8, device=DEV)
    out = torch.zeros((4, 4), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_verify_logprobs(x, tok, top_n=20, workspace=ws, logprobs=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.logprobs)
    assert not ws[: 256 * 1024].any()


def test_refusals():
    x, tok = rows(2, 3, 101, BF)
    with pytest.raises(TypeError):
        sv.spec_verify_logprobs(x.half(), tok)
    with pytest.raises(TypeError):
        sv.spec_verify_logprobs(x, tok.long())
    with pytest.raises(ValueError):
        sv.spec_verify_logprobs(x.transpose(0, 1), tok)
    with pytest.raises(ValueError):
        sv.spec_verify_logprobs(x, tok, row_index=tok[:, :2])
    with pytest.raises(ValueError):
        sv.spec_verify_logprobs(x, tok, logprobs=torch.zeros((2, 2), device=DEV))
    for kw in (dict(top_n=33), dict(temperature=-1.0), dict(temperature=float("nan")),
               dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_verify_logprobs(x, tok, **kw)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_verify_logprobs(x, torch.zeros((2, 4), dtype=torch.int32, device=DEV))  # more tokens than rows


@pytest.mark.parametrize("dtype", [BF, FP32])
def test_more_rows_than_are_listed_at_once(dtype):
    """Hundreds of rows for every CTA and of entries for every thread, a third of them absent."""
    B, T, V = 700, 64, 41
    x, tok = rows(B, T, V, dtype, seed=12)
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    absent = torch.rand((B, T), generator=g, device=DEV) < 0.33
    tok = tok.masked_fill(absent, -1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv.spec_verify_logprobs(x, tok, top_n=3, temperature=0.9, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    raw = x.double()
    d = raw / 0.9 - (raw / 0.9).amax(-1, keepdim=True)
    lnz = d.exp().sum(-1).log()
    at = tok.clamp(min=0).long()[..., None]
    base = 2.0 ** -20 + (V / 4096 + 32) * 2.0 ** -23
    w = d.gather(2, at)[..., 0]
    near(got.logprobs, torch.where(absent, 0.0, w - lnz), base + 2.0 ** -22 * (w.abs() + lnz))
    near(got.entropy, torch.where(absent, 0.0, lnz - (d.exp() * d).sum(-1) / lnz.exp()), base * (4 + 2 * lnz))
    ranks = 1 + (raw > raw.gather(2, at)).sum(-1)
    assert torch.equal(got.ranks.long(), torch.where(absent, 0, ranks))
    order = torch.sort(raw, dim=-1, descending=True, stable=True).indices[..., :3]
    assert torch.equal(got.top_ids.long(), torch.where(absent[..., None], -1, order))
    y = d.gather(2, order)
    near(got.top_logprobs, torch.where(absent[..., None], -math.inf, y - lnz[..., None]),
         base + 2.0 ** -22 * (y.abs() + lnz[..., None]))
