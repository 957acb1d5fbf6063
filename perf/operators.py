"""The operators around one verification step, as cases to measure.

  append     spec_verify_kv_append: the verify forward's rotated keys and values into the paged cache
  attention  spec_verify_attention: the nodes' attention over that cache and over their ancestors
  logprobs   spec_verify_logprobs: what is answered beside the emitted tokens

`own` selects the form that `run` computes: the library's kernels, or the same operators in elementary
torch operations in 32 bits.  `exact` gives them in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # Plain decoding of one request: one new token, a short context; latency is what counts.
        dict(name="attention b1 n1", op="attention", dtype="bf16", B=1, N=1, Hq=32, Hkv=8, D=128, lo=701, hi=701,
             tree=False, ragged=False),
        # The tree-verification workload's cache: 48 requests of 8 nodes, contexts within 512 positions.
        dict(name="attention b48 tree8", op="attention", dtype="bf16", B=48, N=8, Hq=32, Hkv=8, D=128, lo=1, hi=504,
             tree=True, ragged=False),
        # The chain workload's batch (64 requests, 7 drafts) in a serving mix of context lengths.
        dict(name="attention b64 chain8 8k", op="attention", dtype="bf16", B=64, N=8, Hq=32, Hkv=8, D=128, lo=509,
             hi=8192, tree=False, ragged=True),
        # One request with a very long context and a wide tree: only a split over the length fills the GPU.
        dict(name="attention b1 tree16 128k", op="attention", dtype="bf16", B=1, N=16, Hq=32, Hkv=8, D=128, lo=131000,
             hi=131000, tree=True, ragged=False),
        # A small draft model decoding token by token for a batch: every head has its own keys.
        dict(name="attention b96 n1 d64", op="attention", dtype="fp16", B=96, N=1, Hq=12, Hkv=12, D=64, lo=1, hi=4001,
             tree=False, ragged=False),
        # One token of one request appended.
        dict(name="append b1 n1", op="append", dtype="bf16", B=1, N=1, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             lo=701, hi=701, tree=False),
        # The tree workload's nodes: positions by depth, slots by node.
        dict(name="append b48 tree8", op="append", dtype="bf16", B=48, N=8, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, lo=1, hi=504, tree=True),
        # Two prompts written at once, behind a long shared conversation; adjacent pairs, half of the head rotated.
        dict(name="append b2 n4097", op="append", dtype="fp16", B=2, N=4097, Hq=32, Hkv=8, D=128, rot=64,
             interleaved=True, lo=126000, hi=126000, tree=False),
        # One request's verified positions (k = 3) at the sampling temperature.
        dict(name="logprobs b1k3", op="logprobs", dtype="bf16", B=1, rows=4, V=128256, T=0.8, top=5, tree=False,
             ragged=False, masked=False),
        # Every position of the headline batch, with the most alternatives that serving interfaces give.
        dict(name="logprobs b64k7 top20", op="logprobs", dtype="bf16", B=64, rows=8, V=128256, T=1.0, top=20, tree=False,
             ragged=False, masked=False),
        # The emitted tokens of the tree batch alone, under grammar masks.
        dict(name="logprobs b48 tree8", op="logprobs", dtype="bf16", B=48, rows=8, V=151936, T=1.0, top=5, tree=True,
             ragged=True, masked=True),
        # A head with an odd vocabulary in 32 bits: no row but the first starts on a vector boundary.
        dict(name="logprobs fp32 v32003", op="logprobs", dtype="fp32", B=16, rows=5, V=32003, T=0.7, top=8, tree=False,
             ragged=True, masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "logprobs"])
    while True:
        if op == "logprobs":
            B, rows = _log_int(rng, 1, 64), rng.randint(1, 16)
            V = _log_int(rng, 1000, 160000)
            c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), B=B, rows=rows, V=V,
                     T=round(rng.uniform(0.5, 1.5), 2), top=rng.choice([0, 1, 5, 8, 20, 32]), tree=rng.random() < 0.4,
                     ragged=rng.random() < 0.5, masked=rng.random() < 0.3)
            if V == 3072 or B * rows * V * (2 if c["dtype"] == "bf16" else 4) > 512 * 128256 * 2:
                continue
            return c
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        D = rng.choice([64, 80, 96, 128, 128])
        B = _log_int(rng, 1, 64)
        tree = rng.random() < 0.5
        if 3072 in (Hkv * G * D, Hkv * D, (Hkv * G + 2 * Hkv) * D):
            continue
        if op == "append":
            N = _log_int(rng, 2, 64) if tree else _log_int(rng, 1, 4097)
            lo = _log_int(rng, 1, 100000)
            hi = _log_int(rng, lo, 120000)
            if N == 3072 or B * N * (G + 2) * Hkv * D > 2 * 4097 * 48 * 128:
                continue
            return dict(op=op, dtype=rng.choice(["bf16", "fp16"]), B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D,
                        rot=rng.choice([D, D, 32, 64]), interleaved=rng.random() < 0.4, lo=lo, hi=hi, tree=tree)
        N = rng.choice([1, 1, _log_int(rng, 2, 64)])
        hi = _log_int(rng, 1, 131072)
        lo = _log_int(rng, 1, hi)
        c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, lo=lo, hi=hi,
                 tree=tree and N > 1, ragged=rng.random() < 0.4)
        w = work(c)
        if w["bytes"] > 6.5e8 or w["flops"] > 7e10 or B * (hi + N) * Hkv * D > 64 * 8200 * 1024 \
                or B * Hkv * G * N * (hi + N) > 64 * 8200 * 256:
            continue
        return c


def _lengths(case):
    """(committed positions, nodes) of each request: the same lengths whatever the seed, in another order."""
    B, lo, hi, N = case["B"], case["lo"], case["hi"], case["N"]
    got = []
    for i in range(B):
        c = int(round(lo * (hi / lo) ** (i / (B - 1)))) if B > 1 else hi
        c += c == 3072
        got.append((c, 1 + (i * 7 + 2) % N if case.get("ragged") else N))
    return got


def _emitted(case):
    """Tokens emitted by each request of a logprobs case."""
    return [1 + (i * 5) % case["rows"] if case["ragged"] else case["rows"] for i in range(case["B"])]


def work(case):
    """Bytes that have to be read and written, and arithmetic, of one pass."""
    if case["op"] == "logprobs":
        n, elt = sum(_emitted(case)), 4 if case["dtype"] == "fp32" else 2
        out = case["B"] * case["rows"] * (4 + 12 + 8 * case["top"])
        return {"bytes": n * case["V"] * elt + out, "flops": 6 * n * case["V"]}
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    if case["op"] == "append":
        rows = B * N
        return {"bytes": rows * (2 * (Hq + 2 * Hkv) * D * 2 + 4) + B * N * case["rot"] * 4, "flops": 3 * rows * (Hq + Hkv) * D}
    cells = [(c + n, n) for c, n in _lengths(case)]
    kv = sum(t for t, _ in cells)
    return {"bytes": kv * (2 * Hkv * D * 2 + 4) + 2 * B * N * Hq * D * 2 + B * N * Hq * 4,
            "flops": sum(4 * t * n for t, n in cells) * Hq * D}


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _parents(B, N, g):
    """Random trees: every node's parent is an earlier node, the nearer ones likelier."""
    j = torch.arange(N, device="cuda")
    u = torch.rand((B, N), generator=g, device="cuda").sqrt()
    p = torch.minimum((u * j).long(), (j - 1).clamp(min=0))
    p[:, 0] = -1
    return p.int()


def _cache(case, g, positions):
    """A layer's K and V pool, each position of each request at a random slot; slots that nobody holds are NaN."""
    B, Hkv, D, dt = case["B"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    slots = B * positions + 17
    table = torch.randperm(slots, generator=g, device="cuda")[: B * positions].view(B, positions).int()
    k = torch.randn((slots, Hkv, D), generator=g, device="cuda", dtype=dt)
    v = torch.randn((slots, Hkv, D), generator=g, device="cuda", dtype=dt)
    free = torch.ones(slots, dtype=torch.bool, device="cuda")
    free[table.view(-1).long()] = False
    k[free], v[free] = math.nan, math.nan
    return k, v, table


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    B = case["B"]
    order = torch.randperm(B, generator=g, device="cuda")
    s = dict(case, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "logprobs":
        R, V, T = case["rows"], case["V"], case["rows"]
        x = torch.randn((B, R, V), generator=g, device="cuda") * 3.0
        x.scatter_add_(2, torch.randint(0, V, (B, R, 1), generator=g, device="cuda"),
                       torch.full((B, R, 1), 8.0, device="cuda"))
        keep = torch.randint(0, V, (B, R, 1), generator=g, device="cuda")
        if case["masked"]:  # a grammar leaves a tenth of the vocabulary to every other request
            out = torch.rand((B, R, V), generator=g, device="cuda") < 0.9
            out[1::2] = False
            x.masked_fill_(out.scatter_(2, keep, False), -math.inf)
        logits = x.to(dt)
        index = None
        if case["tree"]:  # the accepted path: the root, then nodes in ascending order
            index = torch.rand((B, R), generator=g, device="cuda").argsort(1).int()
            index[:, 0] = 0
        n = torch.tensor(_emitted(case), device="cuda")[order][:, None]
        t = torch.arange(T, device="cuda")[None]
        rows = logits if index is None else logits.gather(1, index.long()[:, :, None].expand(B, R, V))
        hit = torch.rand((B, T), generator=g, device="cuda") < 0.7
        tok = torch.where(hit, rows.float().argmax(-1), keep[:, :, 0])
        s.update(logits=logits, tokens=torch.where(t < n, tok, -1).int(),
                 index=None if index is None else torch.where(t < n, index, -1).int())
        f = lambda *d: torch.empty(d, device="cuda")  # noqa: E731
        s["out"] = dict(logprobs=f(B, T), entropy=f(B, T), ranks=f(B, T).int(), top_ids=f(B, T, case["top"]).int(),
                        top_logprobs=f(B, T, case["top"]))
        return s
    N, Hq, Hkv, D = (case[k] for k in ("N", "Hq", "Hkv", "D"))
    lengths = torch.tensor(_lengths(case), device="cuda")[order].int()
    s["committed"] = lengths[:, 0].contiguous()
    s["num_nodes"] = lengths[:, 1].contiguous() if case.get("ragged") else None
    s["parents"] = _parents(B, N, g) if case["tree"] else None
    qkv = torch.randn((B, N, (Hq + 2 * Hkv) * D), generator=g, device="cuda", dtype=dt)  # the projections' one output
    s["q"], s["k"], s["v"] = (t.unflatten(2, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 2))
    if case["op"] == "attention":
        s["q"].mul_(2.0)
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, g, case["hi"] + N + 1)
        s["positions"] = max(c + n for c, n in _lengths(case))
        s["out"] = torch.empty((B, N, Hq, D), device="cuda", dtype=dt)
        s["lse"] = torch.empty((B, N, Hq), device="cuda")
        return s
    # The new positions have slots of their own; the tables' other entries are not used by this operator.
    positions = case["hi"] + N + 1
    slots = B * N + 17
    mine = torch.randperm(slots, generator=g, device="cuda")[: B * N].view(B, N).int()
    s["table"] = torch.zeros((B, positions), dtype=torch.int32, device="cuda")
    s["table"].scatter_(1, s["committed"].long()[:, None] + torch.arange(N, device="cuda"), mine)
    s["k_cache"] = torch.randn((slots, Hkv, D), generator=g, device="cuda", dtype=dt)
    s["v_cache"] = torch.randn((slots, Hkv, D), generator=g, device="cuda", dtype=dt)
    freq = 500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["out"] = torch.empty((B, N, Hq, D), device="cuda", dtype=dt)
    return s


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_append(s):
    import speculative_decoding_verification_verify_gb300 as sv

    q = sv.spec_verify_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["committed"],
                                 s["cos_sin"], parents=s["parents"], interleaved=s["interleaved"], q_out=s["out"],
                                 dev_status=s["status"])
    return q, s["k_cache"], s["v_cache"]


def _own_attention(s):
    import speculative_decoding_verification_verify_gb300 as sv

    return tuple(sv.spec_verify_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["committed"],
                                          parents=s["parents"], num_nodes=s["num_nodes"], scale=s["D"] ** -0.5,
                                          out=s["out"], lse=s["lse"], dev_status=s["status"]))


def _own_logprobs(s):
    import speculative_decoding_verification_verify_gb300 as sv

    r = sv.spec_verify_logprobs(s["logits"], s["tokens"], row_index=s["index"], temperature=s["T"], top_n=s["top"],
                                dev_status=s["status"], **s["out"])
    return _said(r.logprobs, r.entropy, r.ranks, r.top_ids, r.top_logprobs)


def _said(logprobs, entropy, ranks, top_ids, top_logprobs):
    got = dict(logprobs=logprobs, entropy=entropy, ranks=ranks)
    return dict(got, top_ids=top_ids, top_logprobs=top_logprobs) if top_ids is not None and top_ids.shape[-1] else got


def _ancestors(parents):
    """[B, N, N] truth values: whether node a is node n or an ancestor of it."""
    N = parents.shape[1]
    step = (parents[:, :, None] == torch.arange(N, device="cuda")).float() + torch.eye(N, device="cuda")
    return torch.linalg.matrix_power(step, 64) > 0


def _plain_append(s):
    B, N, Hq, D = s["q"].shape
    node = torch.arange(N, device="cuda")
    depth = node.expand(B, N) if s["parents"] is None else _ancestors(s["parents"]).sum(-1) - 1
    slot = s["table"].gather(1, s["committed"].long()[:, None] + node).long()
    cs = s["cos_sin"][s["committed"].long()[:, None] + depth][:, :, None]
    c, sn = cs.chunk(2, -1)

    def turn(x):
        y = x.float()
        r, rest = y[..., : s["rot"]], y[..., s["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else r.chunk(2, -1)
        a, b = a * c - b * sn, b * c + a * sn
        r = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    s["k_cache"][slot] = turn(s["k"])
    s["v_cache"][slot] = s["v"]
    return turn(s["q"]), s["k_cache"], s["v_cache"]


def _plain_attention(s):
    B, N, Hq, D = s["q"].shape
    Hkv, L = s["Hkv"], s["positions"]
    pos, node = torch.arange(L, device="cuda"), torch.arange(N, device="cuda")
    committed = s["committed"].long()[:, None]
    nodes = (torch.full((B,), N, device="cuda") if s["num_nodes"] is None else s["num_nodes"].long())[:, None]
    held = pos < committed + nodes
    slot = torch.where(held, s["table"][:, :L], s["table"][:, :1]).long()
    k = s["k_cache"][slot].float()
    v = s["v_cache"][slot].float().masked_fill_(~held[:, :, None, None], 0.0)
    above = (node[:, None] >= node).expand(B, N, N) if s["parents"] is None else _ancestors(s["parents"])
    at = (pos - committed).clamp(0, N - 1)
    seen = (pos < committed)[:, None] | above.gather(2, at[:, None].expand(B, N, L)) & (pos >= committed)[:, None]
    seen = seen & held[:, None] & (node < nodes)[:, :, None]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D) * D ** -0.5
    x = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, -1, N, L).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = x.sub_(m).exp_()
    z = e.sum(-1, keepdim=True)
    o = (e.reshape(B, Hkv, -1, L) @ v.permute(0, 2, 1, 3)).view(B, Hkv, -1, N, D) / z
    o = o.masked_fill(z == 0, 0.0).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)
    lse = (m + z.log())[..., 0].permute(0, 3, 1, 2).reshape(B, N, Hq)
    return o.to(s["q"].dtype), lse


def _plain_logprobs(s):
    logits, tokens, n = s["logits"], s["tokens"].long(), s["top"]
    B, R, V = logits.shape
    if s["index"] is not None:
        logits = logits.gather(1, s["index"].long().clamp(min=0)[:, :, None].expand(B, tokens.shape[1], V))
    here = tokens >= 0
    x = logits.float()
    own_x = x.gather(2, tokens.clamp(min=0)[:, :, None])
    ranks = torch.where(here, (x > own_x).sum(-1) + 1, 0).int()
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :, :n]
    top = x.gather(2, ids)
    m = x.amax(-1, keepdim=True)
    d = (x - m) / s["T"]
    e = d.exp()
    z = e.sum(-1, keepdim=True)
    entropy = z.log() - (e * d.masked_fill_(e == 0, 0.0)).sum(-1, keepdim=True) / z
    said = lambda y: (y - m) / s["T"] - z.log()  # noqa: E731
    there = here[:, :, None] & (top > -math.inf)
    return _said(said(own_x)[..., 0].masked_fill(~here, 0.0), entropy[..., 0].masked_fill(~here, 0.0), ranks,
                 torch.where(there, ids, -1).int(), said(top).masked_fill(~there, -math.inf))


_run_own = {"append": _own_append, "attention": _own_attention, "logprobs": _own_logprobs}
_run_plain = {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs}


# --------------------------------------------------------------------------------------------
# The same in 64 bits, request by request from the definitions
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["op"]](s)


def _path(parents, n):
    """The nodes from n up to the root."""
    got = [n]
    while parents[got[-1]] >= 0:
        got.append(parents[got[-1]])
    return got


def _exact_append(s):
    B, N, Hq, D = s["q"].shape
    half = s["rot"] // 2
    k, v = s["k_cache"].double(), s["v_cache"].double()
    q_out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    i = torch.arange(half, device="cuda")
    at, to = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    for b in range(B):
        c = int(s["committed"][b])
        up = None if s["parents"] is None else s["parents"][b].tolist()
        pos = torch.tensor([c + (n if up is None else len(_path(up, n)) - 1) for n in range(N)], device="cuda")
        cos, sin = s["cos_sin"][pos, :half].double()[:, None], s["cos_sin"][pos, half:].double()[:, None]
        slot = s["table"][b, c:c + N].long()
        got = []
        for x in (s["q"][b].double(), s["k"][b].double()):
            y = x.clone()
            y[..., at] = x[..., at] * cos - x[..., to] * sin
            y[..., to] = x[..., at] * sin + x[..., to] * cos
            got.append(y)
        q_out[b], k[slot], v[slot] = got[0], got[1], s["v"][b].double()
    return q_out, k, v


def _exact_attention(s):
    B, N, Hq, D = s["q"].shape
    if work({k: s[k] for k in ("op", "B", "N", "Hq", "Hkv", "D", "lo", "hi", "ragged")})["flops"] > 2e12:
        return None
    G = Hq // s["Hkv"]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        c = int(s["committed"][b])
        nodes = N if s["num_nodes"] is None else int(s["num_nodes"][b])
        up = list(range(-1, N - 1)) if s["parents"] is None else s["parents"][b].tolist()
        seen = torch.zeros((nodes, c + nodes), dtype=torch.bool)
        seen[:, :c] = True
        for n in range(nodes):
            seen[n, [c + a for a in _path(up, n)]] = True
        hidden = ~seen.cuda().repeat_interleave(G, 0)
        slot = s["table"][b, :c + nodes].long()
        for h in range(s["Hkv"]):
            k, v = s["k_cache"][slot, h].double(), s["v_cache"][slot, h].double()
            q = s["q"][b, :nodes, h * G:(h + 1) * G].double().reshape(-1, D)
            x = (q @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, 1)
            out[b, :nodes, h * G:(h + 1) * G] = ((x - z[:, None]).exp() @ v).view(nodes, G, D)
            lse[b, :nodes, h * G:(h + 1) * G] = z.view(nodes, G)
    return out, lse


def _exact_logprobs(s):
    B, T = s["tokens"].shape
    n = s["top"]
    lp = torch.zeros((B, T), dtype=torch.float64, device="cuda")
    ent, top = torch.zeros_like(lp), torch.full((B, T, n), -math.inf, dtype=torch.float64, device="cuda")
    tokens = s["tokens"].tolist()
    for b in range(B):
        for t in range(T):
            if tokens[b][t] < 0:
                continue
            row = s["logits"][b, t if s["index"] is None else int(s["index"][b, t])].double() / s["T"]
            y = torch.log_softmax(row, 0)
            lp[b, t] = y[tokens[b][t]]
            fine = y[y > -math.inf]
            ent[b, t] = -(fine.exp() * fine).sum()
            best = fine.topk(min(n, fine.numel())).values
            top[b, t, :best.numel()] = best
    got = dict(logprobs=lp, entropy=ent, ranks=None)
    return dict(got, top_ids=None, top_logprobs=top) if n else got
