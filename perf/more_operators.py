"""The operators of a target forward over a cache that is kept in 8 bits, from prompt to verification, as cases to
measure.

  append  spec_verify_kv_append_ex: heads' norms, position rotation and the paged append in one pass, the cache's rows
          in 16 bits or as e4m3 with a power of two for each head
  read    spec_verify_kv_read: positions of the paged cache as contiguous rows of 16 bits
  nodes   spec_verify_attention_e4m3: tree nodes, chain positions or single tokens over the 8-bit cache
  chunk   spec_verify_attention_chunk: a chunk of a prompt over either cache, causal

`own` selects the form that `run` computes: the library's kernels, or the same operators in elementary torch
operations in 32 bits.  `exact` gives them in 64 bits.

An 8-bit row of a slot is [Hkv][D] e4m3, then a byte for each head (its power of two's exponent + 127), then zeros up to
a multiple of 16 bytes.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LARGEST = 448.0   # of e4m3
EXP_HI = 7        # of a row's power of two: larger values saturate
EXP_LO = {"bf16": -126, "fp16": -15}


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # One new token of one request, heads normalised, into the 8-bit cache: latency is what counts.
        dict(name="append b1 n1 e4m3", op="append", dtype="bf16", cache="e4m3", B=1, N=1, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, norm=True, lo=701, hi=701, tree=False),
        # The tree workload's nodes into a 16-bit cache, heads normalised.
        dict(name="append b48 tree8", op="append", dtype="bf16", cache="half", B=48, N=8, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, norm=True, lo=1, hi=504, tree=True),
        # Two prompts' chunks behind a long shared conversation into the 8-bit cache, and the rows read back as
        # a caller's own attention would; adjacent pairs, half of the head rotated.
        dict(name="append b2 n4097 e4m3", op="append", dtype="fp16", cache="e4m3", B=2, N=4097, Hq=32, Hkv=8, D=128,
             rot=64, interleaved=True, norm=True, lo=126000, hi=126000, tree=False),
        # The tree workload's cache handed out whole: 48 requests of up to 504 positions.
        dict(name="read b48 504", op="read", dtype="bf16", cache="e4m3", B=48, N=504, Hkv=8, D=128, lo=0,
             hi=0, ragged=True),
        # What one long conversation has added behind a shared prefix, of a model with few, odd-sized heads.
        dict(name="read b1 60001 d80", op="read", dtype="fp16", cache="e4m3", B=1, N=60001, Hkv=4, D=80, lo=1021,
             hi=1021, ragged=False),
        # Plain decoding of one request: one new token, a short context.
        dict(name="nodes b1 n1", op="nodes", dtype="bf16", cache="e4m3", B=1, N=1, Hq=32, Hkv=8, D=128, lo=701, hi=701,
             tree=False, ragged=False),
        # The chain workload's batch (64 requests, 7 drafts) in a serving mix of context lengths.
        dict(name="nodes b64 chain8 8k", op="nodes", dtype="bf16", cache="e4m3", B=64, N=8, Hq=32, Hkv=8, D=128, lo=509,
             hi=8192, tree=False, ragged=True),
        # One request with a very long context and a wide tree: only a split over the length fills the GPU.
        dict(name="nodes b1 tree16 128k", op="nodes", dtype="fp16", cache="e4m3", B=1, N=16, Hq=32, Hkv=8, D=128,
             lo=131000, hi=131000, tree=True, ragged=False),
        # What is left of three prompts behind shared prefixes: few rows, odd heads.
        dict(name="chunk b3 n67 d80", op="chunk", dtype="fp16", cache="half", B=3, N=67, Hq=14, Hkv=2, D=80, lo=901,
             hi=9001, ragged=True),
        # Eight fresh prompts of different lengths in one padded batch, a small model's heads.
        dict(name="chunk b8 prompts d64", op="chunk", dtype="fp16", cache="half", B=8, N=4096, Hq=32, Hkv=8, D=64, lo=0,
             hi=0, ragged=True),
        # A chunk of a long prompt behind what earlier chunks wrote.
        dict(name="chunk b1 n2048 14k", op="chunk", dtype="bf16", cache="half", B=1, N=2048, Hq=32, Hkv=8, D=128,
             lo=14337, hi=14337, ragged=False),
        # The same in large, over the 8-bit cache.
        dict(name="chunk b1 n4096 28k e4m3", op="chunk", dtype="bf16", cache="e4m3", B=1, N=4096, Hq=32, Hkv=8, D=128,
             lo=28001, hi=28001, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "nodes", "nodes", "chunk", "chunk"])
    while True:
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        D = rng.choice([64, 80, 96, 128, 128])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), cache="e4m3", B=_log_int(rng, 1, 64), Hkv=Hkv, D=D)
        if op == "read":
            hi = rng.choice([0, _log_int(rng, 1, 60000)])
            c.update(N=_log_int(rng, 1, 60001), ragged=rng.random() < 0.5, cache=rng.choice(["e4m3", "e4m3", "half"]),
                     lo=_log_int(rng, 1, hi) if hi else 0, hi=hi)
            if c["B"] * c["N"] * Hkv * D > 48 * 504 * 8 * 128 or c["B"] * (hi + c["N"]) * Hkv * D > 64 * 8200 * 1024:
                continue
            return c
        c["Hq"] = Hkv * G
        if op == "append":
            tree = rng.random() < 0.4
            N = _log_int(rng, 2, 64) if tree else _log_int(rng, 1, 4097)
            lo = _log_int(rng, 1, 100000)
            c.update(N=N, rot=rng.choice([D, D, 32, 64]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                     lo=lo, hi=_log_int(rng, lo, 120000), tree=tree, cache=rng.choice(["e4m3", "half"]))
            if not c["norm"]:
                c["cache"] = "e4m3"
            if c["B"] * N * (G + 2) * Hkv * D > 2 * 4097 * 48 * 128:
                continue
            return c
        if op == "nodes":
            N = rng.choice([1, 1, _log_int(rng, 2, 64)])
            hi = _log_int(rng, 1, 131072)
            c.update(N=N, lo=_log_int(rng, 1, hi), hi=hi, tree=N > 1 and rng.random() < 0.5, ragged=rng.random() < 0.4)
            w = work(c)
            if w["bytes"] > 3.2e8 or w["flops"] > 7e10 or c["B"] * (hi + N) * Hkv * D > 64 * 8200 * 1024 \
                    or c["B"] * Hkv * G * N * (hi + N) > 64 * 8200 * 256:
                continue
            return c
        N = _log_int(rng, 2, 8192)
        hi = rng.choice([0, _log_int(rng, 1, 60000)])
        c.update(N=N, lo=_log_int(rng, 1, hi) if hi else 0, hi=hi, ragged=rng.random() < 0.5,
                 cache=rng.choice(["half", "half", "e4m3"]))
        # (The plain form takes a request and a key head at a time, so many requests cost it time.)
        if work(c)["flops"] > 1.5e12 or c["B"] * Hkv > 128 or c["B"] * (hi + N) * Hkv * D > 64 * 8200 * 1024 \
                or c["B"] * N * Hkv * G * D > 8 * 4096 * 32 * 128 or G * N * (hi + N) > 4 * 4096 * 32100:
            continue
        return c


def _lengths(case):
    """(committed positions, nodes) of each request: the same lengths whatever the seed, in another order."""
    B, N = case["B"], case["N"]
    lo, hi = case.get("lo", 0), case.get("hi", 0)
    got = []
    for i in range(B):
        c = int(round(lo * (hi / lo) ** (i / (B - 1)))) if B > 1 and lo else hi
        # Chunks and rows to read of a ragged batch: from an eighth of N to all of it.  Nodes: any number.
        n = N
        if case.get("ragged"):
            n = 1 + (i * 7 + 2) % N if case["op"] == "nodes" else max(1, N * (8 - (i * 3) % 8) // 8)
        got.append((c, n))
    return got


def _row_bytes(case):
    """Of one position's keys (or values) in the cache."""
    return case["Hkv"] * (case["D"] + 1) if case["cache"] == "e4m3" else case["Hkv"] * case["D"] * 2


def work(case):
    """Bytes that have to be read and written, and arithmetic, of one pass."""
    B, N, Hkv, D = (case[k] for k in ("B", "N", "Hkv", "D"))
    lens, row = _lengths(case), _row_bytes(case)
    if case["op"] == "read":
        n = sum(m for _, m in lens)
        return {"bytes": n * (2 * row + 4) + B * N * 2 * Hkv * D * 2, "flops": 2 * n * Hkv * D}
    Hq = case["Hq"]
    if case["op"] == "append":
        rows = B * N
        back = 2 * row + 2 * Hkv * D * 2 if case["cache"] == "e4m3" else 0  # the rows read back
        return {"bytes": rows * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * row + 4 + back) + rows * case["rot"] * 4,
                "flops": 8 * rows * (Hq + Hkv) * D}
    kv = sum(c + n for c, n in lens)
    pairs = sum((c + n) * n if case["op"] == "nodes" else c * n + n * (n + 1) // 2 for c, n in lens)
    return {"bytes": kv * (2 * row + 4) + sum(n for _, n in lens) * Hq * D * 2 + B * N * Hq * (D * 2 + 4),
            "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def _parents(B, N, g):
    """Random trees: every node's parent is an earlier node, the nearer ones likelier."""
    j = torch.arange(N, device="cuda")
    u = torch.rand((B, N), generator=g, device="cuda").sqrt()
    p = torch.minimum((u * j).long(), (j - 1).clamp(min=0))
    p[:, 0] = -1
    return p.int()


def _powers(x, dtype):
    """The exponents of heads' powers of two: the smallest with which the largest value fits e4m3."""
    m, e = torch.frexp(x.abs().amax(-1))
    return torch.where(m > LARGEST / 512, e - 8, e - 9).clamp(EXP_LO[dtype], EXP_HI)


def _rounded(x, dtype):
    """x [..., D] in 32 bits as e4m3, and the exponents."""
    e = _powers(x, dtype)
    y = torch.ldexp(x, -e[..., None]).clamp(-LARGEST, LARGEST)
    return y.to(torch.float8_e4m3fn), e


def _pool(case, g, slots):
    """A layer's keys or values with random rows: [slots, Hkv, D], or 8-bit rows as bytes."""
    Hkv, D = case["Hkv"], case["D"]
    x = torch.randn((slots, Hkv, D), generator=g, device="cuda", dtype=DTYPES[case["dtype"]])
    if case["cache"] != "e4m3":
        return x
    pool = torch.zeros((slots, (Hkv * (D + 1) + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
    for s in range(0, slots, 1 << 16):
        y, e = _rounded(x[s:s + (1 << 16)].float(), case["dtype"])
        pool[s:s + (1 << 16), : Hkv * D] = y.view(torch.uint8).flatten(1)
        pool[s:s + (1 << 16), Hkv * D: Hkv * (D + 1)] = (e + 127).to(torch.uint8)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, N, Hkv, D, op = (case[k] for k in ("B", "N", "Hkv", "D", "op"))
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    lens = [_lengths(case)[i] for i in order]
    s = dict(case, lens=lens, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["committed"] = torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda")
    s["num_nodes"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda") if case.get("ragged") else None
    s["parents"] = _parents(B, N, g) if case.get("tree") else None
    f = lambda *d, t=dt: torch.empty(d, device="cuda", dtype=t)  # noqa: E731
    positions = case.get("hi", 0) + N + 1
    if op == "append":
        # The new positions have slots of their own; the tables' other entries are not used by this operator.
        slots = B * N + 17
        mine = torch.randperm(slots, generator=g, device="cuda")[: B * N].view(B, N).int()
        s["table"] = torch.zeros((B, positions), dtype=torch.int32, device="cuda")
        s["table"].scatter_(1, s["committed"].long()[:, None] + torch.arange(N, device="cuda"), mine)
        qkv = torch.randn((B, N, (case["Hq"] + 2 * Hkv) * D), generator=g, device="cuda", dtype=dt)  # one projection's rows
        s["q"], s["k"], s["v"] = (t.unflatten(2, (-1, D)) for t in qkv.split([case["Hq"] * D, Hkv * D, Hkv * D], 2))
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.1 * torch.randn((2, D), generator=g, device="cuda")).to(dt)
        freq = 500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["k_cache"], s["v_cache"] = _pool(case, g, slots), _pool(case, g, slots)
        s["q_out"], s["k_rows"], s["v_rows"] = f(B, N, case["Hq"], D), f(B, N, Hkv, D), f(B, N, Hkv, D)
        return s
    # Each position of each request has a random slot; slots that nobody holds are NaN.
    slots = B * positions + 17
    s["table"] = torch.randperm(slots, generator=g, device="cuda")[: B * positions].view(B, positions).int()
    s["k_cache"], s["v_cache"] = _pool(case, g, slots), _pool(case, g, slots)
    free = torch.ones(slots, dtype=torch.bool, device="cuda")
    free[s["table"].view(-1).long()] = False
    for cache in (s["k_cache"], s["v_cache"]):
        cache[free] = 0xFF if case["cache"] == "e4m3" else math.nan
    if op == "read":
        s["k_rows"], s["v_rows"] = f(B, N, Hkv, D), f(B, N, Hkv, D)
        return s
    s["q"] = torch.randn((B, N, case["Hq"], D), generator=g, device="cuda", dtype=dt) * 2.0
    s["out"], s["lse"] = f(B, N, case["Hq"], D), f(B, N, case["Hq"], t=torch.float32)
    return s


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_append(s):
    import speculative_decoding_verification_verify_gb300 as sv

    q = sv.spec_verify_kv_append_ex(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["committed"],
                                    s["cos_sin"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, parents=s["parents"],
                                    interleaved=s["interleaved"], q_out=s["q_out"], dev_status=s["status"])
    if s["cache"] != "e4m3":
        return q, s["k_cache"], s["v_cache"]
    k, v = sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["table"], s["committed"], s["N"], kv_heads=s["Hkv"],
                                  head_dim=s["D"], dtype=DTYPES[s["dtype"]], k_out=s["k_rows"], v_out=s["v_rows"],
                                  dev_status=s["status"])
    return q, k, v


def _own_read(s):
    import speculative_decoding_verification_verify_gb300 as sv

    return tuple(sv.spec_verify_kv_read(s["k_cache"], s["v_cache"], s["table"], s["committed"], s["N"],
                                        num_rows=s["num_nodes"], kv_heads=s["Hkv"], head_dim=s["D"],
                                        dtype=DTYPES[s["dtype"]], k_out=s["k_rows"], v_out=s["v_rows"],
                                        dev_status=s["status"]))


def _own_nodes(s):
    import speculative_decoding_verification_verify_gb300 as sv

    return tuple(sv.spec_verify_attention_e4m3(s["q"], s["k_cache"], s["v_cache"], s["table"], s["committed"],
                                               kv_heads=s["Hkv"], parents=s["parents"], num_nodes=s["num_nodes"],
                                               scale=s["D"] ** -0.5, out=s["out"], lse=s["lse"], dev_status=s["status"]))


def _own_chunk(s):
    import speculative_decoding_verification_verify_gb300 as sv

    return tuple(sv.spec_verify_attention_chunk(s["q"], s["k_cache"], s["v_cache"], s["table"], s["committed"],
                                                kv_heads=s["Hkv"], num_nodes=s["num_nodes"], scale=s["D"] ** -0.5,
                                                out=s["out"], lse=s["lse"], dev_status=s["status"]))


def _values(s, cache, slot):
    """Rows of the cache in 32 bits, [..., Hkv, D]."""
    if s["cache"] != "e4m3":
        return cache[slot].float()
    Hkv, D = s["Hkv"], s["D"]
    rows = cache[slot]
    x = rows[..., : Hkv * D].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (Hkv, D))
    return torch.ldexp(x, rows[..., Hkv * D: Hkv * (D + 1)].int()[..., None] - 127)


def _depth(parents):
    return _ancestors(parents).sum(-1) - 1


def _ancestors(parents):
    """[B, N, N] truth values: whether node a is node n or an ancestor of it."""
    N = parents.shape[1]
    step = (parents[:, :, None] == torch.arange(N, device="cuda")).float() + torch.eye(N, device="cuda")
    return torch.linalg.matrix_power(step, 64) > 0


def _plain_append(s):
    B, N, Hq, D = s["q"].shape
    dt = s["q"].dtype
    node = torch.arange(N, device="cuda")
    at = s["committed"].long()[:, None] + node
    slot = s["table"].gather(1, at).long()
    pos = at if s["parents"] is None else s["committed"].long()[:, None] + _depth(s["parents"])
    c, sn = s["cos_sin"][pos][:, :, None].chunk(2, -1)

    def turn(x, weight):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r, rest = y[..., : s["rot"]], y[..., s["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else r.chunk(2, -1)
        a, b = a * c - b * sn, b * c + a * sn
        r = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1)

    q, k, v = turn(s["q"], s["q_norm"]).to(dt), turn(s["k"], s["k_norm"]), s["v"].float()
    if s["cache"] != "e4m3":
        s["k_cache"][slot], s["v_cache"][slot] = k.to(dt), v.to(dt)
        return q, s["k_cache"], s["v_cache"]
    Hkv, back = s["Hkv"], []
    for x, cache in ((k, s["k_cache"]), (v, s["v_cache"])):
        y, e = _rounded(x, s["dtype"])
        rows = torch.zeros((B, N, cache.shape[1]), dtype=torch.uint8, device="cuda")
        rows[..., : Hkv * D] = y.view(torch.uint8).flatten(2)
        rows[..., Hkv * D: Hkv * (D + 1)] = (e + 127).to(torch.uint8)
        cache[slot] = rows
        back.append(_values(s, cache, slot).to(dt))
    return q, back[0], back[1]


def _plain_read(s):
    N = s["N"]
    pos = torch.arange(N, device="cuda")
    n = torch.full_like(s["committed"], N) if s["num_nodes"] is None else s["num_nodes"]
    here = pos < n[:, None]
    slot = s["table"].gather(1, torch.where(here, s["committed"].long()[:, None] + pos, 0)).long()
    return tuple(_values(s, cache, slot).masked_fill_(~here[:, :, None, None], 0.0).to(DTYPES[s["dtype"]])
                 for cache in (s["k_cache"], s["v_cache"]))


def _plain_nodes(s):
    B, N, Hq, D = s["q"].shape
    Hkv, L = s["Hkv"], max(c + n for c, n in s["lens"])
    pos, node = torch.arange(L, device="cuda"), torch.arange(N, device="cuda")
    committed = s["committed"].long()[:, None]
    nodes = (torch.full((B,), N, device="cuda") if s["num_nodes"] is None else s["num_nodes"].long())[:, None]
    held = pos < committed + nodes
    slot = torch.where(held, s["table"][:, :L], s["table"][:, :1]).long()
    k = _values(s, s["k_cache"], slot)
    v = _values(s, s["v_cache"], slot).masked_fill_(~held[:, :, None, None], 0.0)
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


def _plain_chunk(s):
    B, N, Hq, D = s["q"].shape
    Hkv, G = s["Hkv"], Hq // s["Hkv"]
    out, lse = torch.zeros_like(s["q"]), torch.full((B, N, Hq), -math.inf, device="cuda")
    for b, (c, n) in enumerate(s["lens"]):
        slot = s["table"][b, : c + n].long()
        k, v = _values(s, s["k_cache"], slot), _values(s, s["v_cache"], slot)
        hidden = (torch.arange(c + n, device="cuda") > c + torch.arange(n, device="cuda")[:, None])
        for h in range(Hkv):
            q = s["q"][b, :n, h * G:(h + 1) * G].transpose(0, 1).reshape(G * n, D).float() * D ** -0.5
            x = (q @ k[:, h].T).view(G, n, c + n).masked_fill_(hidden, -math.inf)
            m = x.amax(-1, keepdim=True)
            e = x.sub_(m).exp_()
            z = e.sum(-1, keepdim=True)
            o = (e.view(G * n, c + n) @ v[:, h]).view(G, n, D) / z
            out[b, :n, h * G:(h + 1) * G] = o.transpose(0, 1).to(out.dtype)
            lse[b, :n, h * G:(h + 1) * G] = (m + z.log())[..., 0].T
    return out, lse


_run_own = {"append": _own_append, "read": _own_read, "nodes": _own_nodes, "chunk": _own_chunk}
_run_plain = {"append": _plain_append, "read": _plain_read, "nodes": _plain_nodes, "chunk": _plain_chunk}


# --------------------------------------------------------------------------------------------
# The same in 64 bits, request by request from the definitions
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("nodes", "chunk") and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "nodes": _exact_attention, "chunk": _exact_attention}[s["op"]](s)


def _path(parents, n):
    """The nodes from n up to the root."""
    got = [n]
    while parents[got[-1]] >= 0:
        got.append(parents[got[-1]])
    return got


def _e4m3_grid():
    """The 127 finite values of e4m3 from 0 on, by their bits."""
    got = []
    for bits in range(127):
        e, m = bits >> 3, bits & 7
        got.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _nearest(x, dtype):
    """x [..., D] in 64 bits: the values that an 8-bit row holds for it."""
    grid = _e4m3_grid()
    mid = (grid[1:] + grid[:-1]) / 2
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / grid[-1])
    p = (e - (m == 0.5).int()).double()  # the smallest power that is no smaller
    step = 2.0 ** p.clamp(EXP_LO[dtype], EXP_HI)
    y = (x.abs() / step).clamp(max=float(grid[-1]))
    lower, upper = torch.bucketize(y, mid), torch.bucketize(y, mid, right=True)
    at = torch.where(lower % 2 == 0, lower, upper)  # they differ at a tie: the even one
    return grid[at] * x.sign() * step


def _exact_rows(s, cache, slot):
    if s["cache"] != "e4m3":
        return cache[slot].double()
    Hkv, D, grid = s["Hkv"], s["D"], _e4m3_grid()
    rows = cache[slot]
    bits = rows[:, : Hkv * D].long()
    x = grid[(bits & 127).clamp(max=126)] * (1 - 2 * (bits >> 7))
    x = torch.where(bits & 127 == 127, math.nan, x)
    return x.view(-1, Hkv, D) * 2.0 ** (rows[:, Hkv * D: Hkv * (D + 1)].double() - 127)[:, :, None]


def _exact_append(s):
    B, N, Hq, D = s["q"].shape
    half = s["rot"] // 2
    i = torch.arange(half, device="cuda")
    at, to = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    e4m3 = s["cache"] == "e4m3"
    q_out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    shape = (B, N, s["Hkv"], D)
    k, v = (torch.zeros(shape, dtype=torch.float64, device="cuda") if e4m3 else s[x].double() for x in ("k_cache", "v_cache"))
    for b in range(B):
        c = int(s["committed"][b])
        up = None if s["parents"] is None else s["parents"][b].tolist()
        pos = torch.tensor([c + (n if up is None else len(_path(up, n)) - 1) for n in range(N)], device="cuda")
        cos, sin = s["cos_sin"][pos, :half].double()[:, None], s["cos_sin"][pos, half:].double()[:, None]
        slot = s["table"][b, c:c + N].long()
        got = []
        for x, w in ((s["q"][b].double(), s["q_norm"]), (s["k"][b].double(), s["k_norm"])):
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            y = x.clone()
            y[..., at] = x[..., at] * cos - x[..., to] * sin
            y[..., to] = x[..., at] * sin + x[..., to] * cos
            got.append(y)
        q_out[b] = got[0]
        if e4m3:
            k[b], v[b] = _nearest(got[1], s["dtype"]), _nearest(s["v"][b].double(), s["dtype"])
        else:
            k[slot], v[slot] = got[1], s["v"][b].double()
    return q_out, k, v


def _exact_read(s):
    got = []
    for cache in (s["k_cache"], s["v_cache"]):
        out = torch.zeros((s["B"], s["N"], s["Hkv"], s["D"]), dtype=torch.float64, device="cuda")
        for b, (c, n) in enumerate(s["lens"]):
            out[b, :n] = _exact_rows(s, cache, s["table"][b, c:c + n].long())
        got.append(out)
    return tuple(got)


def _exact_attention(s):
    B, N, Hq, D = s["q"].shape
    G = Hq // s["Hkv"]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (c, n) in enumerate(s["lens"]):
        if s["parents"] is None:
            hidden = torch.arange(c + n, device="cuda")[None] > c + torch.arange(n, device="cuda")[:, None]
        else:
            up = s["parents"][b].tolist()
            hidden = torch.ones((n, c + n), dtype=torch.bool)
            hidden[:, :c] = False
            for i in range(n):
                hidden[i, [c + a for a in _path(up, i)]] = False
            hidden = hidden.cuda()
        slot = s["table"][b, : c + n].long()
        k, v = _exact_rows(s, s["k_cache"], slot), _exact_rows(s, s["v_cache"], slot)
        for h in range(Hq):
            for r in range(0, n, 2048):  # rows at a time
                q = s["q"][b, r:r + 2048, h].double()
                x = (q[:n - r] @ k[:, h // G].T / math.sqrt(D)).masked_fill_(hidden[r:r + 2048], -math.inf)
                z = torch.logsumexp(x, 1)
                out[b, r:r + len(x), h] = x.sub_(z[:, None]).exp_() @ v[:, h // G]
                lse[b, r:r + len(x), h] = z
    return out, lse
