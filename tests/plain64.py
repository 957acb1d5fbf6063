"""Plain 64-bit implementations of the operators around verification, for the GPU tests: the
definitions written out request by request, sharing nothing with the kernels.  With each value comes
the size that roundings act on, from which the tests derive their tolerances."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALLEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def path_of(parents, n):
    """The nodes from n up to the root; parents None: a chain."""
    if parents is None:
        return list(range(n, -1, -1))
    got = [n]
    while parents[got[-1]] >= 0:
        got.append(parents[got[-1]])
    return got


def rotate(x, cos, sin, rot, interleaved):
    """x [..., D] in 64 bits; cos, sin [rot / 2].  Returns the rotated vector and, per element, the sum
    of the two products' magnitudes."""
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, size = x.clone(), x.abs()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    size[..., a] = (x[..., a] * cos).abs() + (x[..., b] * sin).abs()
    size[..., b] = (x[..., b] * cos).abs() + (x[..., a] * sin).abs()
    return y, size


def attention(q, k_cache, v_cache, slot_table, committed, parents=None, num_nodes=None, scale=None):
    """(out, lse, out_tol, lse_tol), all in 64 bits.  A node's row is computed from the positions that
    it sees alone.

    Tolerances, with u the half step of q's type: each weight is rounded to that type once and the sum
    that divides them is of the rounded or the unrounded ones (2 u sum p |v|), the result is rounded
    (u |out|); a score's fp32 dot product is off by at most (D + 2) 2^-24 sum |q k| scale, in whatever
    order it is summed; 2^x by 2^-21 relative, the sums by (positions / 16 + 32) 2^-24."""
    B, N, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    u = HALF_STEP[q.dtype]
    scale = D ** -0.5 if scale is None else scale
    f = dict(dtype=torch.float64, device=q.device)
    out, tol = torch.zeros((B, N, Hq, D), **f), torch.zeros((B, N, Hq, D), **f)
    lse, lse_tol = torch.full((B, N, Hq), -math.inf, **f), torch.zeros((B, N, Hq), **f)
    for b in range(B):
        c = int(committed[b])
        nodes = N if num_nodes is None else int(num_nodes[b])
        up = None if parents is None else parents[b].tolist()
        for n in range(nodes):
            pos = list(range(c)) + sorted(c + a for a in path_of(up, n))
            slot = slot_table[b].long()[torch.tensor(pos, device=q.device)]
            k = k_cache[slot].double().repeat_interleave(G, 1)  # [L, Hq, D]
            v = v_cache[slot].double().repeat_interleave(G, 1)
            x = q[b, n].double()
            s = (x * k).sum(-1) * scale
            size = ((x * k).abs().sum(-1) * scale).amax(0)
            m = s.amax(0)
            e = (s - m).exp()
            z = e.sum(0)
            p = e / z
            out[b, n] = torch.einsum("lh,lhd->hd", p, v)
            lse[b, n] = m + z.log()
            d = (D + 2) * 2.0 ** -24 * size + (m.abs() + 2) * 2.0 ** -23 + 2.0 ** -21 + (len(pos) / 16 + 32) * 2.0 ** -24
            mass = torch.einsum("lh,lhd->hd", p, v.abs())
            tol[b, n] = 2 * u * mass + u * out[b, n].abs() + 3 * d[:, None] * mass + SMALLEST[q.dtype]
            lse_tol[b, n] = 2 * d + 2.0 ** -23 * lse[b, n].abs()
    return out, lse, tol, lse_tol


def logprobs(logits, tokens, row_index=None, temperatures=None, temperature=1.0, top_n=0):
    """Dict of logprobs, entropy, ranks, top_ids, top_logprobs, and tol / entropy_tol.

    Tolerances: (x - m) / T carries the scale's and the product's rounding (2^-23 of it), the sum's
    logarithm the exponentials' 2^-21 and the sum's (V / 4096 + 32) 2^-24; the entropy's second sum
    has terms up to ln Z + 1 in size."""
    B, T = tokens.shape
    V = logits.shape[2]
    f = dict(dtype=torch.float64, device=logits.device)
    got = dict(logprobs=torch.zeros((B, T), **f), entropy=torch.zeros((B, T), **f),
               ranks=torch.zeros((B, T), dtype=torch.int32, device=logits.device),
               top_ids=torch.full((B, T, top_n), -1, dtype=torch.int32, device=logits.device),
               top_logprobs=torch.full((B, T, top_n), -math.inf, **f), tol=torch.zeros((B, T), **f),
               entropy_tol=torch.zeros((B, T), **f), top_tol=torch.zeros((B, T, top_n), **f))
    base = 2.0 ** -20 + (V / 4096 + 32) * 2.0 ** -23
    for b in range(B):
        temp = float(temperature if temperatures is None else temperatures[b]) or 1.0
        for t in range(T):
            tok = int(tokens[b, t])
            r = t if row_index is None else int(row_index[b, t])
            if tok < 0 or r < 0:
                continue
            raw = logits[b, r].double()
            x = raw / temp
            m = x.max()
            e = (x - m).exp()
            z = e.sum()
            lnz = z.log()
            d = torch.where(e > 0, x - m, torch.zeros_like(x))
            got["logprobs"][b, t] = x[tok] - m - lnz
            got["entropy"][b, t] = lnz - (e * d).sum() / z
            got["ranks"][b, t] = 1 + int((raw > raw[tok]).sum())
            w = x[tok] - m
            got["tol"][b, t] = base + 2.0 ** -22 * (0.0 if math.isinf(w) else float(w.abs()) + float(lnz))
            got["entropy_tol"][b, t] = base * (4 + 2 * float(lnz))
            order = torch.sort(raw, descending=True, stable=True).indices[:top_n]
            order = order[raw[order] > -math.inf]
            got["top_ids"][b, t, :order.numel()] = order.int()
            y = x[order] - m
            got["top_logprobs"][b, t, :order.numel()] = y - lnz
            got["top_tol"][b, t, :order.numel()] = base + 2.0 ** -22 * (y.abs() + lnz)
    return got
