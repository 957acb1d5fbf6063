"""spec_verify_attention_chunk's definition in 64 bits, for the GPU tests."""
import math

import torch

from plain64 import HALF_STEP, SMALLEST


def chunk(q, k_val, v_val, slot_table, committed, num_nodes=None, scale=None):
    """(out, lse, out_tol, lse_tol) in 64 bits, key head by key head; k_val, v_val [slots, Hkv, D] are what the cache's
    rows stand for.  A row is computed from the positions that it sees alone: what lies behind is replaced by zeros
    before the products.

    Tolerances, with u the half step of q's type: each weight is rounded to that type once, the sum that divides is of
    the unrounded ones (u sum p |v|, and as much again for the sum), the result is rounded (u |out|); a score's fp32 dot
    product is off by at most (D + 2) 2^-24 sum |q k| scale, in whatever order it is summed; 2^x by 2^-21 relative;
    a row's sum goes through 32 adds a lane of a tile and one per tile, the products' accumulators through one add per 16
    positions: (positions / 16 + 64) 2^-24."""
    B, N, Hq, D = q.shape
    Hkv = k_val.shape[1]
    G = Hq // Hkv
    u = HALF_STEP[q.dtype]
    scale = D ** -0.5 if scale is None else scale
    f = dict(dtype=torch.float64, device=q.device)
    out, tol = torch.zeros((B, N, Hq, D), **f), torch.zeros((B, N, Hq, D), **f)
    lse, lse_tol = torch.full((B, N, Hq), -math.inf, **f), torch.zeros((B, N, Hq), **f)
    for b in range(B):
        c = int(committed[b])
        n = N if num_nodes is None else int(num_nodes[b])
        L = c + n
        if n == 0:
            continue
        slot = slot_table[b, :L].long()
        pos, at = torch.arange(L, device=q.device), c + torch.arange(n, device=q.device)
        hidden = (pos > at[:, None]).repeat_interleave(G, 0)
        for h in range(Hkv):
            k, v = k_val[slot, h].double(), v_val[slot, h].double()
            x = q[b, :n, h * G:(h + 1) * G].double().reshape(n * G, D)
            fk, fv = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
            s = x @ fk.T * scale
            odd = ~torch.isfinite(k).all(1)
            if odd.any():
                s[:, odd] = (x[:, None] * k[odd]).sum(-1) * scale
            s = s.masked_fill(hidden, -math.inf)
            size = (x.abs() @ fk.abs().T * scale).masked_fill(hidden, 0).amax(1)
            m = s.amax(1)
            e = (s - m[:, None]).exp()
            z = e.sum(1)
            p = e / z[:, None]
            o = p @ fv
            mass = p @ fv.abs()
            for y in (~torch.isfinite(v).all(1)).nonzero()[:, 0].tolist():
                bad = ~torch.isfinite(v[y])
                sees = ~hidden[:, y]
                o[sees] = o[sees] + torch.where(bad, v[y], 0.0)
            l = m + z.log()
            d = (D + 2) * 2.0 ** -24 * size + (m.abs() + 2) * 2.0 ** -23 + 2.0 ** -21 + (L / 16 + 64) * 2.0 ** -24
            t = 2 * u * mass + u * o.abs() + 3 * d[:, None] * mass + SMALLEST[q.dtype]
            to = (b, slice(0, n), slice(h * G, (h + 1) * G))
            out[to], tol[to] = o.view(n, G, D), t.view(n, G, D)
            lse[to], lse_tol[to] = l.view(n, G), (2 * d + 2.0 ** -23 * l.abs()).view(n, G)
    return out, lse, tol, lse_tol
