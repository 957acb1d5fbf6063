"""The decoder of tree_verify_step.py with normalised heads and a cache of 8-bit rows, from prompt to verification:

    prompt, chunk by chunk   spec_verify_kv_append_ex      heads' norms, rotation, e4m3 rows with a power of two per head
                             spec_verify_attention_chunk   the chunk over what the chunks before it wrote
    a step's tree            spec_verify_kv_append_ex, spec_verify_attention_e4m3
    then                     spec_verify_tree, spec_verify_logprobs
                             spec_verify_kv_compact        the accepted path's rows, their powers of two with them
    at the end               spec_verify_kv_read           the cache as 16-bit rows

It decodes token by token, then again with trees, and the two have to agree.

    python examples/cache8_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import tree_verify_step as base  # noqa: E402

sv = base.sv


class Decoder(base.Decoder):
    """Prompts go through in chunks of `chunk` tokens; the cache is one pool of bytes, [planes, slots, row bytes]."""

    def __init__(self, chunk=16, **kw):
        super().__init__(**kw)
        self.chunk = chunk
        g = torch.Generator(device="cuda")
        g.manual_seed(99)
        for w in self.layers:
            w["q_norm"], w["k_norm"] = (1 + 0.1 * torch.randn((2, self.head_dim), generator=g, device="cuda")).bfloat16()

    def cache(self, B, max_pos, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        row = sv.spec_verify_kv_e4m3_row_bytes(self.kv_heads, self.head_dim)
        pool = torch.zeros((2 * len(self.layers), B * max_pos, row), dtype=torch.uint8, device="cuda")
        return pool, torch.randperm(B * max_pos, generator=g, device="cuda").view(B, max_pos).int()

    def forward(self, tokens, pool, slot_table, committed, parents=None, status=None):
        """Logits [B, N, vocab]; a prompt (no tree, more than one token) goes through in chunks."""
        B, N = tokens.shape
        if parents is None and N > 1:
            return torch.cat([self.nodes(tokens[:, n:n + self.chunk], pool, slot_table, committed + n, None, status)
                              for n in range(0, N, self.chunk)], 1)
        return self.nodes(tokens, pool, slot_table, committed, parents, status)

    def nodes(self, tokens, pool, slot_table, committed, parents, status):
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        H, K, D = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens.long()]
        for i, w in enumerate(self.layers):
            qkv = (norm(x) @ w["qkv"]).to(torch.bfloat16)
            q, k, v = (t.unflatten(2, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 2))
            kc, vc = pool[2 * i], pool[2 * i + 1]
            q = sv.spec_verify_kv_append_ex(q, k, v, kc, vc, slot_table, committed, self.cos_sin, q_norm=w["q_norm"],
                                            k_norm=w["k_norm"], parents=parents, dev_status=status)
            if parents is None and tokens.shape[1] > 1:
                a = sv.spec_verify_attention_chunk(q, kc, vc, slot_table, committed, kv_heads=K, dev_status=status).out
            else:
                a = sv.spec_verify_attention_e4m3(q, kc, vc, slot_table, committed, kv_heads=K, parents=parents,
                                                  dev_status=status).out
            x = x + a.float().flatten(2) @ w["out"]
            x = x + torch.nn.functional.silu(norm(x) @ w["up"]) @ w["down"]
        return norm(x) @ self.head


def run(B=3, prompt_len=37, steps=48, N=8, vocab=997, seed=0, verbose=False):
    """As tree_verify_step.run, and the first layer's keys at the end as 16-bit rows."""
    g = torch.Generator()
    g.manual_seed(seed)
    model = Decoder(vocab=vocab, seed=seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prompt = torch.randint(0, vocab, (B, prompt_len), generator=g).int().cuda()
    text, said = base.decode(model, prompt, steps, status)
    host = text.cpu()

    pool, table = model.cache(B, prompt_len + steps + 2 * N, seed=2)
    committed = torch.zeros(B, dtype=torch.int32, device="cuda")
    model.forward(prompt, pool, table, committed, status=status)
    committed += prompt_len
    got, at, rounds = [[int(host[b, 0])] for b in range(B)], [0] * B, 0
    while min(at) < steps - 1:
        tokens, parents = base.draft(host, at, N, vocab, g)
        logits = model.forward(tokens, pool, table, committed, parents, status)
        r = sv.spec_verify_tree(logits, tokens, parents, mode=0, dev_status=status)
        sv.spec_verify_logprobs(logits, r.out_tokens, row_index=r.accept_index, top_n=4, dev_status=status)
        committed, _ = sv.spec_verify_kv_compact(pool, table, committed, r.accept_index, r.accept_len, stacked=True,
                                                 dev_status=status)
        new, n = r.out_tokens.tolist(), r.accept_len.tolist()
        for b in range(B):
            if at[b] < steps - 1:
                got[b] += new[b][: n[b] + 1]
            at[b] = min(at[b] + n[b] + 1, steps - 1)
            committed[b] = min(int(committed[b]), prompt_len + steps)  # requests that are done wait for the others
        rounds += 1
        if verbose:
            print(f"round {rounds}: accepted {n}")
    first = torch.zeros(B, dtype=torch.int32, device="cuda")
    keys = sv.spec_verify_kv_read(pool[0], pool[1], table, first, int(committed.max()), num_rows=committed,
                                  kv_heads=model.kv_heads, head_dim=model.head_dim, dtype=torch.bfloat16,
                                  dev_status=status).k
    assert int(status) == 0, sv.spec_verify_strerror(int(status))
    return host, torch.tensor([x[:steps] for x in got]), keys, committed.cpu(), (steps - 1) / rounds


if __name__ == "__main__":
    text, got, keys, committed, rate = run(verbose=True)
    same = float((text == got).float().mean())
    print(f"tokens that agree with token-by-token decoding: {same:.3f}; tokens per step of the slowest request {rate:.2f}")
    sys.exit(0 if same == 1.0 else 1)
