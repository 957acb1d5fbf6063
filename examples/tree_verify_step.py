"""Speculative decoding with a tree of drafts, a small decoder end to end through the library:

    for each layer   spec_verify_kv_append   the nodes' rotated keys and values into the paged cache
                     spec_verify_attention   the nodes over the committed prefix and their ancestors
    then             spec_verify_tree        the accepted path and the emitted tokens
                     spec_verify_logprobs    their log probabilities and alternatives
                     spec_verify_kv_compact  the accepted path's cache rows behind the prefix

The decoder's weights are random.  It first decodes token by token (N = 1, the same calls), then again
with trees whose drafts follow that text at random, and the two have to agree.

    python examples/tree_verify_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import speculative_decoding_verification_verify_gb300 as sv  # noqa: E402


class Decoder:
    """A decoder with grouped key heads.  Linear layers in fp32, cache and attention in bf16."""

    def __init__(self, vocab=997, width=256, layers=2, heads=8, kv_heads=2, head_dim=64, max_pos=256, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.embed, self.head = r(vocab, width), r(width, vocab) * 0.5
        rows = (heads + 2 * kv_heads) * head_dim
        self.layers = [dict(qkv=r(width, rows) / width ** 0.5, out=r(heads * head_dim, width) / width ** 0.5,
                            up=r(width, 2 * width) / width ** 0.5, down=r(2 * width, width) / width ** 0.5)
                       for _ in range(layers)]
        freq = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64, device="cuda") / head_dim)
        angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    def cache(self, B, max_pos, seed=0):
        """One pool for all layers' keys and values ([planes, slots, row]), slots in random order."""
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        row = self.kv_heads * self.head_dim
        pool = torch.zeros((2 * len(self.layers), B * max_pos, row), dtype=torch.bfloat16, device="cuda")
        return pool, torch.randperm(B * max_pos, generator=g, device="cuda").view(B, max_pos).int()

    def forward(self, tokens, pool, slot_table, committed, parents=None, status=None):
        """Logits [B, N, vocab] of new nodes behind each request's committed positions."""
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        B, N = tokens.shape
        H, K, D = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens.long()]
        for i, w in enumerate(self.layers):
            qkv = (norm(x) @ w["qkv"]).to(torch.bfloat16)
            q, k, v = (t.unflatten(2, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 2))
            kc, vc = pool[2 * i].view(-1, K, D), pool[2 * i + 1].view(-1, K, D)
            q = sv.spec_verify_kv_append(q, k, v, kc, vc, slot_table, committed, self.cos_sin, parents=parents,
                                         dev_status=status)
            a = sv.spec_verify_attention(q, kc, vc, slot_table, committed, parents=parents, dev_status=status).out
            x = x + a.float().flatten(2) @ w["out"]
            x = x + torch.nn.functional.silu(norm(x) @ w["up"]) @ w["down"]
        return norm(x) @ self.head


def decode(model, prompt, steps, status):
    """Greedy decoding token by token: the continuation [B, steps] and its log probabilities."""
    B, P = prompt.shape
    pool, table = model.cache(B, P + steps + 1, seed=1)
    committed = torch.zeros(B, dtype=torch.int32, device="cuda")
    logits = model.forward(prompt, pool, table, committed, status=status)[:, -1:]
    committed += P
    out, said = [], []
    for _ in range(steps):
        token = logits.argmax(-1).int()
        out.append(token)
        said.append(sv.spec_verify_logprobs(logits.contiguous(), token, dev_status=status).logprobs)
        logits = model.forward(token, pool, table, committed, status=status)
        committed += 1
    return torch.cat(out, 1), torch.cat(said, 1)


def draft(text, at, N, vocab, g):
    """A random tree behind each request's last token: node tokens [B, N] and parents [B, N].  A node's
    token is the text's next one with probability 0.7."""
    B = text.shape[0]
    tokens, parents = torch.zeros((B, N), dtype=torch.int32), torch.full((B, N), -1, dtype=torch.int32)
    for b in range(B):
        depth, used = [0] * N, [set() for _ in range(N)]
        tokens[b, 0] = text[b, at[b]]
        for j in range(1, N):
            p = int(torch.randint(max(0, j - 3), j, (1,), generator=g))
            depth[j] = depth[p] + 1
            want = int(text[b, min(at[b] + depth[j], text.shape[1] - 1)])
            while want in used[p] or float(torch.rand(1, generator=g)) > 0.7:
                want = int(torch.randint(0, vocab, (1,), generator=g))
                if want not in used[p]:
                    break
            used[p].add(want)
            tokens[b, j], parents[b, j] = want, p
    return tokens.cuda(), parents.cuda()


def run(B=3, prompt_len=37, steps=48, N=8, vocab=997, seed=0, verbose=False):
    """Decode, then decode with trees; returns (text, log probabilities, both again from the trees, tokens per step)."""
    g = torch.Generator()
    g.manual_seed(seed)
    model = Decoder(vocab=vocab, seed=seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prompt = torch.randint(0, vocab, (B, prompt_len), generator=g).int().cuda()
    text, said = decode(model, prompt, steps, status)
    host = text.cpu()

    pool, table = model.cache(B, prompt_len + steps + 2 * N, seed=2)
    committed = torch.zeros(B, dtype=torch.int32, device="cuda")
    model.forward(prompt, pool, table, committed, status=status)
    committed += prompt_len
    got, got_said, at, rounds = [[int(host[b, 0])] for b in range(B)], [[] for _ in range(B)], [0] * B, 0
    while min(at) < steps - 1:
        tokens, parents = draft(host, at, N, vocab, g)
        logits = model.forward(tokens, pool, table, committed, parents, status)
        r = sv.spec_verify_tree(logits, tokens, parents, mode=0, dev_status=status)
        lp = sv.spec_verify_logprobs(logits, r.out_tokens, row_index=r.accept_index, top_n=4, dev_status=status)
        committed, _ = sv.spec_verify_kv_compact(pool, table, committed, r.accept_index, r.accept_len, stacked=True,
                                                 dev_status=status)
        new, logp, n = r.out_tokens.tolist(), lp.logprobs.tolist(), r.accept_len.tolist()
        for b in range(B):
            if at[b] < steps - 1:
                got[b] += new[b][: n[b] + 1]
                got_said[b] += logp[b][: n[b] + 1]
            at[b] = min(at[b] + n[b] + 1, steps - 1)
            committed[b] = min(int(committed[b]), prompt_len + steps)  # requests that are done wait for the others
        rounds += 1
        if verbose:
            print(f"round {rounds}: accepted {n}")
    assert int(status) == 0, sv.spec_verify_strerror(int(status))
    got = torch.tensor([x[:steps] for x in got])
    got_said = torch.tensor([x[: steps - 1] for x in got_said])
    return host, said.cpu(), got, got_said, (steps - 1) / rounds


if __name__ == "__main__":
    text, said, got, got_said, rate = run(verbose=True)
    same = float((text == got).float().mean())
    print(f"tokens that agree with token-by-token decoding: {same:.3f}; largest difference of their log probabilities "
          f"{float((said[:, 1:] - got_said).abs().max()):.4f}; tokens per step of the slowest request {rate:.2f}")
    sys.exit(0 if same == 1.0 else 1)
