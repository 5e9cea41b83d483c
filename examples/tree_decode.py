"""Decoding with trees of drafted tokens: every step on the operators of this
package, over a small random target model.

A round: `plan` gives pages, slots, positions and ancestor masks; per layer
`append` norms and rotates queries and keys and writes the cache, `attend` runs
the tree over context and ancestors; `spec_lmhead_logits` gives the logits of all
nodes; a greedy `Verifier` run accepts along each path of the tree; `keep` moves
the longest accepted path's keys and values together.  The prompt is a round
too: a chain without drafts.

    python examples/tree_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_42_gb300 as sv  # noqa: E402

# node 0 is the last emitted token; its three likeliest successors, two of each of theirs
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3]
PATHS = [[0, 1, 4], [0, 1, 5], [0, 2, 6], [0, 2, 7], [0, 3, 8], [0, 3, 9]]


class Target:
    """A random decoder with per-head norms and rotary positions, bf16."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, head_dim=64, vocab=512, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers, self.hq, self.hkv, self.d, self.vocab = layers, q_heads, kv_heads, head_dim, vocab
        h = self.hidden = q_heads * head_dim

        def w(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.embed = w(vocab, h, std=1.0)
        self.qkv = [w(h, (q_heads + 2 * kv_heads) * head_dim, std=h ** -0.5) for _ in range(layers)]
        self.proj = [w(h, h, std=h ** -0.5) for _ in range(layers)]
        self.norms = [(1 + 0.1 * w(2, head_dim, std=1.0)) for _ in range(layers)]
        self.head = w(h, vocab, std=2 * h ** -0.5)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()

    @staticmethod
    def unit(x):
        f = x.float()
        return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """The target with its paged cache, for a batch of requests."""

    def __init__(self, model: Target, batch: int, max_tokens: int, page_size=16, table_width=32):
        self.m, self.batch = model, batch
        pages = batch * table_width
        self.tc = sv.TreeCache(max_batch=batch, max_tokens=max_tokens, q_heads=model.hq, kv_heads=model.hkv,
                               head_dim=model.d, dtype="bf16", page_size=page_size, num_pages=pages,
                               table_width=table_width)
        shape = (model.layers, pages, page_size, model.hkv, model.d)
        self.k, self.v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.pool = self.tc.new_pool(batch)
        self.ctx = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.ver = sv.Verifier(vocab=model.vocab, max_batch=batch * len(PATHS), max_k=2, dtype=torch.float32)

    def forward(self, tokens, n_tokens, parents=None):
        """Logits [B, T, vocab] of the nodes' tokens, their keys and values in the cache, and
        the plan's status: where it is not 0 the request got no pages, and its logits mean nothing."""
        m, pool = self.m, self.pool
        B, T = tokens.shape
        plan = self.tc.plan(self.ctx, n_tokens, pool["held"], pool["ring"], pool["free_pages"],
                            pool["block_table"], parents=parents, max_tokens=T)
        pool["held"], pool["ring"] = plan["held"], plan["ring"]
        x = m.embed[tokens.long()]
        for i in range(m.layers):
            qkv = m.unit(x) @ m.qkv[i]
            q, k, v = (y.unflatten(-1, (-1, m.d)) for y in
                       qkv.split([m.hq * m.d, m.hkv * m.d, m.hkv * m.d], dim=-1))
            q = self.tc.append(q, k, v, self.k[i], self.v[i], plan["slot_map"], plan["positions"], n_tokens,
                               q_weight=m.norms[i][0], k_weight=m.norms[i][1], cos_sin=m.cos_sin)
            a = self.tc.attend(q, self.k[i], self.v[i], pool["block_table"], self.ctx, n_tokens,
                               tree_mask=plan.get("tree_mask"), lse=False)["out"]
            x = x + a.reshape(B, T, -1) @ m.proj[i]
        h = m.unit(x).reshape(B * T, -1).contiguous()
        logits = torch.empty(B * T, m.vocab, device="cuda")
        sv.spec_lmhead_logits(h.data_ptr(), m.head.data_ptr(), B * T, m.hidden, m.vocab, logits.data_ptr(),
                              torch.cuda.current_stream().cuda_stream)
        return logits.view(B, T, -1), plan["row_status"]

    def prompt(self, tokens, n_tokens):
        """Takes the prompts in; the token that follows each."""
        logits, status = self.forward(tokens, n_tokens)
        if status.any():
            raise RuntimeError("the cache has too few pages for these prompts")
        self.ctx = self.ctx + n_tokens
        return logits[torch.arange(self.batch), n_tokens.long() - 1].argmax(-1).int()

    def draft(self, root):
        """Tokens [B, nodes] of the tree under root: a cheap bigram guess (embedding times LM head)."""
        m = self.m

        def top(tokens, k):
            return (m.unit(m.embed[tokens.long()]) @ m.head).float().topk(k, -1).indices.int()

        first = top(root, 3)
        return torch.cat([root[:, None], first, top(first, 2).flatten(1)], 1)

    def round(self, root):
        """One tree: the accepted tokens and the next root, [B, 3] padded with -1, and their number
        (0 for a request that the cache has no pages for: it waits)."""
        B, T = self.batch, len(PARENTS)
        tokens = self.draft(root)
        n = torch.full((B,), T, dtype=torch.int32, device="cuda")
        parents = torch.tensor(PARENTS, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
        logits, status = self.forward(tokens, n, parents)
        # every root-to-leaf path is a sequence of the verify step
        paths = torch.tensor(PATHS, device="cuda")
        out = self.ver.run(logits[:, paths].flatten(0, 1).contiguous(), None,
                           tokens[:, paths[:, 1:]].flatten(0, 1).contiguous(), temperature=0.0)
        accepted = out["num_accepted"].view(B, -1)
        best = accepted.argmax(1)  # the first of the longest
        rows = torch.arange(B, device="cuda")
        kept = accepted[rows, best] + 1  # the root is kept in any case
        path = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        path[:, :3] = paths[best]
        self.ctx = self.tc.keep(self.k, self.v, self.pool["block_table"], self.ctx, n, path, kept,
                                plan_status=status)["ctx_len"]
        emitted = out["tokens"].view(B, len(PATHS), 3)[rows, best]
        return emitted, torch.where(status == 0, kept, 0)

    def close(self):
        self.tc.close()
        self.ver.close()


def decode(prompts, lengths, steps, model=None):
    """`steps` rounds; the emitted tokens of every request (lists, the first from the prompt)."""
    dec = Decoder(model or Target(), prompts.shape[0], prompts.shape[1])
    root = dec.prompt(prompts, lengths)
    texts = [[int(t)] for t in root]
    for _ in range(steps):
        emitted, n = dec.round(root)
        for b, (row, k) in enumerate(zip(emitted.tolist(), n.tolist())):
            texts[b] += row[:k]
        last = emitted[torch.arange(len(texts), device="cuda"), n.long().clamp(min=1) - 1]
        root = torch.where(n > 0, last, root)
    assert dec.tc.check() == sv.SPEC_OK
    dec.close()
    return texts


if __name__ == "__main__":
    lens = torch.tensor([5, 40, 17, 1], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 512, (4, 40), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(1))
    for line in decode(ids, lens, 12):
        print(len(line), "tokens in 12 rounds:", line)
