"""Decoding rounds of a small target model with random weights: every step between the
drafter's logits and the user's tokens runs in the library.

A round for a batch of requests of different lengths:
  build_tree_mask    the draft tree of every request, its ancestor mask and positions
  tree_attention     in each layer, all rows of the trees over the paged e4m3 context
  verify             the accepted path and the next token (greedy)
  kv_append          in each layer, the path's keys and values join the context
  token_logprobs     log-probability, rank and best alternatives of what was emitted
Prompts go through the same attention (mask None: a chain) and the same append, and
plain decoding is the tree of one node.  The model's own products are torch's.

    python examples/decode_rounds.py [--rounds N]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_draft_bf16_gb300 import dtree  # noqa: E402

V, H, LAYERS, HQ, HKV, D, PAGE = 2048, 256, 2, 8, 2, 64, 16
L, K, BUDGET = 8, 16, 40


class Model:
    """Attention layers between an embedding and a head; follow[token] is a likely next token."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.emb = torch.randn((V, H), generator=g).to(**bf16)
        self.head = (torch.randn((H, V), generator=g) / math.sqrt(H)).to(**bf16)
        self.qkv = [(torch.randn((H, (HQ + 2 * HKV) * D), generator=g) / math.sqrt(H)).to(**bf16) for _ in range(LAYERS)]
        self.out = [(torch.randn((HQ * D, H), generator=g) / math.sqrt(HQ * D)).to(**bf16) for _ in range(LAYERS)]
        self.follow = torch.randperm(V, generator=g).to(device)
        at = torch.arange(4096, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        self.rope = dtree.Rope(at.cos().float().to(device), at.sin().float().to(device))

    def forward(self, tokens, caches, workspace, status, **tree):
        """Logits [b, M, V] of the rows `tokens` [b, M] and each layer's keys and values, not in the caches yet."""
        x, kv = self.emb[tokens], []
        b, M = tokens.shape
        for i in range(LAYERS):
            y = torch.nn.functional.rms_norm(x, (H,)) @ self.qkv[i]
            q, k, v = (t.unflatten(-1, (-1, D)) for t in y.split((HQ * D, HKV * D, HKV * D), -1))  # slices, no copies
            o = dtree.tree_attention(caches[i], q, k, v, rope=self.rope, workspace=workspace, status=status, **tree)
            x = x + o.view(b, M, HQ * D) @ self.out[i]
            kv.append((k, v))
        logits = torch.nn.functional.rms_norm(x, (H,)) @ self.head
        return logits + 4.0 * torch.nn.functional.one_hot(self.follow[tokens], V).to(logits.dtype), kv

    def draft(self, tokens, generator):
        """A drafter's logits [b, L, V] for the L positions after `tokens` [b]: the likely chain under noise."""
        rows = []
        for _ in range(L):
            tokens = self.follow[tokens]
            rows.append(4.0 * torch.nn.functional.one_hot(tokens, V))
        noise = torch.randn((tokens.shape[0], L, V), generator=generator, device=tokens.device)
        return (torch.stack(rows, 1) + noise).to(torch.bfloat16)


def new_caches(batch, tokens, device="cuda"):
    """A cache per layer with pages for `tokens` tokens of each request; they share lengths and pages' numbers."""
    pages = -(-tokens // PAGE)
    caches = [dtree.PagedCache.empty(batch * pages, PAGE, HKV, D, batch, pages, device) for _ in range(LAYERS)]
    for c in caches:
        c.table.copy_(torch.randperm(batch * pages, generator=torch.Generator().manual_seed(1)).view(batch, pages))
    return caches


def append(model, caches, kv, length, status, **rows):
    """Every layer appends at the same length, which moves on once they all have."""
    for c, (k, v) in zip(caches, kv):
        dtree.kv_append(c, k, v, rope=model.rope, len_out=length, status=status, **rows)
    for c in caches:
        c.len.copy_(length)


def prefill(model, prompts, caches, status):
    """Prompts [b, P] padded with -1: all but each one's last token into the caches; returns those [b]."""
    count = (prompts >= 0).sum(1).to(torch.int32) - 1
    length = torch.empty_like(count)
    ws = dtree.attention_workspace(caches[0], prompts.shape[1], HQ)
    _, kv = model.forward(prompts.clamp(min=0), caches, ws, status, n_nodes=count)
    append(model, caches, kv, length, status, count=count)
    return prompts.gather(1, count[:, None].long())[:, 0]


def decode(model, prompts, rounds, top=4, seed=0):
    """Rounds of draft, verify and append.  Returns, per request, the emitted tokens and their
    log-probabilities and ranks, the caches, and the status words (all zero)."""
    b, dev = prompts.shape[0], prompts.device
    caches = new_caches(b, prompts.shape[1] + rounds * (L + 1), dev)
    status = torch.zeros((b,), dtype=torch.int32, device=dev)
    length = torch.empty((b,), dtype=torch.int32, device=dev)
    last = prefill(model, prompts, caches, status)
    p = dtree.Params(mode="ddtree", batch=b, L=L, V=V, K=K, B=BUDGET)
    tree = dtree.TreeBuffers.for_params(p, device=dev)
    mask, pos = dtree.alloc_mask(tree, dev)
    ws = dtree.attention_workspace(caches[0], tree.max_nodes, HQ)
    gen = torch.Generator(device=dev).manual_seed(seed)
    step = torch.arange(L + 1, device=dev)
    got = [[] for _ in range(b)]
    for _ in range(rounds):
        dtree.build_tree_mask(p, model.draft(last, gen), tree, mask, pos)
        tokens = tree.node_tok.long()
        tokens[:, 0] = last  # the root
        logits, kv = model.forward(tokens.clamp(min=0), caches, ws, status, mask=mask, pos=pos, n_nodes=tree.n_nodes)
        path, acc, nxt = dtree.verify(tree, logits.contiguous())
        append(model, caches, kv, length, status, rows=path, count=acc, count_add=1)
        # emitted: the accepted nodes' tokens, then the next one; token i comes from path node i's logits
        used = step <= acc[:, None]
        after = torch.cat((path[:, 1:], path[:, :1]), 1).clamp(min=0).long()
        said = torch.where(step < acc[:, None], tokens.gather(1, after), nxt[:, None].long())
        said = torch.where(used, said, -1).to(torch.int32)
        lp = dtree.token_logprobs(logits, said, top=top, rows=torch.where(used, path, -1).to(torch.int32))
        last = nxt.long()
        for i in range(b):
            n = int(acc[i]) + 1
            got[i] += list(zip(said[i, :n].tolist(), lp.logprob[i, :n].tolist(), lp.rank[i, :n].tolist()))
    return got, caches, status | tree.status


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=8)
    rounds = ap.parse_args().rounds
    model = Model()
    prompts = torch.full((3, 50), -1, device="cuda")
    for i, n in enumerate((1, 17, 50)):
        prompts[i, :n] = torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(i)).cuda()
    got, caches, status = decode(model, prompts, rounds)
    print("status", status.tolist(), "tokens held", caches[0].len.tolist())
    for i, g in enumerate(got):
        print("request %d: %d tokens in %d rounds, mean log-probability %.3f: %s"
              % (i, len(g), rounds, sum(x[1] for x in g) / len(g), [x[0] for x in g]))


if __name__ == "__main__":
    main()
