"""One step of speculative decoding with a draft tree, attention and cache included.

    python examples/cached_tree_step.py

A toy target model of one attention layer (random weights) holds its context in the 8-bit cache.  The step:

  candidates --spec_tree_rerank--> draft tree and its ancestor mask
  nodes' keys and values --spec_cache_append--> behind the context
  nodes' queries --spec_cache_attend, with the mask--> the target's logits of every node
  --spec_verify_tree--> accepted path and the target's own token
  accepted rows --spec_cache_append, index = path--> committed over the draft's rows
  --spec_cache_weights, of the accepted rows--> accumulated weight of every cached token
  --spec_cache_evict--> the drafter's small cache of the heaviest and the latest tokens
  drafter's single token --spec_cache_attend over the small cache--> its next distribution

The drafter's cache is lossy; verification keeps the target's distribution all the same.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verification_02_gb300 import api  # noqa: E402


class Toy:
    """Embedding, one attention layer with grouped heads, output head."""

    def __init__(self, vocab, heads, kv_heads, head_dim, device, g):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        width = heads * head_dim
        def w(*s):
            return (torch.randn(s, generator=g, device=device) / s[0] ** 0.5).bfloat16()
        self.embed = torch.randn((vocab, width), generator=g, device=device).bfloat16()
        self.wq, self.wk, self.wv = w(width, width), w(width, kv_heads * head_dim), w(width, kv_heads * head_dim)
        self.head = w(width, vocab) * 4

    def project(self, tokens):
        x = self.embed[tokens]
        B, n = tokens.shape
        q = (x @ self.wq).view(B, n, self.heads, self.head_dim)
        k = (x @ self.wk).view(B, n, self.kv_heads, self.head_dim)
        v = (x @ self.wv).view(B, n, self.kv_heads, self.head_dim)
        return q, k, v

    def logits(self, attended):
        return (attended.flatten(2) @ self.head).contiguous()


def step(B=4, context=700, candidates=96, nodes=24, depth=5, vocab=2048, heads=8, kv_heads=2, head_dim=128, page=64, keep=256,
         recent=64, temperature=1.0, seed=0, device="cuda"):
    """Returns what the step made, by name."""
    g = torch.Generator(device=device).manual_seed(seed)
    toy = Toy(vocab, heads, kv_heads, head_dim, device, g)
    per_request = -(-(context + nodes) // page)
    small = -(-keep // page)
    cache = api.spec_cache_new(B * (per_request + small), kv_heads, page, head_dim, device)
    pages = torch.randperm(B * (per_request + small), generator=g, device=device).to(torch.int32)
    table = pages[:B * per_request].view(B, per_request)
    small_table = pages[B * per_request:].view(B, small)

    # the prompts, of different lengths
    lens = torch.randint(context // 2, context + 1, (B,), generator=g, device=device, dtype=torch.int32)
    prompt = torch.randint(0, vocab, (B, context), generator=g, device=device)
    _, k, v = toy.project(prompt)
    done = api.spec_cache_append(cache, table, torch.zeros_like(lens), k, v, counts=lens)
    length = done["new_len"]

    # candidate nodes in the order they were made, every parent one of the nodes before; the drafter's confidence in each
    parents = torch.full((B, candidates), -1, dtype=torch.int32, device=device)
    level = torch.zeros((B, candidates), dtype=torch.int32, device=device)
    for i in range(1, candidates):
        p = torch.randint(max(0, (i - 1) // 3 - 2), (i - 1) // 3 + 1, (B,), generator=g, device=device)
        p = torch.where(level.gather(1, p[:, None])[:, 0] < depth, p, 0)
        parents[:, i] = p
        level[:, i] = level.gather(1, p[:, None])[:, 0] + 1
    conf = 0.3 + 0.7 * torch.rand((B, candidates), generator=g, device=device)
    tokens = torch.randint(0, vocab, (B, candidates), generator=g, device=device).to(torch.int32)
    tree = api.spec_tree_rerank(parents, conf, nodes, depth, node_tok=tokens)

    # the target's forward over the tree
    q, k, v = toy.project(tree["sel_tok"].long())
    api.spec_cache_append(cache, table, length, k, v)
    attended = api.spec_cache_attend(q, cache, table, length, mask=tree["mask"])
    target = toy.logits(attended["out"])
    draft = (target.float() + torch.randn(target.shape, generator=g, device=device)).bfloat16()  # a drafter that is nearly right
    u = torch.rand((B, nodes + 1), generator=g, device=device)
    verdict = api.spec_verify_tree(target, draft, tree["sel_parents"], tree["sel_tok"], u, temperature, depth)

    # commit the accepted path, and count what its rows looked at
    path, rows = verdict["path_nodes"], verdict["n_emit"]
    committed = api.spec_cache_append(cache, table, length, k, v, index=path, counts=rows)
    weights = api.spec_cache_weights(q, attended["lse"], cache, table, length, index=path, counts=rows)

    # the drafter's cache, and its next token's attention
    kept = api.spec_cache_evict(cache, table, committed["new_len"], weights["weights"], keep, recent, small_table)
    last = verdict["out_tokens"].gather(1, (rows - 1).clamp(min=0).long()[:, None])
    q1, k1, v1 = toy.project(last.long())
    drafted = None
    if keep % page:  # room for the token in the last page
        api.spec_cache_append(cache, small_table, kept["new_len"], k1, v1)
        drafted = api.spec_cache_attend(q1, cache, small_table, kept["new_len"])
    return dict(cache=cache, table=table, small_table=small_table, length=length, tree=tree, attended=attended, q=q, k=k, v=v,
                verdict=verdict, committed=committed, weights=weights, kept=kept, drafted=drafted, q1=q1, k1=k1, v1=v1)


if __name__ == "__main__":
    r = step(keep=250)
    torch.cuda.synchronize()
    print("contexts          ", r["length"].tolist())
    print("accepted nodes    ", r["verdict"]["accepted_len"].tolist())
    print("emitted tokens    ", [t[:n] for t, n in zip(r["verdict"]["out_tokens"].tolist(), r["verdict"]["n_emit"].tolist())])
    print("committed contexts", r["committed"]["new_len"].tolist())
    print("drafter's cache   ", r["kept"]["new_len"].tolist(), "of the heaviest and latest tokens")
    print("drafter attends   ", tuple(r["drafted"]["out"].shape), "log-sum-exp", [round(x, 3) for x in r["drafted"]["lse"][:, 0, 0].tolist()])
