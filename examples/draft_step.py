"""Speculative decoding steps over a paged 8-bit cache, on a toy model.

Each step of each sequence: its last token and a block of drafts get their
places in the cache (``sv_kv_plan``), their keys and values are written
(``sv_kv_append``), their queries read the cache (``sv_kv_attention``), and one
token is drawn from each position's filtered logits (``sv_sample_rows``).  The
drafts that equal the draws before them are kept; the first other draw is the
next token.  The drafter draws with the same uniforms, so that it agrees often.

The model is one attention layer with random weights: it shows the calls, not
language.  Run: python examples/draft_step.py
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_block_verification_gb300 as dbv  # noqa: E402


class Toy:
    def __init__(self, V, Hq, H, D, seed, dev):
        g = torch.Generator(device=dev).manual_seed(seed)
        E = 256
        w = lambda *s: (torch.randn(s, generator=g, device=dev) * s[0] ** -0.5).bfloat16()  # noqa: E731
        self.Hq, self.H, self.D = Hq, H, D
        self.embed = (torch.randn((V, E), generator=g, device=dev)).bfloat16()
        self.q, self.kv, self.o = w(E, Hq * D), w(E, 2 * H * D), w(Hq * D, E)
        self.head = w(E, V) * 3

    def keys_values(self, x):
        return (x @ self.kv).unflatten(1, (2, self.H, self.D)).unbind(1)

    def queries(self, x):
        return (x @ self.q).unflatten(1, (self.Hq, self.D))

    def logits(self, x, mixed=None):
        return (x if mixed is None else x + mixed.flatten(1) @ self.o) @ self.head


def run(steps=6, B=8, K=4, V=32000, Hq=8, H=2, D=128, block=16, pages=256, seed=0):
    """Returns (tokens of each sequence, state of the cache, accepted drafts)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    i32 = torch.int32
    m = Toy(V, Hq, H, D, seed, dev)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    cols = pages // B
    cache = [torch.zeros((pages, H, block, D), dtype=torch.float8_e4m3fn, device=dev)
             for _ in range(2)]
    scale = [torch.ones((pages, H), device=dev) for _ in range(2)]
    table = torch.full((B, cols), -1, dtype=i32, device=dev)
    free_ids = torch.arange(pages, dtype=i32, device=dev)
    free_pos = torch.tensor([0, pages], dtype=torch.int64, device=dev)
    cached, held = (torch.zeros(B, dtype=i32, device=dev) for _ in range(2))
    n = K + 1
    new = torch.full((B,), n, dtype=i32, device=dev)
    last = torch.randint(0, V, (B,), generator=g, device=dev, dtype=i32)
    filters = dict(temperature=torch.full((B * n,), 0.8, device=dev),
                   top_k=torch.full((B * n,), 50, dtype=i32, device=dev),
                   top_p=torch.full((B * n,), 0.95, device=dev))
    draft_filters = {k: v[:B].contiguous() for k, v in filters.items()}
    told, accepted = [[] for _ in range(B)], 0
    for _ in range(steps):
        u = torch.rand((B, n), generator=g, device=dev)
        # the drafter: the same embedding and head, without attention
        block_ids = [last]
        for i in range(K):
            x = m.embed[block_ids[-1].long()]
            block_ids.append(dbv.sv_sample_rows(m.logits(x), u[:, i].contiguous(),
                                                **draft_filters)["token"])
        ids = torch.stack(block_ids, 1)
        x = m.embed[ids.reshape(-1).long()]
        plan = dbv.sv_kv_plan(cached, new, held, table, free_ids, free_pos, block, B * n)
        held, free_pos = plan["held"], plan["free_pos"]
        k, v = m.keys_values(x)
        dbv.sv_kv_append(k, v, plan["slot"], *cache, *scale)
        mixed = dbv.sv_kv_attention(m.queries(x), *cache, *scale, table, plan["kv_len"],
                                    plan["cu_new"])["out"]
        out = dbv.sv_sample_rows(m.logits(x, mixed), u.reshape(-1), **filters)
        token = out["token"].reshape(B, n)
        agree = torch.cumprod((token[:, :K] == ids[:, 1:]).to(i32), 1).sum(1, dtype=i32)
        # the block's last token and the agreed drafts stay; the rest are overwritten
        cached = cached + 1 + agree
        last = token.gather(1, agree[:, None].long())[:, 0]
        for b, a in enumerate(agree.tolist()):
            told[b] += token[b, :a + 1].tolist()
            accepted += a
    # the sequences end: their pages go back to the queue
    zero = torch.zeros_like(cached)
    end = dbv.sv_kv_plan(zero, zero, held, table, free_ids, free_pos, block, 0)
    dbv.default_handle(dev).sync_status()
    state = dict(cached=cached, held=held, free_pos=free_pos, end_free=end["free_pos"],
                 end_held=end["held"], pages=pages, block=block, free_ids=free_ids)
    return told, state, accepted


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=6)
    a = p.parse_args()
    told, state, accepted = run(steps=a.steps)
    for b, t in enumerate(told):
        print("sequence %d: %s" % (b, t))
    print("%d tokens in %d steps, %d drafts kept" % (sum(map(len, told)), a.steps, accepted))
