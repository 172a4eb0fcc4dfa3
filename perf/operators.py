"""The serving operators around the verify calls: cases, inputs and plain forms.

A draft block goes through four operators between two verify calls: the plan
that gives the block's tokens their places in the paged cache, the append that
writes their keys and values in 8 bits, the attention that reads the cache,
and the draw of tokens from filtered logit rows.  Each case here is one call
of one of them.

``run(state)`` computes it in elementary torch operations where ``own`` is
false and through the package's entry points where it is true; ``exact`` is
the same result from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
SCALE_EXP = 40          # cache scales are powers of two in [2^-40, 2^40]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 64 sequences with up to 16 drafts and the next token each
        dict(name="plan_draft_64", op="plan", B=64, block=64, ctx=4096, new=17, mix=1),
        # a large mixed batch: some sequences bring long prompts, some only a token
        dict(name="plan_mixed_1024", op="plan", B=1024, block=16, ctx=16384, new=96, mix=2),
        # one token for each of eight sequences: the call's latency
        dict(name="append_8x1", op="append", B=8, block=64, ctx=2048, new=1, Hkv=8, D=128,
             dtype="bf16", mix=3),
        # the draft blocks of 64 sequences
        dict(name="append_64x17", op="append", B=64, block=64, ctx=4096, new=17, Hkv=8, D=128,
             dtype="bf16", mix=4),
        # prompts of several thousand tokens
        dict(name="append_prompts", op="append", B=8, block=32, ctx=1024, new=6144, Hkv=8, D=128,
             dtype="bf16", mix=5),
        # one token of one sequence: the call's latency
        dict(name="attend_1x1", op="attend", B=1, block=16, ctx=1024, new=1, Hq=32, Hkv=8, D=128,
             tree=False, mix=6),
        # single-token decoding of 128 sequences of unequal length
        dict(name="attend_128x1", op="attend", B=128, block=64, ctx=8192, new=1, Hq=32, Hkv=8,
             D=128, tree=False, mix=7),
        # draft blocks of 16 tokens and one more, 64 sequences
        dict(name="attend_64x17", op="attend", B=64, block=64, ctx=4096, new=17, Hq=32, Hkv=8,
             D=128, tree=False, mix=8),
        # draft trees of up to 64 nodes
        dict(name="attend_tree_32x64", op="attend", B=32, block=32, ctx=2048, new=64, Hq=32,
             Hkv=8, D=128, tree=True, mix=9),
        # few sequences, long contexts, small heads
        dict(name="attend_long_4x5", op="attend", B=4, block=128, ctx=131072, new=5, Hq=48,
             Hkv=8, D=64, tree=False, mix=10),
        # one row of the smallest vocabulary: the call's latency
        dict(name="sample_1", op="sample", rows=1, V=32000, dtype="f32", spread=3.0, mix=11),
        # the rows of 64 sequences with 16 drafts each
        dict(name="sample_1088", op="sample", rows=1088, V=128256, dtype="bf16", spread=2.0,
             mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "attend", "attend", "sample"))
    block = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    if op == "plan":
        return dict(op=op, B=_log_int(rng, 1, 1024), block=block, ctx=_log_int(rng, 1, 16384),
                    new=_log_int(rng, 1, 96), mix=mix)
    if op == "append":
        B, H, D = _log_int(rng, 1, 256), rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128))
        new = _log_int(rng, 1, max(2, min(4096, 6144 * 8 * 8 * 128 // (B * H * D * 2))))
        return dict(op=op, B=B, block=block, ctx=_log_int(rng, 1, 4096), new=new, Hkv=H, D=D,
                    dtype=rng.choice(("bf16", "f32")), mix=mix)
    if op == "attend":
        H, G, D = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 6, 7, 8, 12)), \
            rng.choice((64, 128))
        B, new = _log_int(rng, 1, 160), _log_int(rng, 1, 72)
        room = min((1 << 28) // (B * H * D), (1 << 27) // (B * H * G * new))
        return dict(op=op, B=B, block=block, ctx=_log_int(rng, 1, max(2, min(131072, room))),
                    new=new, Hq=H * G, Hkv=H, D=D, tree=new > 1 and rng.random() < 0.4, mix=mix)
    V = rng.choice((rng.randrange(5, 2000), rng.randrange(30000, 34000), 32000, 50257, 128256,
                    151936))
    dtype = rng.choice(("bf16", "f32"))
    most = 1088 * 128256 // V // (1 if dtype == "bf16" else 2)
    return dict(op=op, rows=_log_int(rng, 1, min(1200, most)), V=V, dtype=dtype,
                spread=rng.choice((1.0, 2.0, 3.0, 5.0)), mix=mix)


def _lengths(case):
    """(tokens in the cache, tokens that come) of each sequence; by the case alone."""
    r = random.Random(case["mix"])
    B, ctx, new = case["B"], case["ctx"], case["new"]
    cached = [r.randint((ctx + 1) // 2, ctx) for _ in range(B)]
    fresh = [r.randint((new + 1) // 2, new) for _ in range(B)]
    cached[0], fresh[0] = ctx, new
    if case["op"] == "plan" and B > 3:
        # a sequence that has ended, one that waits, one that starts
        cached[1], fresh[1] = 0, 0
        fresh[2] = 0
        cached[3] = 0
    return cached, fresh


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(pages, H, bs, D, g):
    """Stored keys or values (float8) and scales of ordinary size."""
    x = torch.empty((pages, H, bs, D), dtype=torch.float8_e4m3fn, device=DEV)
    x.copy_((torch.randn(x.shape, generator=g, device=DEV) * 90).clamp_(-448, 448))
    e = torch.randint(-8, -5, (pages, H), generator=g, device=DEV).float()
    return x, torch.exp2(e)


def _paged(case, seed, g):
    """Lengths, a table of shuffled pages, and the places of the new tokens."""
    cached, fresh = _lengths(case)
    B, bs = case["B"], case["block"]
    want = [(c + n + bs - 1) // bs for c, n in zip(cached, fresh)]
    pages = sum(want) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    cols = max(max(want), 1)
    w = _i32(want)
    start = torch.cumsum(w, 0) - w
    j = torch.arange(cols, device=DEV)
    at = (start[:, None] + j).clamp_(max=pages - 1)
    table = torch.where(j < w[:, None], order[at], -1)
    n = _i32(fresh)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(n, 0)
    T = sum(fresh)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = _i32(cached)[b] + t - cu[b]
    slot = (table[b, pos // bs] * bs + pos % bs).to(torch.int32)
    return dict(table=table.contiguous(), cu=cu, slot=slot.contiguous(),
                kv_len=_i32([c + f for c, f in zip(cached, fresh)]), pages=pages, T=T)


def _trees(case, seed, cu_rows):
    """Ancestor bits of random draft trees, and which new tokens each token sees."""
    cached, fresh = _lengths(case)
    words = (case["new"] + 31) // 32
    r = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))
    bits = np.zeros((cu_rows, words), np.uint32)
    at = 0
    for n in fresh:
        for i in range(n):
            if i and r.rand() < 0.95:
                bits[at + i] = bits[at + r.randint(max(0, i - 6), i)]
            bits[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += n
    return torch.from_numpy(bits.view(np.int32)).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "plan":
        cached, fresh = _lengths(case)
        B, bs = case["B"], case["block"]
        r = random.Random(int(seed) * 13 + case["mix"])
        # drafts rejected by the last step leave pages over; most need more
        held = [max(0, (c + r.randint(0, case["new"]) + bs - 1) // bs) if r.random() < 0.3
                else (c + bs - 1) // bs for c in cached]
        if B > 3:
            held[1] = r.randint(0, (case["ctx"] + bs - 1) // bs)
        most = [(c + case["new"] + bs - 1) // bs for c in cached]
        if B > 3:
            most[1] = (case["ctx"] + bs - 1) // bs
        cols, ring = max(most), sum(most) + 5
        ids = torch.randperm(ring, generator=g, device=DEV).to(torch.int32)
        h = _i32(held)
        start = torch.cumsum(h, 0) - h
        j = torch.arange(cols, device=DEV)
        table = torch.where(j < h[:, None], ids[(start[:, None] + j).clamp_(max=ring - 1)], -1)
        used = sum(held)
        first = r.randrange(ring)
        free = torch.full((ring,), -1, dtype=torch.int32, device=DEV)
        free[(first + torch.arange(ring - used, device=DEV)) % ring] = ids[used:]
        s.update(cached=_i32(cached), new=_i32(fresh), held=h, table=table.contiguous(),
                 free_ids=free, max_tokens=sum(fresh) + 7,
                 free_pos=torch.tensor([first, first + ring - used], dtype=torch.int64,
                                       device=DEV))
        return s
    if op == "append":
        s.update(_paged(case, seed, g))
        H, D = case["Hkv"], case["D"]
        dt = DTYPES[case["dtype"]]
        for n in "kv":
            # channels of unequal size, as keys have them
            gain = torch.exp(torch.randn((1, H, D), generator=g, device=DEV) * 0.5)
            s[n] = (torch.randn((s["T"], H, D), generator=g, device=DEV) * gain).to(dt)
            s[n + "_cache"], s[n + "_scale"] = _cache(s["pages"], H, case["block"], D, g)
        return s
    if op == "attend":
        s.update(_paged(case, seed, g))
        H, D = case["Hkv"], case["D"]
        for n in "kv":
            s[n + "_cache"], s[n + "_scale"] = _cache(s["pages"], H, case["block"], D, g)
        s["q"] = (torch.randn((s["T"], case["Hq"], D), generator=g, device=DEV) * 1.5).to(
            torch.bfloat16)
        s["mask"] = _trees(case, seed, s["T"]) if case["tree"] else None
        return s
    R, V = case["rows"], case["V"]
    x = torch.randn((R, V), generator=g, device=DEV) * case["spread"]
    # a few likely tokens in most rows
    top = torch.randint(0, V, (R, 12), generator=g, device=DEV)
    lift = torch.rand((R, 12), generator=g, device=DEV) * 10 * \
        (torch.rand((R, 1), generator=g, device=DEV) < 0.8)
    x.scatter_add_(1, top, lift)
    s["logits"] = x.to(DTYPES[case["dtype"]])
    pick = lambda v: torch.tensor(v, device=DEV)[torch.randint(  # noqa: E731
        0, len(v), (R,), generator=g, device=DEV)]
    s["u"] = torch.rand(R, generator=g, device=DEV)
    s["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2])
    s["top_k"] = pick([0, 0, 0, 20, 40, 50, 1000]).to(torch.int32)
    s["top_p"] = pick([1.0, 0.8, 0.9, 0.95, 0.95, 0.99])
    s["min_p"] = pick([0.0, 0.0, 0.0, 0.02, 0.1])
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _plan_plain(s):
    bs, table, ring = s["case"]["block"], s["table"], s["free_ids"]
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    R, (B, cols) = ring.numel(), table.shape
    total = cached + new
    want = (total + bs - 1) // bs
    take, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    t0, g0 = torch.cumsum(take, 0) - take, torch.cumsum(give, 0) - give
    head, tail = s["free_pos"][0], s["free_pos"][1]
    j = torch.arange(cols, device=DEV)
    gets = (j >= held[:, None]) & (j < want[:, None])
    src = (head + t0[:, None] + j - held[:, None]) % R
    out_table = torch.where(gets, ring[src], table)
    gives = (j >= want[:, None]) & (j < held[:, None])
    dst = torch.where(gives, (tail + g0[:, None] + j - want[:, None]) % R, R)
    out_ring = torch.cat([ring, ring[:1]]).scatter_(0, dst.reshape(-1), table.reshape(-1))[:R]
    cu = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(s["max_tokens"], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = cached[b] + t - cu[b]
    live = t < cu[B]
    page = out_table[b, (pos // bs).clamp(max=cols - 1)].long()
    i = lambda v: v.to(torch.int32)  # noqa: E731
    return dict(table=out_table, free_ids=out_ring, held=i(want), kv_len=i(total), cu_new=i(cu),
                free_pos=torch.stack([head + take.sum(), tail + give.sum()]),
                slot=i(torch.where(live, page * bs + pos % bs, -1)),
                pos=i(torch.where(live, pos, -1)))


def _needed_exp(amax):
    """Least e with amax <= 448 * 2^e, within the range of the scales."""
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax == 0, -SCALE_EXP, e).clamp(-SCALE_EXP, SCALE_EXP)


def _append_plain(s):
    bs, slot = s["case"]["block"], s["slot"].long()
    page, off = slot // bs, slot % bs
    pages = s["pages"]
    first = torch.full((pages,), bs, device=DEV).scatter_reduce(0, page, off, "amin")
    hit = first < bs
    row = torch.arange(bs, device=DEV)
    kept = hit[:, None] & (row < first[:, None])
    out = {}
    for n in "kv":
        x, cache, scale = s[n].float(), s[n + "_cache"], s[n + "_scale"]
        H = x.shape[1]
        amax = torch.zeros((pages, H), device=DEV).scatter_reduce(
            0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        need = torch.exp2(_needed_exp(amax).float())
        grown = torch.where((first > 0)[:, None], torch.maximum(scale, need), need)
        new_scale = torch.where(hit[:, None], grown, scale)
        ratio = (scale / new_scale)[:, :, None, None]
        again = (cache.float() * ratio).to(torch.float8_e4m3fn)
        mixed = torch.where(kept[:, None, :, None], again.view(torch.uint8),
                            cache.view(torch.uint8))
        fresh = (x / new_scale[page][:, :, None]).to(torch.float8_e4m3fn)
        mixed[page, :, off] = fresh.view(torch.uint8)
        out[n + "_cache"], out[n + "_scale"] = mixed.view(torch.float8_e4m3fn), new_scale
    return out


def _visible(s, L):
    """[B, new, L] : whether token i of sequence b sees cache position p."""
    cu, kv = s["cu"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["case"]["new"], device=DEV)
    p = torch.arange(L, device=DEV)
    ctx = (kv - n)[:, None, None]
    real = i[None, :, None] < n[:, None, None]
    if s["mask"] is None:
        sees = p <= ctx + i[None, :, None]
    else:
        rows = (cu[:-1, None] + i).clamp(max=s["T"] - 1)
        j = p - ctx
        word = s["mask"][rows].gather(
            2, (j // 32).clamp(0, s["mask"].shape[1] - 1).expand(-1, i.numel(), -1))
        sees = (j < 0) | (((word >> (j % 32)) & 1) == 1)
    return sees & real & (p < kv[:, None, None])


def _attend_plain(s):
    case = s["case"]
    bs, Hq, H, D = case["block"], case["Hq"], case["Hkv"], case["D"]
    B, G, cols, new = case["B"], Hq // H, s["table"].shape[1], case["new"]
    L = cols * bs
    cu, kv = s["cu"].long(), s["kv_len"].long()
    at = s["table"].long().clamp(min=0)
    read = {}
    for n in "kv":
        x = s[n + "_cache"].float() * s[n + "_scale"][:, :, None, None]
        read[n] = x[at].permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
    live = torch.arange(L, device=DEV) < kv[:, None]
    read["v"] = torch.where(live[:, None, :, None], read["v"], 0.0)
    i = torch.arange(new, device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][rows].float().reshape(B, new, H, G, D).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.reshape(B, H, G * new, D), read["k"].transpose(2, 3)) / math.sqrt(D)
    sees = _visible(s, L)[:, None, None].expand(B, 1, G, new, L).reshape(B, 1, G * new, L)
    z = z.masked_fill_(~sees, -math.inf)
    top = z.amax(-1, keepdim=True)
    w = torch.exp_(z.sub_(torch.where(top == -math.inf, 0.0, top)))
    mass = w.sum(-1, keepdim=True)
    o = torch.matmul(w, read["v"]) / torch.where(mass == 0, 1.0, mass)
    o = o.reshape(B, H, G, new, D).permute(0, 3, 1, 2, 4).reshape(B, new, Hq, D)
    real = i < (cu[1:] - cu[:-1])[:, None]
    return o[real].to(s["q"].dtype)


def _sample_plain(s):
    x, T = s["logits"].double(), s["temperature"].double()[:, None]
    R, V = x.shape
    greedy = T == 0
    val, idx = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((val - val[:, :1]) / torch.where(greedy, 1.0, T))
    cum = torch.cumsum(w, 1)
    k = s["top_k"].long()[:, None]
    k = torch.where(k == 0, V, k.clamp(max=V))
    mass = cum.gather(1, k - 1)
    p = s["top_p"].double()[:, None]
    n_p = torch.where(p >= 1, V, (cum < p * mass).sum(1, keepdim=True) + 1)
    n_m = (w >= s["min_p"].double()[:, None]).sum(1, keepdim=True)
    n = torch.minimum(torch.minimum(k, n_p), n_m).clamp(min=1)
    n = torch.where(greedy, 1, n)
    w = torch.where(torch.arange(V, device=DEV) < n, w, 0.0)
    by_id = torch.zeros_like(w).scatter_(1, idx, w)
    cum = torch.cumsum(by_id, 1)
    goal = s["u"].double()[:, None] * cum[:, -1:]
    token = (cum <= goal).sum(1, keepdim=True).clamp(max=V - 1)
    prob = by_id.gather(1, token) / cum[:, -1:]
    return dict(token=token[:, 0].to(torch.int32), prob=prob[:, 0].float(),
                kept=n[:, 0].to(torch.int32))


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain,
                "sample": _sample_plain}[op](s)
    import draft_block_verification_gb300 as dbv
    if op == "plan":
        out = dbv.sv_kv_plan(s["cached"], s["new"], s["held"], s["table"], s["free_ids"],
                             s["free_pos"], case["block"], s["max_tokens"])
        out.update(table=s["table"], free_ids=s["free_ids"])
        return out
    if op == "append":
        dbv.sv_kv_append(s["k"], s["v"], s["slot"], s["k_cache"], s["v_cache"], s["k_scale"],
                         s["v_scale"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if op == "attend":
        return dbv.sv_kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                   s["v_scale"], s["table"], s["kv_len"], s["cu"],
                                   mask=s["mask"])["out"]
    return dbv.sv_sample_rows(s["logits"], s["u"], temperature=s["temperature"],
                              top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "sample":
        esz = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["V"]
        return {"bytes": n * esz + case["rows"] * 32, "flops": 4 * n}
    cached, fresh = _lengths(case)
    B, bs, T = case["B"], case["block"], sum(fresh)
    pages = sum((c + f + bs - 1) // bs for c, f in zip(cached, fresh))
    if op == "plan":
        # lengths and counts in, counts out, the new table entries and two words a token
        fresh_pages = sum((c + f + bs - 1) // bs - (c + bs - 1) // bs
                          for c, f in zip(cached, fresh))
        return {"bytes": 24 * B + 8 * fresh_pages + 8 * T, "flops": 10 * (B + T)}
    H, D = case["Hkv"], case["D"]
    if op == "append":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * T * H * D * (esz + 1) + 4 * T, "flops": 4 * T * H * D}
    Hq = case["Hq"]
    pairs = sum(f * c + f * (f + 1) // 2 for c, f in zip(cached, fresh))
    return {"bytes": 2 * sum(c + f for c, f in zip(cached, fresh)) * H * D + 8 * pages * H
            + 4 * pages + 4 * T * Hq * D, "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def _exact_plan(s):
    bs = s["case"]["block"]
    cached, new, held = (s[n].tolist() for n in ("cached", "new", "held"))
    table, ring = s["table"].cpu().numpy().copy(), s["free_ids"].cpu().numpy().copy()
    head, tail = s["free_pos"].tolist()
    R = len(ring)
    cu, slot, pos, kv, after = [0], [], [], [], []
    for b, (c, n, h) in enumerate(zip(cached, new, held)):
        w = -(-(c + n) // bs)
        for j in range(h, w):
            table[b, j] = ring[head % R]
            head += 1
        for j in range(w, h):
            ring[tail % R] = table[b, j]
            tail += 1
        p = np.arange(c, c + n)
        slot.append(table[b][p // bs].astype(np.int64) * bs + p % bs)
        pos.append(p)
        cu.append(cu[-1] + n)
        kv.append(c + n)
        after.append(w)
    pad = np.full(s["max_tokens"] - cu[-1], -1)
    cat = lambda v: torch.from_numpy(np.concatenate(v + [pad]).astype(np.int32))  # noqa: E731
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(table=torch.from_numpy(table), free_ids=torch.from_numpy(ring), held=i(after),
                kv_len=i(kv), cu_new=i(cu), free_pos=torch.tensor([head, tail]), slot=cat(slot),
                pos=cat(pos))


# The magnitudes that 8 bits with 4 of exponent (bias 7) and 3 of fraction stand for.
_STEPS = sorted((m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
                for e in range(16) for m in range(8) if (e, m) != (15, 7))


def _nearest8(x):
    """The nearest 8-bit value of each element, ties to the even code."""
    table = torch.tensor(_STEPS, dtype=torch.float64, device=x.device)
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(table, a).clamp(max=len(_STEPS) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    pick = torch.where(up < down, hi, torch.where(down < up, lo,
                                                  torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(table[pick], x)


def _exact_append(s):
    bs, slot = s["case"]["block"], s["slot"].tolist()
    runs, at = [], 0
    while at < len(slot):
        end = at + 1
        while end < len(slot) and slot[end] == slot[end - 1] + 1 and slot[end] % bs:
            end += 1
        runs.append((at, end, slot[at] // bs, slot[at] % bs))
        at = end
    if len(runs) * s["case"]["Hkv"] > 60000:
        return None
    out = {}
    for n in "kv":
        cache, scale = s[n + "_cache"].double(), s[n + "_scale"].double()
        x = s[n].double()
        for a, b, page, off in runs:
            amax = x[a:b].abs().amax(dim=(0, 2))
            e = torch.ceil(torch.log2(amax / E4M3_MAX))
            e = e + (amax > E4M3_MAX * torch.exp2(e)).double()
            e = e - (amax <= E4M3_MAX * torch.exp2(e - 1)).double()
            need = torch.exp2(e.clamp(-SCALE_EXP, SCALE_EXP))
            if off:
                need = torch.maximum(need, scale[page])
                cache[page, :, :off] = _nearest8(
                    cache[page, :, :off] * (scale[page] / need)[:, None, None])
            cache[page, :, off:off + b - a] = _nearest8(
                (x[a:b] / need[:, None]).transpose(0, 1))
            scale[page] = need
        out[n + "_cache"], out[n + "_scale"] = cache, scale
    return out


def _exact_attend(s):
    case = s["case"]
    H, D, G = case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    cu, kv = s["cu"].tolist(), s["kv_len"].tolist()
    out = torch.zeros((s["T"], case["Hq"], D), dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, L = cu[b + 1] - cu[b], kv[b]
        if n == 0:
            continue
        pages = s["table"][b, :-(-L // case["block"])].long()
        K, V = ((s[m + "_cache"][pages].double() * s[m + "_scale"][pages].double()[..., None,
                 None]).transpose(0, 1).reshape(H, -1, D)[:, :L] for m in "kv")
        sees = torch.ones((n, L), dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            sees = sees.tril(L - n)
        else:
            w = s["mask"][cu[b]:cu[b + 1]].cpu().numpy().view(np.uint32)
            block = np.unpackbits(w.view(np.uint8), axis=1, bitorder="little")[:, :n]
            sees[:, L - n:] = torch.from_numpy(block.astype(bool)).to(DEV)
        q = s["q"][cu[b]:cu[b + 1]].double().reshape(n, H, G, D)
        z = torch.einsum("nhgd,hld->hgnl", q, K) * D ** -0.5
        z = torch.where(sees, z, torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
        p = torch.softmax(z, -1)
        p = torch.where(sees.any(-1)[:, None], p, 0.0)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgnl,hld->nhgd", p, V).reshape(n, -1, D)
    return out


def _exact_sample(s):
    token, prob, kept = [], [], []
    par = [s[n].tolist() for n in ("u", "temperature", "top_k", "top_p", "min_p")]
    for r, (u, T, k, p, m) in enumerate(zip(*par)):
        x = s["logits"][r].double()
        if T == 0:
            token.append(int((x == x.max()).nonzero()[0]))
            prob.append(1.0)
            kept.append(1)
            continue
        w = torch.exp((x - x.max()) / T)
        order = torch.argsort(-x, stable=True)
        n = x.numel() if k == 0 else min(k, x.numel())
        run_ = torch.cumsum(w[order[:n]], 0)
        if p < 1:
            n = int((run_ >= p * run_[-1]).nonzero()[0]) + 1
        n = max(1, min(n, int((w >= m).sum())))
        ids = order[:n].sort().values
        run_ = torch.cumsum(w[ids], 0)
        past = (run_ > u * run_[-1]).nonzero()
        at = int(past[0]) if len(past) else n - 1
        token.append(int(ids[at]))
        prob.append(float(w[ids[at]] / run_[-1]))
        kept.append(n)
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(token=i(token), prob=torch.tensor(prob, dtype=torch.float64), kept=i(kept))


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend,
            "sample": _exact_sample}[case["op"]](s)
