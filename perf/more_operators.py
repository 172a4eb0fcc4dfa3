"""More serving operators around the paged cache: cases, inputs and plain forms.

Before a draft block's keys go into the cache, its queries and keys are
normalised for each head and rotated by their positions; a batch whose
sequences share a long prefix attends to it once for all; and stored tokens
are read back from the cache's 8 bits.  Each case here is one call of one of
the three.

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
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence before its decode step: the call's latency
        dict(name="rope_1", op="rope", T=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, norm=True,
             din="bf16", dout="bf16", base=500000.0, far=4096, mix=1),
        # the draft blocks of 64 sequences, 16 drafts and the next token each
        dict(name="rope_64x17", op="rope", T=1088, Hq=32, Hkv=8, D=128, rot=128, inter=False,
             norm=True, din="bf16", dout="bf16", base=500000.0, far=32768, mix=2),
        # a projection left in 32 bits, heads of 96 of which a part is rotated, neighbours paired
        dict(name="rope_part_777", op="rope", T=777, Hq=14, Hkv=2, D=96, rot=48, inter=True,
             norm=False, din="f32", dout="bf16", base=10000.0, far=1000000, mix=3),
        # prompts of several sequences at once
        dict(name="rope_prompts", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128, inter=False,
             norm=True, din="bf16", dout="bf16", base=500000.0, far=131072, mix=4),
        # the last draft block of one sequence: the call's latency
        dict(name="read_1x17", op="read", B=1, block=64, ctx=4096, n=17, Hkv=8, D=128,
             dtype="bf16", mix=5),
        # ragged pieces of 37 sequences, small heads, into 32 bits
        dict(name="read_37", op="read", B=37, block=16, ctx=3000, n=1999, Hkv=3, D=64,
             dtype="f32", mix=6),
        # long sequences, whole, for a second pass in 16 bits
        dict(name="read_8x16384", op="read", B=8, block=64, ctx=16384, n=16384, Hkv=8, D=128,
             dtype="bf16", mix=7),
        # four sequences behind a short system prompt: the call's latency
        dict(name="prefix_4x1", op="prefix", groups=1, B=4, block=64, prefix=1024, after=64,
             new=1, Hq=32, Hkv=8, D=128, tree=False, mix=8),
        # single tokens of 128 sequences behind a long instruction
        dict(name="prefix_128x1", op="prefix", groups=1, B=128, block=64, prefix=8192, after=512,
             new=1, Hq=32, Hkv=8, D=128, tree=False, mix=9),
        # draft blocks of 16 tokens and one more, 64 sequences behind one prompt
        dict(name="prefix_64x17", op="prefix", groups=1, B=64, block=64, prefix=8192, after=512,
             new=17, Hq=32, Hkv=8, D=128, tree=False, mix=10),
        # draft trees of up to 64 nodes, two prompts
        dict(name="prefix_tree_32x64", op="prefix", groups=2, B=32, block=32, prefix=4096,
             after=1024, new=64, Hq=32, Hkv=8, D=128, tree=True, mix=11),
        # questions to three long documents, small heads, seven to a stored one
        dict(name="prefix_long_24x5", op="prefix", groups=3, B=24, block=128, prefix=131072,
             after=2048, new=5, Hq=56, Hkv=8, D=64, tree=False, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "read", "prefix", "prefix", "prefix"))
    block = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    if op == "rope":
        H, G = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8))
        D = rng.choice((64, 64, 128, 128, 128, 80, 96, 256, 2 * rng.randrange(8, 100)))
        rot = D if rng.random() < 0.6 else 2 * rng.randrange(1, D // 2 + 1)
        din = rng.choice(("bf16", "bf16", "f32"))
        dout = "bf16" if din == "bf16" else rng.choice(("bf16", "f32"))
        room = 16384 * 40 * 128 // (H * (G + 1) * D * (1 if din == "bf16" else 2))
        return dict(op=op, T=_log_int(rng, 1, min(room, 65536)), Hq=H * G, Hkv=H, D=D, rot=rot,
                    inter=rng.random() < 0.3, norm=rng.random() < 0.7, din=din, dout=dout,
                    base=rng.choice((10000.0, 500000.0, 1000000.0)),
                    far=_log_int(rng, 1, 1 << 20), mix=mix)
    if op == "read":
        B, H, D = _log_int(rng, 1, 256), rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 128))
        dtype = rng.choice(("bf16", "f32"))
        room = 8 * 16384 * 8 * 128 // (B * H * D * (1 if dtype == "bf16" else 2))
        ctx = _log_int(rng, 1, max(2, min(65536, room)))
        return dict(op=op, B=B, block=block, ctx=ctx, n=_log_int(rng, 1, ctx), Hkv=H, D=D,
                    dtype=dtype, mix=mix)
    H, G, D = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 7, 8, 12)), \
        rng.choice((64, 128, 128))
    B, new = _log_int(rng, 2, 160), _log_int(rng, 1, 72)
    groups = min(B, rng.choice((1, 1, 1, 2, 3, 5)))
    rows = B * H * G * new
    after = _log_int(rng, 1, max(2, min(4096, (1 << 27) // (B * H * D), (1 << 27) // rows)))
    room = min((1 << 27) // (groups * H * D), (1 << 28) // rows)
    return dict(op=op, groups=groups, B=B, block=block,
                prefix=_log_int(rng, 16, max(32, min(131072, room))), after=after, new=new,
                Hq=H * G, Hkv=H, D=D, tree=new > 1 and rng.random() < 0.4, mix=mix)


def _read_lengths(case):
    """(first position, tokens) that are read of each sequence; by the case alone."""
    r = random.Random(case["mix"])
    n = [r.randint((case["n"] + 1) // 2, case["n"]) for _ in range(case["B"])]
    n[0] = case["n"]
    if case["B"] > 3:
        n[1] = 0
    return [r.choice((0, r.randint(0, case["ctx"] - k))) for k in n], n


def _prefix_lengths(case):
    """Prefix of each group; group, tokens after the prefix (the new ones among them)
    and new tokens of each sequence; by the case alone."""
    r = random.Random(case["mix"])
    N, B, bs = case["groups"], case["B"], case["block"]
    prefix = [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(N)]
    prefix[0] = case["prefix"]
    # (every group has a sequence at least)
    edge = [0] + sorted(r.sample(range(1, B), N - 1)) + [B]
    of = [g for g in range(N) for _ in range(edge[g], edge[g + 1])]
    new = [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(B)]
    new[0] = case["new"]
    after = [n + r.randint(case["after"] // 4, case["after"]) for n in new]
    return prefix, edge, of, after, new


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(s, pages, case, g):
    """Stored keys and values (float8) and scales of ordinary size."""
    shape = (pages, case["Hkv"], case["block"], case["D"])
    for n in "kv":
        x = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
        x.copy_((torch.randn(shape, generator=g, device=DEV) * 90).clamp_(-448, 448))
        e = torch.randint(-8, -5, shape[:2], generator=g, device=DEV).float()
        s[n + "_cache"], s[n + "_scale"] = x, torch.exp2(e)
    s["pages"] = pages


def _sums(n):
    cu = torch.zeros(len(n) + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(_i32(n), 0)
    return cu


def _own_pages(want, cols, g):
    """Table of shuffled pages, want[b] of sequence b's own."""
    pages = sum(want) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    w = _i32(want)
    j = torch.arange(cols, device=DEV)
    at = (torch.cumsum(w, 0) - w)[:, None] + j
    return torch.where(j < w[:, None], order[at.clamp_(max=pages - 1)], -1), order, pages


def _trees(case, seed, new):
    """Ancestor bits of random draft trees, a row for each new token."""
    words = (case["new"] + 31) // 32
    r = np.random.RandomState((int(seed) * 37 + 11) % (1 << 31))
    bits = np.zeros((sum(new), words), np.uint32)
    at = 0
    for n in new:
        for i in range(n):
            if i and r.rand() < 0.95:
                bits[at + i] = bits[at + r.randint(max(0, i - 6), i)]
            bits[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += n
    return torch.from_numpy(bits.view(np.int32)).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op, D, H = case["op"], case["D"], case["Hkv"]
    s = dict(case=case)
    if op == "rope":
        T, Hq = case["T"], case["Hq"]
        # one projection's output: queries, keys and values side by side; channels of
        # unequal size, as queries and keys have them
        x = torch.randn((T, (Hq + 2 * H), D), generator=g, device=DEV)
        x *= torch.exp(torch.randn((1, Hq + 2 * H, D), generator=g, device=DEV) * 0.5)
        x = x.to(DTYPES[case["din"]])
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + H]
        far = case["far"]
        s["pos"] = torch.randint(0, far, (T,), generator=g, device=DEV).to(torch.int32)
        s["pos"][0] = far - 1
        r = case["rot"]
        e = torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r
        s["inv_freq"] = (case["base"] ** -e).float()
        for n in "qk":
            s[n + "_weight"] = None
            if case["norm"]:
                s[n + "_weight"] = torch.rand(D, generator=g, device=DEV) * 1.5 + 0.25
        return s
    bs = case["block"]
    if op == "read":
        first, n = _read_lengths(case)
        want = [(f + k + bs - 1) // bs for f, k in zip(first, n)]
        cols = (case["ctx"] + bs - 1) // bs
        s["table"], _, pages = _own_pages(want, cols, g)
        _cache(s, pages, case, g)
        s.update(first=_i32(first), cu=_sums(n), T=sum(n))
        return s
    prefix, edge, of, after, new = _prefix_lengths(case)
    B = case["B"]
    # whole pages of a prefix are the group's; what is left of it is each sequence's own
    shared = [p // bs for p in prefix]
    kv = [prefix[of[b]] + after[b] for b in range(B)]
    want = [(kv[b] + bs - 1) // bs - shared[of[b]] for b in range(B)]
    cols = max((k + bs - 1) // bs for k in kv)
    pages = sum(want) + sum(shared) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    start = [0]
    for n in shared + want:
        start.append(start[-1] + n)
    j = torch.arange(cols, device=DEV)
    sh, wn = _i32([shared[of[b]] for b in range(B)])[:, None], _i32(want)[:, None]
    at_p = _i32([start[of[b]] for b in range(B)])[:, None] + j
    at_o = _i32(start[len(shared):-1])[:, None] + j - sh
    at = torch.where(j < sh, at_p, at_o).clamp_(0, pages - 1)
    s["table"] = torch.where(j < sh + wn, order[at], -1).contiguous()
    _cache(s, pages, case, g)
    T = sum(new)
    s.update(kv_len=_i32(kv), cu=_sums(new), T=T, cu_group=_i32(edge), prefix_len=_i32(prefix))
    s["q"] = (torch.randn((T, case["Hq"], D), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    s["mask"] = _trees(case, seed, new) if case["tree"] else None
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _rope_plain(s):
    case = s["case"]
    r, h = case["rot"], case["rot"] // 2
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    c, d = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = {}
    for n in "qk":
        x, w = s[n].float(), s[n + "_weight"]
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["inter"] else (x[..., :h], x[..., h:r])
        p, m = a * c - b * d, b * c + a * d
        y = torch.stack((p, m), -1).flatten(-2) if case["inter"] else torch.cat((p, m), -1)
        out[n] = torch.cat((y, x[..., r:]), -1).to(DTYPES[case["dout"]])
    return out


def _read_plain(s):
    bs, T = s["case"]["block"], s["T"]
    cu = s["cu"].long()
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = s["first"].long()[b] + t - cu[b]
    page = s["table"][b, pos // bs].long()
    out = {}
    for n in "kv":
        x = s[n + "_cache"][page, :, pos % bs].float() * s[n + "_scale"][page][:, :, None]
        out[n] = x.to(DTYPES[s["case"]["dtype"]])
    return out


def _prefix_plain(s):
    case = s["case"]
    bs, Hq, H, D = case["block"], case["Hq"], case["Hkv"], case["D"]
    G, new = Hq // H, case["new"]
    prefix, edge, _, _, _ = _prefix_lengths(case)
    cu, kv, table = s["cu"].long(), s["kv_len"].long(), s["table"].long()
    i = torch.arange(new, device=DEV)
    parts = []
    for g, P in enumerate(prefix):
        lo, hi, P = edge[g], edge[g + 1], P // bs * bs
        n = cu[lo + 1:hi + 1] - cu[lo:hi]
        real = i < n[:, None]
        B = hi - lo
        rows = (cu[lo:hi, None] + i).clamp(max=s["T"] - 1)
        q = s["q"][rows].float().reshape(B, new, H, G, D).permute(2, 0, 3, 1, 4)
        # the pages that all share: one product for the rows of the whole group
        at = table[lo, :P // bs]
        keys, vals = ((s[m + "_cache"][at].float() * s[m + "_scale"][at][:, :, None, None])
                      .transpose(0, 1).reshape(H, P, D) for m in "kv")
        z = torch.matmul(q.reshape(H, -1, D), keys.transpose(1, 2)) / math.sqrt(D)
        # each sequence's own
        cols = (case["after"] + new) // bs + 2
        j = torch.arange(P // bs, P // bs + cols, device=DEV)
        at = table[lo:hi][:, j.clamp(max=table.shape[1] - 1)].clamp(min=0)
        pos = P + torch.arange(cols * bs, device=DEV)
        live = pos < kv[lo:hi, None]
        mine, theirs = ((s[m + "_cache"][at].float() * s[m + "_scale"][at][..., None, None])
                        .transpose(1, 2).reshape(B, H, -1, D) for m in "kv")
        theirs = torch.where(live[:, None, :, None], theirs, 0.0)
        y = torch.matmul(q.transpose(0, 1).reshape(B, H, G * new, D), mine.transpose(2, 3))
        y /= math.sqrt(D)
        ctx = (kv[lo:hi] - n)[:, None, None]
        if s["mask"] is None:
            sees = pos <= ctx + i[None, :, None]
        else:
            k = pos - ctx
            word = s["mask"][rows].gather(
                2, (k // 32).clamp(0, s["mask"].shape[1] - 1).expand(-1, new, -1))
            sees = (k < 0) | (((word >> (k % 32)) & 1) == 1)
        sees = sees & live[:, None]
        sees = sees[:, None, None].expand(B, 1, G, new, -1).reshape(B, 1, G * new, -1)
        y = y.masked_fill_(~sees, -math.inf)
        # [H, B, G new, .] both
        z, y = z.reshape(H, B, G * new, P), y.transpose(0, 1)
        top = y.amax(-1, keepdim=True)
        if P:
            top = torch.maximum(top, z.amax(-1, keepdim=True))
        top = torch.where(top == -math.inf, 0.0, top)
        z, y = torch.exp_(z.sub_(top)), torch.exp_(y - top)
        mass = z.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.matmul(z.reshape(H, B * G * new, P), vals).reshape(H, B, G * new, D)
        o = o + torch.matmul(y, theirs.transpose(0, 1))
        o = o / torch.where(mass == 0, 1.0, mass)
        o = o.reshape(H, B, G, new, D).permute(1, 3, 0, 2, 4).reshape(B, new, Hq, D)
        parts.append(o[real].to(s["q"].dtype))
    return torch.cat(parts)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rope": _rope_plain, "read": _read_plain, "prefix": _prefix_plain}[op](s)
    import draft_block_verification_gb300 as dbv
    if op == "rope":
        return dbv.sv_qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                   interleaved=case["inter"], dtype=DTYPES[case["dout"]])
    if op == "read":
        return dbv.sv_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                              s["cu"], s["T"], first=s["first"], dtype=DTYPES[case["dtype"]])
    return dbv.sv_kv_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                      s["v_scale"], s["table"], s["kv_len"], s["cu"],
                                      s["prefix_len"], cu_group=s["cu_group"],
                                      mask=s["mask"])["out"]


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, H, D = case["op"], case["Hkv"], case["D"]
    size = {"bf16": 2, "f32": 4}
    if op == "rope":
        n = case["T"] * (case["Hq"] + H) * D
        return {"bytes": n * (size[case["din"]] + size[case["dout"]]) + 4 * case["T"]
                + 2 * case["rot"] + (8 * D if case["norm"] else 0),
                "flops": n * (7 if case["norm"] else 3)}
    if op == "read":
        first, n = _read_lengths(case)
        T, bs = sum(n), case["block"]
        pages = sum((f + k + bs - 1) // bs - f // bs for f, k in zip(first, n) if k)
        return {"bytes": 2 * T * H * D * (1 + size[case["dtype"]]) + pages * (4 + 8 * H)
                + 8 * case["B"], "flops": 2 * T * H * D}
    prefix, _, of, after, new = _prefix_lengths(case)
    Hq, bs, T = case["Hq"], case["block"], sum(new)
    once = [p // bs * bs for p in prefix]
    kv = [prefix[g] + a for g, a in zip(of, after)]
    tokens = sum(once) + sum(k - once[g] for k, g in zip(kv, of))
    pairs = sum(n * (k - n) + n * (n + 1) // 2 for k, n in zip(kv, new))
    return {"bytes": 2 * tokens * H * D + (tokens // bs) * (4 + 8 * H) + 4 * T * Hq * D,
            "flops": 4 * pairs * Hq * D}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
# The magnitudes that 8 bits with 4 of exponent (bias 7) and 3 of fraction stand for.
_STEPS = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
          for e in range(16) for m in range(8)]


def _decode(x):
    code = x.view(torch.uint8).long()
    mag = torch.tensor(_STEPS, dtype=torch.float64, device=x.device)[code & 127]
    return torch.where(code >= 128, -mag, mag)


def _exact_rope(s):
    case = s["case"]
    r = case["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["pos"].double()[:, None] * s["inv_freq"].double())[:, None]
    out = {}
    for n in "qk":
        x = s[n].double()
        if s[n + "_weight"] is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt()
            x = x * s[n + "_weight"].double()
        y = x.clone()
        if case["inter"]:
            first, second = slice(0, r, 2), slice(1, r, 2)
        else:
            first, second = slice(0, r // 2), slice(r // 2, r)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out[n] = y
    return out


def _exact_read(s):
    bs, cu, first = s["case"]["block"], s["cu"].tolist(), s["first"].tolist()
    out = {}
    for n in "kv":
        rows = []
        for b, f in enumerate(first):
            k = cu[b + 1] - cu[b]
            if not k:
                continue
            pages = s["table"][b, f // bs:(f + k + bs - 1) // bs].long()
            x = _decode(s[n + "_cache"][pages]) * s[n + "_scale"][pages].double()[..., None, None]
            rows.append(x.transpose(1, 2).flatten(0, 1)[f % bs:f % bs + k])
        out[n] = torch.cat(rows) if rows else torch.zeros(
            (0, s["case"]["Hkv"], s["case"]["D"]), dtype=torch.float64, device=DEV)
    return out


def _exact_prefix(s):
    case = s["case"]
    H, D, G = case["Hkv"], case["D"], case["Hq"] // case["Hkv"]
    cu, kv = s["cu"].tolist(), s["kv_len"].tolist()
    if 4 * sum((cu[b + 1] - cu[b]) * kv[b] for b in range(case["B"])) * case["Hq"] * D > 2e12:
        return None
    out = torch.zeros((s["T"], case["Hq"], D), dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, L = cu[b + 1] - cu[b], kv[b]
        pages = s["table"][b, :-(-L // case["block"])].long()
        K, V = ((_decode(s[m + "_cache"][pages])
                 * s[m + "_scale"][pages].double()[..., None, None])
                .transpose(0, 1).reshape(H, -1, D)[:, :L] for m in "kv")
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


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "read": _exact_read, "prefix": _exact_prefix}[case["op"]](s)
