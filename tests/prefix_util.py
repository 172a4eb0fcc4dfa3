"""Cases of attention over a shared prefix, and their values in 64 bits (not
collected)."""
import numpy as np
import torch

import kv_util


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device="cuda")


def make(seed, prefix, sizes, after, new, H, G, D, block, tree=False, pow2=True, spread=1.0,
         far=0):
    """Groups of sizes[g] sequences behind prefix[g] tokens each; after[b] tokens
    come between the prefix and the new[b] new ones.  Whole pages of a prefix are
    shared.  Every byte that no token may see is NaN.  far: the value scales of
    every other page are 2^far times as large."""
    r = np.random.RandomState(seed)
    of = np.repeat(np.arange(len(sizes)), sizes)
    B = len(of)
    L = np.array([prefix[of[b]] + after[b] + new[b] for b in range(B)])
    shared = [p // block for p in prefix]
    need = [int(-(-L[b] // block)) - shared[of[b]] for b in range(B)]
    pages = sum(shared) + sum(need) + 2
    ids = r.permutation(pages).astype(np.int32)
    cols = int(max(-(-L // block))) + 1
    table = np.full((B, cols), -1, np.int32)
    at, first = 0, []
    for n in shared:
        first.append(ids[at:at + n])
        at += n
    for b in range(B):
        s = first[of[b]]
        table[b, :len(s)] = s
        table[b, len(s):len(s) + need[b]] = ids[at:at + need[b]]
        at += need[b]
    codes = [kv_util.e4m3_encode(r.randn(pages, H, block, D) * 60) for _ in range(2)]
    scale = [(2.0 ** r.randint(-8, -3, (pages, H)) if pow2 else
              np.exp(r.uniform(-5, -3, (pages, H)))).astype(np.float32) for _ in range(2)]
    scale[1][1::2] *= np.float32(2.0 ** far)
    live = np.zeros((pages, block), bool)
    for b in range(B):
        p = np.arange(L[b])
        live[table[b, p // block], p % block] = True
    for c in codes:
        c[~np.broadcast_to(live[:, None], (pages, H, block))] = 0x7F
    T = int(np.sum(new))
    cu = np.append(0, np.cumsum(new)).astype(np.int32)
    q = torch.as_tensor(r.randn(T, H * G, D) * spread, dtype=torch.bfloat16, device="cuda")
    mask = None
    if tree:
        words = max(1, -(-max(new) // 32))
        mask = np.zeros((T, words), np.uint32)
        for b, n in enumerate(new):
            for i in range(n):
                t = cu[b] + i
                if i and r.rand() < 0.9:
                    mask[t] = mask[cu[b] + r.randint(i)]
                if r.rand() < 0.9:
                    mask[t, i // 32] |= np.uint32(1 << (i % 32))
    return dict(q=q, codes=codes, scale=scale, table=table, kv=L.astype(np.int32), cu=cu,
                mask=mask, block=block, group=np.append(0, np.cumsum(sizes)).astype(np.int32),
                prefix=np.array(prefix, np.int32))


def tensors(c):
    k, v = (dev(a, torch.uint8).view(torch.float8_e4m3fn) for a in c["codes"])
    ks, vs = (dev(a, torch.float32) for a in c["scale"])
    return [c["q"], k, v, ks, vs, dev(c["table"]), dev(c["kv"]), dev(c["cu"])], dict(
        mask=None if c["mask"] is None else dev(c["mask"].view(np.int32)), want_lse=True)


def run(dbv, c, prefix_len="given", cu_group="given", **kw):
    a, k = tensors(c)
    p = dev(c["prefix"]) if isinstance(prefix_len, str) else prefix_len
    g = dev(c["group"]) if isinstance(cu_group, str) else cu_group
    return dbv.sv_kv_prefix_attention(*a, p, cu_group=g, **k, **kw)


def exact(c, scale=None):
    """(out, lse, sum w|v| / sum w, largest sum |q||k| |scale|) in 64 bits."""
    q = c["q"].double()
    T, Hq, D = q.shape
    H = c["codes"][0].shape[1]
    G, block = Hq // H, c["block"]
    s = D ** -0.5 if scale is None else scale
    val = torch.tensor(np.append(kv_util.MAGNITUDES, np.nan), device="cuda")
    full = []
    for x, f in zip(c["codes"], c["scale"]):
        x = dev(x, torch.int64)
        v = val[x & 127]
        full.append(torch.where(x >= 128, -v, v) * dev(f, torch.float64)[:, :, None, None])
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(lse)
    for b in range(len(c["kv"])):
        L, lo, hi = int(c["kv"][b]), int(c["cu"][b]), int(c["cu"][b + 1])
        n = hi - lo
        if not n:
            continue
        pages = dev(c["table"][b, :-(-L // block)]).long()
        k, v = (x[pages].transpose(0, 1).reshape(H, -1, D)[:, :L] for x in full)
        sees = torch.stack([dev(kv_util.sees(i, n, L - n, L, None if c["mask"] is None else
                                             c["mask"][lo + i]), torch.bool) for i in range(n)])
        x = q[lo:hi].reshape(n, H, G, D)
        z = torch.einsum("nhgd,hld->hgnl", x, k) * s
        far = torch.einsum("nhgd,hld->hgnl", x.abs(), k.abs()) * abs(s)
        size[lo:hi] = torch.where(sees, far, 0.0).amax(-1).permute(2, 0, 1).reshape(n, Hq)
        z = torch.where(sees, z, -float("inf"))
        lse[lo:hi] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(n, Hq)
        w = torch.where(sees.any(-1)[:, None], torch.softmax(z, -1), 0.0)
        v = torch.where(sees.any(0)[:, None], v, 0.0)
        out[lo:hi] = torch.einsum("hgnl,hld->nhgd", w, v).reshape(n, Hq, D)
        mag[lo:hi] = torch.einsum("hgnl,hld->nhgd", w, v.abs()).reshape(n, Hq, D)
    return out, lse, mag, size


def check(c, got, scale=None, rows=slice(None)):
    """Tolerances.  The output is rounded to bf16 (2^-8 of its size); a weight is
    held to 2^-8 on shared pages and to 2^-8 + 2^-11 on the others (of sum w|v| /
    sum w), there down to 2^-24 of the largest; a score is a sum of up to 256
    exact products in fp32 (2^-16 of sum |q||k| at worst), its exponential within
    2^-20 of a score's size."""
    want, lse, mag, size = exact(c, scale)
    out = got["out"].double()
    L = float(c["kv"].max())
    top = 448.0 * float(max(s.max() for s in c["scale"]))
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15 * size[..., None]) * mag + \
        L * 2.0 ** -24 * top * (mag > 0)
    bad = ~((out - want).abs() <= tol)[rows]
    assert not bad.any(), (bad.nonzero()[:4], out[rows][bad][:4], want[rows][bad][:4],
                           tol[rows][bad][:4])
    gl = got["lse"].double()
    assert torch.equal(torch.isinf(gl[rows]), torch.isinf(lse[rows]))
    ok = torch.isfinite(lse)
    ok &= torch.isfinite(gl)
    near = (gl - lse).abs() <= 2.0 ** -16 * size + 2.0 ** -19 * (1 + lse.abs())
    assert near[rows][ok[rows]].all()
