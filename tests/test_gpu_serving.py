"""The operators around the paged cache as a serving step uses them together:
places, norms with the rotation, the cache's write, attention over the shared
prefix and the new tokens read back, eager and from a captured graph."""
import numpy as np
import pytest
import torch

import prefix_util as pu
from test_gpu_qk_rope import formula

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def dbv():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import draft_block_verification_gb300 as m
    return m


class Server:
    """B sequences behind one prompt of whole pages, whose page ids their table rows
    share.  step() is one serving step on fixed buffers, so that it can be captured."""

    def __init__(self, dbv, B, H, G, D, block, prompt, cap, dtype):
        g = torch.Generator(device="cuda").manual_seed(B + D)
        self.dbv, self.B, self.H, self.G, self.D, self.block, self.cap = dbv, B, H, G, D, block, cap
        self.gen, self.pages, cols = g, 40 + B * 8, 40
        shape = (self.pages, H, block, D)
        self.cache = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(
            torch.float8_e4m3fn) for _ in range(2)]
        self.scale = [torch.ones((self.pages, H), device="cuda") for _ in range(2)]
        self.table = torch.full((B, cols), -1, dtype=I32, device="cuda")
        self.free_ids = torch.randperm(self.pages, generator=g, device="cuda").to(I32)
        self.free_pos = torch.tensor([0, self.pages], dtype=torch.int64, device="cuda")
        self.held, self.cached, self.new = (torch.zeros(B, dtype=I32, device="cuda")
                                            for _ in range(3))
        self.f = (10000.0 ** -(torch.arange(0, D, 2, device="cuda") / D)).float()
        self.w = [torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2)]
        self.dtype = dtype
        self.x = torch.zeros((cap, H * (G + 2), D), dtype=dtype, device="cuda")
        # the prompt, by the first sequence alone; its pages then stand in all rows
        self.prompt = prompt
        self.new[0] = prompt
        self.cap = prompt
        x, self.x = self.x, torch.randn((prompt, H * (G + 2), D), generator=g,
                                        device="cuda").to(dtype)
        self.advance(self.step(), [prompt] + [0] * (B - 1))
        self.x, self.cap = x, cap
        self.table[:, :prompt // block] = self.table[0, :prompt // block].clone()
        self.held.fill_(prompt // block)
        self.cached.fill_(prompt)

    def fill(self, new):
        self.new.copy_(torch.tensor(new, dtype=I32))
        self.x.copy_(torch.randn(self.x.shape, generator=self.gen, device="cuda"))

    def step(self):
        d, q = self.dbv, self.H * self.G
        p = d.sv_kv_plan(self.cached, self.new, self.held, self.table, self.free_ids,
                         self.free_pos, self.block, self.cap)
        qk = d.sv_qk_norm_rope(self.x[:, :q], self.x[:, q:q + self.H], p["pos"], self.f,
                               q_weight=self.w[0], k_weight=self.w[1], dtype=torch.bfloat16)
        v = self.x[:, q + self.H:].to(torch.bfloat16)
        d.sv_kv_append(qk["k"], v, p["slot"], *self.cache, *self.scale)
        a = d.sv_kv_prefix_attention(qk["q"], *self.cache, *self.scale, self.table, p["kv_len"],
                                     p["cu_new"], want_lse=True)
        back = d.sv_kv_read(*self.cache, *self.scale, self.table, p["cu_new"], self.cap,
                            first=self.cached)
        return dict(p, v=v, q=qk["q"], kk=qk["k"], out=a["out"], lse=a["lse"], rk=back["k"],
                    rv=back["v"])

    def advance(self, r, kept):
        self.held.copy_(r["held"])
        self.free_pos.copy_(r["free_pos"])
        self.cached += torch.tensor(kept, dtype=I32, device="cuda")

    def check(self, r):
        T = int(r["cu_new"][-1])
        assert T == int(self.new.sum()) and (r["pos"][T:] == -1).all()
        nq = self.H * self.G
        for n, lo, hi, w in (("q", 0, nq, 0), ("kk", nq, nq + self.H, 1)):
            want, size = formula(self.x[:T, lo:hi], r["pos"][:T], self.f, self.w[w], 1e-6, False)
            near = (r[n][:T].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size
            assert near.all()
        # read back: half a step of e4m3 (2^-4 of the value; below 2^-6 of its scale
        # half of steps of 2^-9)
        slot = r["slot"][:T].long()
        for n, of, s in (("rk", "kk", self.scale[0]), ("rv", "v", self.scale[1])):
            x, y = r[of][:T].double(), r[n][:T].double()
            step = s[slot // self.block].double()[:, :, None]
            assert ((x - y).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * step).all()
        c = dict(q=r["q"][:T], codes=[a.view(torch.uint8).cpu().numpy() for a in self.cache],
                 scale=[a.cpu().numpy() for a in self.scale], table=self.table.cpu().numpy(),
                 kv=r["kv_len"].cpu().numpy(), cu=r["cu_new"].cpu().numpy(), mask=None,
                 block=self.block)
        pu.check(c, dict(out=r["out"][:T], lse=r["lse"][:T]))


@pytest.mark.parametrize("B,H,G,D,block,prompt,dtype", [
    (5, 2, 4, 64, 32, 96, torch.bfloat16), (3, 1, 7, 128, 16, 48, torch.float32),
    (9, 2, 5, 128, 64, 1280, torch.bfloat16)])
def test_steps(dbv, B, H, G, D, block, prompt, dtype):
    """Blocks of drafts of which a part is kept, sequences that pause, one with more
    rows than the others, and the sequences' end."""
    r = np.random.RandomState(B)
    s = Server(dbv, B, H, G, D, block, prompt, 13 * B, dtype)
    h = dbv.default_handle(torch.device("cuda", 0))
    graph, got = None, None
    for i in range(6):
        new = r.randint(1, 6, B)
        new[i % B] = 0
        new[(i + 1) % B] = 12
        s.fill(new.tolist())
        if i < 2:
            got = s.step()
        else:
            if graph is None:
                state = [t.clone() for t in (*s.cache, *s.scale, s.table, s.free_ids)]
                want = s.step()
                for t, o in zip((*s.cache, *s.scale, s.table, s.free_ids), state):
                    t.copy_(o)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    got = s.step()
                graph.replay()
                T = int(new.sum())
                for n in want:
                    m = T if want[n].shape[:1] == (s.cap,) else None
                    assert torch.equal(got[n][:m], want[n][:m]), n
            else:
                graph.replay()
        s.check(got)
        s.advance(got, [int(r.randint(1, n + 1)) if n else 0 for n in new])
    h.sync_status()
    # The end.  All but one sequence first go back to the prompt: what they hold beyond
    # it is free again.  The last one gives back the prompt's pages.
    s.cached.fill_(prompt)
    s.new.zero_()
    end = dbv.sv_kv_plan(s.cached, s.new, s.held, s.table, s.free_ids, s.free_pos, block, 0)
    assert (end["held"] == prompt // block).all()
    held = end["held"].clone()
    held[1:] = 0
    s.cached.zero_()
    end = dbv.sv_kv_plan(s.cached, s.new, held, s.table, s.free_ids, end["free_pos"], block, 0)
    h.sync_status()
    lo, hi = end["free_pos"].tolist()
    assert hi - lo == s.pages
    left = s.free_ids.cpu().numpy()[np.arange(lo, hi) % s.pages]
    assert sorted(left.tolist()) == list(range(s.pages))
