"""Decoding steps of block-sparse attention in the ways a server issues them: call by call, back to back without
waiting, and as one captured graph whose inputs are replaced from step to step. All give the same bits."""
import pytest
import torch

from chunk_harness import BF, F8, SCALE
from mla_paged_decode_02_gb300 import api

pytestmark = pytest.mark.gpu

B, P, PAGES, HI, K, STEPS = 6, 64, 30, 64, 6, 12


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


class Server:
    """Caches of B sequences, and the buffers of a step of one token each."""

    def __init__(self, kv, H, block):
        gen = torch.Generator(device="cuda").manual_seed(H)
        self.kv, self.block = kv, block
        self.table = torch.randperm(B * PAGES, generator=gen, device="cuda").int().view(B, PAGES)
        self.cache = torch.randn(B * PAGES, P, 576, generator=gen, device="cuda").to(torch.bfloat16)
        self.scale = None
        if kv == F8:
            self.scale = torch.tensor([0.01], device="cuda")
            self.cache = (self.cache.float() / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.icache = torch.randn(B * PAGES, P, 128, generator=gen, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        self.iscale = torch.rand(B * PAGES, P, generator=gen, device="cuda")
        angle = torch.rand(P * PAGES, 32, generator=gen, device="cuda")
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1)
        bf = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
        lengths = torch.tensor([1, 63, 700, 1500, 64, 1200], device="cuda")
        self.inputs = []
        for k in range(STEPS):
            pos = lengths + k
            slots = self.table.long().gather(1, pos[:, None] // P)[:, 0] * P + pos % P
            self.inputs.append([pos, slots, (pos + 1).int(), bf(B, 512), bf(B, 64), bf(B, H, 576), bf(B, HI, 128), bf(B, 128),
                                torch.randn(B, HI, generator=gen, device="cuda")])
        self.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        self.q8, self.qw = torch.zeros(B, HI, 128, dtype=torch.uint8, device="cuda"), torch.zeros(B, HI, device="cuda")
        self.scores = torch.zeros(B, PAGES * P // block, device="cuda")
        self.chosen = torch.zeros(B, K, dtype=torch.int32, device="cuda")
        self.out, self.lse = torch.zeros(B, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, device="cuda")
        self.workspace = api.alloc_sparse_workspace(api.make_sparse_params(B, B, H, P, B * PAGES, PAGES, PAGES * P, block, K, kv))

    def step(self, pos, slots, lens, latent, rope, q, iq, ik, w, after=lambda: None):
        kw = dict(max_seq_len=PAGES * P, block_size=self.block)
        api.rope_cache_write(latent, rope, pos, self.cos_sin, slots, self.cache, self.scale, q_rope=q[..., 512:].clone(), q=q)
        after()
        api.index_cache_write(ik, pos, self.cos_sin, slots, self.icache, self.iscale, queries=iq, weights=w, q_index=self.q8,
                              q_weights=self.qw)
        after()
        api.index_scores(self.q8, self.qw, self.icache, self.iscale, self.table, lens, self.cu, out=self.scores, **kw)
        after()
        api.select_blocks(self.scores, lens, self.cu, K, block_size=self.block, keep_first=1, keep_last=2, out=self.chosen)
        after()
        api.sparse_attention(q, self.cache, self.table, lens, self.cu, self.chosen, SCALE, self.scale, out=self.out, lse=self.lse,
                             workspace=self.workspace, **kw)
        after()

    def results(self):
        return self.out.clone(), self.lse.clone(), self.chosen.clone(), self.scores.clone()

    def run(self, way):
        got = []
        if way == "graph":
            held = [t.clone() for t in self.inputs[0]]
            saved = [t.clone() for t in (self.cache, self.icache, self.iscale)]
            self.step(*held)                       # (the first call of a form prepares its kernels)
            for t, s in zip((self.cache, self.icache, self.iscale), saved):
                t.copy_(s)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                self.step(*held)
        for values in self.inputs:
            if way == "graph":
                for t, v in zip(held, values):
                    t.copy_(v)
                graph.replay()
            else:
                self.step(*values, after=torch.cuda.synchronize if way == "waiting" else lambda: None)
            got.append(self.results())
        torch.cuda.synchronize()
        assert api.decode_check(self.workspace) == (0, 0)
        return got, (self.cache, self.icache, self.iscale)


@pytest.mark.parametrize("kv,H,block", [(F8, 16, 64), (BF, 16, 64), (BF, 128, 32), (F8, 40, 16)])
def test_steps_give_the_same_bits_however_they_are_issued(kv, H, block):
    want, caches = Server(kv, H, block).run("waiting")
    assert any((a[2] != b[2]).any() for a, b in zip(want, want[1:]))          # the choice changes from step to step
    for way in ("back to back", "graph"):
        got, written = Server(kv, H, block).run(way)
        for k, (a, b) in enumerate(zip(want, got)):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), (way, k)
        assert all(torch.equal(a, b) for a, b in zip(caches, written)), way
