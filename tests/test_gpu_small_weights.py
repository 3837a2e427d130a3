"""The E4M3 cache with one strong key over a long even context: most of the softmax's weight lies in
keys that are each far below the largest one, and the values have a common component, so that a
weight that is lost or rounded the same way for all of them shows in the result.

The scores come from one rope column alone (the others of q are zero), so that they are known
exactly: code c of the strong key and codes 0 of the rest, times head-dependent queries that set
the strong key 6 to 13 natural-log units above the rest.

Bound, whatever the length. With x the weights in units where the reference weight is 2^4, and
A = sum_j w_j |v_j|: P's two terms are off by 2^-8 x where x >= 2^-6 and by at most 2^-14 below; the
reference follows the largest score of 2048 keys, so that the even keys are below 2^-6 for the 2048
keys with the strong one only: 2048 x 2^-14 = 2^-3 next to a weight of 2^4, i.e. 2^-7 A. With the fp16
rounding of x (2^-11 A), the result's own (2^-8 |out|) and the factor 1.05 of the other tests for
float32: 1.05 (2^-8 (A + |out|) + 2^-11 A + 2^-7 A). The 2-norm is held to 1e-2, the decode tests'
contract for this cache.
"""
import math

import pytest
import torch

from chunk_harness import F8, LSE_ABS, SCALE
from mla_paged_decode_02_gb300 import api

pytestmark = pytest.mark.gpu
P = 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


class Sink:
    """keys [L, 576] E4M3 codes in scattered pages; q [H, 576] with a gap per head."""

    def __init__(self, L, H, strong, spread=0.0, seed=0, gaps=(6.0, 13.0)):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.L, self.H = L, H
        self.scale = torch.tensor([1.0 / 64], device="cuda")
        values = torch.randn((L, 576), generator=gen, device="cuda") + 0.5
        values[:, 512:] = 0
        values[strong, 512] = 4.0
        if spread:
            values[:, 513] = torch.randn(L, generator=gen, device="cuda")
            values[strong, 513] = 0
        codes = (values / self.scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.k = codes.float().double() * self.scale.double()
        pages = -(-L // P)
        order = torch.randperm(pages + 2, generator=gen, device="cuda")[:pages]
        self.cache = torch.full(((pages + 2) * P, 576), 0x7F, dtype=torch.uint8, device="cuda")
        j = torch.arange(L, device="cuda")
        self.cache[order[j // P] * P + j % P] = codes.view(torch.uint8)
        self.cache = self.cache.view(-1, P, 576)
        self.table = order.int()[None]
        self.q = torch.zeros((H, 576), dtype=torch.bfloat16, device="cuda")
        self.q[:, 512] = (torch.linspace(*gaps, H, device="cuda") / (4.0 * SCALE)).to(torch.bfloat16)
        self.q[:, 513] = spread / SCALE

    def exact(self):
        s = (self.q.double() @ self.k.T) * SCALE
        lse = torch.logsumexp(s, dim=1)
        w = torch.exp(s - lse[:, None])
        v = self.k[:, :512]
        return w @ v, lse, w @ v.abs()

    def check(self, out, lse):
        r, rl, A = self.exact()
        for b in range(out.shape[0]):
            err = (out[b].double() - r).abs()
            rel = (err.norm(dim=1) / r.norm(dim=1)).max().item()
            assert rel <= 1e-2, (b, rel)
            bound = 1.05 * (2.0 ** -8 * (A + r.abs()) + (2.0 ** -11 + 2.0 ** -7) * A) + 1e-6
            assert (err <= bound).all(), (b, ((err - bound).max().item()))
            assert (lse[b].double() - rl).abs().max().item() <= LSE_ABS[F8]


def place(L, where):
    return {"first": [0], "middle": [L // 2 + 7], "last": [L - 1], "often": list(range(5, L, 4096))}[where]


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "middle", "last", "often"])
@pytest.mark.parametrize("L,copies", [(32768, 1), (32768, 90), (131072, 1), (131072, 90)])
def test_chunk_attention(L, copies, where, spread):
    """One token (its block is cut over all workers) and 90 sequences over the same pages (more
    blocks than workers: most are whole)."""
    c = Sink(L, 16, place(L, where), spread, seed=L + copies)
    i32 = lambda t: torch.as_tensor(t, dtype=torch.int32, device="cuda")
    out, lse = api.chunk_attention(c.q[None].expand(copies, -1, -1).contiguous(), c.cache,
                                   c.table.expand(copies, -1).contiguous(), i32([L] * copies),
                                   i32(list(range(copies + 1))), SCALE, c.scale, max_seq_len=L)
    c.check(out, lse)


def test_chunk_attention_with_a_key_far_above_all_others():
    """Gaps of 40 to 400: the rest has no weight that counts, and the reference, which moves down by
    a limited amount, keeps every sum finite."""
    c = Sink(32768, 16, [3], 1.0, seed=5, gaps=(40.0, 400.0))
    i32 = lambda t: torch.as_tensor(t, dtype=torch.int32, device="cuda")
    for copies in (1, 90):
        out, lse = api.chunk_attention(c.q[None].expand(copies, -1, -1).contiguous(), c.cache,
                                       c.table.expand(copies, -1).contiguous(), i32([c.L] * copies),
                                       i32(list(range(copies + 1))), SCALE, c.scale, max_seq_len=c.L)
        c.check(out, lse)


def test_chunk_attention_with_scores_that_fall_and_rise():
    """Scores that wander over 60 natural-log units: the reference moves down and up again."""
    L, H = 65536, 16
    c = Sink(L, H, [0], seed=6)
    t = torch.arange(L, device="cuda", dtype=torch.float64)
    wave = torch.sin(2 * math.pi * t / 20000)
    codes = (wave / 1.0 * 4.0 / c.scale).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    flat = c.cache.view(-1, 576)
    slots = c.table[0].long()[t.long() // P] * P + t.long() % P
    flat[slots, 512] = codes.view(torch.uint8)
    c.k[:, 512] = codes.float().double() * c.scale.double()
    c.q[:, 512] = (torch.linspace(1, 30, H, device="cuda") / (4.0 * SCALE)).to(torch.bfloat16)
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")
    for copies in (1, 90):
        out, lse = api.chunk_attention(c.q[None].expand(copies, -1, -1).contiguous(), c.cache,
                                       c.table.expand(copies, -1).contiguous(), i32([L] * copies),
                                       i32(list(range(copies + 1))), SCALE, c.scale, max_seq_len=L)
        c.check(out, lse)
