"""The E4M3 cache with one strong key over a long even context: most of the softmax's weight lies in
keys that are each far below the largest one, and the values have a common component, so that a
weight that is lost or rounded the same way for all of them shows in the result.

The scores come from one rope column alone (the others of q are zero), so that they are known
exactly: code c of the strong key and codes 0 of the rest, times head-dependent queries that set
the strong key 6 to 13 natural-log units above the rest.

Bound, whatever the length. With x the weights in units where the reference weight is 2^4, and
A = sum_j w_j |v_j|: P's two terms are off by 2^-8 x where x >= 2^-6 and by at most 2^-14 below. The
reference moves down at the end of every 1024 keys (decode, and 128 heads' 2048) whose largest score
lies below it, so that the even keys stay below 2^-6 for the 2048 keys around a strong one only. A strong key of weight w has x >= 2^4 (the
reference never lies above the largest score), so that those keys' errors, in weights, are at most
2^-18 w each, and sum to 2^-18 w S with S their sum of |v_j|. That happens once per strong key, at
most, and the strong keys' weights add up to at most 1: at most 2^-18 W S with W the strong keys'
weight and S the largest sum of |v_j| over 2048 keys in a row. (Where a block is cut, each piece has
this bound with weights and sums of its own.) With the fp16 rounding of x (2^-11 A), the result's own
(2^-8 |out|) and the factor 1.05 of the other tests for float32:
1.05 (2^-8 (A + |out|) + 2^-11 A + 2^-18 W S) + 1e-6. The 2-norm is held to 1e-2, the decode tests'
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
        self.L, self.H, self.strong = L, H, strong
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
        rows = torch.cat([torch.zeros((1, 512), dtype=torch.float64, device="cuda"), v.abs().cumsum(0)])
        most = (rows[2048:] - rows[:-2048]).amax(0)
        return w @ v, lse, w @ v.abs(), w[:, self.strong].sum(1, keepdim=True) * most

    def check(self, out, lse):
        r, rl, A, strong = self.exact()
        for b in range(out.shape[0]):
            err = (out[b].double() - r).abs()
            rel = (err.norm(dim=1) / r.norm(dim=1)).max().item()
            assert rel <= 1e-2, (b, rel)
            bound = 1.05 * (2.0 ** -8 * (A + r.abs()) + 2.0 ** -11 * A + 2.0 ** -18 * strong) + 1e-6
            assert (err <= bound).all(), (b, ((err - bound).max().item()))
            assert (lse[b].double() - rl).abs().max().item() <= LSE_ABS[F8]


def place(L, where):
    return {"first": [0], "middle": [L // 2 + 7], "last": [L - 1], "often": list(range(5, L, 4096))}[where]


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


def chunk(c, copies):
    """One token of each of `copies` sequences over the same pages."""
    q = c.q[None].expand(copies, -1, -1).contiguous()
    return api.chunk_attention(q, c.cache, c.table.expand(copies, -1).contiguous(), i32([c.L] * copies),
                               i32(list(range(copies + 1))), SCALE, c.scale, max_seq_len=c.L)


def decode(c, copies):
    q = c.q[None, None].expand(copies, -1, -1, -1).contiguous()
    out, lse = api.decode(q, c.cache, c.table.expand(copies, -1).contiguous(), i32([c.L] * copies), SCALE, c.scale,
                          max_seq_len=c.L)
    return out[:, 0], lse[:, 0]


def wave(H):
    """Scores that wander over 2 to 60 natural-log units."""
    L = 65536
    c = Sink(L, H, [0], seed=6)
    t = torch.arange(L, device="cuda")
    codes = (4.0 * torch.sin(2 * math.pi * t.double() / 20000) / c.scale).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    slots = c.table[0].long()[t // P] * P + t % P
    c.cache.view(-1, 576)[slots, 512] = codes.view(torch.uint8)
    c.k[:, 512] = codes.float().double() * c.scale.double()
    c.q[:, 512] = (torch.linspace(1, 30, H, device="cuda") / (4.0 * SCALE)).to(torch.bfloat16)
    return c


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "middle", "last", "often"])
@pytest.mark.parametrize("L", [32768, 131072])
@pytest.mark.parametrize("copies", [1, 90])
def test_chunk_attention(copies, L, where, spread):
    """One block, cut over all workers, and more blocks than workers: most are whole."""
    c = Sink(L, 16, place(L, where), spread, seed=L + copies)
    c.check(*chunk(c, copies))


def test_chunk_attention_with_a_key_far_above_all_others():
    """Gaps of 40 to 400: the rest has no weight that counts, and the reference, which moves down by
    a limited amount, keeps every sum finite."""
    c = Sink(32768, 16, [3], 1.0, seed=5, gaps=(40.0, 400.0))
    for copies in (1, 90):
        c.check(*chunk(c, copies))


def test_chunk_attention_with_scores_that_fall_and_rise():
    """The reference moves down and up again."""
    c = wave(16)
    for copies in (1, 90):
        c.check(*chunk(c, copies))


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("where", ["first", "middle", "last", "often"])
@pytest.mark.parametrize("L", [32768, 131072])
@pytest.mark.parametrize("H,copies", [(16, 1), (16, 170), (32, 170), (64, 1), (64, 170), (128, 1), (128, 90)])
def test_decode(H, copies, L, where, spread):
    """16, 32 and 64 heads (one SM each) and 128 (SM pairs), cut sequences and whole ones."""
    c = Sink(L, H, place(L, where), spread, seed=L + copies + H)
    c.check(*decode(c, copies))


@pytest.mark.parametrize("H,copies", [(16, 170), (32, 170), (64, 170), (128, 90)])
def test_decode_with_far_keys_and_wandering_scores(H, copies):
    c = Sink(32768, H, [3], 1.0, seed=5, gaps=(40.0, 400.0))
    c.check(*decode(c, copies))
    c = wave(H)
    c.check(*decode(c, copies))


def causal_check(c, q, out, lse):
    """Rows of the last n tokens, each over the keys up to its own."""
    n = q.shape[0]
    v = c.k[:, :512]
    sums = torch.cat([torch.zeros((1, 512), dtype=torch.float64, device="cuda"), v.abs().cumsum(0)])
    most = (sums[2048:] - sums[:-2048]).amax(0)
    for i in range(n):
        vis = c.L - n + 1 + i
        s = (q[i].double() @ c.k[:vis].T) * SCALE
        rl = torch.logsumexp(s, dim=1)
        w = torch.exp(s - rl[:, None])
        r, A = w @ v[:vis], w @ v[:vis].abs()
        err = (out[i].double() - r).abs()
        bound = 1.05 * (2.0 ** -8 * (A + r.abs()) + 2.0 ** -11 * A + 2.0 ** -18 * w[:, c.strong].sum(1, keepdim=True) * most) + 1e-6
        assert (err <= bound).all(), (i, (err - bound).max().item())
        assert (lse[i].double() - rl).abs().max().item() <= LSE_ABS[F8]


@pytest.mark.parametrize("where", ["first", "middle"])
@pytest.mark.parametrize("H,n,copies", [(16, 150, 1), (16, 150, 6), (3, 300, 4), (128, 9, 10)])
def test_chunk_attention_of_many_causal_tokens(H, n, copies, where):
    """Rows that see different numbers of keys share a block, and its last tiles are masked."""
    c = Sink(9001, H, place(9001, where), 1.0, seed=n + H)
    gain = torch.linspace(0.7, 1.2, n, device="cuda")[:, None, None]
    q = (c.q.float()[None] * gain).to(torch.bfloat16)
    out, lse = api.chunk_attention(q.repeat(copies, 1, 1), c.cache, c.table.expand(copies, -1).contiguous(),
                                   i32([c.L] * copies), i32([n * b for b in range(copies + 1)]), SCALE, c.scale, max_seq_len=c.L)
    for b in range(copies):
        causal_check(c, q, out[n * b:n * (b + 1)], lse[n * b:n * (b + 1)])


@pytest.mark.parametrize("where", ["first", "middle"])
@pytest.mark.parametrize("H,n,copies", [(8, 2, 170), (16, 2, 170), (16, 4, 170), (128, 3, 90), (128, 3, 1)])
def test_decode_of_several_tokens(H, n, copies, where):
    c = Sink(9001, H, place(9001, where), 1.0, seed=n + H + 1)
    gain = torch.linspace(0.7, 1.2, n, device="cuda")[:, None, None]
    q = (c.q.float()[None] * gain).to(torch.bfloat16)
    out, lse = api.decode(q[None].repeat(copies, 1, 1, 1), c.cache, c.table.expand(copies, -1).contiguous(),
                          i32([c.L] * copies), SCALE, c.scale, max_seq_len=c.L)
    for b in range(0, copies, 13):
        causal_check(c, q, out[b], lse[b])
