"""The rotating cache write against the same float32 steps done one by one (bit for bit) and
against float64, and the state merge against float64.

Bounds. The rotation's products and sums round in float32 (2^-24 of |a| + |b| each, 2^-22
together) and the result once: bf16 2^-8, E4M3 2^-4 relative or half its smallest step, 2^-10, of
the quotient. The merge: float32 weights (2^-20 of the terms' sizes) and one bf16 rounding.
"""
import math

import numpy as np
import pytest
import torch

from chunk_harness import bf16_normal
from mla_paged_decode_02_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def table(max_pos):
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def rotate(x, cs, interleaved):
    """x [..., 64], cs [..., 64] (cosines, sines) of one floating type, elementary steps."""
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    r0, r1 = a * c - b * s, b * c + a * s
    return torch.stack([r0, r1], -1).flatten(-2) if interleaved else torch.cat([r0, r1], -1)


class Append:
    def __init__(self, n, H, P, fp8, interleaved, seed, max_pos=5000, views=True):
        rng = np.random.default_rng(seed)
        self.n, self.H, self.P, self.fp8, self.interleaved, self.max_pos = n, H, P, fp8, interleaved, max_pos
        self.pages = max(2, -(-n * 2 // P))
        self.slots = torch.from_numpy(rng.permutation(self.pages * P)[:n].astype(np.int64))
        self.pos = torch.from_numpy(rng.integers(0, max_pos, n).astype(np.int64))
        if views:
            kv = bf16_normal(rng, n, 600)
            self.latent, self.rope = kv[:, 8:520], kv[:, 528:592]
            self.q_rope = bf16_normal(rng, n, max(H, 1), 192)[:, :H, 128:]
        else:
            self.latent, self.rope = bf16_normal(rng, n, 512), bf16_normal(rng, n, 64)
            self.q_rope = bf16_normal(rng, n, H, 64)
        self.q = bf16_normal(rng, n, H, 576)
        self.cs = table(max_pos)
        self.scale = torch.tensor([0.0123]) if fp8 else None
        self.cache = (torch.full((self.pages, P, 576), 0x55, dtype=torch.uint8) if fp8 else
                      torch.full((self.pages, P, 576), 3.0, dtype=torch.bfloat16))
        self.err = torch.zeros(1, dtype=torch.int32)

    def run(self, queries=True):
        def dev(t):
            """The same strides on the GPU."""
            if t is None:
                return None
            base = t._base if t._base is not None else t
            return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())
        self.g = {k: dev(getattr(self, k)) for k in ("latent", "rope", "pos", "cs", "slots", "cache", "scale", "q_rope", "q", "err")}
        g = self.g
        api.rope_cache_write(g["latent"], g["rope"], g["pos"], g["cs"], g["slots"], g["cache"], g["scale"],
                             q_rope=g["q_rope"] if queries else None, q=g["q"] if queries else None,
                             interleaved=self.interleaved, device_error=g["err"])
        torch.cuda.synchronize()

    def expected(self):
        """(cache, q) by the float32 steps; tokens with a bad position or slot skipped."""
        cache, q = self.cache.clone(), self.q.clone()
        ok = (self.pos >= 0) & (self.pos < self.max_pos)
        put = ok & (self.slots >= 0) & (self.slots < self.pages * self.P)
        cs = self.cs[self.pos.clamp(0, self.max_pos - 1)]
        row = torch.cat([self.latent.float(), rotate(self.rope.float(), cs, self.interleaved)], dim=1)
        if self.fp8:
            row = (row / self.scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            row = row.to(torch.bfloat16)
        cache.view(-1, 576)[self.slots[put]] = row[put]
        q[ok, :, 512:] = rotate(self.q_rope.float(), cs[:, None], self.interleaved).to(torch.bfloat16)[ok]
        return cache, q

    def check(self, queries=True):
        cache, q = self.expected()
        bits = lambda t: t.contiguous().view(torch.uint8 if t.dtype == torch.uint8 else torch.int16)
        assert torch.equal(bits(self.g["cache"].cpu()), bits(cache))
        assert torch.equal(bits(self.g["q"].cpu()), bits(q if queries else self.q))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,H,P,views", [(1, 1, 64, True), (3, 16, 64, True), (129, 20, 16, True), (70, 128, 128, True),
                                         (33, 33, 24, False), (1000, 5, 8, True)])
def test_rows_and_queries(n, H, P, views, interleaved, fp8):
    a = Append(n, H, P, fp8, interleaved, seed=n + H, views=views)
    a.run()
    a.check()
    assert int(a.g["err"].item()) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
def test_against_float64(interleaved, fp8):
    a = Append(200, 16, 64, fp8, interleaved, seed=1, max_pos=131072)
    a.run()
    cs = a.cs.double()[a.pos]
    turn = torch.complex(cs[:, :32].contiguous(), cs[:, 32:].contiguous())

    def exact(x, turn):
        x = x.double()
        z = (torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) if interleaved else
             torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous())) * turn
        return torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)

    rq = exact(a.q_rope, turn[:, None])
    size = a.q_rope.double().abs().amax(dim=-1, keepdim=True) * 2
    err = (a.g["q"].cpu()[:, :, 512:].double() - rq).abs()
    assert (err <= 2.0 ** -8 * rq.abs() + 2.0 ** -22 * size).all()
    rk = exact(a.rope, turn)
    row = a.g["cache"].cpu().view(-1, 576)[a.slots][:, 512:]
    if fp8:
        rk = (rk / a.scale.double()).clamp(-448, 448)
        err = (row.contiguous().view(torch.float8_e4m3fn).double() - rk).abs()
        assert (err <= 2.0 ** -4 * rk.abs() * (1 + 1e-5) + 2.0 ** -10).all()
    else:
        err = (row.double() - rk).abs()
        assert (err <= 2.0 ** -8 * rk.abs() + 2.0 ** -22 * a.rope.double().abs().amax(dim=-1, keepdim=True) * 2).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_bad_indices(fp8):
    a = Append(40, 16, 64, fp8, True, seed=2)
    a.pos[3], a.slots[3] = -1, -1                 # a padding token
    a.slots[7] = -1                               # its row is cached already, its queries turn
    a.pos[11] = -5
    a.run()
    a.check()
    assert int(a.g["err"].item()) == 0
    a.slots[20] = a.pages * a.P
    a.run()
    a.check()
    assert int(a.g["err"].item()) == 0x10
    a.pos[21] = a.max_pos
    a.run()
    a.check()
    assert int(a.g["err"].item()) == 0x50


def test_without_queries_and_in_place_queries():
    a = Append(50, 16, 64, False, False, seed=3)
    a.run(queries=False)
    a.check(queries=False)
    for interleaved in (True, False):
        a = Append(50, 40, 64, True, interleaved, seed=4)
        a.q_rope = a.q[:, :, 512:].clone()        # the expected values' input
        want = a.expected()[1]
        q = a.q.cuda()
        g = [t.cuda() for t in (a.latent.contiguous(), a.rope.contiguous(), a.pos, a.cs, a.slots, a.cache, a.scale)]
        api.rope_cache_write(*g, q_rope=q[:, :, 512:], q=q, interleaved=interleaved)
        assert torch.equal(q.cpu().view(torch.int16), want.view(torch.int16))


def test_an_unrotated_position_matches_cache_write():
    """At position 0 the rotation is the identity: the same cache bytes as cache_write."""
    for fp8 in (False, True):
        a = Append(300, 1, 64, fp8, True, seed=5)
        a.pos.zero_()
        a.run()
        other = a.cache.cuda()
        api.cache_write(a.latent.contiguous().cuda(), a.rope.contiguous().cuda(), a.slots.cuda(), other,
                        None if a.scale is None else a.scale.cuda())
        assert torch.equal(other.view(torch.uint8), a.g["cache"].view(torch.uint8))


def test_no_tokens():
    a = Append(1, 4, 64, False, True, seed=6)
    z = lambda t: t[:0].cuda()
    cache = a.cache.cuda()
    api.rope_cache_write(z(a.latent), z(a.rope), z(a.pos), a.cs.cuda(), z(a.slots), cache, q_rope=z(a.q_rope), q=z(a.q))
    assert torch.equal(cache.cpu(), a.cache)


# ------------------------------------------------------------------------------------ merge
def merge_exact(oa, la, ob, lb):
    la, lb = la.double(), lb.double()
    m = torch.maximum(la, lb)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    wa, wb = torch.exp(la - m0), torch.exp(lb - m0)
    z = wa + wb
    inv = torch.where(z == 0, torch.zeros_like(z), 1 / z)
    ta = torch.where((wa == 0)[..., None], torch.zeros(()).double(), (wa * inv)[..., None] * oa.double())
    tb = torch.where((wb == 0)[..., None], torch.zeros(()).double(), (wb * inv)[..., None] * ob.double())
    return ta + tb, m0 + torch.log(z), ta.abs() + tb.abs()


@pytest.mark.parametrize("shape", [(1,), (7, 3), (128, 16), (2, 3, 5), (33, 128)])
def test_merge(shape):
    rng = np.random.default_rng(sum(shape))
    oa, ob = bf16_normal(rng, *shape, 512), bf16_normal(rng, *shape, 512)
    la = torch.from_numpy(rng.normal(5, 4, shape).astype(np.float32))
    lb = torch.from_numpy(rng.normal(5, 4, shape).astype(np.float32))
    fa, fb = la.view(-1), lb.view(-1)
    n = fa.numel()
    if n > 6:
        fa[0] = -math.inf                          # nothing attended: its rows may hold NaN
        oa.view(-1, 512)[0] = float("nan")
        fb[1] = -math.inf
        ob.view(-1, 512)[1] = float("inf")
        fa[2] = fb[2] = -math.inf
        fa[3], fb[3] = 300.0, -300.0
        fa[4], fb[4] = -3e38, -3e38
    out, lse = api.merge_states(oa.cuda(), la.cuda(), ob.cuda(), lb.cuda())
    r, rl, size = merge_exact(oa, la, ob, lb)
    o, l = out.double().cpu(), lse.double().cpu()
    assert ((o - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -19 * size).all()
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(l), none)
    assert ((l - rl)[~none].abs() <= 2.0 ** -22 * rl[~none].abs() + 1e-6).all()
    # in place of either input
    for which in (0, 1):
        g = [t.cuda() for t in (oa, la, ob, lb)]
        api.merge_states(*g, out=g[2 * which], lse=g[2 * which + 1])
        assert torch.equal(g[2 * which], out) and torch.equal(g[2 * which + 1], lse)


def test_merge_of_nothing():
    z = torch.empty((0, 4, 512), dtype=torch.bfloat16, device="cuda")
    l = torch.empty((0, 4), dtype=torch.float32, device="cuda")
    out, lse = api.merge_states(z, l, z, l)
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)
