"""Calls at the documented limits of the chunked-prefill operators: queries that are not finite,
more heads than a block has rows, the longest sequence, pages and queries used more than once."""
import numpy as np
import pytest
import torch

from chunk_harness import BF, F8, LSE_ABS, SCALE, ChunkCase, bf16_normal
from mla_paged_decode_02_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("lens", [[(6, 300), (1, 90)], [(1, 9000)]])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_makes_its_row_nan(kv, lens, value):
    """Some scores of the row are +inf or NaN (its keys have both signs), so its softmax is NaN; all
    other rows of the block are as they are without it."""
    H, head = 16, 5
    c = ChunkCase(lens, H, 64, kv, seed=41)
    c.run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    c.q[0, head, 40] = value
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    assert torch.isnan(c.out[0, head]).all() and torch.isnan(c.lse[0, head])
    keep = torch.ones((c.T, H), dtype=torch.bool, device="cuda")
    keep[0, head] = False
    assert torch.equal(c.out[keep], out[keep]) and torch.equal(c.lse[keep], lse[keep])


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [129, 300])
def test_more_heads_than_a_block_has_rows(kv, H):
    c = ChunkCase([(3, 290), (1, 33), (2, 2)], H, 64, kv, pad=1, seed=42)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_the_longest_sequence(kv):
    """2^20 keys: the last token against the value in float64, by pieces of the keys."""
    L, H, P = 1 << 20, 16, 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(43)
    pages = L // P
    values = torch.empty((pages, P, 576), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    scale = None
    if kv == F8:
        scale = torch.tensor([1.0 / 64], dtype=torch.float32, device="cuda")
        values = (values.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    table = torch.randperm(pages, device="cuda", generator=gen)
    q = torch.empty((2, H, 576), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out, lse = api.chunk_attention(q, values if kv == BF else values.view(torch.uint8), table.int()[None], i32([L]),
                                   i32([0, 2]), SCALE, scale, max_seq_len=L)
    step = 1 << 15
    qd = q[1].double()
    score, num, absn, absv, kmax = [], torch.zeros((H, 512), dtype=torch.float64, device="cuda"), 0, 0, 0.0
    for a in range(0, L, step):
        k = values[table[a // P:(a + step) // P]].reshape(step, 576).float().double()
        k = k if scale is None else k * scale.double()
        s = (qd @ k.T) * SCALE
        w = torch.exp(s)                               # |s| is a few units for these inputs
        score.append(w.sum(1))
        num += w @ k[:, :512]
        absn = absn + w @ k[:, :512].abs()
        absv = absv + k[:, :512].abs().sum(0)
        kmax = max(kmax, k.abs().sum(1).max().item())
        m = s.amax(1) if a == 0 else torch.maximum(m, s.amax(1))
    z = torch.stack(score).sum(0)[:, None]
    r, A = num / z, absn / z
    # the bound of tests/chunk_harness.py, with e^m / z the largest weight
    t = 2.0 ** -8 * (A + r.abs())
    if kv == F8:
        d = 2.0 ** -17 * qd.abs().amax(1, keepdim=True) * SCALE * kmax
        t = t + 2.0 ** -11 * A + 2.0 ** -13 * absv[None] * torch.exp(m)[:, None] / z + 2 * d * A
    bound = 1.05 * t + 1e-6
    assert ((out[1].double() - r).abs() <= bound).all()
    assert ((lse[1].double() - torch.log(z[:, 0])).abs() <= LSE_ABS[kv]).all()


@pytest.mark.parametrize("kv", [BF, F8])
def test_pages_shared_by_sequences_and_within_one(kv):
    """One page in several sequences, and twice in one: the same keys again."""
    c = ChunkCase([(5, 192), (3, 130)], 16, 64, kv, seed=44)
    c.table[1, :3] = c.table[0, :3]
    c.keys[1] = c.keys[0][:130]
    c.table[0, 2] = c.table[0, 0]
    c.keys[0] = torch.cat([c.keys[0][:128], c.keys[0][:64]])
    c.run()
    c.check()


def test_one_query_rope_part_for_all_heads_and_tokens():
    """q_rope with strides of zero."""
    rng = np.random.default_rng(45)
    n, H = 70, 40
    lat, rope, part = bf16_normal(rng, n, 512).cuda(), bf16_normal(rng, n, 64).cuda(), bf16_normal(rng, 64).cuda()
    cs = torch.rand((100, 64), device="cuda")
    pos = torch.arange(n, device="cuda") % 100
    cache = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda")
    got = []
    for q_rope in (part.expand(n, H, 64), part.expand(n, H, 64).contiguous()):
        q = torch.zeros((n, H, 576), dtype=torch.bfloat16, device="cuda")
        api.rope_cache_write(lat, rope, pos, cs, torch.arange(n, device="cuda"), cache, q_rope=q_rope, q=q)
        got.append(q)
    assert torch.equal(got[0], got[1]) and (got[0][..., :512] == 0).all() and got[0][..., 512:].abs().sum() > 0


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("lens", [[(6, 300), (1, 90)], [(1, 9000)]])
def test_an_output_that_starts_between_two_32_byte_boundaries(kv, lens):
    """out needs 16-byte alignment only: a contiguous view that starts 8 elements into a buffer, for
    blocks that are written directly and for blocks that are cut and merged."""
    H = 16
    c = ChunkCase(lens, H, 64, kv, pad=1, seed=46)
    n = c.T * H * 512
    flat = torch.full((n + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:8 + n].view(c.T, H, 512)
    assert out.data_ptr() % 32 == 16
    c.run(out=out, lse=torch.full((c.T, H), -3.5, dtype=torch.float32, device="cuda"))
    c.check()
    assert (flat[:8] == 7.0).all() and (flat[8 + n:] == 7.0).all()
    aligned = ChunkCase(lens, H, 64, kv, pad=1, seed=46)
    aligned.run()
    assert torch.equal(aligned.out, c.out) and torch.equal(aligned.lse, c.lse)
