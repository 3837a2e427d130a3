"""Ragged chunk attention against float64, within the bounds of tests/chunk_harness.py: head
counts that leave blocks ragged, page sizes from 8 rows, lengths around the tile and block
edges, idle sequences, rows that see no key, single-token rows, and NaN or infinities wherever
a row does not look."""
import numpy as np
import pytest
import torch

from chunk_harness import BF, F8, SCALE, ChunkCase
from mla_paged_decode_02_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H,P,lens", [
    (128, 64, [(1, 1)]),                                  # a single key
    (128, 64, [(1, 256), (1, 257), (1, 255)]),            # tile edges
    (128, 128, [(5, 300), (0, 77), (3, 3)]),              # an idle sequence
    (16, 64, [(17, 274), (1, 100)]),                      # ragged blocks
    (16, 64, [(8, 8), (9, 9), (1, 1), (130, 130)]),       # whole prompts
    (16, 64, [(40, 1000)] + [(1, 500 + 61 * i) for i in range(9)]),
    (1, 64, [(200, 333), (1, 1025)]),                     # 128 tokens in a block
    (3, 64, [(50, 513)]),
    (20, 64, [(13, 770), (7, 31)]),
    (100, 64, [(3, 600)]),
    (128, 64, [(20, 1100)]),
])
def test_lengths_and_heads(kv, H, P, lens):
    c = ChunkCase(lens, H, P, kv, seed=len(lens) + H)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("P", [8, 16, 24, 32, 48, 96, 256, 1024])
def test_page_sizes(kv, P):
    c = ChunkCase([(6, 530), (1, 41), (10, 10)], 16, P, kv, seed=P)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_no_key(kv, causal):
    """A sequence shorter than its new tokens leaves its first rows without a key (causal); one
    without any key leaves all of them."""
    c = ChunkCase([(9, 4), (3, 0), (5, 260), (2, 2)], 16, 64, kv, causal=causal, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_shared_prefix_without_a_mask(kv):
    c = ChunkCase([(33, 1500)], 16, 64, kv, causal=False, seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_padding_rows_before_and_behind_are_left(kv):
    c = ChunkCase([(4, 90), (11, 400)], 16, 64, kv, pad=9, lead=5, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("H", [1, 16, 20])
def test_masked_keys_may_hold_anything(kv, H):
    """NaN and infinities in the keys of the last tokens: tokens before them are exact, tokens that
    see them are not finite."""
    bad = ([torch.tensor(v, dtype=torch.bfloat16) for v in (float("nan"), float("inf"), float("-inf"))]
           if kv == BF else [torch.tensor(0x7F, dtype=torch.uint8), torch.tensor(0xFF, dtype=torch.uint8)])
    n, L = 150, 700
    for v in bad:
        c = ChunkCase([(n, L), (2, 50)], H, 64, kv, seed=6)
        for j in (L - 1, L - 40, L - 41):
            c.set_key(0, j, v)
        c.run()
        torch.cuda.synchronize()
        assert api.decode_check(c.workspace) == (0, 0)
        clean = n - 41                                   # tokens that see none of the three
        out, lse = c.out.double().cpu(), c.lse.double().cpu()
        r, rl, bound = c.exact(0)
        assert ((out[:clean] - r[:clean]).abs() <= bound[:clean]).all()
        assert (lse[:clean] - rl[:clean]).abs().max() <= 1e-3
        assert torch.isfinite(out[n:]).all()
        assert torch.isnan(out[clean:n]).any(dim=-1).all()


@pytest.mark.parametrize("kv", [BF, F8])
def test_few_rows_over_a_long_context_are_split(kv):
    c = ChunkCase([(2, 20000), (1, 9000)], 16, 64, kv, seed=7)
    c.run()
    c.check()


@pytest.mark.parametrize("kv,H", [(BF, 128), (F8, 128), (BF, 16), (F8, 16)])
def test_many_blocks(kv, H):
    """More blocks than workers: units that start and end inside a worker's range."""
    lens = [(60, 60 + 97 * i) for i in range(6)] if H == 128 else [(300, 300 + 211 * i) for i in range(8)]
    c = ChunkCase(lens, H, 64, kv, seed=8)
    c.run()
    c.check(seqs=[0, len(lens) - 1])


def test_growing_scores_move_the_reference():
    """Keys whose scores grow along the sequence: the running reference moves in every tile."""
    for kv in (BF, F8):
        c = ChunkCase([(4, 2000)], 16, 64, kv, seed=9)
        q = c.q.float()
        q[:, :, :] = q[:1, :1, :]                         # one direction for all rows
        c.q = q.to(torch.bfloat16)
        d = c.q[0, 0].double() / c.q[0, 0].double().norm()
        k = c.keys[0]
        amp = torch.linspace(-20, 20, 2000, dtype=torch.float64)[:, None]
        if kv == BF:
            rows = (0.2 * k + amp * d[None, :]).to(torch.bfloat16)
            c.keys[0] = rows.double()
        else:
            rows = ((0.2 * k + amp * d[None, :]).float() / c.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            c.keys[0] = rows.float().double() * c.kv_scale.double()
        for j in range(2000):
            c.set_key(0, j, rows[j] if kv == BF else rows[j].view(torch.uint8))
        c.run()
        c.check()


def test_garbage_after_repeats_changes_nothing():
    """The same call on a used workspace gives the same bits."""
    for kv in (BF, F8):
        c = ChunkCase([(37, 3000), (1, 700), (5, 5)], 16, 64, kv, seed=10)
        c.run()
        o, l = c.out.clone(), c.lse.clone()
        for _ in range(5):
            c.run(out=c.out, lse=c.lse, workspace=c.workspace)
            torch.cuda.synchronize()
            assert torch.equal(c.out, o) and torch.equal(c.lse, l)
