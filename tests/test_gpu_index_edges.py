"""Edges of the block scores and the block selection."""
import pytest
import torch

from mla_paged_decode_02_gb300 import api
from sparse_harness import ScoreCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


@pytest.mark.parametrize("lens", [[(1, 700)] * 40, [(3, 1500), (37, 90)]])
@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_scores_with_weights_by_one_copy_and_by_loads(H, lens):
    """Heads that fill a token's columns: weights on a 16-byte boundary come by a bulk copy into memory that nothing
    else has written, others by loads. Few units, so that each fills a buffer for the first time, and repeated, as
    what could go wrong is a matter of order."""
    c = ScoreCase(lens, H, 64, 32, seed=H)
    c.run()
    c.check()
    assert c.dev[1].data_ptr() % 16 == 0
    shifted = torch.empty(c.w.numel() + 1, device="cuda")[1:].view(c.w.shape)
    shifted.copy_(c.w)
    kw = dict(max_seq_len=c.max_seq_len, block_size=32)
    for weights in (c.dev[1], shifted) * 20:
        out = torch.full_like(c.out, 7.5)
        assert torch.equal(api.index_scores(c.dev[0], weights, *c.dev[2:], out=out, **kw), c.out)


def guarded(c):
    """(scores with 9 rows on either side that nothing may write, the rows themselves)"""
    rows = torch.full((c.T + 18, -(-c.max_seq_len // c.block)), 7.5, device="cuda")
    return rows[9:-9], rows


LENS = [(2, 100), (1, 64), (40, 300)]


def test_scores_of_a_bad_page_are_page_0s():
    bad, page0 = ScoreCase(LENS, 8, 16, 16, seed=4, pad=2), ScoreCase(LENS, 8, 16, 16, seed=4, pad=2)
    bad.table[0, 2], bad.table[2, 18] = 1 << 20, -1
    page0.table[0, 2], page0.table[2, 18] = 0, 0
    page0.slots[0][32:48] = torch.arange(16)
    page0.slots[2][288:300] = torch.arange(12)
    out, rows = guarded(bad)
    bad.run(out=out)
    page0.run()
    page0.check()
    assert bad.error.item() == 0x1 and torch.equal(out, page0.out)
    assert (rows[:9] == 7.5).all() and (rows[-9:] == 7.5).all()


def test_scores_of_a_bad_length_are_those_of_the_clamped_one():
    """A length above max_seq_len is that limit's, one above the table's that of its pages, a negative one none."""
    for limit, want in ((208, 208), (1000, 320)):
        lens = [(2, 100), (3, 320)]
        bad, good = ScoreCase(lens, 8, 16, 16, seed=5, max_seq_len=limit), ScoreCase(lens, 8, 16, 16, seed=5, max_seq_len=limit)
        for c in (bad, good):
            c.table = c.table[:, :20].contiguous()                  # the pages of 320 keys
        bad.seq_lens[1] = 1 << 19
        good.lens, good.seq_lens[1] = [(2, 100), (3, want)], want
        out, rows = guarded(bad)
        bad.run(out=out)
        good.run()
        good.check()
        assert bad.error.item() == 0x2 and torch.equal(out, good.out)
        assert (rows[:9] == 7.5).all() and (rows[-9:] == 7.5).all()
    bad = ScoreCase(LENS, 8, 16, 16, seed=4, pad=1)
    bad.seq_lens[1] = -5
    bad.run()
    torch.cuda.synchronize()
    assert bad.error.item() == 0x2 and (bad.out[2] == -float("inf")).all()
    assert torch.isfinite(bad.out[0, 0]) and torch.isfinite(bad.out[3, 0]) and (bad.out[-1] == 7.5).all()


OFFSETS = [[-1, 2, 3, 43], [-40, 2, 3, 43], [0, 9, 3, 43], [0, -7, 3, 43], [0, 2, 3, 46], [0, 2, 3, 1 << 30], [5, 2, 3, 43],
           [43, 3, 2, 0], [-(1 << 31), 2, 3, (1 << 31) - 1], [50, 60, 70, 80]]


@pytest.mark.parametrize("cu", OFFSETS)
def test_scores_and_selections_of_bad_offsets_stay_within_their_rows(cu):
    c = ScoreCase(LENS, 8, 16, 16, seed=6, pad=2)
    assert c.T == 45
    c.cu = torch.tensor(cu, dtype=torch.int32)
    out, rows = guarded(c)
    c.run(out=out)
    torch.cuda.synchronize()
    assert c.error.item() & 0x20
    assert (rows[:9] == 7.5).all() and (rows[-9:] == 7.5).all()
    for columns in (20, 1500):                                      # a warp for each row, or a block
        scores = torch.randn(45, columns, device="cuda")
        rows = torch.full((45 + 18, 6), 77, dtype=torch.int32, device="cuda")
        error = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.select_blocks(scores, c.dev[5], c.dev[6], 6, block_size=16, out=rows[9:-9], device_error=error)
        assert error.item() & 0x20
        assert (rows[:9] == 77).all() and (rows[-9:] == 77).all()
        inside = rows[9:-9]                                         # rows left alone, or filled within the columns
        assert ((inside == 77) | ((inside >= -1) & (inside < columns))).all()


def test_selection_of_a_bad_length_is_that_of_the_clamped_one():
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 4], **i32)
    for columns in (10, 2000):
        s = torch.randn(4, columns, device="cuda")
        limit = 8 * columns
        for length, same in ((limit + 20, limit), (1 << 30, limit), (-3, 0)):
            error = torch.zeros(1, **i32)
            got = api.select_blocks(s, torch.tensor([length, 64], **i32), cu, 4, block_size=8, device_error=error)
            assert error.item() == 0x2
            error.zero_()
            want = api.select_blocks(s, torch.tensor([same, 64], **i32), cu, 4, block_size=8, device_error=error)
            assert error.item() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("H", [8, 64])
def test_scores_of_large_weights(H):
    """Sums over heads up to 2^127 are finite, whatever the head: a quarter of the heads is added doubled."""
    c = ScoreCase([(1, 64)], H, 64, 64, seed=7)
    c.q[:], c.cache[:], c.scale[:] = 0x7E, 0x7E, 2.0 ** -120        # 448 everywhere
    for used in (range(H), [6], [H - 1], [0]):
        c.w[:] = 0.0
        c.w[0, list(used)] = 0.999 * 2.0 ** 127 / (128 * 448.0 ** 2 * len(used))
        c.run()
        c.check()
        assert 0.99 * 2.0 ** 7 < c.out[0, 0].item() < 2.0 ** 7
