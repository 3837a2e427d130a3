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
