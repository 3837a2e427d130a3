"""Index cache write, block scores and block selection against plain implementations."""
import math

import numpy as np
import pytest
import torch

from chunk_harness import bf16_normal
from mla_paged_decode_02_gb300 import api
from sparse_harness import INF, ScoreCase, seen_keys, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


# ------------------------------------------------------------------------- index cache write
def rotated(x, cs, interleaved):
    """x [..., 128] float32 with its last 64 values turned, each product and sum rounded on its own."""
    x = x.float().clone()
    c, s = cs[..., :32], cs[..., 32:]
    t = x[..., 64:].clone()
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :32], t[..., 32:])
    y, z = a * c - b * s, b * c + a * s
    x[..., 64:] = torch.stack([y, z], dim=-1).flatten(-2) if interleaved else torch.cat([y, z], dim=-1)
    return x


def quantise(x):
    top = torch.tensor(448.0)
    m = torch.clamp(x.abs().amax(dim=-1), min=448 * 2.0 ** -126)
    return (x * (top / m)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), m / top


def table(n, seed=0):
    a = torch.from_numpy(np.random.default_rng(seed).uniform(0, 6.28, (n, 32)))
    return torch.cat([a.cos(), a.sin()], dim=1).float()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,H,P", [(1, 1, 8), (5, 3, 16), (64, 16, 64), (33, 17, 48), (7, 64, 64), (130, 128, 128)])
def test_index_write_equals_single_steps(n, H, P, interleaved):
    rng = np.random.default_rng(n * 1000 + H)
    keys, queries = bf16_normal(rng, n, 128), bf16_normal(rng, n, H, 128)
    keys[0, 5] = 300.0
    queries[0, 0] = 0.0                                   # a row of zeros
    weights = torch.from_numpy(rng.standard_normal((n, H), dtype=np.float32))
    cs = table(50)
    pos = torch.from_numpy(rng.integers(0, 50, n))
    pages = -(-n // P) + 2
    slots = torch.from_numpy(rng.permutation(pages * P)[:n].astype(np.int64))
    if n > 4:
        pos[3] = -1                                       # a padding token
        slots[1] = -1                                     # its queries alone
    d = lambda t: t.cuda()
    cache = torch.full((pages, P, 128), 0xEE, dtype=torch.uint8, device="cuda")
    scale = torch.full((pages, P), -5.0, device="cuda")
    qi = torch.full((n, H, 128), 0xDD, dtype=torch.uint8, device="cuda")
    qw = torch.full((n, H), -6.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.index_cache_write(d(keys), d(pos), d(cs), d(slots), cache, scale, queries=d(queries), weights=d(weights), q_index=qi,
                          q_weights=qw, interleaved=interleaved, device_error=err)
    want_cache, want_scale = torch.full_like(cache.cpu(), 0xEE), torch.full((pages, P), -5.0)
    want_qi, want_qw = torch.full((n, H, 128), 0xDD, dtype=torch.uint8), torch.full((n, H), -6.0)
    for t in range(n):
        if pos[t] < 0:
            continue
        if slots[t] >= 0:
            want_cache.view(-1, 128)[slots[t]], want_scale.view(-1)[slots[t]] = quantise(rotated(keys[t], cs[pos[t]], interleaved))
        want_qi[t], s = quantise(rotated(queries[t], cs[pos[t]], interleaved))
        want_qw[t] = weights[t] * s
    assert err.item() == 0
    same = lambda a, b: torch.equal(a.cpu() & 0x7F, b & 0x7F) and torch.equal((a.cpu() ^ b) & 0x80 & -((b & 0x7F) != 0).to(torch.uint8), torch.zeros_like(b))
    assert same(cache, want_cache) and same(qi, want_qi)  # a zero's sign aside
    assert torch.equal(scale.cpu(), want_scale) and torch.equal(qw.cpu(), want_qw)


def test_index_write_views_keys_alone_and_float8_tensors():
    rng = np.random.default_rng(3)
    n, H = 9, 4
    proj, qproj = bf16_normal(rng, n, 576 + 128).cuda(), bf16_normal(rng, n, H, 192).cuda()
    cs, pos, slots = table(20).cuda(), torch.arange(n).cuda(), torch.arange(n).flip(0).cuda()
    w = torch.ones(n, H, device="cuda")
    make = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    a, sa, qa, wa = make(1, 16, 128), torch.zeros(1, 16, device="cuda"), make(n, H, 128), torch.zeros(n, H, device="cuda")
    b, sb, qb, wb = make(1, 16, 128), torch.zeros(1, 16, device="cuda"), make(n, H, 128), torch.zeros(n, H, device="cuda")
    api.index_cache_write(proj[:, 576:], pos, cs, slots, a, sa, queries=qproj[..., 64:], weights=w, q_index=qa, q_weights=wa)
    api.index_cache_write(proj[:, 576:].contiguous(), pos, cs, slots, b.view(torch.float8_e4m3fn), sb)
    assert torch.equal(a, b) and torch.equal(sa, sb)
    api.index_cache_write(proj[:, 576:].contiguous(), pos, cs, slots, b, sb, queries=qproj[..., 64:].contiguous(), weights=w,
                          q_index=qb.view(torch.float8_e4m3fn), q_weights=wb)
    assert torch.equal(a, b) and torch.equal(qa, qb) and torch.equal(wa, wb)
    # one key and one query head for all
    api.index_cache_write(proj[:1, 576:].expand(1, 128), pos[:1], cs, slots[:1], a, sa)
    api.index_cache_write(proj[:, 576:], pos, cs, slots, a, sa, queries=qproj[:1, :1, 64:].expand(n, H, 128), weights=w, q_index=qa,
                          q_weights=wa)
    api.index_cache_write(proj[:, 576:], pos, cs, slots, b, sb, queries=qproj[:1, :1, 64:].expand(n, H, 128).contiguous(), weights=w,
                          q_index=qb, q_weights=wb)
    assert torch.equal(qa, qb) and torch.equal(wa, wb) and torch.equal(a, b)
    api.index_cache_write(proj[:0, 576:], pos[:0], cs, slots[:0], a, sa)


def test_index_write_reports_bad_slots_and_positions_and_marks_rows_that_are_not_finite():
    rng = np.random.default_rng(4)
    n = 6
    keys, queries = bf16_normal(rng, n, 128), bf16_normal(rng, n, 2, 128)
    keys[0, 3], keys[1, 100], queries[2, 1, 7] = float("nan"), float("inf"), float("-inf")
    keys[5] = 3e38                                        # the rotation overflows
    pos, slots = torch.tensor([0, 1, 2, 99, 3, 4]), torch.tensor([0, 1, 2, 3, 16, 5])
    cache, scale = torch.zeros(1, 16, 128, dtype=torch.uint8, device="cuda"), torch.full((1, 16), -1.0, device="cuda")
    qi, qw = torch.zeros(n, 2, 128, dtype=torch.uint8, device="cuda"), torch.full((n, 2), -1.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = torch.full((9, 64), 0.9)
    api.index_cache_write(keys.cuda(), pos.cuda(), cs.cuda(), slots.cuda(), cache, scale, queries=queries.cuda(),
                          weights=torch.ones(n, 2, device="cuda"), q_index=qi, q_weights=qw, device_error=err)
    assert err.item() == 0x10 | 0x40
    s = scale.cpu()[0]
    assert torch.isnan(s[[0, 1, 5]]).all() and s[2] > 0 and (s[[3, 4]] == -1).all() and (s[6:] == -1).all()
    w = qw.cpu()
    assert math.isnan(w[2, 1]) and (w[[0, 1, 4, 5]] > 0).all() and w[2, 0] > 0 and (w[3] == -1).all()


def test_index_write_past_two_to_the_31_bytes():
    P, pages = 64, (1 << 25) // 64 * 65 // 64             # more than 2^32 bytes of codes
    cache = torch.empty((pages, P, 128), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, P), device="cuda")
    cache[-1], scale[-1] = 0, 0.0
    keys = bf16_normal(np.random.default_rng(5), 2, 128).cuda()
    slots = torch.tensor([pages * P - 1, 1 << 25], device="cuda")
    api.index_cache_write(keys, torch.zeros(2, dtype=torch.int64, device="cuda"), table(1).cuda(), slots, cache, scale)
    code, s = quantise(rotated(keys.cpu(), table(1)[0], True))
    assert torch.equal(scale.view(-1)[slots].cpu(), s)
    assert ((cache.view(-1, 128)[slots].cpu() == code) | (code & 0x7F == 0)).all()
    # and the scores of blocks there
    q = torch.full((1, 8, 128), 0x38, dtype=torch.uint8, device="cuda")          # ones
    i32 = dict(dtype=torch.int32, device="cuda")
    got = api.index_scores(q, torch.ones(1, 8, device="cuda"), cache, scale, torch.tensor([[pages - 1]], **i32),
                           torch.tensor([64], **i32), torch.tensor([0, 1], **i32), max_seq_len=64, block_size=64)
    row = code[0].view(torch.float8_e4m3fn).double()
    want = max(0.0, row.sum().item()) * 8 * s[0].item()
    assert abs(got.item() - want) <= (128 + 8 + 3) * 2.0 ** -23 * row.abs().sum().item() * 8 * s[0].item()


# -------------------------------------------------------------------------------- scores
SCORES = [
    # lens, H, P, block, causal, pad, lead
    ([(1, 1)], 1, 8, 8, True, 0, 0),
    ([(1, 100), (1, 257)], 64, 64, 64, True, 0, 0),
    ([(3, 3), (0, 70), (5, 40), (1, 1), (0, 0)], 16, 16, 8, True, 3, 2),
    ([(9, 200)], 5, 24, 24, True, 0, 0),
    ([(4, 300), (2, 129)], 128, 32, 16, True, 1, 0),
    ([(130, 700)], 32, 64, 32, True, 0, 0),
    ([(20, 1100), (1, 2500)], 64, 128, 128, True, 0, 1),
    ([(7, 640)], 33, 64, 64, False, 0, 0),
    ([(5, 3)], 8, 8, 8, True, 0, 0),                       # more new tokens than keys: rows that see none
    ([(2, 2048)], 96, 1024, 1024, True, 0, 0),
    ([(6, 500)], 12, 200, 40, True, 2, 0),
    ([(17, 390)], 127, 48, 48, True, 0, 0),
    ([(33, 65)] * 3 + [(1, 17)] * 5, 2, 16, 16, True, 4, 0),
    ([(300, 300)], 1, 64, 8, True, 0, 0),
]


@pytest.mark.parametrize("lens,H,P,block,causal,pad,lead", SCORES)
def test_scores_match_float64(lens, H, P, block, causal, pad, lead):
    c = ScoreCase(lens, H, P, block, causal, pad, lead, seed=len(lens) + H)
    c.run()
    c.check()


def test_scores_of_many_sequences_with_idle_ones_and_long_contexts():
    rng = np.random.default_rng(1)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(3, 120))) for _ in range(1100)] + [(2, 9000)]
    c = ScoreCase(lens, 4, 16, 16, seed=9)
    c.run()
    c.check(list(range(0, 1100, 41)) + [1100])


@pytest.mark.parametrize("P,block", [(64, 8), (24, 24), (40, 40), (1000, 1000), (1024, 512)])
def test_scores_of_long_and_short_contexts_together(P, block):
    """Few sequences, whose units are sized by their lengths."""
    c = ScoreCase([(4, 33001), (0, 700), (2, 70001), (1, 5), (3, 1)], 3, P, block, seed=P, pad=1)
    c.run()
    c.check()


def test_scores_of_short_contexts_under_a_long_limit():
    c = ScoreCase([(1, 40), (0, 9), (2, 300), (1, 1)], 64, 16, 8, seed=7, max_seq_len=1 << 20)
    c.run()
    c.check()


def test_scores_with_weights_between_16_byte_boundaries():
    c = ScoreCase([(3, 400)], 64, 64, 64, seed=8)
    c.run()
    shifted = torch.empty(c.w.numel() + 1, device="cuda")[1:].view(c.w.shape)
    shifted.copy_(c.w)
    assert shifted.data_ptr() % 16 == 4
    got = api.index_scores(c.dev[0], shifted, *c.dev[2:], max_seq_len=c.max_seq_len, block_size=64)
    assert torch.equal(got, c.out)


def test_scores_of_calls_at_once():
    cases = [ScoreCase([(60, 900), (1, 2000)], 64, 64, 64, seed=20 + i) for i in range(3)]
    for c in cases:
        c.run()
    want = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(cases, streams):
            c.out.fill_(7.5)
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            api.index_scores(*c.dev, max_seq_len=c.max_seq_len, block_size=64, out=c.out, device_error=c.error, stream=s)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)
    cases[0].check()


def test_scores_of_keys_and_queries_that_are_not_finite():
    c = ScoreCase([(3, 200)], 16, 64, 64, seed=2)
    j = c.slots[0]
    c.scale.view(-1)[j[10]] = float("nan")                 # a key whose row was not finite
    c.cache.view(-1, 128)[j[10]] = 0x7F
    c.scale.view(-1)[j[70]] = float("inf")
    c.cache.view(-1, 128)[j[71]] = 0x7F                    # NaN codes under a finite scale
    c.w[1, 4] = float("nan")                               # a query head whose row was not finite
    c.run()
    torch.cuda.synchronize()
    out = c.out.cpu()
    assert not torch.isnan(out).any() and (out[1] == -INF).all()
    r, bound = c.exact(0)
    for i in (0, 2):
        for col in range(4):
            assert out[i, col] == r[i, col] if math.isinf(r[i, col]) else abs(out[i, col] - r[i, col]) <= bound[i, col]


def test_scores_all_negative_or_zero():
    c = ScoreCase([(4, 150)], 8, 16, 16, seed=3)
    c.w[:] = -c.w.abs()
    c.run()
    c.check()
    assert (c.out[0][torch.isfinite(c.out[0])] <= 0).all()


def test_scores_report_device_errors():
    c = ScoreCase([(2, 100), (1, 64)], 8, 16, 16, seed=4)
    c.table[0, 2] = 1 << 20                                # read as page 0
    c.run()
    torch.cuda.synchronize()
    assert c.error.item() == 0x1
    c = ScoreCase([(2, 100), (1, 64)], 8, 16, 16, seed=4)
    c.seq_lens[1] = 1 << 19
    c.run()
    torch.cuda.synchronize()
    assert c.error.item() & 0x2
    c = ScoreCase([(2, 100), (1, 64)], 8, 16, 16, pad=2, seed=4)
    c.cu[1] = 9
    c.run()
    torch.cuda.synchronize()
    assert c.error.item() & 0x20
    c = ScoreCase([(2, 100), (1, 64)], 8, 16, 16, seed=4)
    c.run()
    c.check()


def test_scores_of_a_stalled_pipeline_time_out_and_the_next_call_is_clean():
    c = ScoreCase([(3, 3000), (1, 700)], 64, 64, 64, seed=6)
    api.test_set_hooks(20_000_000, True)
    try:
        c.run()
        torch.cuda.synchronize()
        assert c.error.item() == 0x8
    finally:
        api.test_set_hooks(0, False)
    c.run()
    c.check()


def test_scores_default_output_strided_streams_and_graph():
    c = ScoreCase([(5, 300), (1, 90)], 64, 64, 32, seed=5)
    c.run()
    want = c.out.clone()
    got = api.index_scores(*c.dev, max_seq_len=c.max_seq_len, block_size=32)
    assert torch.equal(got, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.index_scores(*c.dev, max_seq_len=c.max_seq_len, block_size=32, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(g):
        api.index_scores(*c.dev, max_seq_len=c.max_seq_len, block_size=32, out=out)
    for n in (301, 290):
        c.dev[5][0] = n - 1
        g.replay()
        assert torch.equal(out, api.index_scores(*c.dev, max_seq_len=c.max_seq_len, block_size=32))
        assert torch.equal(out, want) == (n == 301)


# ------------------------------------------------------------------------------- selection
def run_select(scores, lens, block, K, first, last, causal=True, lead=0, pad=0, wide=0, stream=None):
    """lens as the score cases; scores [T, C] float32 on the CPU. Checks every row."""
    starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32) + lead
    T = int(starts[-1]) + pad
    assert scores.shape[0] == T
    dev = torch.full((T, scores.shape[1] + wide), 1e9, device="cuda")
    dev[:, :scores.shape[1]] = scores.cuda()
    out = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    api.select_blocks(dev[:, :scores.shape[1]], torch.tensor([L for _, L in lens], **i32), torch.tensor(starts.tolist(), **i32), K,
                      block_size=block, keep_first=first, keep_last=last, causal=causal, out=out, device_error=err, stream=stream)
    torch.cuda.synchronize()
    got = out.cpu().tolist()
    assert err.item() == 0
    for b, (n, L) in enumerate(lens):
        for i in range(n):
            t = int(starts[b]) + i
            want = selection(scores[t].tolist(), seen_keys(n, L, i, causal), block, K, first, last)
            assert got[t] == want, (b, i)
    for t in list(range(lead)) + list(range(int(starts[-1]), T)):
        assert got[t] == [77] * K
    return out


def ragged_scores(rng, lens, block, C, lead=0, pad=0, ties=False):
    T = sum(n for n, _ in lens) + lead + pad
    s = torch.from_numpy(rng.standard_normal((T, C), dtype=np.float32))
    return torch.round(s * 2) / 2 if ties else s


SELECTS = [
    # lens, block, C, K, first, last
    ([(1, 1)], 8, 1, 1, 0, 0),
    ([(1, 1)], 8, 1, 5, 1, 1),
    ([(1, 6000), (1, 2048), (1, 100), (0, 50), (3, 3)], 64, 96, 16, 1, 2),
    ([(4, 4000)], 64, 63, 8, 0, 0),
    ([(40, 40)], 8, 5, 3, 1, 1),
    ([(5, 3)], 8, 4, 4, 1, 0),                              # rows that see nothing
    ([(2, 33 * 8), (2, 32 * 8), (2, 31 * 8 + 1)], 8, 33, 16, 2, 2),
    ([(3, 8200)], 8, 1030, 64, 1, 1),
    ([(2, 20000)], 8, 2500, 700, 3, 5),
    ([(2, 100000)], 24, 4200, 64, 1, 4),
    ([(1, 1 << 20), (1, 500000)], 8, 131072, 1000, 1, 1),
    ([(9, 1025 * 16)], 16, 1025, 1024, 0, 3),
    ([(70, 3000)], 16, 188, 187, 1, 0),
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,block,C,K,first,last", SELECTS)
def test_selection_equals_sorting(lens, block, C, K, first, last, ties):
    s = ragged_scores(np.random.default_rng(K), lens, block, C, lead=1, pad=2, ties=ties)
    run_select(s, lens, block, K, first, last, lead=1, pad=2, wide=3)
    run_select(s, lens, block, K, first, last, causal=False, lead=1, pad=2)


@pytest.mark.parametrize("C", [20, 300, 1500, 9000])
def test_selection_of_special_values(C):
    rng = np.random.default_rng(C)
    lens = [(1, C * 16)] * 9
    s = torch.from_numpy(rng.standard_normal((9, C), dtype=np.float32))
    s[0, ::3] = float("nan")
    s[1, :] = -INF
    s[2, :] = float("nan")
    s[3, ::2] = INF
    s[4, :] = 0.0
    s[4, ::2] = -0.0
    s[5, 1::2] = -INF
    s[6, :] = -torch.finfo(torch.float32).max
    s[6, C // 2:] = -INF
    s[7, :] = 2.0 ** -149                                   # the smallest numbers are told apart
    s[7, C // 3] = 2.0 ** -148
    s[7, C // 2] = -2.0 ** -149
    s[8, :] = 1.0
    s[8, 7] = 1.0 + 2.0 ** -23
    for K in (1, 7, C // 2, C - 1):
        run_select(s, lens, 16, K, 0, 0)
        if K > 3:
            run_select(s, lens, 16, K, 1, 2)


def test_selection_of_many_rows_default_output_stream_and_graph():
    rng = np.random.default_rng(8)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(3, 5000))) for _ in range(1500)]
    s = ragged_scores(rng, lens, 32, 157)
    want = run_select(s, lens, 32, 24, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    seq = torch.tensor([L for _, L in lens], **i32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in lens])]).tolist(), **i32)
    dev = s.cuda()
    got = api.select_blocks(dev, seq, cu, 24, block_size=32, keep_first=1, keep_last=1)
    assert torch.equal(got, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = api.select_blocks(dev, seq, cu, 24, block_size=32, keep_first=1, keep_last=1, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(g):
        api.select_blocks(dev, seq, cu, 24, block_size=32, keep_first=1, keep_last=1, out=out)
    dev.mul_(-1.0)
    g.replay()
    assert torch.equal(out, api.select_blocks(dev, seq, cu, 24, block_size=32, keep_first=1, keep_last=1))


def test_selection_reports_device_errors():
    i32 = dict(dtype=torch.int32, device="cuda")
    s = torch.randn(4, 10, device="cuda")
    for seq, cu, bit in (([100, 81], [0, 2, 4], 0x2), ([80, -1], [0, 2, 4], 0x2), ([80, 80], [0, 5, 4], 0x20),
                         ([80, 80], [3, 1, 4], 0x20), ([80, 80], [-1, 1, 4], 0x20), ([80, 80], [0, 1, 5], 0x20)):
        err = torch.zeros(1, **i32)
        api.select_blocks(s, torch.tensor(seq, **i32), torch.tensor(cu, **i32), 3, block_size=8, device_error=err)
        assert err.item() & bit, (seq, cu)
