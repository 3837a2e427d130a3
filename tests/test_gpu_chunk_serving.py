"""The chunked-prefill operators together, as a serving engine calls them, against the float64
oracle of the decode tests; CUDA graphs, streams, shared workspaces, device-side errors."""
import numpy as np
import pytest
import torch

from chunk_harness import BF, F8, SCALE, ChunkCase, bf16_normal
from mla_paged_decode_02_gb300 import api
from oracle import mla_oracle as O
from test_gpu_append_merge import rotate, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


def close(out, lse, r, rl, kv):
    """The decode tests' contract: per element and relative L2 (bf16), relative L2 and cosine (FP8)."""
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    err = np.linalg.norm(o - r) / np.linalg.norm(r)
    assert err <= (5e-3 if kv == BF else 1e-2), err
    if kv == BF:
        assert np.abs(o - r).max() <= 2e-2
    else:
        assert O.cos_diff(o, r) < 1e-4
    assert np.abs(l - rl).max() <= 1e-3


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_serving_run(kv):
    """Prompts arrive in pieces, are appended and attended step by step beside decoding
    sequences, then decode: every step's rows equal the oracle's attention over the cache that the
    float64 rotation of all tokens so far would give (up to the cache's own rounding, which the
    oracle reads back)."""
    rng = np.random.default_rng(11)
    B, H, P, pages = 3, 16, 32, 40
    cs = table(4096)
    total = [0] * B
    perm = rng.permutation(pages)
    bt = np.zeros((B, 12), dtype=np.int32)
    for b in range(B):
        bt[b] = perm[12 * b:12 * b + 12]
    scale = torch.tensor([6.0 / 448], device="cuda") if kv == F8 else None
    cache = (torch.full((pages, P, 576), 0x7F, dtype=torch.uint8, device="cuda") if kv == F8 else
             torch.full((pages, P, 576), float("nan"), dtype=torch.bfloat16, device="cuda"))
    steps = [[70, 1, 0], [60, 33, 1], [0, 100, 1], [1, 1, 200], [1, 1, 1]]
    for news in steps:
        T = sum(news)
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        pos = np.concatenate([np.arange(total[b], total[b] + news[b]) for b in range(B)]).astype(np.int64)
        seq = np.repeat(np.arange(B), news)
        slots = bt[seq, pos // P].astype(np.int64) * P + pos % P
        kvp, qp = bf16_normal(rng, T, 576), bf16_normal(rng, T, H, 192)
        q = bf16_normal(rng, T, H, 576).cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        g = kvp.cuda()
        api.rope_cache_write(g[:, :512], g[:, 512:], torch.from_numpy(pos).cuda(), cs.cuda(), torch.from_numpy(slots).cuda(),
                             cache, scale, q_rope=qp.cuda()[:, :, 128:], q=q, interleaved=True, device_error=err)
        total = [t + n for t, n in zip(total, news)]
        ws = None
        out, lse = api.chunk_attention(q, cache, torch.from_numpy(bt).cuda(), torch.tensor(total, dtype=torch.int32).cuda(),
                                       torch.from_numpy(starts).cuda(), SCALE, scale, max_seq_len=400, workspace=ws)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        # the queries' rope part
        want = rotate(qp[:, :, 128:].float(), cs[torch.from_numpy(pos)][:, None], True).to(torch.bfloat16)
        assert torch.equal(q[:, :, 512:].cpu().view(torch.int16), want.view(torch.int16))
        # each token as a one-token decode of the oracle over the keys it sees
        bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
        cn = cache.cpu().numpy() if kv == F8 else bits(cache)
        lens = (pos + 1).astype(np.int32)
        r, rl = O.mla_decode(bits(q)[:, None], cn, bt[seq], lens, P, SCALE, kv, 6.0 / 448 if kv == F8 else None, True)
        close(out, lse, r[:, 0], rl[:, 0], kv)


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_shared_prefix_and_the_rest_merge_into_the_whole(kv):
    """All queries over the shared prefix in one chunk call without a mask, each over its own rest by
    decode, joined: the attention over prefix and rest together. One request has an empty prefix."""
    rng = np.random.default_rng(12)
    H, P, prefix, rest = 16, 64, 512, [100, 1, 64, 333]
    B = len(rest)
    lens = [(1, prefix + r) for r in rest]
    whole = ChunkCase(lens, H, P, kv, seed=13)
    pages = prefix // P
    # the prefix pages of sequence 0 are everyone's
    for b in range(1, B):
        for j in range(prefix):
            whole.set_key(b, j, whole.cache.view(-1, 576)[int(whole.table[0, j // P]) * P + j % P].clone())
        whole.keys[b] = torch.cat([whole.keys[0][:prefix], whole.keys[b][prefix:]])
    whole.run()
    whole.check()
    q, cache, bt, sl, cu = whole.dev
    one = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    oa, la = api.chunk_attention(q, cache, bt[:1, :pages].contiguous(), one([prefix]), one([0, B]), SCALE, whole.dscale,
                                 max_seq_len=prefix, causal=False)
    ob, lb = api.decode(q[:, None].contiguous(), cache, bt[:, pages:-1].contiguous(), one(rest), SCALE, whole.dscale,
                        max_seq_len=max(rest))
    out, lse = api.merge_states(oa, la, ob[:, 0], lb[:, 0])
    for b in range(B):
        r, rl, bound = whole.exact(b)
        # one more rounding of each part and of the result
        size = (oa[b].double().cpu().abs() + ob[b, 0].double().cpu().abs())
        assert ((out[b].double().cpu() - r[0]).abs() <= 2 * bound[0] + 2.0 ** -8 * size + 2.0 ** -8 * r[0].abs()).all()
        assert (lse[b].double().cpu() - rl[0]).abs().max() <= 1e-3
    none = torch.full_like(la, float("-inf"))
    out, lse = api.merge_states(torch.full_like(oa, float("nan")), none, ob[:, 0], lb[:, 0])
    assert torch.equal(out, ob[:, 0]) and torch.equal(lse, lb[:, 0])


def test_a_prompt_attended_in_two_pieces_of_context():
    """Chunk attention over the first keys without a mask and over the rest with one, merged."""
    c = ChunkCase([(40, 700)], 20, 64, BF, seed=14)
    c.run()
    c.check()
    q, cache, bt, sl, cu = c.dev
    one = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    split = 448
    oa, la = api.chunk_attention(q, cache, bt[:, :split // 64].contiguous(), one([split]), cu, SCALE, max_seq_len=split, causal=False)
    ob, lb = api.chunk_attention(q, cache, bt[:, split // 64:].contiguous(), one([700 - split]), cu, SCALE, max_seq_len=700)
    out, lse = api.merge_states(oa, la, ob, lb)
    r, rl, bound = c.exact(0)
    size = oa.double().cpu().abs() + ob.double().cpu().abs()
    assert ((out.double().cpu() - r).abs() <= 2 * bound + 2.0 ** -8 * size + 2.0 ** -8 * r.abs()).all()
    assert (lse.double().cpu() - rl).abs().max() <= 1e-3


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_single_token_each_equals_decode(kv):
    """n_b = 1 everywhere is a decode step."""
    lens = [(1, L) for L in (1, 63, 64, 65, 300, 1000, 2049)]
    c = ChunkCase(lens, 16, 64, kv, seed=15)
    c.run()
    c.check()
    q, cache, bt, sl, cu = c.dev
    od, ld = api.decode(q[:, None].contiguous(), cache, bt[:, :-1].contiguous(), sl, SCALE, c.dscale, max_seq_len=2049)
    for b in range(len(lens)):
        r, rl, bound = c.exact(b)
        assert ((c.out[b] - od[b, 0]).double().cpu().abs() <= 2 * bound[0]).all()
        assert (c.lse[b] - ld[b, 0]).abs().max().item() <= 2e-3


def test_one_capture_replays_with_new_lengths_queries_and_offsets():
    """A batch padded to 64 tokens: one graph serves other splits of the rows among the sequences."""
    for kv in (BF, F8):
        a = ChunkCase([(30, 700), (1, 300), (8, 8)], 16, 64, kv, pad=25, seed=16)
        a.run()
        a.check()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        q, cache, bt, sl, cu = a.dev
        with torch.cuda.graph(graph, stream=side):
            api.chunk_attention(q, cache, bt, sl, cu, SCALE, a.dscale, max_seq_len=a.max_seq_len, out=a.out, lse=a.lse,
                                workspace=a.workspace)
        torch.cuda.current_stream().wait_stream(side)
        o, l = a.out.clone(), a.lse.clone()
        a.out.fill_(7.0)
        a.lse.fill_(-3.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, o) and torch.equal(a.lse, l)
        # other rows: the first sequence brings 3, the second is idle, the third brings all of its 8
        a.lens = [(3, 650), (0, 300), (8, 8)]
        a.starts = np.array([0, 3, 3, 11], dtype=np.int32)
        a.q[:11] = bf16_normal(np.random.default_rng(17), 11, 16, 576)
        a.keys[0] = a.keys[0][:650]
        q.copy_(a.q)
        sl.copy_(torch.tensor([L for _, L in a.lens], dtype=torch.int32))
        cu.copy_(torch.from_numpy(a.starts))
        a.out.fill_(7.0)
        a.lse.fill_(-3.5)
        graph.replay()
        a.check()


def test_two_streams_with_workspaces_of_their_own():
    cases = [ChunkCase([(100, 3000), (7, 500)], 16, 64, BF, seed=18), ChunkCase([(20, 5000), (3, 64)], 16, 64, F8, seed=19)]
    for c in cases:
        c.run()
        c.check()
    streams = [torch.cuda.Stream() for _ in cases]
    want = [(c.out.clone(), c.lse.clone()) for c in cases]
    spaces = [torch.empty_like(c.workspace) for c in cases]
    torch.cuda.synchronize()
    got = []
    for rep in range(4):
        for c, s, w in zip(cases, streams, spaces):
            q, cache, bt, sl, cu = c.dev
            got.append(api.chunk_attention(q, cache, bt, sl, cu, SCALE, c.dscale, max_seq_len=c.max_seq_len, workspace=w, stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_calls_without_a_workspace_on_another_stream():
    """Tensors the call allocates stay alive until its stream is done with them."""
    c = ChunkCase([(50, 2000)], 16, 64, BF, seed=20)
    c.run()
    c.check()
    q, cache, bt, sl, cu = c.dev
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [api.chunk_attention(q, cache, bt, sl, cu, SCALE, max_seq_len=2000, stream=s) for _ in range(6)]
    junk = [torch.full((1 << 22,), 1.0, device="cuda") for _ in range(4)]     # takes freed memory, if any
    merged = api.merge_states(*outs[0], *outs[1], stream=s)
    torch.cuda.synchronize()
    del junk
    for o, l in outs:
        assert torch.equal(o, c.out) and torch.equal(l, c.lse)
    assert torch.equal(merged[0], c.out)          # two equal halves of the weight: the same rows
    assert (merged[1] - c.lse - np.log(2)).abs().max().item() <= 1e-5


# ------------------------------------------------------------------------- device-side errors
@pytest.mark.parametrize("kv", [BF, F8])
def test_bad_pages_lengths_and_offsets_are_reported(kv):
    c = ChunkCase([(5, 300), (2, 70)], 16, 64, kv, seed=21)
    c.table[0, 2] = c.num_pages                    # a page outside the pool: page 0 is read instead
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (-6, 0x1)
    c.table[0, 2] = -1
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (-6, 0x1)

    c = ChunkCase([(5, 300), (2, 70)], 16, 64, kv, seed=21)
    c.seq_lens[0] = c.max_seq_len + 1              # clamped
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (-6, 0x2)
    c.seq_lens[0] = -4
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (-6, 0x2)

    for cu in ([0, 8, 7], [-1, 5, 7], [0, 5, 99], [3, 2, 7]):
        c = ChunkCase([(5, 300), (2, 70)], 16, 64, kv, seed=21)
        c.cu = torch.tensor(cu, dtype=torch.int32)
        c.run()
        torch.cuda.synchronize()
        assert api.decode_check(c.workspace) == (-6, 0x20)
        assert (c.out == 7.0).all() and (c.lse == -3.5).all()
    c = ChunkCase([(5, 300), (2, 70)], 16, 64, kv, seed=21)
    c.run()
    c.check()


def test_no_tokens_at_all():
    c = ChunkCase([(0, 300), (0, 0)], 16, 64, BF, seed=22)
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    c = ChunkCase([(0, 300), (0, 0)], 16, 64, BF, seed=22, pad=3)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_stalled_pipeline_times_out_and_the_next_call_is_clean(kv):
    c = ChunkCase([(40, 900), (1, 300)], 16, 64, kv, seed=23)
    c.run()
    c.check()
    try:
        api.test_set_hooks(wait_limit_ns=20_000_000, stall=True)
        c.run(out=c.out, lse=c.lse, workspace=c.workspace)
        st, bits = api.decode_check(c.workspace)
    finally:
        api.test_set_hooks()
    assert st == -5 and bits & 0x8
    c.run()
    c.check()


# ----------------------------------------------------------------------------- sizes, extremes
def test_many_sequences():
    """More sequences than the scheduler has threads, most of them idle or single tokens."""
    rng = np.random.default_rng(24)
    lens = [(int(n), int(n + c)) for n, c in zip(rng.integers(0, 3, 1500), rng.integers(0, 40, 1500))]
    c = ChunkCase(lens, 4, 8, BF, seed=25)
    c.run()
    c.check(seqs=[b for b in range(1500) if b % 50 < 2 or b > 1490])


@pytest.mark.parametrize("scale", [0.0, -0.07])
def test_scales_of_any_sign(scale):
    """A zero scale averages the values; a negative one turns the scores around."""
    import chunk_harness
    c = ChunkCase([(9, 520)], 16, 64, BF, seed=26)
    old = chunk_harness.SCALE
    try:
        chunk_harness.SCALE = scale
        c.run()
        c.check()
    finally:
        chunk_harness.SCALE = old


def test_large_and_tiny_queries_over_an_fp8_cache():
    """The two-term split of q scales each row by itself: rows of very different magnitudes."""
    c = ChunkCase([(6, 400)], 16, 64, F8, seed=27)
    q = c.q.float()
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] = 0
    q[3, :, 100] = 3e4
    c.q = q.to(torch.bfloat16)
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    r, rl, bound = c.exact(0)
    o = c.out.double().cpu()
    assert torch.isfinite(o).all()
    # rows whose scores stay moderate keep the usual bounds; the first attends one key (its scores
    # differ by more than any rounding of them)
    for i in (1, 2, 4, 5):
        assert ((o[i] - r[i]).abs() <= bound[i]).all(), i
    assert ((o[0] - r[0]).abs() <= 2.0 ** -7 * r[0].abs() + 1e-6).float().mean() > 0.99


def test_a_long_cache_beyond_31_bits_of_bytes():
    """A pool whose byte offsets pass 2^31 (and whose element offsets do, for the bf16 cache)."""
    P, pages, H = 128, 32768, 16
    cache = torch.zeros((pages, P, 576), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(28)
    L = 500
    where = [pages - 1, pages - 5, 7, pages - 100]
    rows = bf16_normal(rng, L, 576)
    for i, pg in enumerate(where):
        n = min(P, L - i * P)
        cache[pg, :n] = rows[i * P:i * P + n].cuda()
    q = bf16_normal(rng, 3, H, 576)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out, lse = api.chunk_attention(q.cuda(), cache, i32([where]), i32([L]), i32([0, 3]), SCALE, max_seq_len=L)
    c = ChunkCase([(3, L)], H, P, BF, seed=29)
    c.q[:3] = q
    c.keys[0] = rows.double()
    r, rl, bound = c.exact(0)
    assert ((out.double().cpu() - r).abs() <= bound).all()
    # and appending to the last slot
    lat, rope = bf16_normal(rng, 1, 512).cuda(), bf16_normal(rng, 1, 64).cuda()
    one = lambda v: torch.tensor([v], dtype=torch.int64, device="cuda")
    api.rope_cache_write(lat, rope, one(0), table(4).cuda(), one(pages * P - 1), cache)
    assert torch.equal(cache[-1, -1, :512], lat[0]) and torch.equal(cache[-1, -1, 512:], rope[0])
