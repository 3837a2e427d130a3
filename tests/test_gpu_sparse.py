"""Block-sparse attention against float64, and the four operators together as a serving step runs them."""
import math

import numpy as np
import pytest
import torch

from chunk_harness import BF, F8, LSE_ABS, SCALE, ChunkCase, bf16_normal
from mla_paged_decode_02_gb300 import api
from sparse_harness import INF, SparseCase, attended, selection

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.lib()


CASES = [
    # lens, H, P, block, K, causal, pad, lead
    ([(1, 100), (1, 257)], 16, 64, 64, 4, True, 0, 0),
    ([(1, 1)], 1, 8, 8, 1, True, 0, 0),
    ([(3, 3), (0, 70), (5, 40), (1, 1), (0, 0)], 16, 16, 8, 3, True, 3, 2),
    ([(9, 700)], 128, 64, 32, 7, True, 0, 0),
    ([(2, 1000), (1, 900)], 130, 24, 24, 9, True, 2, 0),
    ([(4, 1100)], 20, 128, 128, 3, True, 0, 1),
    ([(3, 2100)], 64, 1024, 1024, 2, True, 0, 0),
    ([(6, 640)], 8, 64, 16, 5, False, 0, 0),
    ([(5, 3)], 4, 8, 8, 2, True, 0, 0),                     # rows that see no key
    ([(2, 600)], 300, 64, 64, 4, True, 0, 0),
    ([(20, 333)], 3, 48, 48, 20, True, 0, 0),               # lists longer than the context
    ([(7, 500)], 33, 200, 40, 6, True, 1, 0),
    ([(5, 3), (2, 200), (0, 9), (3, 700)], 16, 64, 64, 3, True, 2, 1),
    ([(300, 400)], 7, 128, 64, 2, True, 1, 0),
    ([(1, 5000), (2, 3000)], 9, 128, 128, 20, True, 0, 0),
]


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("lens,H,P,block,K,causal,pad,lead", CASES)
def test_sparse_matches_float64(lens, H, P, block, K, causal, pad, lead, kv):
    c = SparseCase(lens, H, P, block, K, kv, causal, pad, seed=H + K, lead=lead)
    c.run()
    c.check()


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("kv", [BF, F8])
def test_lists_are_sets(kv, P):
    """Any order, repetitions, negative numbers, blocks past the context, empty lists, and lists whose
    blocks a token does not see yet."""
    lens = [(4, 300 * P // 16), (3, 8 * P + 2)]
    big = 1 << 30
    lists = [[3, 0, 7, 3, 3, 0], [18, 1, -5, big, -big - 1, 2], [-1] * 6, [big] * 6, [8, 8, 8, 8, 8, 8], [0, 8, 9, 10, -1, 4],
             [8, 7, 6, 5, 4, 3]]
    c = SparseCase(lens, 16, P, P, 6, kv, seed=5, selected=lists)
    c.run()
    c.check()
    assert math.isinf(c.lse[2, 0].item()) and math.isinf(c.lse[3, 0].item())
    # sequence 1 sees 8 P, 8 P + 1 and 8 P + 2 keys: its first token does not see block 8
    assert math.isinf(c.lse[4, 0].item()) and not math.isinf(c.lse[5, 0].item())
    again = SparseCase(lens, 16, P, P, 6, kv, seed=5, selected=[sorted(r, reverse=True) for r in lists])
    again.run()
    torch.cuda.synchronize()
    assert torch.equal(again.out, c.out) and torch.equal(again.lse, c.lse)


@pytest.mark.parametrize("kv", [BF, F8])
def test_all_blocks_are_chunk_attention(kv):
    lens = [(6, 500), (0, 9), (1, 333), (40, 40)]
    full = [[c for c in range(32)] for n, _ in lens for _ in range(n)]
    s = SparseCase(lens, 32, 64, 16, 32, kv, seed=6, selected=full)
    s.run()
    s.check()
    d = ChunkCase(lens, 32, 64, kv, seed=6)
    d.run()
    torch.cuda.synchronize()
    assert (s.lse - d.lse).abs().max().item() <= LSE_ABS[kv]
    assert (s.out.float() - d.out.float()).abs().max().item() <= 2.0 ** -6


def test_keys_outside_the_lists_may_hold_anything():
    for kv in (BF, F8):
        c = SparseCase([(3, 400)], 16, 32, 16, 5, kv, seed=7)
        used = set()
        for i in range(3):
            used |= set(c.keys_of(0, i))
        nan = torch.full((576,), float("nan"), dtype=torch.bfloat16) if kv == BF else torch.full((576,), 0x7F, dtype=torch.uint8)
        for j in range(400):
            if j not in used:
                c.set_key(0, j, nan)
        c.run()
        c.check()


def test_many_tokens_and_sequences():
    rng = np.random.default_rng(2)
    lens = [(int(rng.integers(0, 4)), int(rng.integers(4, 90))) for _ in range(700)]
    c = SparseCase(lens, 2, 16, 8, 4, BF, seed=8, pad=3)
    c.run()
    c.check(list(range(0, 700, 23)))


@pytest.mark.parametrize("kv,H", [(F8, 16), (BF, 16), (F8, 130)])
@pytest.mark.parametrize("n", [20, 38, 64, 76, 101, 152, 153])
def test_decode_batches_of_uneven_lengths(n, kv, H):
    """One token each: as many pieces as workers or fewer, around the sizes at which the shares change, with
    sequences without keys, short ones and one far longer than the rest."""
    rng = np.random.default_rng(n)
    lens = [(1, int(x)) for x in rng.integers(1, 2600, n)]
    lens[3], lens[n // 2], lens[n - 1], lens[7] = (1, 9000), (1, 1), (1, 64), (0, 40)
    c = SparseCase(lens, H, 64, 64, 150, kv, seed=n)
    c.run()
    c.check()


@pytest.mark.parametrize("kv,H", [(BF, 130), (F8, 130), (F8, 16)])
def test_whole_blocks_of_many_tokens(kv, H):
    """Shares of six row blocks or more are not cut; lists of all lengths, rows that see nothing among them."""
    rng = np.random.default_rng(3)
    lens = [(400, 900), (0, 30), (300, 250), (37, 37), (1500 if H == 16 else 200, 2000)]
    c = SparseCase(lens, H, 64, 64 if H == 16 else 32, 3, kv, seed=12, pad=5, lead=3)
    c.selected[::7] = -1
    c.selected[5] = torch.tensor([2, 1, 0])
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    for b, (n, _) in enumerate(lens):
        for i in sorted(set(rng.integers(0, n, 12).tolist()) | {0, n - 1}) if n else ():
            t = c.starts[b] + i
            keys = c.keys_of(b, i)
            out, lse = c.out[t].double().cpu(), c.lse[t].double().cpu()
            if not keys:
                assert (out == 0).all() and (lse == -INF).all()
                continue
            r, rl, bound = attended(c.q[t].double(), c.keys[b][keys], kv)
            assert ((out - r).abs() <= bound).all() and (lse - rl).abs().max() <= LSE_ABS[kv]
    assert (c.out[:3] == 7.0).all() and (c.out[-5:] == 7.0).all() and (c.lse[-5:] == -3.5).all()


def test_more_tokens_than_lengths_fit_shared_memory():
    lens = [(4000, 4000), (5000, 5100), (1, 70)]
    c = SparseCase(lens, 1, 16, 16, 2, BF, seed=13)
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    for b, i in ((0, 0), (0, 1), (0, 3999), (1, 0), (1, 2500), (1, 4999), (2, 0)):
        t = c.starts[b] + i
        r, rl, bound = attended(c.q[t].double(), c.keys[b][c.keys_of(b, i)], BF)
        assert ((c.out[t].double().cpu() - r).abs() <= bound).all()
        assert (c.lse[t].double().cpu() - rl).abs().max() <= LSE_ABS[BF]


@pytest.mark.parametrize("kv", [BF, F8])
def test_more_positions_than_32_bits_might_hold(kv):
    """Lists long enough that the tokens' tiles could pass 2^30, though few entries are used."""
    T, K, P = 1 << 18, 1024, 1024
    gen = torch.Generator(device="cuda").manual_seed(2)
    cache = torch.randn((3, P, 576), generator=gen, device="cuda").to(torch.bfloat16)
    scale = None
    if kv == F8:
        cache, scale = cache.to(torch.float8_e4m3fn), torch.ones(1, device="cuda")
    q = torch.randn((T, 1, 576), generator=gen, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((1, 1024), -1, **i32)
    table[0, :3] = torch.tensor([2, 0, 1], **i32)
    sel = torch.full((T, K), -1, **i32)
    sel[:, 5] = torch.arange(T, device="cuda").int() % 3
    sel[::3, 9] = 1
    out, lse = api.sparse_attention(q, cache, table, torch.tensor([3 * P], **i32), torch.tensor([0, T], **i32), sel, SCALE, scale,
                                    max_seq_len=1 << 20, block_size=P, causal=False)
    rows = cache[[2, 0, 1]].double()
    for t in (0, 1, 2, 3, 77777, T - 2, T - 1):
        k = torch.cat([rows[c] for c in sorted({t % 3} | ({1} if t % 3 == 0 else set()))])
        r, rl, bound = attended(q[t].double(), k, kv)
        assert ((out[t].double() - r).abs() <= bound).all() and (lse[t].double() - rl).abs().max() <= LSE_ABS[kv]


def test_a_long_context():
    L = (1 << 20) - 3
    pages = L // 64 + 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.empty((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    cache.normal_(generator=gen)
    q = torch.randn((2, 16, 576), generator=gen, device="cuda").to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, generator=gen, device="cuda").int()[None]
    nb = -(-L // 32)
    sel = torch.tensor([[nb - 1, 5, 70000, 0, 32766, -1], [1, 32767, nb - 1, nb - 2, 3, 20000]], **i32)
    out, lse = api.sparse_attention(q, cache, table, torch.tensor([L], **i32), torch.tensor([0, 2], **i32), sel, SCALE,
                                    max_seq_len=1 << 20, block_size=32)
    for i, n in ((0, L - 1), (1, L)):
        rows = [j for c in sorted(set(sel[i].tolist())) if 0 <= c < nb for j in range(32 * c, min(n, 32 * c + 32))]
        j = torch.tensor(rows, device="cuda")
        k = cache.view(-1, 576)[table[0].long()[j // 64] * 64 + j % 64].double()
        r, rl, bound = attended(q[i].double(), k, BF)
        assert ((out[i].double() - r).abs() <= bound).all() and (lse[i].double() - rl).abs().max() <= LSE_ABS[BF]


@pytest.mark.parametrize("kv,P", [(BF, 16), (F8, 64)])
def test_device_errors(kv, P):
    def run(**change):
        c = SparseCase([(2, 100 * P // 16), (1, 64)], 8, P, P, 7, kv, seed=4, pad=2)
        for k, v in change.items():
            if k == "page":
                c.table[0, 3] = v
            elif k == "length":
                c.seq_lens[1] = v
            elif k == "offset":
                c.cu[1] = v
        c.run()
        torch.cuda.synchronize()
        return c, api.decode_check(c.workspace)
    c, (st, bits) = run(page=1 << 20)
    assert st == -6 and bits == 0x1 and not torch.isnan(c.out[:3]).all()
    c, (st, bits) = run(length=1 << 19)
    assert st == -6 and bits & 0x2
    c, (st, bits) = run(length=-3)
    assert st == -6 and bits == 0x2 and (c.lse[2] == -INF).all() and (c.out[2] == 0).all()
    for v in (9, -1, 4):
        c, (st, bits) = run(offset=v)
        assert st == -6 and bits & 0x20
        assert (c.out == 7.0).all() and (c.lse == -3.5).all()
    c, _ = run()
    c.check()


@pytest.mark.parametrize("H,block", [(48, 32), (16, 64)])
def test_default_buffers_streams_and_two_graphs(H, block):
    c = SparseCase([(5, 300), (1, 90), (2, 700)], H, 64, block, 4, F8, seed=9)
    c.run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    kw = dict(max_seq_len=c.max_seq_len, block_size=block)
    o, l = api.sparse_attention(*c.dev, SCALE, c.dscale, **kw)
    assert torch.equal(o, out) and torch.equal(l, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, l = api.sparse_attention(*c.dev, SCALE, c.dscale, stream=s, **kw)
    s.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    graphs = []
    for _ in range(2):                                     # each with a workspace of its own
        ws = api.alloc_sparse_workspace(c.params)
        buf = (torch.zeros_like(out), torch.zeros_like(lse))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.sparse_attention(*c.dev, SCALE, c.dscale, out=buf[0], lse=buf[1], workspace=ws, **kw)
        graphs.append((g, buf, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, buf, ws in graphs:
        assert torch.equal(buf[0], out) and torch.equal(buf[1], lse) and api.decode_check(ws) == (0, 0)
    # other lists and lengths, in place, in a replayed graph
    c.dev[5][:, 0] = 1
    c.dev[3][0] = 250
    graphs[0][0].replay()
    o, l = api.sparse_attention(*c.dev, SCALE, c.dscale, **kw)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1][0], o) and torch.equal(graphs[0][1][1], l)


@pytest.mark.parametrize("kv", [BF, F8])
def test_a_stalled_pipeline_times_out_and_the_next_call_is_clean(kv):
    c = SparseCase([(2, 300)], 16, 64, 64, 3, kv, seed=10)
    api.test_set_hooks(20_000_000, True)
    try:
        c.run()
        torch.cuda.synchronize()
        assert api.decode_check(c.workspace)[0] == -5
    finally:
        api.test_set_hooks(0, False)
    c.run(workspace=c.workspace)
    c.check()


@pytest.mark.parametrize("kv", [BF, F8])
def test_no_tokens_and_no_blocks(kv):
    c = SparseCase([(0, 100), (0, 0)], 16, 64, 64, 3, kv, seed=11)
    c.run()
    torch.cuda.synchronize()
    assert api.decode_check(c.workspace) == (0, 0)
    c = SparseCase([(3, 100), (2, 0), (1, 64)], 16, 64, 64, 3, kv, seed=11, pad=1, selected=[[-1, 9, -7]] * 7)
    c.run()
    c.check()


# --------------------------------------------------------------- the operators as they are used
@pytest.mark.parametrize("kv", [BF, F8])
def test_a_serving_run(kv):
    """A prompt in two pieces beside another sequence, then decoding steps: rows and index keys are
    appended, blocks scored and selected, and attended; every step is checked against float64 on what
    the caches hold, the selection given the scores that the GPU computed."""
    rng = np.random.default_rng(21)
    H, HI, P, block, K, first, last = 16, 8, 32, 16, 6, 1, 2
    pages = 24
    table = torch.from_numpy(rng.permutation(pages)[:20].reshape(2, 10).astype(np.int32))
    kvs = torch.tensor([6.0 / 448.0])
    cache = torch.zeros(pages, P, 576, dtype=torch.bfloat16 if kv == BF else torch.uint8, device="cuda")
    icache, iscale = torch.zeros(pages, P, 128, dtype=torch.uint8, device="cuda"), torch.zeros(pages, P, device="cuda")
    a = torch.from_numpy(rng.uniform(0, 6.28, (400, 32)))
    cs = torch.cat([a.cos(), a.sin()], dim=1).float().cuda()
    lengths = [0, 0]
    i32 = dict(dtype=torch.int32, device="cuda")
    for new in ((90, 0), (70, 33), (1, 1), (1, 0), (2, 3)):
        n = sum(new)
        pos = torch.tensor([lengths[b] + i for b in (0, 1) for i in range(new[b])])
        owner = torch.tensor([b for b in (0, 1) for _ in range(new[b])])
        slots = table[owner, pos // P].long() * P + pos % P
        lengths = [lengths[b] + new[b] for b in (0, 1)]
        seq, cu = torch.tensor(lengths, **i32), torch.tensor([0, new[0], n], **i32)
        latent, rope = bf16_normal(rng, n, 512).cuda(), bf16_normal(rng, n, 64).cuda()
        q = bf16_normal(rng, n, H, 576).cuda()
        scale = kvs.cuda() if kv == F8 else None
        api.rope_cache_write(latent, rope, pos.cuda(), cs, slots.cuda(), cache, scale, q_rope=q[..., 512:].clone(), q=q)
        qi, qw = torch.empty(n, HI, 128, dtype=torch.uint8, device="cuda"), torch.empty(n, HI, device="cuda")
        api.index_cache_write(bf16_normal(rng, n, 128).cuda(), pos.cuda(), cs, slots.cuda(), icache, iscale,
                              queries=bf16_normal(rng, n, HI, 128).cuda(), weights=torch.randn(n, HI, device="cuda"), q_index=qi,
                              q_weights=qw)
        kw = dict(max_seq_len=10 * P, block_size=block)
        scores = api.index_scores(qi, qw, icache, iscale, table.cuda(), seq, cu, **kw)
        chosen = api.select_blocks(scores, seq, cu, K, block_size=block, keep_first=first, keep_last=last)
        out, lse = api.sparse_attention(q, cache, table.cuda(), seq, cu, chosen, SCALE, scale, **kw)
        torch.cuda.synchronize()
        rows = cache.cpu().view(-1, 576)
        rows = rows.double() if kv == BF else rows.view(torch.float8_e4m3fn).double() * kvs.double()
        ikeys = icache.cpu().view(-1, 128).view(torch.float8_e4m3fn).double() * iscale.cpu().view(-1, 1).double()
        for t in range(n):
            b, vis = int(owner[t]), int(pos[t]) + 1
            where = torch.arange(vis)
            where = table[b, where // P].long() * P + where % P
            s = (torch.relu(qi[t].cpu().view(torch.float8_e4m3fn).double() @ ikeys[where].T) * qw[t].cpu().double()[:, None]).sum(dim=0)
            nb = -(-vis // block)
            best = torch.tensor([s[c * block:(c + 1) * block].max() for c in range(nb)])
            assert (scores[t, :nb].cpu() - best).abs().max() <= 1e-4 * s.abs().max()
            assert (scores[t, nb:] == -INF).all()
            want = selection(scores[t].tolist(), vis, block, K, first, last)
            assert chosen[t].tolist() == want
            keys = torch.tensor([j for c in want if c >= 0 for j in range(c * block, min(vis, c * block + block))])
            k = rows[table[b, keys // P].long() * P + keys % P]
            r, rl, bound = attended(q[t].cpu().double(), k, kv)
            assert ((out[t].cpu().double() - r).abs() <= bound).all()
            assert (lse[t].cpu().double() - rl).abs().max() <= LSE_ABS[kv]
