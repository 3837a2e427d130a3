"""Workloads of the block-sparse operators: cases, inputs, plain forms and exact values.

Four operators around the paged latent cache, in the order a serving step calls them when each
query attends only to the blocks of its context that a cheap score selects:

* write — the new tokens' index keys are rotated, quantised to 8 bits with a scale for each row
  and written into a paged index cache; their index queries are rotated and quantised beside it;
* scores — each new token scores every block of its context: the largest, over the block's keys,
  of a weighted sum over the index heads of the positive parts of query times key;
* select — for each new token the blocks with the largest scores, the first and the latest blocks
  always among them;
* sparse — each new token attends over its selected blocks of the paged latent cache.

``own`` selects this package's kernels; otherwise ``run`` computes the same in elementary torch
operations in 32 bits. Batches, lengths and heads are those of this package's decode workloads
(16 or 128 heads, pages of 64 or 128 rows, contexts to 131072 tokens); 64 index heads of 128.
"""
import math
import random

import numpy
import torch

own = False

D_LATENT, D_ROPE, D_INDEX = 512, 64, 128
D_QK = D_LATENT + D_ROPE
SCALE = 1.0 / math.sqrt(192.0)
MAX_WRITE = 4096 * 64              # tokens x index heads of the largest write
MAX_SCORE_FLOPS = 1.0e12           # of the largest scoring
MAX_SELECT = 2048 * 512            # scores of the largest selection
MAX_SPARSE_FLOPS = 2.9e11          # of the largest sparse attention
MAX_CONTEXT = 400_000              # tokens in the cache of a drawn case


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's new tokens: the latency of a small write
        dict(name="write_step_t128_h64", op="write", tokens=128, heads=64, page=64, interleaved=True,
             max_pos=8192, pad=0, lens_seed=1),
        # a prefill chunk of 4096 tokens, rows padded to the chunk's size: bandwidth
        dict(name="write_chunk_t4096_h64", op="write", tokens=4096, heads=64, page=64, interleaved=False,
             max_pos=131072, pad=100, lens_seed=2),
        # one decode step of the ragged 128-sequence batch, padded to its graph's batch size
        dict(name="scores_step_b128_h64", op="scores", heads=64, page=64, block=64, causal=True, batch=120,
             new_lo=1, new_hi=1, ctx_lo=2048, ctx_hi=6144, long_new=0, long_ctx=0, pad=8, lens_seed=3),
        # four long sequences with four new tokens each, small blocks
        dict(name="scores_long_b4_h64", op="scores", heads=64, page=64, block=32, causal=True, batch=3,
             new_lo=4, new_hi=4, ctx_lo=32768, ctx_hi=100000, long_new=4, long_ctx=131000, pad=0, lens_seed=4),
        # a 2048-token piece of a long prompt over 24 K of context: arithmetic
        dict(name="scores_chunk_t2048_h64", op="scores", heads=64, page=128, block=64, causal=True, batch=0,
             new_lo=0, new_hi=0, ctx_lo=0, ctx_hi=0, long_new=2048, long_ctx=24576, pad=0, lens_seed=5),
        # one decode step of the ragged batch: up to 96 scores for each token
        dict(name="select_step_t128", op="select", tokens=128, block=64, ctx_lo=2048, ctx_hi=6144, max_len=6144,
             top_k=16, keep_first=1, keep_last=2, pad=8, lens_seed=6),
        # four long sequences with four new tokens each, blocks of 32: up to 4096 scores for each
        dict(name="select_long_t16", op="select", tokens=16, block=32, ctx_lo=32768, ctx_hi=131072, max_len=131072,
             top_k=64, keep_first=1, keep_last=4, pad=0, lens_seed=7),
        # a 2048-token prefill chunk over up to 32 K
        dict(name="select_chunk_t2048", op="select", tokens=2048, block=64, ctx_lo=24576, ctx_hi=32768, max_len=32768,
             top_k=32, keep_first=1, keep_last=1, pad=0, lens_seed=8),
        # two short requests whose context the selection covers: the latency of a small call
        dict(name="sparse_tiny_b2_h16_bf16", op="sparse", heads=16, page=64, block=64, kv="bf16", causal=True, top_k=16,
             batch=2, new_lo=1, new_hi=1, ctx_lo=99, ctx_hi=256, long_new=0, long_ctx=0, pad=0, lens_seed=9),
        # one decode step of 64 sequences, 16 heads, FP8 cache, 2048 keys for each token
        dict(name="sparse_step_b64_h16_fp8", op="sparse", heads=16, page=64, block=64, kv="fp8", causal=True, top_k=32,
             batch=64, new_lo=1, new_hi=1, ctx_lo=1500, ctx_hi=12000, long_new=0, long_ctx=0, pad=0, lens_seed=10),
        # four long sequences with four new tokens each, 128 heads, FP8 cache, small blocks
        dict(name="sparse_long_b4_h128_fp8", op="sparse", heads=128, page=64, block=32, kv="fp8", causal=True, top_k=64,
             batch=3, new_lo=4, new_hi=4, ctx_lo=32768, ctx_hi=100000, long_new=4, long_ctx=131000, pad=4, lens_seed=11),
        # a 512-token piece of a prompt over 16 K of context, 128 heads: arithmetic
        dict(name="sparse_chunk_t512_h128_bf16", op="sparse", heads=128, page=128, block=64, kv="bf16", causal=True,
             top_k=32, batch=0, new_lo=0, new_hi=0, ctx_lo=0, ctx_hi=0, long_new=512, long_ctx=16384, pad=0, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "scores", "select", "sparse", "sparse"])
    page = rng.choice([8, 16, 24, 32, 48, 64, 64, 128, 256])
    block = rng.choice([b for b in (8, 16, 24, 32, 48, 64, 128, 256) if page % b == 0])
    seed = rng.randrange(1 << 30)
    pad = rng.choice([0, 0, rng.randint(1, 31)])
    if op == "write":
        heads = rng.choice([16, 64, _log_int(rng, 1, 128)])
        return dict(op=op, tokens=min(_log_int(rng, 1, 4096), MAX_WRITE // heads), heads=heads, page=page,
                    interleaved=rng.random() < 0.5, max_pos=_log_int(rng, 64, 131072), pad=pad, lens_seed=seed)
    if op == "select":
        tokens = _log_int(rng, 1, 2048)
        blocks = min(_log_int(rng, 24, 16384), MAX_SELECT // tokens)
        max_len = blocks * block - rng.randrange(block)
        return dict(op=op, tokens=tokens, block=block, ctx_lo=max_len // rng.choice([2, 3]), ctx_hi=max_len,
                    max_len=max_len, top_k=_log_int(rng, 6, max(6, min(256, blocks // 4))), keep_first=rng.choice([0, 1, 2]),
                    keep_last=rng.choice([0, 1, 3]), pad=min(pad, tokens - 1), lens_seed=seed)
    case = dict(op=op, heads=rng.choice([16, 64, 128, _log_int(rng, 1, 128)]), page=page, block=block,
                causal=rng.random() < 0.85, batch=_log_int(rng, 1, 96) - 1, new_lo=rng.choice([0, 1]),
                new_hi=_log_int(rng, 1, 64), ctx_lo=rng.choice([0, 0, 100]), ctx_hi=_log_int(rng, 100, 16384),
                long_new=_log_int(rng, 1, 1024), long_ctx=_log_int(rng, 1, 65536) - 1, pad=pad, lens_seed=seed)
    if op == "sparse":
        case["kv"] = rng.choice(["bf16", "fp8"])
        case["top_k"] = max(2, _log_int(rng, 64, 4096) // block)
    most = MAX_SCORE_FLOPS if op == "scores" else MAX_SPARSE_FLOPS
    while work(case)["flops"] > most:
        for k in ("new_hi", "long_new"):
            case[k] = max(1, case[k] // 2)
        if case["new_hi"] == 1 and case["long_new"] == 1:
            case["batch"] //= 2
    while sum(a + c for a, c in _lens(case)) > MAX_CONTEXT:
        case["batch"] //= 2
    return case


def _lens(case):
    """[(new tokens, tokens in the cache before them)] of the sequences of a scores or sparse case."""
    rng = random.Random(case["lens_seed"])
    out = [(rng.randint(case["new_lo"], case["new_hi"]), rng.randint(case["ctx_lo"], case["ctx_hi"]))
           for _ in range(case["batch"])]
    if case["long_new"] > 0:
        out.insert(len(out) // 2, (case["long_new"], case["long_ctx"]))
    return out


def _seen(case):
    """The number of keys that each new token of a scores or sparse case sees."""
    out = []
    for new, ctx in _lens(case):
        out += [ctx + 1 + i if case["causal"] else ctx + new for i in range(new)]
    return out


def _select_lens(case):
    """The context of each token of a select case that is not padding."""
    rng = random.Random(case["lens_seed"])
    return [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["tokens"] - case["pad"])]


def _real_tokens(case):
    """Tokens of a write that are not padding."""
    return max(1, case["tokens"] - case["pad"])


def _score_columns(case):
    longest = max([a + c for a, c in _lens(case)] + [1])
    return -(-longest // case["block"])


def work(case):
    if case["op"] == "write":
        n, h = _real_tokens(case), case["heads"]
        # a key in and out with its scale, its position, slot, cosines and sines; each head's query in
        # and out, its weight in and out
        return {"bytes": n * (D_INDEX * 3 + 4 + 16 + D_ROPE * 4 + h * (D_INDEX * 3 + 8)),
                "flops": n * (h + 1) * (D_ROPE * 3 + 2 * D_INDEX)}
    if case["op"] == "select":
        blocks = [-(-n // case["block"]) for n in _select_lens(case)]
        return {"bytes": 4 * sum(blocks) + len(blocks) * 4 * (case["top_k"] + 2), "flops": 2 * sum(blocks)}
    h = case["heads"]
    if case["op"] == "scores":
        keys = sum(a + c for a, c in _lens(case) if a > 0)
        seen = _seen(case)
        return {"bytes": keys * (D_INDEX + 4) + len(seen) * (h * (D_INDEX + 4) + 4 * _score_columns(case)),
                "flops": sum(seen) * h * (2 * D_INDEX + 2)}
    attended, rows, t0, seen = 0, 0, 0, _seen(case)
    for new, ctx in _lens(case):
        mine = sum(_attended(case, n) for n in seen[t0:t0 + new])
        attended += mine
        rows += min(mine, new + ctx)
        t0 += new
    row = D_QK * (2 if case["kv"] == "bf16" else 1)
    return {"bytes": rows * row + len(seen) * (h * (D_QK * 2 + D_LATENT * 2 + 4) + 4 * case["top_k"]),
            "flops": 2 * (D_QK + D_LATENT) * h * attended}


def _attended(case, n):
    """Keys of the selected blocks (the latest among them) of a token that sees n keys."""
    blocks = -(-n // case["block"])
    return min(case["top_k"], blocks) * case["block"] - (blocks * case["block"] - n)


# ---------------------------------------------------------------------------- the inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    return {"write": _prepare_write, "scores": _prepare_scores, "select": _prepare_select,
            "sparse": _prepare_sparse}[case["op"]](case, gen, rng)


def _prepare_write(case, gen, rng):
    n, h, p = case["tokens"], case["heads"], case["page"]
    real = _real_tokens(case)
    pages = (real * 11 // 10 + p) // p + 1
    # slots of as many scattered rows of the pool; padding tokens carry -1 in both
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[:real] = torch.randperm(pages * p, generator=gen, device="cuda")[:real]
    positions = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    positions[:real] = torch.randint(0, case["max_pos"], (real,), generator=gen, device="cuda")
    # cos | sin of position x base^(-2i/64), in 64 bits and rounded once
    inv = 10000.0 ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64, device="cuda") / D_ROPE)
    angle = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return dict(op="write", keys=_normal(gen, n, D_INDEX), queries=_normal(gen, n, h, D_INDEX),
                weights=torch.randn((n, h), generator=gen, device="cuda") * h ** -0.5 * D_INDEX ** -0.5,
                slots=slots, positions=positions, real=real, interleaved=case["interleaved"],
                cos_sin=torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous(),
                index_cache=torch.zeros((pages, p, D_INDEX), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                index_scale=torch.zeros((pages, p), dtype=torch.float32, device="cuda"),
                q_index=torch.zeros((n, h, D_INDEX), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                q_weights=torch.zeros((n, h), dtype=torch.float32, device="cuda"))


def _paged(case, rng):
    """Lengths, block table and row offsets of a ragged batch over a shuffled pool of pages."""
    lens = _lens(case)
    p = case["page"]
    new = [a for a, _ in lens]
    total = [a + c for a, c in lens]
    need = [-(-t // p) for t in total]
    pages = max(1, sum(need) * 11 // 10 + 1)
    perm = list(range(pages))
    rng.shuffle(perm)
    width = max([1] + need)
    table, at = [], 0
    for k in need:
        table.append(perm[at:at + k] + [0] * (width - k))
        at += k
    starts = [0]
    for a in new:
        starts.append(starts[-1] + a)
    rows = max(1, starts[-1] + case["pad"])
    return pages, rows, dict(new=new, total=total, block_table=_int32(table or [[0]]), seq_lens=_int32(total or [0]),
                             starts=_int32(starts if lens else [0, 0]), max_seq_len=max([1] + total),
                             block=case["block"], causal=case["causal"])


def _row_quantised(x):
    """E4M3 codes of the last dimension and their float32 scales."""
    x = x.float()
    scale = x.abs().amax(dim=-1) / 448.0
    return (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _prepare_scores(case, gen, rng):
    h = case["heads"]
    pages, rows, st = _paged(case, rng)
    st["q_index"], q_scale = _row_quantised(_normal(gen, rows, h, D_INDEX))
    st["q_weights"] = torch.randn((rows, h), generator=gen, device="cuda") * h ** -0.5 * D_INDEX ** -0.5 * q_scale
    st["index_cache"], st["index_scale"] = _row_quantised(_normal(gen, pages, case["page"], D_INDEX))
    # rows behind the last sequence are left as they are
    st["out"] = torch.zeros((rows, _score_columns(case)), dtype=torch.float32, device="cuda")
    return dict(st, op="scores")


def _prepare_select(case, gen, rng):
    lens = _select_lens(case)
    n, columns = case["tokens"], -(-case["max_len"] // case["block"])
    # each token ends a sequence of its own; blocks past its context score minus infinity
    scores = torch.randn((n, columns), generator=gen, device="cuda")
    blocks = _int32([-(-m // case["block"]) for m in lens] + [0] * (n - len(lens)))
    scores.masked_fill_(torch.arange(columns, device="cuda")[None, :] >= blocks[:, None], float("-inf"))
    return dict(op="select", scores=scores, seq_lens=_int32(lens), starts=_int32(list(range(len(lens) + 1))), lens=lens,
                block=case["block"], top_k=case["top_k"], keep_first=case["keep_first"], keep_last=case["keep_last"],
                out=torch.full((n, case["top_k"]), -1, dtype=torch.int32, device="cuda"))


def _prepare_sparse(case, gen, rng):
    h, k, block = case["heads"], case["top_k"], case["block"]
    pages, rows, st = _paged(case, rng)
    st["q"] = _normal(gen, rows, h, D_QK)
    kv = _normal(gen, pages, case["page"], D_QK)
    st["kv_scale"] = None
    if case["kv"] == "fp8":
        st["kv_scale"] = (kv.abs().max().float() / 448.0).reshape(1)
        kv = (kv.float() / st["kv_scale"]).to(torch.float8_e4m3fn)
    st["cache"] = kv
    # a random choice for each token, its first and its latest block among it, ascending, -1 behind
    seen = torch.tensor(_seen(case), dtype=torch.int64, device="cuda")
    blocks = (seen + block - 1) // block
    columns = torch.arange(max(k, -(-st["max_seq_len"] // block)), device="cuda")
    st["selected"] = torch.full((rows, k), -1, dtype=torch.int32, device="cuda")
    for i in range(0, len(seen), 256):
        nb = blocks[i:i + 256, None]
        taste = torch.rand((len(nb), len(columns)), generator=gen, device="cuda")
        taste = torch.where((columns == 0) | (columns == nb - 1), taste + 2.0, taste)
        taste = torch.where(columns < nb, taste, -1.0)
        best, at = taste.topk(k, dim=1)
        at = torch.where(best >= 0, at, len(columns)).sort(dim=1).values
        st["selected"][i:i + len(nb)] = torch.where(at < len(columns), at, -1).int()
    # rows behind the last sequence are left as they are
    st["out"] = torch.zeros((rows, h, D_LATENT), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros((rows, h), dtype=torch.float32, device="cuda")
    if own:
        from mla_paged_decode_02_gb300 import api
        kvd = api.KV_BF16 if st["kv_scale"] is None else api.KV_FP8_E4M3
        params = api.make_sparse_params(len(st["seq_lens"]), rows, h, case["page"], pages, st["block_table"].shape[1],
                                        st["max_seq_len"], block, k, kvd, st["causal"])
        st["workspace"] = api.alloc_sparse_workspace(params, "cuda")
    return dict(st, op="sparse")


# ------------------------------------------------------------------------------- the runs
def run(st):
    if own:
        return {"write": _own_write, "scores": _own_scores, "select": _own_select, "sparse": _own_sparse}[st["op"]](st)
    return {"write": _plain_write, "scores": _plain_scores, "select": _plain_select, "sparse": _plain_sparse}[st["op"]](st)


def _own_write(st):
    from mla_paged_decode_02_gb300 import api
    api.index_cache_write(st["keys"], st["positions"], st["cos_sin"], st["slots"], st["index_cache"], st["index_scale"],
                          queries=st["queries"], weights=st["weights"], q_index=st["q_index"],
                          q_weights=st["q_weights"], interleaved=st["interleaved"])
    return st["index_cache"], st["index_scale"], st["q_index"], st["q_weights"]


def _own_scores(st):
    from mla_paged_decode_02_gb300 import api
    return api.index_scores(st["q_index"], st["q_weights"], st["index_cache"], st["index_scale"], st["block_table"],
                            st["seq_lens"], st["starts"], max_seq_len=st["max_seq_len"], block_size=st["block"],
                            causal=st["causal"], out=st["out"])


def _own_select(st):
    from mla_paged_decode_02_gb300 import api
    return api.select_blocks(st["scores"], st["seq_lens"], st["starts"], st["top_k"], block_size=st["block"],
                             keep_first=st["keep_first"], keep_last=st["keep_last"], out=st["out"])


def _own_sparse(st):
    from mla_paged_decode_02_gb300 import api
    return api.sparse_attention(st["q"], st["cache"], st["block_table"], st["seq_lens"], st["starts"], st["selected"],
                                SCALE, st["kv_scale"], max_seq_len=st["max_seq_len"], block_size=st["block"],
                                causal=st["causal"], out=st["out"], lse=st["lse"], workspace=st["workspace"])


def _rotated(x, cos, sin, interleaved):
    """x [..., 128] in 32 bits, its last 64 values turned; pairs are neighbours, or a half apart."""
    x = x.float()
    keep, x = x[..., : D_INDEX - D_ROPE], x[..., D_INDEX - D_ROPE:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.cat([keep, torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)], dim=-1)
    a, b = x[..., : D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat([keep, a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_write(st):
    real = st["real"]
    cs = st["cos_sin"][st["positions"][:real]]
    cos, sin = cs[:, : D_ROPE // 2], cs[:, D_ROPE // 2:]
    code, scale = _row_quantised(_rotated(st["keys"][:real], cos, sin, st["interleaved"]))
    st["index_cache"].view(torch.uint8).view(-1, D_INDEX)[st["slots"][:real]] = code.view(torch.uint8)
    st["index_scale"].view(-1)[st["slots"][:real]] = scale
    code, scale = _row_quantised(_rotated(st["queries"][:real], cos[:, None], sin[:, None], st["interleaved"]))
    st["q_index"][:real] = code
    st["q_weights"][:real] = st["weights"][:real] * scale
    return st["index_cache"], st["index_scale"], st["q_index"], st["q_weights"]


def _sequence_pages(st, cache, b, length):
    """The pages of `cache` that hold the first `length` tokens of sequence b."""
    return cache[st["block_table"][b, : -(-length // cache.shape[1])].long()]


def _plain_scores(st):
    out, block = st["out"], st["block"]
    h = st["q_index"].shape[1]
    t0 = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        if new == 0:
            continue
        codes = _sequence_pages(st, st["index_cache"].view(torch.uint8), b, total).reshape(-1, D_INDEX)[:total]
        keys = codes.view(torch.float8_e4m3fn).float()
        key_scale = _sequence_pages(st, st["index_scale"], b, total).reshape(-1)[:total]
        blocks = -(-total // block)
        step = max(1, (1 << 29) // (h * total))
        for i in range(0, new, step):
            n = min(step, new - i)
            q = st["q_index"][t0 + i:t0 + i + n].float()
            s = (q.reshape(n * h, D_INDEX) @ keys.T).clamp_(min=0.0).view(n, h, total)
            s = (s.mul_(st["q_weights"][t0 + i:t0 + i + n, :, None])).sum(dim=1) * key_scale
            if st["causal"]:
                seen = torch.arange(total, device="cuda")[None, :] < (total - new + 1 + i + torch.arange(n, device="cuda"))[:, None]
                s.masked_fill_(~seen, float("-inf"))
            full = torch.full((n, blocks * block), float("-inf"), device="cuda")
            full[:, :total] = s
            out[t0 + i:t0 + i + n, :blocks] = full.view(n, blocks, block).amax(dim=-1)
        out[t0:t0 + new, blocks:] = float("-inf")
        t0 += new
    return out


def _plain_select(st):
    n, columns = len(st["lens"]), st["scores"].shape[1]
    at = torch.arange(columns, device="cuda")[None, :]
    blocks = ((st["seq_lens"] + st["block"] - 1) // st["block"])[:, None]
    inside = at < blocks
    kept = inside & ((at < st["keep_first"]) | (at >= blocks - st["keep_last"]))
    # kept blocks first, then by descending score, then by ascending index (the sorts are stable)
    order = st["scores"][:n].masked_fill(~inside, float("-inf")).sort(dim=1, descending=True, stable=True).indices
    rank = (~kept).int() + (~inside).int()
    order = order.gather(1, rank.gather(1, order).sort(dim=1, stable=True).indices)[:, : st["top_k"]]
    order = torch.where(inside.gather(1, order), order, columns).sort(dim=1).values
    st["out"][:n, : order.shape[1]] = torch.where(order < columns, order, -1).int()
    st["out"][:n, order.shape[1]:] = -1
    return st["out"]


def _plain_sparse(st):
    q, out, lse, block = st["q"], st["out"], st["lse"], st["block"]
    h, k = q.shape[1], st["selected"].shape[1]
    inside = torch.arange(block, device="cuda")
    t0 = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        if new == 0:
            continue
        page = st["cache"].shape[1]
        step = max(1, (1 << 28) // (k * block * (D_QK + 2 * h)))
        for i in range(0, new, step):
            n = min(step, new - i)
            rows = slice(t0 + i, t0 + i + n)
            chosen = st["selected"][rows].long()
            where = (chosen[:, :, None] * block + inside).view(n, k * block)
            sees = (total - new + 1 + i + torch.arange(n, device="cuda"))[:, None] if st["causal"] else total
            seen = (where >= 0) & (where < sees)
            where = where.clamp(0, total - 1)
            where = st["block_table"][b].long()[where // page] * page + where % page
            if st["kv_scale"] is None:
                keys = st["cache"].view(-1, D_QK)[where].float()
            else:
                codes = st["cache"].view(torch.uint8).view(-1, D_QK)[where]
                keys = codes.view(torch.float8_e4m3fn).float() * st["kv_scale"]
            s = (q[rows].float() @ keys.transpose(1, 2)).mul_(SCALE)
            s.masked_fill_(~seen[:, None, :], float("-inf"))
            m = s.amax(dim=-1, keepdim=True)
            w = (s - m).exp_()
            z = w.sum(dim=-1, keepdim=True)
            out[rows] = ((w @ keys[:, :, :D_LATENT]) / z).to(torch.bfloat16)
            lse[rows] = (m + z.log())[..., 0]
        t0 += new
    return out, lse


# --------------------------------------------------------------------------- exact values
def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return {"write": _exact_write, "scores": _exact_scores, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](st)


def _exact_write(st):
    # each pair is a complex number times exp(i angle)
    real = st["real"]
    half = D_ROPE // 2
    table = st["cos_sin"].double()[st["positions"][:real]]
    turn = torch.complex(table[:, :half].contiguous(), table[:, half:].contiguous())

    def rotate(x, turn):
        x = x.double()
        tail = x[..., D_INDEX - D_ROPE:]
        if st["interleaved"]:
            z = torch.view_as_complex(tail.reshape(*tail.shape[:-1], half, 2).contiguous()) * turn
            tail = torch.view_as_real(z).reshape(tail.shape)
        else:
            z = torch.complex(tail[..., :half].contiguous(), tail[..., half:].contiguous()) * turn
            tail = torch.cat([z.real, z.imag], dim=-1)
        return torch.cat([x[..., : D_INDEX - D_ROPE], tail], dim=-1)

    key = rotate(st["keys"][:real], turn)
    scale = key.abs().max(dim=-1).values / 448
    cache = torch.zeros(st["index_cache"].shape, dtype=torch.float64, device="cuda")
    cache.view(-1, D_INDEX).index_copy_(0, st["slots"][:real], key / scale[:, None])
    scales = torch.zeros(st["index_scale"].shape, dtype=torch.float64, device="cuda")
    scales.view(-1).index_copy_(0, st["slots"][:real], scale)
    query = rotate(st["queries"][:real], turn[:, None, :])
    scale = query.abs().max(dim=-1).values / 448
    q_index = torch.zeros(st["q_index"].shape, dtype=torch.float64, device="cuda")
    q_index[:real] = query / scale[..., None]
    q_weights = torch.zeros(st["q_weights"].shape, dtype=torch.float64, device="cuda")
    q_weights[:real] = st["weights"][:real].double() * scale
    return cache, scales, q_index, q_weights


def _exact_scores(st):
    out = st["out"].double()
    h, p, block = st["q_index"].shape[1], st["index_cache"].shape[1], st["block"]
    flat = st["index_cache"].view(torch.uint8).view(-1, D_INDEX)
    at = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        if new == 0:
            continue
        where = torch.arange(total, device="cuda")
        owner = where // block
        where = st["block_table"][b].long()[where // p] * p + where % p
        k = flat[where].view(torch.float8_e4m3fn).double() * st["index_scale"].view(-1)[where].double()[:, None]
        chunk = max(1, (1 << 26) // (h * total))
        for lo in range(at, at + new, chunk):
            hi = min(at + new, lo + chunk)
            dots = torch.einsum("thd,kd->tkh", st["q_index"][lo:hi].double(), k)
            score = torch.einsum("tkh,th->tk", torch.relu(dots), st["q_weights"][lo:hi].double())
            last = total - new + torch.arange(lo - at, hi - at, device="cuda") if st["causal"] else torch.full((hi - lo,), total - 1, device="cuda")
            score = torch.where(torch.arange(total, device="cuda") <= last[:, None], score,
                                torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            best = torch.full((hi - lo, out.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
            out[lo:hi] = best.scatter_reduce(1, owner.expand(hi - lo, -1), score, "amax")
        at += new
    return out


def _exact_select(st):
    out = st["out"].cpu().numpy().copy()
    scores = st["scores"].double().cpu().numpy()
    for t, n in enumerate(st["lens"]):
        blocks = -(-n // st["block"])
        index = numpy.arange(blocks)
        kept = (index < st["keep_first"]) | (index >= blocks - st["keep_last"])
        chosen = numpy.sort(numpy.lexsort((index, -scores[t, :blocks], ~kept))[: st["top_k"]])
        out[t] = -1
        out[t, : len(chosen)] = chosen
    return torch.from_numpy(out).cuda()


def _exact_sparse(st):
    h = st["q"].shape[1]
    out, lse = st["out"].double(), st["lse"].double()
    p, block = st["cache"].shape[1], st["block"]
    selected = st["selected"].cpu().tolist()
    t = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        table = st["block_table"][b].long()
        for i in range(new):
            last = total - new + 1 + i if st["causal"] else total
            spans = [torch.arange(j * block, min((j + 1) * block, last), device="cuda") for j in selected[t] if j >= 0]
            where = torch.cat(spans)
            where = table[where // p] * p + where % p
            if st["kv_scale"] is None:
                k = st["cache"].view(-1, D_QK)[where].double()
            else:
                k = st["cache"].view(torch.uint8).view(-1, D_QK)[where].view(torch.float8_e4m3fn).double()
                k = k * st["kv_scale"].double()
            score = torch.einsum("hd,kd->hk", st["q"][t].double(), k) * SCALE
            norm = torch.logsumexp(score, dim=-1)
            out[t] = torch.einsum("hk,kd->hd", torch.exp(score - norm[:, None]), k[:, :D_LATENT])
            lse[t] = norm
            t += 1
    return out, lse
