"""Workloads of the chunked-prefill operators: cases, inputs, plain forms and exact values.

Three operators around the paged latent cache, in the order a serving step calls them:

* append — new tokens' rows go into the paged cache with the position rotation applied on the
  way, and the rotated rope part of their queries goes next to the absorbed part;
* chunk — a ragged batch of new tokens (whole prompts, pieces of prompts, single tokens)
  attends over the paged cache, causal within the new tokens or over a shared prefix;
* merge — two attention results over disjoint keys (a shared prefix and the rest) are joined
  by their log-sum-exps.

``own`` selects this package's kernels; otherwise ``run`` computes the same in elementary
torch operations in 32 bits. Shapes are those of this package's decode workloads: 576-wide
cache rows (512 latent, 64 rope), 16 or 128 heads, pages of 64 or 128 rows.
"""
import math
import random

import torch

own = False

D_LATENT, D_ROPE = 512, 64
D_QK = D_LATENT + D_ROPE
SCALE = 1.0 / math.sqrt(192.0)
MAX_APPEND = 4096 * 128            # tokens x heads of the largest append
MAX_CHUNK_FLOPS = 2.2e12           # of the largest chunk attention
MAX_MERGE_ROWS = 2048 * 128        # rows of the largest merge


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step's new tokens, 16 heads, FP8 cache: the latency of a small append
        dict(name="append_step_t128_h16_fp8", op="append", tokens=128, heads=16, page=64, kv="fp8",
             interleaved=True, max_pos=8192, pad=0, lens_seed=1),
        # one decode step of a full 512-sequence batch with 128 heads, padded to the batch size
        # its graph was captured for
        dict(name="append_step_t512_h128_bf16", op="append", tokens=512, heads=128, page=128, kv="bf16",
             interleaved=True, max_pos=4096, pad=24, lens_seed=2),
        # a prefill chunk of 4096 tokens with 128 heads: bandwidth
        dict(name="append_chunk_t4096_h128_fp8", op="append", tokens=4096, heads=128, page=64, kv="fp8",
             interleaved=False, max_pos=131072, pad=0, lens_seed=3),
        # two short requests: the latency of a small call
        dict(name="chunk_tiny_b2_h16_bf16", op="chunk", heads=16, page=64, kv="bf16", causal=True, batch=2,
             new_lo=1, new_hi=17, ctx_lo=100, ctx_hi=257, long_new=0, long_ctx=0, pad=0, lens_seed=4),
        # a mixed serving step: 64 sequences decode one token each beside a 448-token piece of a
        # prompt, rows padded to a multiple of 64 tokens
        dict(name="chunk_mixed_b65_h16_fp8", op="chunk", heads=16, page=64, kv="fp8", causal=True, batch=64,
             new_lo=1, new_hi=1, ctx_lo=2048, ctx_hi=6144, long_new=448, long_ctx=4096, pad=64, lens_seed=5),
        # whole prompts from an empty cache, 16 heads, ragged lengths
        dict(name="chunk_prompts_b8_h16_bf16", op="chunk", heads=16, page=64, kv="bf16", causal=True, batch=8,
             new_lo=150, new_hi=2000, ctx_lo=0, ctx_hi=0, long_new=0, long_ctx=0, pad=0, lens_seed=6),
        # a 512-token piece of a long prompt over 8 K of context, 128 heads
        dict(name="chunk_t512_h128_bf16", op="chunk", heads=128, page=128, kv="bf16", causal=True, batch=0,
             new_lo=0, new_hi=0, ctx_lo=0, ctx_hi=0, long_new=512, long_ctx=8192, pad=0, lens_seed=7),
        # two 128-token pieces and two idle sequences over 20 to 32 K of context, 128 heads, FP8
        dict(name="chunk_long_h128_fp8", op="chunk", heads=128, page=64, kv="fp8", causal=True, batch=3,
             new_lo=0, new_hi=128, ctx_lo=20000, ctx_hi=32768, long_new=128, long_ctx=32768, pad=0, lens_seed=8),
        # one token of each of 128 requests over their shared 16 K prefix (one sequence, no mask)
        dict(name="chunk_prefix_t128_h16_bf16", op="chunk", heads=16, page=64, kv="bf16", causal=False, batch=0,
             new_lo=0, new_hi=0, ctx_lo=0, ctx_hi=0, long_new=128, long_ctx=16256, pad=0, lens_seed=9),
        # shared-prefix decode of the ragged 16-head batch: the smallest merge
        dict(name="merge_t128_h16", op="merge", tokens=128, heads=16, empty=16, lens_seed=10),
        # shared-prefix decode of a 512-sequence batch with 128 heads
        dict(name="merge_t512_h128", op="merge", tokens=512, heads=128, empty=0, lens_seed=11),
        # a prefill chunk of 2048 tokens attended in two pieces of context
        dict(name="merge_t2048_h128", op="merge", tokens=2048, heads=128, empty=64, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "merge"])
    heads = rng.choice([16, 128, _log_int(rng, 1, 128), _log_int(rng, 1, 128)])
    page = rng.choice([8, 16, 24, 32, 48, 64, 64, 128, 256])
    kv = rng.choice(["bf16", "fp8"])
    seed = rng.randrange(1 << 30)
    if op == "append":
        tokens = min(_log_int(rng, 1, 4096), MAX_APPEND // heads)
        return dict(op=op, tokens=tokens, heads=heads, page=page, kv=kv, interleaved=rng.random() < 0.5,
                    max_pos=_log_int(rng, 64, 131072), pad=rng.choice([0, 0, rng.randint(1, 31)]), lens_seed=seed)
    if op == "merge":
        tokens = min(_log_int(rng, 1, 4096), MAX_MERGE_ROWS // heads)
        return dict(op=op, tokens=tokens, heads=heads, empty=rng.choice([0, 2, 16, 64]), lens_seed=seed)
    case = dict(op=op, heads=heads, page=page, kv=kv, causal=rng.random() < 0.75, batch=_log_int(rng, 1, 96) - 1,
                new_lo=rng.choice([0, 1]), new_hi=_log_int(rng, 1, 256), ctx_lo=rng.choice([0, 0, 100]),
                ctx_hi=_log_int(rng, 100, 16384), long_new=_log_int(rng, 1, 2048), long_ctx=_log_int(rng, 1, 32768) - 1,
                pad=rng.choice([0, 0, rng.randint(1, 63)]), lens_seed=seed)
    while work(case)["flops"] > MAX_CHUNK_FLOPS:
        for k in ("new_hi", "long_new"):
            case[k] = max(1, case[k] // 2)
        if case["new_hi"] == 1 and case["long_new"] == 1:
            case["batch"] //= 2
    return case


def _lens(case):
    """[(new tokens, tokens in the cache before them)] of the sequences of a chunk case."""
    rng = random.Random(case["lens_seed"])
    out = [(rng.randint(case["new_lo"], case["new_hi"]), rng.randint(case["ctx_lo"], case["ctx_hi"]))
           for _ in range(case["batch"])]
    if case["long_new"] > 0:
        out.insert(len(out) // 2, (case["long_new"], case["long_ctx"]))
    return out


def _real_tokens(case):
    """Tokens of an append that are not padding."""
    return max(1, case["tokens"] - case["pad"])


def work(case):
    h = case["heads"]
    if case["op"] == "append":
        n = _real_tokens(case)
        row = D_QK * (2 if case["kv"] == "bf16" else 1)
        # a token's row in and out, its position, slot and cosines and sines, its queries' rope part in and out
        return {"bytes": n * (D_QK * 2 + row + 8 + 8 + D_ROPE * 4 + 2 * h * D_ROPE * 2), "flops": n * (h + 1) * 96 * 2}
    if case["op"] == "merge":
        rows = case["tokens"] * h
        return {"bytes": rows * (3 * D_LATENT * 2 + 3 * 4), "flops": rows * D_LATENT * 3}
    byts, flops = 0, 0
    for new, ctx in _lens(case):
        if new == 0:
            continue
        total = new + ctx
        pairs = new * ctx + new * (new + 1) // 2 if case["causal"] else new * total
        flops += 2 * (D_QK + D_LATENT) * h * pairs
        byts += total * D_QK * (2 if case["kv"] == "bf16" else 1) + new * h * (D_QK * 2 + D_LATENT * 2 + 4)
    return {"bytes": byts, "flops": flops}


# ---------------------------------------------------------------------------- the inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _quantised(x, scale):
    return (x.float() / scale).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    return {"append": _prepare_append, "chunk": _prepare_chunk, "merge": _prepare_merge}[case["op"]](case, gen, rng)


def _prepare_append(case, gen, rng):
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
    cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    # the key-value projection's output, latent beside rope, and the query projection's, whose
    # last 64 columns of each head rotate; q's first 512 columns hold the absorbed queries
    kv_proj = _normal(gen, n, D_QK)
    q_proj = _normal(gen, n, h, 128 + D_ROPE)
    q = torch.zeros((n, h, D_QK), dtype=torch.bfloat16, device="cuda")
    if case["kv"] == "fp8":
        kv_scale = torch.full((1,), 6.0 / 448.0, dtype=torch.float32, device="cuda")
        cache = torch.zeros((pages, p, D_QK), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    else:
        kv_scale = None
        cache = torch.zeros((pages, p, D_QK), dtype=torch.bfloat16, device="cuda")
    return dict(op="append", kv_proj=kv_proj, q_proj=q_proj, q=q, cache=cache, kv_scale=kv_scale, slots=slots,
                positions=positions, cos_sin=cos_sin, interleaved=case["interleaved"], real=real)


def _prepare_chunk(case, gen, rng):
    lens = _lens(case)
    h, p = case["heads"], case["page"]
    new = [a for a, _ in lens]
    total = [a + c for a, c in lens]
    need = [-(-t // p) for t in total]
    pages = max(1, sum(need) * 11 // 10 + 1)
    perm = list(range(pages))
    rng.shuffle(perm)
    mb = max(1, max(need, default=1))
    table, at = [], 0
    for k in need:
        table.append(perm[at:at + k] + [0] * (mb - k))
        at += k
    starts = [0]
    for a in new:
        starts.append(starts[-1] + a)
    rows = starts[-1] + case["pad"]
    q = _normal(gen, max(1, rows), h, D_QK)
    kv = _normal(gen, pages, p, D_QK)
    kv_scale = None
    if case["kv"] == "fp8":
        kv_scale = (kv.abs().max().float() / 448.0).reshape(1)
        kv = _quantised(kv, kv_scale)
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(op="chunk", q=q, cache=kv, kv_scale=kv_scale, new=new, total=total, causal=case["causal"],
              block_table=torch.tensor(table or [[0]], **i32), seq_lens=torch.tensor(total or [0], **i32),
              starts=torch.tensor(starts if lens else [0, 0], **i32), max_seq_len=max(1, max(total, default=1)),
              # rows behind the last sequence are left as they are
              out=torch.zeros((q.shape[0], h, D_LATENT), dtype=torch.bfloat16, device="cuda"),
              lse=torch.zeros((q.shape[0], h), dtype=torch.float32, device="cuda"))
    if own:
        from mla_paged_decode_02_gb300 import api
        kvd = api.KV_BF16 if kv_scale is None else api.KV_FP8_E4M3
        params = api.make_chunk_params(len(st["seq_lens"]), q.shape[0], h, p, pages, st["block_table"].shape[1],
                                       st["max_seq_len"], kvd, st["causal"])
        st["workspace"] = api.alloc_chunk_workspace(params, "cuda")
    return st


def _prepare_merge(case, gen, rng):
    n, h = case["tokens"], case["heads"]
    st = dict(op="merge")
    for k in ("a", "b"):
        st["out_" + k] = _normal(gen, n, h, D_LATENT)
        st["lse_" + k] = 8.0 + 2.0 * torch.randn((n, h), generator=gen, device="cuda")
    if case["empty"]:
        # requests without a prefix: nothing attended, a log-sum-exp of minus infinity
        none = torch.randperm(n, generator=gen, device="cuda")[: -(-n // case["empty"])]
        st["out_a"][none] = 0
        st["lse_a"][none] = float("-inf")
    st["out"] = torch.empty_like(st["out_a"])
    st["lse"] = torch.empty_like(st["lse_a"])
    return st


# ------------------------------------------------------------------------------- the runs
def run(st):
    if own:
        return {"append": _own_append, "chunk": _own_chunk, "merge": _own_merge}[st["op"]](st)
    return {"append": _plain_append, "chunk": _plain_chunk, "merge": _plain_merge}[st["op"]](st)


def _own_append(st):
    from mla_paged_decode_02_gb300 import api
    api.rope_cache_write(st["kv_proj"][:, :D_LATENT], st["kv_proj"][:, D_LATENT:], st["positions"], st["cos_sin"],
                         st["slots"], st["cache"], st["kv_scale"], q_rope=st["q_proj"][:, :, 128:], q=st["q"],
                         interleaved=st["interleaved"])
    return st["cache"], st["q"]


def _own_chunk(st):
    from mla_paged_decode_02_gb300 import api
    return api.chunk_attention(st["q"], st["cache"], st["block_table"], st["seq_lens"], st["starts"], SCALE,
                               st["kv_scale"], max_seq_len=st["max_seq_len"], causal=st["causal"], out=st["out"],
                               lse=st["lse"], workspace=st["workspace"])


def _own_merge(st):
    from mla_paged_decode_02_gb300 import api
    return api.merge_states(st["out_a"], st["lse_a"], st["out_b"], st["lse_b"], out=st["out"], lse=st["lse"])


def _rotated(x, cos, sin, interleaved):
    """x [..., 64] in 32 bits; pairs are neighbours, or a half apart."""
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., : D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_append(st):
    real = st["real"]
    cs = st["cos_sin"][st["positions"][:real]]
    cos, sin = cs[:, : D_ROPE // 2], cs[:, D_ROPE // 2:]
    kv = st["kv_proj"][:real]
    row = torch.cat([kv[:, :D_LATENT].float(), _rotated(kv[:, D_LATENT:], cos, sin, st["interleaved"])], dim=1)
    cache = st["cache"]
    if st["kv_scale"] is None:
        cache.view(-1, D_QK)[st["slots"][:real]] = row.to(torch.bfloat16)
    else:
        code = (row / st["kv_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        cache.view(torch.uint8).view(-1, D_QK)[st["slots"][:real]] = code.view(torch.uint8)
    st["q"][:real, :, D_LATENT:] = _rotated(st["q_proj"][:real, :, 128:], cos[:, None], sin[:, None],
                                            st["interleaved"]).to(torch.bfloat16)
    return cache, st["q"]


def _sequence_rows(st, b, length):
    """The first `length` cache rows of sequence b, in 32 bits."""
    cache = st["cache"]
    p = cache.shape[1]
    pages = st["block_table"][b, : -(-length // p)].long()
    if st["kv_scale"] is None:
        return cache[pages].reshape(-1, D_QK)[:length].float()
    codes = cache.view(torch.uint8)[pages].reshape(-1, D_QK)[:length]
    return codes.view(torch.float8_e4m3fn).float() * st["kv_scale"]


def _plain_chunk(st):
    q, out, lse = st["q"], st["out"], st["lse"]
    h = q.shape[1]
    t0 = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        if new == 0:
            continue
        keys = _sequence_rows(st, b, total)
        step = max(1, (1 << 28) // max(1, h * total))
        for i in range(0, new, step):
            n = min(step, new - i)
            s = (q[t0 + i:t0 + i + n].float().reshape(n * h, D_QK) @ keys.T).mul_(SCALE).view(n, h, total)
            if st["causal"]:
                seen = torch.arange(total, device="cuda")[None, :] < (total - new + 1 + i + torch.arange(n, device="cuda"))[:, None]
                s.masked_fill_(~seen[:, None, :], float("-inf"))
            m = s.amax(dim=-1, keepdim=True)
            w = (s - m).exp_()
            z = w.sum(dim=-1, keepdim=True)
            o = (w.view(n * h, total) @ keys[:, :D_LATENT]).view(n, h, D_LATENT) / z
            out[t0 + i:t0 + i + n] = o.to(torch.bfloat16)
            lse[t0 + i:t0 + i + n] = (m + z.log())[..., 0]
        t0 += new
    return out, lse


def _plain_merge(st):
    la, lb = st["lse_a"], st["lse_b"]
    m = torch.maximum(la, lb)
    wa, wb = (la - m).exp(), (lb - m).exp()
    z = wa + wb
    o = (wa / z)[..., None] * st["out_a"].float() + (wb / z)[..., None] * st["out_b"].float()
    st["out"].copy_(o.to(torch.bfloat16))
    st["lse"].copy_(m + z.log())
    return st["out"], st["lse"]


# --------------------------------------------------------------------------- exact values
def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "chunk": _exact_chunk, "merge": _exact_merge}[case["op"]](st)


def _exact_append(st):
    # each pair is a complex number times exp(i angle)
    real = st["real"]
    half = D_ROPE // 2
    table = st["cos_sin"].double()[st["positions"][:real]]
    turn = torch.complex(table[:, :half].contiguous(), table[:, half:].contiguous())

    def rotate(x, turn):
        x = x.double()
        if st["interleaved"]:
            z = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) * turn
            return torch.view_as_real(z).reshape(x.shape)
        z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag], dim=-1)

    rows = st["kv_proj"][:real].double()
    rows[:, D_LATENT:] = rotate(st["kv_proj"][:real, D_LATENT:], turn)
    if st["kv_scale"] is not None:
        rows = (rows / st["kv_scale"].double()).clamp(-448.0, 448.0)
    cache = torch.zeros(st["cache"].shape, dtype=torch.float64, device="cuda")
    cache.view(-1, D_QK).index_copy_(0, st["slots"][:real], rows)
    q = st["q"].double()
    q[:real, :, D_LATENT:] = rotate(st["q_proj"][:real, :, 128:], turn[:, None, :])
    return cache, q


def _exact_chunk(st):
    h = st["q"].shape[1]
    out, lse = st["out"].double(), st["lse"].double()
    p = st["cache"].shape[1]
    at = 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        if new == 0:
            continue
        where = torch.arange(total, device="cuda")
        where = st["block_table"][b].long()[where // p] * p + where % p
        flat = st["cache"].view(-1, D_QK)
        if st["kv_scale"] is None:
            k = flat[where].double()
        else:
            k = flat.view(torch.uint8)[where].view(torch.float8_e4m3fn).float().double() * st["kv_scale"].double()
        block = max(1, (1 << 26) // (h * total))
        for lo in range(0, new, block):
            hi = min(new, lo + block)
            score = torch.einsum("thd,kd->thk", st["q"][at + lo:at + hi].double(), k) * SCALE
            if st["causal"]:
                last = torch.arange(total - new + lo, total - new + hi, device="cuda")
                score = torch.where(torch.arange(total, device="cuda") <= last[:, None, None], score,
                                    torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            norm = torch.logsumexp(score, dim=-1)
            out[at + lo:at + hi] = torch.einsum("thk,kd->thd", torch.exp(score - norm[..., None]), k[:, :D_LATENT])
            lse[at + lo:at + hi] = norm
        at += new
    return out, lse


def _exact_merge(st):
    both = torch.stack([st["lse_a"], st["lse_b"]]).double()
    norm = torch.logsumexp(both, dim=0)
    share = torch.exp(both - norm)
    out = share[0][..., None] * st["out_a"].double() + share[1][..., None] * st["out_b"].double()
    return out, norm
