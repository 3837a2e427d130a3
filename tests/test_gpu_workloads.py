"""The workloads of perf/more_operators.py: their plain forms, their 64-bit values and the package's calls agree.

Bounds. A rotated value is off by at most 2^-23 (|a c| + |b s|), both products and their sum counted, which is within
2^-22 of the row's largest magnitude m (that is at least 1 / sqrt 2 of the pair's largest member): so are m and the
scale, with two quotients 2^-21. A code is off by half a step, 2^-4 of the value or 2^-10 below the normal range,
and by what its row's rounding moves it, 2^-20 of 448. Scores as the harness derives them, with
sum_i |q_i k_i| <= |q| |k|; sparse attention as the harness derives it."""
import random

import pytest
import torch

from chunk_harness import BF, F8, LSE_ABS
from perf import more_operators as workloads
from sparse_harness import attended

pytestmark = pytest.mark.gpu

LISTED = {c["name"]: c for c in workloads.listed()}
NAMES = ["write_step_t128_h64", "scores_long_b4_h64", "select_step_t128", "select_long_t16",
         "select_chunk_t2048", "sparse_tiny_b2_h16_bf16", "sparse_step_b64_h16_fp8", "sparse_long_b4_h128_fp8"]


def small_draws():
    """Six drawn cases of each operator that 64 bits are quick with."""
    rng, found = random.Random(11), {}
    while len(found) < 4 or min(map(len, found.values())) < 6:
        c = workloads.draw(rng)
        mine = found.setdefault(c["op"], [])
        if len(mine) < 6 and workloads.work(c)["flops"] < 1e10:
            mine.append(c)
    return [pytest.param(c, id=f"{op}-{i}") for op, cases in found.items() for i, c in enumerate(cases)]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def outputs(case, seed, own, monkeypatch):
    monkeypatch.setattr(workloads, "own", own)
    state = workloads.prepare(case, seed)
    out = workloads.run(state)
    torch.cuda.synchronize()
    return state, out if isinstance(out, tuple) else (out,)


def check_write(case, st, got, want):
    real = st["real"]
    for code, scale, code_want, scale_want in ((got[0], got[1], want[0], want[1]), (got[2][:real], got[3][:real], want[2][:real], want[3][:real])):
        d = (code.double() - code_want).abs()
        assert (d <= torch.clamp(code_want.abs() * 2.0 ** -4, min=2.0 ** -10) + 448 * 2.0 ** -20).all()
        assert ((scale.double() - scale_want).abs() <= 2.0 ** -21 * scale_want.abs()).all()


def check_scores(case, st, got, want):
    h = case["heads"]
    keys = (st["index_cache"].double().norm(dim=-1) * st["index_scale"].double()).max()
    rows = (st["q_weights"].double().abs() * st["q_index"].double().norm(dim=-1)).sum(dim=1)
    none = torch.isinf(want[0])
    assert torch.equal(torch.isinf(got[0]), none) and (got[0][none] == want[0][none]).all()
    d = torch.where(none, 0.0, got[0].double() - want[0]).abs()
    assert (d <= (128 + h + 3) * 2.0 ** -23 * (rows * keys)[:, None]).all()


def check_select(case, st, got, want):
    assert torch.equal(got[0], want[0])


def check_sparse(case, st, got, want):
    kv = BF if st["kv_scale"] is None else F8
    rows, page, block = st["cache"].view(-1, 576), st["cache"].shape[1], st["block"]
    rng, t0 = random.Random(1), 0
    for b, (new, total) in enumerate(zip(st["new"], st["total"])):
        for i in {0, new - 1, rng.randrange(new)} if new else ():
            t, seen = t0 + i, total - new + 1 + i if st["causal"] else total
            where = torch.tensor([j for c in st["selected"][t].tolist() if c >= 0
                                  for j in range(c * block, min(seen, c * block + block))], device="cuda")
            k = rows[st["block_table"][b].long()[where // page] * page + where % page].double()
            k = k if kv == BF else k * st["kv_scale"].double()
            out, lse, bound = attended(st["q"][t].double(), k, kv)
            # the harness takes the scale as a call does, rounded to float32: scores 2^-24 apart at most, and weights by
            # twice that
            apart = 2.0 ** -24 * (st["q"][t].double() @ k.T).abs().max().item() * workloads.SCALE + 1e-12
            assert ((want[0][t] - out).abs() <= 2 * apart * k[:, :512].abs().max()).all()
            assert ((want[1][t] - lse).abs() <= apart).all()
            assert ((got[0][t].double() - out).abs() <= bound).all(), (b, i)
            assert (got[1][t].double() - lse).abs().max() <= LSE_ABS[kv], (b, i)
        t0 += new
    assert (got[0][t0:] == 0).all() and (got[1][t0:] == 0).all()      # rows behind the last sequence


@pytest.mark.parametrize("case", [pytest.param(LISTED[n], id=n) for n in NAMES] + small_draws())
def test_workloads_agree(case, monkeypatch):
    check = {"write": check_write, "scores": check_scores, "select": check_select, "sparse": check_sparse}[case["op"]]
    want = workloads.exact(case, 3)
    want = want if isinstance(want, tuple) else (want,)
    for own in (True, False):
        st, got = outputs(case, 3, own, monkeypatch)
        check(case, st, got, want)
