"""Calls of the block-sparse operators that are refused before anything is launched; needs no GPU."""
import ctypes
import os

import pytest
import torch

from mla_paged_decode_02_gb300 import api

GOOD = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("libmla.so not built")
    return api.lib()


def index_params(**change):
    p = api.IndexParams(3, 40, 16, 64, 30, 8, 500, 64, 1)
    for k, v in change.items():
        setattr(p, k, v)
    return p


def sparse_params(**change):
    p = api.make_sparse_params(3, 40, 16, 64, 30, 8, 500, 64, 4, api.KV_BF16)
    for k, v in change.items():
        setattr(p, k, v)
    return p


BAD_SIZES = (dict(batch=0), dict(num_tokens=-1), dict(num_heads=0), dict(page_size=0), dict(num_pages=0),
             dict(max_blocks_per_seq=0), dict(max_seq_len=0), dict(block_size=0), dict(causal=2))
UNSUPPORTED = (dict(page_size=12), dict(page_size=1032), dict(block_size=12), dict(block_size=48), dict(block_size=128),
               dict(block_size=4), dict(max_seq_len=(1 << 20) + 1), dict(batch=65537), dict(num_tokens=(1 << 20) + 1),
               dict(num_pages=1 << 26))


def test_index_scores_arguments(lib):
    args = [GOOD] * 8 + [None, None]
    call = lambda p, a=args: lib.mla_index_scores(ctypes.byref(p), *a)
    for bad in BAD_SIZES:
        assert call(index_params(**bad)) == -1, bad
    for bad in UNSUPPORTED + (dict(num_heads=129),):
        assert call(index_params(**bad)) == -2, bad
    assert call(index_params(num_tokens=0)) == 0
    for i in range(8):
        for value in (None, ODD):
            a = list(args)
            a[i] = value
            assert call(index_params(), a) == -1, (i, value)
    assert lib.mla_index_scores(None, *args) == -1


def test_sparse_arguments(lib):
    size = lambda p: lib.mla_sparse_workspace_size(ctypes.byref(p), 152)
    args = [GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, ctypes.c_float(0.1), None, GOOD, GOOD, GOOD, 1 << 34, None]
    call = lambda p, a=args: lib.mla_sparse_attention(ctypes.byref(p), *a)
    assert size(sparse_params()) > 0 and size(sparse_params(num_tokens=0)) > 0
    for bad in BAD_SIZES + (dict(top_k=0), dict(kv_dtype=2)):
        assert size(sparse_params(**bad)) == 0 and call(sparse_params(**bad)) == -1, bad
    for bad in UNSUPPORTED + (dict(top_k=(1 << 20) + 1), dict(num_heads=65537), dict(num_tokens=1 << 20, num_heads=1025)):
        assert size(sparse_params(**bad)) == 0 and call(sparse_params(**bad)) == -2, bad
    assert lib.mla_sparse_workspace_size(None, 152) == 0
    # the table of selected blocks is no wider than the longest context
    assert size(sparse_params(top_k=1 << 20)) == size(sparse_params(top_k=8))
    for i in (0, 1, 2, 3, 4, 5, 8, 9, 10):
        for value in (None, ODD):
            a = list(args)
            a[i] = value
            assert call(sparse_params(), a) == -1, (i, value)
    a = list(args)
    a[6] = ctypes.c_float(float("nan"))
    assert call(sparse_params(), a) == -1
    assert call(sparse_params(kv_dtype=api.KV_FP8_E4M3)) == -1           # without kv_scale


def write_args(**change):
    d = dict(keys=GOOD, ks=128, pos=GOOD, cs=GOOD, max_pos=100, inter=1, slots=GOOD, n=4, cache=GOOD, scale=GOOD, np=10,
             P=64, queries=GOOD, qt=64 * 128, qh=128, w=GOOD, H=64, qi=GOOD, qw=GOOD, err=None, s=None)
    d.update(change)
    return list(d.values())


def test_index_cache_write_arguments(lib):
    f = lib.mla_index_cache_write
    for bad in (dict(n=-1), dict(max_pos=0), dict(np=0), dict(P=0), dict(inter=2), dict(keys=None), dict(pos=None),
                dict(cs=None), dict(slots=None), dict(cache=None), dict(scale=None), dict(queries=None), dict(w=None),
                dict(qi=None), dict(qw=None), dict(H=0), dict(ks=120), dict(ks=132), dict(qt=4), dict(qh=12), dict(qh=-8),
                dict(keys=ODD), dict(cs=ODD), dict(queries=ODD), dict(qi=ODD), dict(cache=ODD), dict(pos=ODD),
                dict(slots=ODD), dict(scale=ODD), dict(w=ODD), dict(qw=ODD), dict(err=ODD)):
        assert f(*write_args(**bad)) == -1, bad
    assert f(*write_args(n=0)) == 0
    assert f(*write_args(H=129)) == -2


def select_args(**change):
    d = dict(scores=GOOD, stride=100, T=4, C=100, seq=GOOD, cu=GOOD, B=2, block=64, K=8, first=1, last=2, causal=1, out=GOOD,
             err=None, s=None)
    d.update(change)
    return list(d.values())


def test_select_blocks_arguments(lib):
    f = lib.mla_select_blocks
    for bad in (dict(T=-1), dict(C=0), dict(B=0), dict(block=0), dict(K=0), dict(first=-1), dict(last=-1), dict(K=2),
                dict(stride=99), dict(causal=2), dict(scores=None), dict(seq=None), dict(cu=None), dict(out=None),
                dict(scores=ODD), dict(seq=ODD), dict(cu=ODD), dict(out=ODD), dict(err=ODD)):
        assert f(*select_args(**bad)) == -1, bad
    for bad in (dict(T=(1 << 20) + 1), dict(B=65537), dict(C=(1 << 20) + 1, stride=1 << 21), dict(K=(1 << 20) + 1),
                dict(block=(1 << 20) + 1)):
        assert f(*select_args(**bad)) == -2, bad
    assert f(*select_args(T=0)) == 0


def tensors():
    i32 = dict(dtype=torch.int32)
    return dict(q=torch.zeros(4, 2, 576, dtype=torch.bfloat16), cache=torch.zeros(3, 64, 576, dtype=torch.bfloat16),
                table=torch.zeros(2, 1, **i32), lens=torch.zeros(2, **i32), cu=torch.zeros(3, **i32),
                sel=torch.zeros(4, 3, **i32))


def test_sparse_attention_tensors():
    def call(max_seq_len=64, block_size=64, out=None, lse=None, workspace=None, **change):
        t = dict(tensors(), **change)
        return api.sparse_attention(t["q"], t["cache"], t["table"], t["lens"], t["cu"], t["sel"], 0.1, max_seq_len=max_seq_len,
                                    block_size=block_size, out=out, lse=lse, workspace=workspace)
    t = tensors()
    for bad in (dict(q=t["q"].float()), dict(q=t["q"][:, :1]), dict(q=t["q"][..., :512]), dict(cache=t["cache"][:, ::2]),
                dict(table=t["table"].long()), dict(table=t["table"][:1]), dict(lens=t["lens"].long()), dict(cu=t["cu"][:2]),
                dict(sel=t["sel"].long()), dict(sel=t["sel"][:3]), dict(sel=t["sel"][:, :2]), dict(sel=t["sel"][0]),
                dict(cache=t["cache"].to(torch.float8_e4m3fn)), dict(max_seq_len=1 << 32), dict(block_size=1 << 32),
                dict(out=torch.zeros(4, 2, 512)), dict(out=torch.zeros(4, 1, 512, dtype=torch.bfloat16)),
                dict(lse=torch.zeros(4, 3)), dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="on the GPU"):
        call()


def test_index_tensors():
    q, w = torch.zeros(4, 2, 128, dtype=torch.uint8), torch.zeros(4, 2)
    cache, scale = torch.zeros(3, 64, 128, dtype=torch.uint8), torch.zeros(3, 64)
    t = tensors()

    def scores(q=q, w=w, cache=cache, scale=scale, table=t["table"], max_seq_len=64, block_size=64, out=None, error=None):
        return api.index_scores(q, w, cache, scale, table, t["lens"], t["cu"], max_seq_len=max_seq_len,
                                block_size=block_size, out=out, device_error=error)
    for bad in (dict(q=q.float()), dict(q=q[:, :1]), dict(q=q[..., :64]), dict(w=w[:3]), dict(w=w.double()),
                dict(cache=cache[..., :64]), dict(cache=cache.float()), dict(scale=scale[:2]), dict(scale=scale.double()),
                dict(table=t["table"].long()), dict(max_seq_len=0), dict(block_size=0), dict(max_seq_len=1 << 32),
                dict(out=torch.zeros(4, 2)), dict(error=torch.zeros(1))):
        with pytest.raises(ValueError):
            scores(**bad)

    def select(s=torch.zeros(4, 9), top_k=3, block_size=64, keep_first=1, keep_last=2, out=None):
        return api.select_blocks(s, t["lens"], t["cu"], top_k, block_size=block_size, keep_first=keep_first,
                                 keep_last=keep_last, out=out)
    for bad in (dict(s=torch.zeros(4, 9).double()), dict(s=torch.zeros(9, 4).T), dict(s=torch.zeros(9)), dict(top_k=0),
                dict(top_k=2), dict(keep_first=-1), dict(top_k=1 << 32), dict(s=torch.zeros(1, 9).expand(4, 9)),
                dict(out=torch.zeros(4, 3)), dict(out=torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            select(**bad)

    keys, pos, cs = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64), torch.zeros(9, 64)
    queries = torch.zeros(4, 2, 128, dtype=torch.bfloat16)

    def write(keys=keys, pos=pos, cs=cs, cache=cache, queries=queries, weights=w, q_index=q, q_weights=w.clone()):
        return api.index_cache_write(keys, pos, cs, pos, cache, scale, queries=queries, weights=weights, q_index=q_index,
                                     q_weights=q_weights)
    for bad in (dict(keys=keys.float()), dict(keys=keys[:, :64]), dict(keys=torch.zeros(4, 132, dtype=torch.bfloat16)[:, :128]),
                dict(pos=pos.int()), dict(cs=cs[:, :32]), dict(cache=cache[:, ::2]), dict(queries=None), dict(weights=None),
                dict(q_index=None), dict(queries=queries[:3]), dict(queries=queries.float()), dict(q_index=q[:, :1]),
                dict(q_weights=w.double()), dict(weights=w.T.contiguous().T)):
        with pytest.raises(ValueError):
            write(**bad)
    with pytest.raises(ValueError, match="on the GPU"):
        write()


@pytest.mark.parametrize("far", [(1 << 31) + 1, (1 << 32) + 1])
def test_sizes_whose_32_bit_fields_would_keep_their_low_bits(far):
    """Tensors of these shapes fit a GPU; the calls must not take them for ones of a few rows or columns."""
    def empty(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")
    t = tensors()
    q, w = torch.zeros(4, 2, 128, dtype=torch.uint8), torch.zeros(4, 2)
    cache, scale = torch.zeros(3, 64, 128, dtype=torch.uint8), torch.zeros(3, 64)

    def scores(table=t["table"], lens=t["lens"], cu=t["cu"]):
        api.index_scores(q, w, cache, scale, table, lens, cu, max_seq_len=64, block_size=64)

    def select(s, lens=t["lens"], cu=t["cu"]):
        api.select_blocks(s, lens, cu, 3, block_size=64)

    def sparse(table=t["table"], lens=t["lens"], cu=t["cu"], sel=t["sel"], max_seq_len=64, block_size=64):
        api.sparse_attention(t["q"], t["cache"], table, lens, cu, sel, 0.1, max_seq_len=max_seq_len, block_size=block_size)
    ragged = dict(lens=empty(far), cu=empty(far + 1))
    for call in (lambda: scores(table=empty(2, far)), lambda: scores(table=empty(far, 1), **ragged),
                 lambda: select(empty(4, far, dtype=torch.float32)), lambda: select(empty(far, 4, dtype=torch.float32)),
                 lambda: select(torch.zeros(4, 9), **ragged), lambda: sparse(table=empty(2, far)),
                 lambda: sparse(table=empty(far, 1), **ragged), lambda: sparse(sel=empty(4, far)),
                 lambda: sparse(max_seq_len=far), lambda: sparse(block_size=far), lambda: sparse(max_seq_len=64 - (1 << 32)),
                 lambda: sparse(block_size=64 - (1 << 32))):
        with pytest.raises(ValueError, match="fit 32 bits"):
            call()
    good = [3, 40, 16, 64, 30, 8, 500, 64, 4, api.KV_BF16]
    for i in range(9):
        for value in (far, -far):
            with pytest.raises(ValueError, match="fit 32 bits"):
                api.make_sparse_params(*good[:i], value, *good[i + 1:])
