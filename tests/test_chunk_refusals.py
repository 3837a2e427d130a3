"""Calls of the chunked-prefill operators that are refused before anything is launched; needs no GPU."""
import ctypes
import os

import pytest
import torch

from mla_paged_decode_02_gb300 import api

GOOD = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("libmla.so not built")
    return api.lib()


def params(**change):
    p = api.make_chunk_params(3, 40, 16, 64, 30, 8, 500, api.KV_BF16)
    for k, v in change.items():
        setattr(p, k, v)
    return p


def test_chunk_workspace(lib):
    assert lib.mla_chunk_workspace_size(ctypes.byref(params()), 152) > 0
    assert lib.mla_chunk_workspace_size(ctypes.byref(params(num_tokens=0)), 152) > 0
    for bad in (dict(batch=0), dict(num_tokens=-1), dict(num_heads=0), dict(page_size=12), dict(page_size=1032),
                dict(num_pages=0), dict(max_blocks_per_seq=0), dict(max_seq_len=0), dict(max_seq_len=(1 << 20) + 1),
                dict(kv_dtype=2), dict(causal=2), dict(num_tokens=1 << 24, num_heads=128), dict(num_heads=65537),
                dict(batch=65537), dict(num_pages=1 << 26)):
        assert lib.mla_chunk_workspace_size(ctypes.byref(params(**bad)), 152) == 0, bad
    assert lib.mla_chunk_workspace_size(None, 152) == 0
    with pytest.raises(api.MLAError):
        api.chunk_workspace_size(params(batch=0), 152)


def test_chunk_pointers(lib):
    args = [GOOD, GOOD, GOOD, GOOD, GOOD, ctypes.c_float(0.1), None, GOOD, GOOD, GOOD, 1 << 34, None]
    call = lambda p, a: lib.mla_chunk_attention(ctypes.byref(p), *a)
    for i in (0, 1, 2, 3, 4, 7, 8, 9):
        a = list(args)
        a[i] = None
        assert call(params(), a) == -1, i
    for i in (0, 1, 7, 9):
        a = list(args)
        a[i] = ODD
        assert call(params(), a) == -1, i
    a = list(args)
    a[5] = ctypes.c_float(float("nan"))
    assert call(params(), a) == -1
    assert call(params(kv_dtype=api.KV_FP8_E4M3), args) == -1          # without kv_scale
    assert call(params(page_size=12), args) == -2


def rope_args(**change):
    d = dict(latent=GOOD, ls=576, rope=GOOD, rs=576, pos=GOOD, cs=GOOD, max_pos=100, inter=1, slots=GOOD, n=4,
             cache=GOOD, np=10, P=64, kvd=0, scale=None, q_rope=GOOD, qt=3 * 192, qh=192, H=3, q=GOOD, err=None, s=None)
    d.update(change)
    return list(d.values())


def test_rope_cache_write_arguments(lib):
    f = lib.mla_rope_cache_write
    for bad in (dict(n=-1), dict(max_pos=0), dict(np=0), dict(P=0), dict(kvd=2), dict(inter=2), dict(latent=None),
                dict(rope=None), dict(pos=None), dict(cs=None), dict(slots=None), dict(cache=None), dict(kvd=1),
                dict(q=None), dict(q_rope=None), dict(H=0), dict(ls=504), dict(rs=56), dict(ls=580), dict(rs=66),
                dict(qt=4), dict(qh=12), dict(qh=-8), dict(latent=ODD), dict(rope=ODD), dict(cs=ODD), dict(q=ODD),
                dict(q_rope=ODD), dict(cache=ODD), dict(pos=ODD), dict(slots=ODD)):
        assert f(*rope_args(**bad)) == -1, bad
    assert f(*rope_args(n=0)) == 0
    assert f(*rope_args(H=70000)) == -2


def test_merge_arguments(lib):
    f = lib.mla_merge_states
    good = [GOOD, GOOD, GOOD, GOOD, 5, GOOD, GOOD, None]
    for i in (0, 1, 2, 3, 5, 6):
        a = list(good)
        a[i] = None
        assert f(*a) == -1, i
    for i in (0, 2, 5):
        a = list(good)
        a[i] = ODD
        assert f(*a) == -1, i
    assert f(GOOD, GOOD, GOOD, GOOD, -1, GOOD, GOOD, None) == -1
    assert f(None, None, None, None, 0, None, None, None) == 0


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def test_chunk_tensors():
    q, kv = bf(10, 4, 576), bf(6, 64, 576)
    bt, sl, cu = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    call = lambda q=q, kv=kv, bt=bt, sl=sl, cu=cu, scale=None, **k: api.chunk_attention(q, kv, bt, sl, cu, 0.1, scale,
                                                                                      max_seq_len=100, **k)
    for bad in (dict(q=bf(10, 4, 575)), dict(q=q.float()), dict(q=bf(10, 8, 576)[:, ::2]), dict(q=bf(10, 576)),
                dict(kv=bf(6, 64, 512)), dict(kv=bf(12, 64, 576)[::2]), dict(bt=bt.long()), dict(sl=sl.long()),
                dict(cu=cu.long()), dict(cu=cu[:2]), dict(bt=bt[:1]), dict(bt=torch.zeros((2, 6), dtype=torch.int32)[:, ::2]),
                dict(kv=torch.zeros((6, 64, 576), dtype=torch.uint8)),                       # FP8 without a scale
                dict(out=bf(10, 4, 576)), dict(out=bf(9, 4, 512)), dict(lse=torch.zeros((10, 5))),
                dict(lse=torch.zeros((10, 4), dtype=torch.float64))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(kv=kv.half())
    with pytest.raises(ValueError, match="GPU"):
        call()


def test_rope_cache_write_tensors():
    n = 5
    base = dict(latent=bf(n, 512), rope=bf(n, 64), positions=torch.zeros(n, dtype=torch.int64),
                cos_sin=torch.zeros((9, 64)), slot_mapping=torch.zeros(n, dtype=torch.int64), kv_cache=bf(3, 64, 576),
                q_rope=bf(n, 4, 64), q=bf(n, 4, 576))

    def call(**change):
        d = {**base, **change}
        pos = [d.pop(k) for k in ("latent", "rope", "positions", "cos_sin", "slot_mapping", "kv_cache")]
        api.rope_cache_write(*pos, **d)

    for bad in (dict(latent=bf(n, 511)), dict(latent=bf(n, 512).float()), dict(latent=bf(n, 516)[:, :512]),
                dict(latent=bf(512, n).T), dict(rope=bf(n, 128)[:, ::2]), dict(rope=bf(n + 1, 64)),
                dict(latent=bf(1, 512).expand(n, 512)), dict(positions=torch.zeros(n, dtype=torch.int32)),
                dict(positions=torch.zeros(n + 1, dtype=torch.int64)), dict(slot_mapping=torch.zeros(2 * n, dtype=torch.int64)[::2]),
                dict(cos_sin=torch.zeros((9, 32))), dict(cos_sin=torch.zeros((9, 64), dtype=torch.float64)),
                dict(kv_cache=bf(3, 64, 512)), dict(kv_cache=torch.zeros((3, 64, 576), dtype=torch.uint8)),
                dict(q=None), dict(q_rope=None), dict(q=bf(n, 4, 512)), dict(q=bf(n, 8, 576)[:, ::2]),
                dict(q_rope=bf(n, 4, 128)[:, :, ::2]), dict(q_rope=bf(n, 3, 64)), dict(q_rope=bf(n, 4, 68)[:, :, :64]),
                dict(device_error=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError, match="GPU"):
        call()


def test_merge_tensors():
    oa, la = bf(4, 3, 512), torch.zeros((4, 3))
    for bad in (dict(out_a=bf(4, 3, 576)), dict(out_b=bf(3, 4, 512)), dict(lse_b=torch.zeros((4, 3), dtype=torch.float64)),
                dict(out=bf(4, 6, 512)[:, ::2]), dict(lse=torch.zeros((3, 4)).T), dict(out_a=oa.float())):
        d = dict(out_a=oa, lse_a=la, out_b=oa, lse_b=la)
        d.update(bad)
        with pytest.raises(ValueError):
            api.merge_states(**d)
    with pytest.raises(ValueError, match="GPU"):
        api.merge_states(oa, la, oa, la)


def test_a_workspace_whose_elements_share_memory():
    """An expanded tensor has as many elements as the call needs and the memory of one."""
    q, kv = bf(10, 4, 576), bf(6, 64, 576)
    bt, sl, cu = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 28), torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            api.chunk_attention(q, kv, bt, sl, cu, 0.1, max_seq_len=100, workspace=ws)


def test_a_length_bound_beyond_32_bits():
    """The parameter structure holds 32 bits: 2^32 + 100 must not become 100."""
    q, kv = bf(10, 4, 576), bf(6, 64, 576)
    bt, sl, cu = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_seq_len"):
        api.chunk_attention(q, kv, bt, sl, cu, 0.1, max_seq_len=(1 << 32) + 100)
    with pytest.raises(ValueError, match="max_seq_len"):
        api.make_chunk_params(2, 10, 4, 64, 6, 3, (1 << 32) + 100, api.KV_BF16)
