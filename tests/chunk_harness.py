"""Shared helpers of the chunk-attention tests: a ragged case with its paged cache, and its
exact result in float64 with per-element error bounds.

The bounds count each rounding of the kernel once (a rounding is off by at most half a step:
bf16 2^-8, fp16 2^-11, relative). With w the normalised weights and A = sum_j w_j |v_j|:

* bf16 cache: P is rounded to bf16 (2^-8 A) and the result to bf16 (2^-8 |out|);
* FP8 cache: P as two E4M3 terms of its fp16 rounding (2^-8 A: the lower term is below 2^-3 of
  the value and has 4 significant bits; at most 2^-11 A for fp16), where the terms run out of
  E4M3's range at most 2^-9 absolute in units where the reference weight is 2^4, i.e.
  2^-13 sum_j |v_j| e^(m - lse); q as two terms, off by at most 2^-17 of its row's largest
  value where they run out, which moves a score by d <= 2^-17 max|q| scale max_j sum_d |k_jd|
  and a result by at most 2 d A.

Float32 accumulation and exp2 (about 1e-4 of A for the scores drawn here) are covered by a
factor of 1.05 and 1e-6.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from mla_paged_decode_02_gb300 import api, synth

SCALE = synth.SOFTMAX_SCALE
BF, F8 = api.KV_BF16, api.KV_FP8_E4M3
LSE_ABS = {BF: 1e-4, F8: 1e-3}


def bf16_normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)


class ChunkCase:
    """lens: [(new tokens, keys in the cache, new ones included)]. The pool starts as NaN; rows
    past a sequence's length, unused pages and padding rows of q stay NaN."""

    def __init__(self, lens, H, P, kv=BF, causal=True, pad=0, seed=0, lead=0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.P, self.kv, self.causal = lens, H, P, kv, causal
        need = [-(-L // P) for _, L in lens]
        self.num_pages = sum(need) + 3
        perm = rng.permutation(self.num_pages)
        mb = max(1, max(need)) + 1
        table = np.full((len(lens), mb), perm[-1], dtype=np.int32)    # a page that stays NaN
        table[:, -1] = -7                                             # never read
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = perm[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32) + lead
        self.T = int(self.starts[-1]) + pad
        self.q = torch.full((self.T, H, 576), float("nan"), dtype=torch.bfloat16)
        self.q[lead:self.starts[-1]] = bf16_normal(rng, int(self.starts[-1]) - lead, H, 576)
        values = bf16_normal(rng, max(1, sum(L for _, L in lens)), 576)
        self.kv_scale = None
        if kv == F8:
            self.kv_scale = torch.tensor([float(np.float32(values.float().abs().max().item()) / np.float32(448))])
            codes = (values.float() / self.kv_scale).to(torch.float8_e4m3fn)
            values = codes
        self.cache = (torch.full((self.num_pages, P, 576), float("nan"), dtype=torch.bfloat16) if kv == BF else
                      torch.full((self.num_pages, P, 576), 0x7F, dtype=torch.uint8))
        flat = self.cache.view(-1, 576)
        self.keys, o = [], 0
        for b, (_, L) in enumerate(lens):
            j = np.arange(L)
            slots = torch.from_numpy(table[b, j // P].astype(np.int64) * P + j % P)
            rows = values[o:o + L]
            flat[slots] = rows if kv == BF else rows.view(torch.uint8)
            self.keys.append(rows.float().double() * (1.0 if kv == BF else self.kv_scale.double()))
            o += L
        self.table = torch.from_numpy(table)
        self.seq_lens = torch.tensor([L for _, L in lens], dtype=torch.int32)
        self.cu = torch.from_numpy(self.starts.copy())
        self.max_seq_len = max(1, max(L for _, L in lens))

    def set_key(self, b, j, row):
        """Overwrite cache row j of sequence b (bf16 values, or E4M3 codes)."""
        slot = int(self.table[b, j // self.P]) * self.P + j % self.P
        self.cache.view(-1, 576)[slot] = row

    def run(self, out=None, lse=None, workspace=None, stream=None):
        dev = lambda t: None if t is None else t.cuda()
        self.params = api.make_chunk_params(len(self.lens), self.T, self.H, self.P, self.num_pages, self.table.shape[1],
                                            self.max_seq_len, self.kv, self.causal)
        if workspace is None:
            workspace = api.alloc_chunk_workspace(self.params)
            workspace.fill_(0xA5)
        self.workspace = workspace
        if out is None:
            out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((self.T, self.H), -3.5, dtype=torch.float32, device="cuda")
        self.dev = [dev(t) for t in (self.q, self.cache, self.table, self.seq_lens, self.cu)]
        self.dscale = dev(self.kv_scale)
        self.out, self.lse = api.chunk_attention(*self.dev, SCALE, self.dscale, max_seq_len=self.max_seq_len,
                                                 causal=self.causal, out=out, lse=lse, workspace=workspace, stream=stream)
        return self.out, self.lse

    def exact(self, b):
        """(out, lse, bound) of sequence b's new tokens, float64 [n, H, ...]."""
        n, L = self.lens[b]
        H = self.H
        q = self.q[self.starts[b]:self.starts[b] + n].double()
        k = self.keys[b]
        out = torch.zeros((n, H, 512), dtype=torch.float64)
        lse = torch.full((n, H), -math.inf, dtype=torch.float64)
        bound = torch.zeros_like(out)
        for i in range(n):
            vis = max(0, min(L, L - n + 1 + i)) if self.causal else L
            if vis == 0:
                continue
            s = (q[i] @ k[:vis].T) * SCALE
            m = s.amax(dim=1, keepdim=True)
            w = torch.exp(s - m)
            z = w.sum(dim=1, keepdim=True)
            v = k[:vis, :512]
            out[i] = (w / z) @ v
            lse[i] = (m + torch.log(z))[:, 0]
            A = (w / z) @ v.abs()
            t = 2.0 ** -8 * (A + out[i].abs())
            if self.kv == F8:
                d = 2.0 ** -17 * q[i].abs().amax(dim=1, keepdim=True) * SCALE * k[:vis].abs().sum(dim=1).max()
                t = t + 2.0 ** -11 * A + 2.0 ** -13 * v.abs().sum(dim=0)[None, :] / z + 2 * d * A
            bound[i] = 1.05 * t + 1e-6
        return out, lse, bound

    def check(self, seqs=None):
        torch.cuda.synchronize()
        assert api.decode_check(self.workspace) == (0, 0)
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        for b in range(len(self.lens)) if seqs is None else seqs:
            n, _ = self.lens[b]
            if n == 0:
                continue
            r, rl, bound = self.exact(b)
            o, l = out[self.starts[b]:self.starts[b] + n], lse[self.starts[b]:self.starts[b] + n]
            none = torch.isinf(rl)
            assert torch.equal(torch.isinf(l) & (l < 0), none), b
            assert (o[none] == 0).all(), b
            assert torch.isfinite(o).all(), b
            worst = ((o - r).abs() - bound).max().item()
            assert worst <= 0, (b, worst, (o - r).abs().max().item())
            if (~none).any():
                assert (l - rl)[~none].abs().max().item() <= LSE_ABS[self.kv], b
        used = torch.zeros(self.T, dtype=torch.bool)
        used[self.starts[0]:self.starts[-1]] = True
        assert (out[~used] == 7.0).all() and (lse[~used] == -3.5).all()
