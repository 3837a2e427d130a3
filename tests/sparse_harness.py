"""Shared helpers of the block-sparse tests: ragged cases with their caches, and exact results in
float64 with bounds on each element.

Sparse attention rounds as chunk attention does, so its bounds are those of the chunk harness, taken
over the keys of the selected blocks.

A score is s sum_h w_h max(0, q_h . k): products of two E4M3 values are exact in float32; each of the
128 additions of a product and of the heads' additions is off by at most one unit in the last place
(2^-23, truncation counted) of the sum of absolute values so far, and three roundings follow. So
|error| <= (128 + H + 3) 2^-23 |s| sum_h |w_h| sum_i |q_hi k_i|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from chunk_harness import BF, F8, SCALE, ChunkCase, bf16_normal
from mla_paged_decode_02_gb300 import api

INF = math.inf


def seen_keys(n, L, i, causal):
    """Keys that new token i of n sees of a sequence of L."""
    return max(0, min(L, L - n + 1 + i)) if causal else L


def random_lists(rng, lens, block, K, causal=True, lead=0, pad=0):
    """Ascending random selections as select_blocks leaves them: the first and the latest block among
    them, -1 behind; rows of no sequence hold a block number that nothing may use."""
    rows = []
    for n, L in lens:
        for i in range(n):
            nb = -(-seen_keys(n, L, i, causal) // block)
            chosen = {0, nb - 1} if nb > 0 else set()
            rest = [c for c in rng.permutation(nb).tolist() if c not in chosen]
            chosen = sorted(chosen | set(rest[:max(0, K - len(chosen))]))[-K:]
            rows.append(chosen + [-1] * (K - len(chosen)))
    return np.array([[12345] * K] * lead + rows + [[54321] * K] * pad, dtype=np.int32).reshape(-1, K)


def attended(q, k, kv):
    """(out, lse, bound) in float64 of one token's queries [H, 576] over its keys [n, 576]; bounds as the chunk
    harness derives them."""
    s = (q @ k.T) * SCALE
    m = s.amax(dim=1, keepdim=True)
    w = torch.exp(s - m)
    z = w.sum(dim=1, keepdim=True)
    v = k[:, :512]
    out, A = (w / z) @ v, (w / z) @ v.abs()
    t = 2.0 ** -8 * (A + out.abs())
    if kv == F8:
        d = 2.0 ** -17 * q.abs().amax(dim=1, keepdim=True) * SCALE * k.abs().sum(dim=1).max()
        t = t + 2.0 ** -11 * A + 2.0 ** -13 * v.abs().sum(dim=0)[None, :] / z + 2 * d * A
    return out, (m + torch.log(z))[:, 0], 1.05 * t + 1e-6


class SparseCase(ChunkCase):
    def __init__(self, lens, H, P, block, K, kv=BF, causal=True, pad=0, seed=0, lead=0, selected=None):
        super().__init__(lens, H, P, kv, causal, pad, seed, lead)
        self.block, self.K = block, K
        if selected is None:
            selected = random_lists(np.random.default_rng(seed + 1), lens, block, K, causal, lead, pad)
        self.selected = torch.from_numpy(np.asarray(selected, dtype=np.int32))

    def run(self, out=None, lse=None, workspace=None, stream=None):
        dev = lambda t: None if t is None else t.cuda()
        self.params = api.make_sparse_params(len(self.lens), self.T, self.H, self.P, self.num_pages, self.table.shape[1],
                                             self.max_seq_len, self.block, self.K, self.kv, self.causal)
        if workspace is None:
            workspace = api.alloc_sparse_workspace(self.params)
            workspace.fill_(0xA5)
        self.workspace = workspace
        if out is None:
            out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((self.T, self.H), -3.5, dtype=torch.float32, device="cuda")
        self.dev = [dev(t) for t in (self.q, self.cache, self.table, self.seq_lens, self.cu, self.selected)]
        self.dscale = dev(self.kv_scale)
        self.out, self.lse = api.sparse_attention(*self.dev, SCALE, self.dscale, max_seq_len=self.max_seq_len,
                                                  block_size=self.block, causal=self.causal, out=out, lse=lse,
                                                  workspace=workspace, stream=stream)
        return self.out, self.lse

    def keys_of(self, b, i):
        """Keys that new token i of sequence b attends to, ascending."""
        n, L = self.lens[b]
        vis = seen_keys(n, L, i, self.causal)
        row = self.selected[self.starts[b] + i].tolist()
        blocks = sorted({c for c in row if 0 <= c and c * self.block < vis})
        return [j for c in blocks for j in range(c * self.block, min(vis, (c + 1) * self.block))]

    def exact(self, b):
        n, _ = self.lens[b]
        H = self.H
        q = self.q[self.starts[b]:self.starts[b] + n].double()
        out = torch.zeros((n, H, 512), dtype=torch.float64)
        lse = torch.full((n, H), -INF, dtype=torch.float64)
        bound = torch.zeros_like(out)
        for i in range(n):
            keys = self.keys_of(b, i)
            if not keys:
                continue
            out[i], lse[i], bound[i] = attended(q[i], self.keys[b][keys], self.kv)
        return out, lse, bound


def quantised(x):
    """E4M3 codes (uint8) of the rows of x and their float32 scales, as index_cache_write() makes them."""
    x, top = x.float(), torch.tensor(448.0)
    m = torch.clamp(x.abs().amax(dim=-1), min=448 * 2.0 ** -126)
    code = (x * (top / m)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return code.view(torch.uint8), m / top


class ScoreCase:
    """lens: [(new tokens, keys in the cache, new ones included)]. Rows past a sequence's length,
    unused pages and rows of no sequence hold NaN codes, scales and weights."""

    def __init__(self, lens, H, P, block, causal=True, pad=0, lead=0, seed=0, max_seq_len=None, extra_columns=2):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.P, self.block, self.causal = lens, H, P, block, causal
        need = [-(-L // P) for _, L in lens]
        self.num_pages = sum(need) + 3
        perm = rng.permutation(self.num_pages)
        table = np.full((len(lens), max([1] + need) + 1), perm[-1], dtype=np.int32)
        table[:, -1] = -7                                             # never read
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = perm[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32) + lead
        self.T = int(self.starts[-1]) + pad
        self.q = torch.full((self.T, H, 128), 0x7F, dtype=torch.uint8)
        self.w = torch.full((self.T, H), float("nan"))
        code, scale = quantised(bf16_normal(rng, self.T - lead - pad, H, 128))
        self.q[lead:self.starts[-1]] = code
        self.w[lead:self.starts[-1]] = torch.from_numpy(rng.standard_normal((self.T - lead - pad, H), dtype=np.float32)) * scale
        self.cache = torch.full((self.num_pages, P, 128), 0x7F, dtype=torch.uint8)
        self.scale = torch.full((self.num_pages, P), float("nan"))
        self.slots = []
        for b, (_, L) in enumerate(lens):
            j = np.arange(L)
            slots = torch.from_numpy(table[b, j // P].astype(np.int64) * P + j % P)
            code, scale = quantised(bf16_normal(rng, L, 128))
            self.cache.view(-1, 128)[slots] = code
            self.scale.view(-1)[slots] = scale
            self.slots.append(slots)
        self.table = torch.from_numpy(table)
        self.seq_lens = torch.tensor([L for _, L in lens], dtype=torch.int32)
        self.cu = torch.from_numpy(self.starts.copy())
        self.max_seq_len = max_seq_len or max([1] + [L for _, L in lens]) + extra_columns * block

    def run(self, out=None, stream=None, error=None):
        self.dev = [t.cuda() for t in (self.q, self.w, self.cache, self.scale, self.table, self.seq_lens, self.cu)]
        self.C = -(-self.max_seq_len // self.block)
        if out is None:
            out = torch.full((self.T, self.C), 7.5, device="cuda")
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda") if error is None else error
        self.out = api.index_scores(*self.dev, max_seq_len=self.max_seq_len, block_size=self.block, causal=self.causal,
                                    out=out, device_error=self.error, stream=stream)
        return self.out

    def exact(self, b):
        """(scores, bounds) of sequence b's new tokens, float64 [n, C]."""
        n, L = self.lens[b]
        out = torch.full((n, self.C), -INF, dtype=torch.float64)
        bound = torch.zeros((n, self.C), dtype=torch.float64)
        k = self.cache.view(-1, 128)[self.slots[b]].view(torch.float8_e4m3fn).double()
        ks = self.scale.view(-1)[self.slots[b]].double()
        for i in range(n):
            vis = seen_keys(n, L, i, self.causal)
            if vis == 0:
                continue
            q = self.q[self.starts[b] + i].view(torch.float8_e4m3fn).double()
            w = self.w[self.starts[b] + i].double()
            s = (torch.relu(q @ k[:vis].T) * w[:, None]).sum(dim=0) * ks[:vis]
            e = ((q.abs() @ k[:vis].abs().T) * w.abs()[:, None]).sum(dim=0) * ks[:vis].abs()
            for c in range(-(-vis // self.block)):
                part = slice(c * self.block, min(vis, (c + 1) * self.block))
                best = torch.where(torch.isnan(s[part]), -INF, s[part])
                out[i, c] = best.max()
                bound[i, c] = torch.nan_to_num(e[part], nan=0.0).max() * (128 + self.H + 3) * 2.0 ** -23
        return out, bound

    def check(self, seqs=None):
        torch.cuda.synchronize()
        assert self.error.item() == 0
        got = self.out.double().cpu()
        assert not torch.isnan(got).any()
        for b in range(len(self.lens)) if seqs is None else seqs:
            r, bound = self.exact(b)
            g = got[self.starts[b]:self.starts[b + 1]]
            none = torch.isinf(r)
            assert torch.equal(torch.isinf(g) & (g < 0), none & (r < 0)), b
            d = torch.where(none, 0.0, g - r).abs()
            assert (d <= bound).all(), (b, (d - bound).max().item())
        used = torch.zeros(self.T, dtype=torch.bool)
        used[self.starts[0]:self.starts[-1]] = True
        assert (got[~used] == 7.5).all()


def selection(scores, seen, block, K, first, last):
    """The selection of one token from its row of scores, by sorting."""
    nb = min(-(-seen // block), len(scores))
    kept = [c for c in range(nb) if c < first or c >= nb - last]
    value = lambda c: -INF if math.isnan(scores[c]) else scores[c]
    rest = sorted((c for c in range(nb) if c not in set(kept)), key=lambda c: (-value(c), c))
    chosen = sorted((kept + rest)[:K])
    return chosen + [-1] * (K - len(chosen))
