"""Shared helpers of the paged key/value tests: caches whose every unseen place holds NaN, a plain
64-bit implementation, and error bounds derived from the formats' half steps."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

import compressed_sparse_kv_overlapped_b200 as csa

SENTINEL = 7.0


@dataclass
class Case:
    seqs: list            # (n, len) of each sequence
    H: int = 8
    H_kv: int = 2
    d: int = 64
    page: int = 16
    dtype: torch.dtype = torch.bfloat16
    W: int = 1 << 20
    S: int = 0
    prefix: int = 0
    heads_first: bool = False   # pages [.., H_kv, slot, d] in memory
    gap: int = 0                # rows of padding behind each sequence's rows
    pad_cols: int = 0           # extra columns in each row of q and out
    scale: float = 0.0
    q_std: float = 1.5
    seed: int = 0

    @property
    def G(self):
        return self.H // self.H_kv


def sees(c: Case, pos: torch.Tensor, t: torch.Tensor) -> torch.Tensor:
    """[len(pos), len(t)] visibility by the definition."""
    far = pos[:, None] - t[None, :]
    return (far >= 0) & ((far < c.W) | (t[None, :] < c.S))


class World:
    """Device tensors of a case.  Only tokens that some query sees (or that `all_live` keeps) hold
    values; every other slot of the pools holds NaN, and pages without such a token are -1 in the
    table."""

    def __init__(self, c: Case, device="cuda", all_live=False):
        g = torch.Generator().manual_seed(1000 + c.seed)
        self.c, B = c, len(c.seqs)
        table_rows, r = [], 0
        for n, m in c.seqs:
            table_rows.append((r, n, m))
            r += n + c.gap
        self.rows, self.seq_rows = r, table_rows
        max_pages = max(1, max((m + c.page - 1) // c.page for _, m in c.seqs), -(-c.prefix // c.page))
        self.K, self.V, live = [], [], []
        for b, (n, m) in enumerate(c.seqs):
            self.K.append(torch.randn(m, c.H_kv, c.d, generator=g, dtype=torch.float64).to(c.dtype))
            self.V.append(torch.randn(m, c.H_kv, c.d, generator=g, dtype=torch.float64).to(c.dtype))
            if b and c.prefix:
                self.K[b][:c.prefix] = self.K[0][:c.prefix]
                self.V[b][:c.prefix] = self.V[0][:c.prefix]
            see = sees(c, torch.arange(m - n, m), torch.arange(m)).any(0) if n else torch.zeros(m, dtype=torch.bool)
            if b == 0:
                see[:c.prefix] = True
            live.append(torch.ones(m, dtype=torch.bool) if all_live else see)
        shared = c.prefix // c.page
        need = [(b, j) for b, (n, m) in enumerate(c.seqs) for j in range((m + c.page - 1) // c.page)
                if live[b][j * c.page:(j + 1) * c.page].any() and not (b and j < shared)]
        num_pages = len(need) + 3
        order = torch.randperm(num_pages, generator=g)
        table = torch.full((B, max_pages), -1, dtype=torch.int32)
        kp = torch.full((num_pages, c.page, c.H_kv, c.d), math.nan, dtype=c.dtype)
        vp = kp.clone()
        for i, (b, j) in enumerate(need):
            pg = int(order[i])
            table[b, j] = pg
            idx = torch.arange(j * c.page, min((j + 1) * c.page, c.seqs[b][1]))
            idx = idx[live[b][idx]]
            kp[pg, idx - j * c.page] = self.K[b][idx]
            vp[pg, idx - j * c.page] = self.V[b][idx]
        if shared:
            table[1:, :shared] = table[0, :shared]
        self.table_cpu = table
        self.table = table.to(device)
        self.seqs = torch.tensor(table_rows, dtype=torch.int64).reshape(B, 3).to(device)
        if c.heads_first:
            self.kp = kp.transpose(1, 2).contiguous().to(device).transpose(1, 2)
            self.vp = vp.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        else:
            self.kp, self.vp = kp.to(device), vp.to(device)
        width = c.H * c.d + c.pad_cols
        q = torch.randn(self.rows, width, generator=g, dtype=torch.float64) * c.q_std
        self.q_full = q.to(c.dtype).to(device)
        self.q = self.q_full[:, :c.H * c.d].unflatten(1, (c.H, c.d))
        self.out_full = torch.full((self.rows, width), SENTINEL, dtype=c.dtype, device=device)
        self.out = self.out_full[:, :c.H * c.d].unflatten(1, (c.H, c.d))
        self.lse = torch.full((self.rows, c.H), SENTINEL, dtype=torch.float32, device=device)
        self.scale = c.scale or c.d ** -0.5
        self.kv = csa.PagedKV(self.kp, self.vp, self.table, self.seqs, c.H)
        self.max_n = max(n for n, _ in c.seqs)
        self.max_len = max(m for _, m in c.seqs)

    def args(self):
        c = self.c
        kw = dict(max_n=self.max_n, max_len=self.max_len, lse=self.lse, scale=self.scale)
        if c.prefix:
            return self.kv.prefix_args(self.q, self.out, prefix_len=c.prefix, **kw)
        return self.kv.window_args(self.q, self.out, W=c.W, S=c.S, **kw)

    def attend(self, args=None, ws=None, stream=None):
        args = self.args() if args is None else args
        ws = self.kv.workspace(args) if ws is None else ws
        (self.kv.prefix_attn if self.c.prefix else self.kv.window_attn)(args, ws, stream)

    def check(self, skip=()):
        """Compare out and lse with the 64-bit reference; rows of no sequence must be untouched."""
        c = self.c
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        touched = torch.zeros(self.rows, dtype=torch.bool)
        for b, (row, n, m) in enumerate(self.seq_rows):
            if n == 0 or b in skip:
                continue
            touched[row:row + n] = True
            ref, ref_lse, tol, tol_lse = reference(c, self.q[row:row + n].double().cpu(), self.K[b].double(),
                                                   self.V[b].double(), m - n, self.scale)
            e, el = (out[row:row + n] - ref).abs(), (lse[row:row + n] - ref_lse).abs()
            assert not e.isnan().any() and not el.isnan().any(), f"sequence {b}: NaN in the output"
            assert (e <= tol).all(), f"sequence {b}: out off by {(e / tol).max():.2f} of the bound, at " \
                                     f"{(e / tol).flatten().argmax().item()} of {tuple(e.shape)}"
            assert (el <= tol_lse).all(), f"sequence {b}: lse off by {(el / tol_lse).max():.2f} of the bound"
        assert (out[~touched] == SENTINEL).all() and (lse[~touched] == SENTINEL).all(), "rows of no sequence were written"
        if c.pad_cols:
            assert (self.out_full[:, c.H * c.d:] == SENTINEL).all(), "columns behind the heads were written"


def reference(c: Case, q, K, V, pos0, scale):
    """out, lse and the bounds of their errors for queries q [n, H, d] at positions pos0..; K, V [m, ..].

    Bounds, with h = eps / 2 of the type (its half step) and u = 2^-24:
      score     |dx| <= scale (d + 8) 2 u sum |q k|       (fp32 products and sums of d terms, scaling, 2^x)
      weight    its own score error, and one rounding to the type: relative h, or 2^-25 below fp16's
                smallest normal number (weights are at most 2^8, so the absolute part is scaled by it at most)
      sums      n terms in fp32: relative 2 n u each for the numerator and the denominator
      output    one rounding: h |out|
    """
    n, H, d = q.shape
    t = torch.arange(K.shape[0])
    see = sees(c, torch.arange(pos0, pos0 + n), t)
    Kh, Vh = K.repeat_interleave(c.G, 1), V.repeat_interleave(c.G, 1)
    x = torch.einsum("nhd,thd->nht", q, Kh) * scale
    mag = torch.einsum("nhd,thd->nht", q.abs(), Kh.abs()) * scale
    x = x.masked_fill(~see[:, None], -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[..., None])
    out = torch.einsum("nht,thd->nhd", w, Vh)
    A = torch.einsum("nht,thd->nhd", w, Vh.abs())
    h, u = torch.finfo(c.dtype).eps / 2, 2.0 ** -24
    dx = (d + 8) * 2 * u * mag.masked_fill(~see[:, None], 0).amax(-1) + 2.0 ** -20
    keys = see.sum(-1).double()[:, None]
    rel = 2 * dx + 4 * keys * u
    sub = keys * 2.0 ** -25 * V.abs().max() if c.dtype == torch.float16 else torch.zeros(n, 1, dtype=torch.float64)
    tol = (h + rel)[..., None] * A + h * out.abs() + sub[..., None] + 1e-30
    tol_lse = rel + 2.0 ** -22 * lse.abs()
    return out, lse, tol, tol_lse


def rotated(x, pos, inv_freq, interleaved):
    """The definition in 64 bits: the first channels of x [n, heads, d] turned in pairs."""
    x, r = x.double(), 2 * inv_freq.numel()
    ang = pos.double()[:, None, None] * inv_freq.double()
    c, s = ang.cos(), ang.sin()
    out = x.clone()
    a = slice(0, r, 2) if interleaved else slice(0, r // 2)
    b = slice(1, r, 2) if interleaved else slice(r // 2, r)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    return out
