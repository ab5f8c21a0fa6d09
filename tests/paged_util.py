"""Inputs and 64-bit oracles of the paged serving tests (plain torch on the CPU)."""
from __future__ import annotations

import math

import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Batch:
    """A ragged batch over a paged pool whose unused places hold NaN."""

    def __init__(self, lens, added, Hq, H, D, page, dtype, seed=0, prefix=0, layers=1, layer=0,
                 unseen=None, scale_q=1.0, extra_rows=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.added, self.Hq, self.H, self.D = list(lens), list(added), Hq, H, D
        self.page, self.dtype, self.prefix, self.layer = page, dtype, prefix, layer
        B = len(lens)
        counts = [-(-x // page) for x in lens]
        ppages = -(-prefix // page)
        pages = sum(counts) + ppages + 3
        perm = torch.randperm(pages, generator=g).tolist()
        self.columns = max(counts + [1]) + 1
        self.tables = torch.full((B, self.columns), -1, dtype=torch.int32)
        pool = torch.full((layers, 2, pages, page, H, D), math.nan, dtype=torch.float32)
        self.keys, self.values = [], []

        def place(table, n, skip):
            k = torch.randn(n, H, D, generator=g).to(dtype)
            v = (torch.randn(n, H, D, generator=g) + 0.25).to(dtype)
            for j in range(n):
                if skip is not None and skip(j):
                    continue  # no row sees it: stays NaN
                pool[layer, 0, table[j // page], j % page] = k[j].float()
                pool[layer, 1, table[j // page], j % page] = v[j].float()
            return k, v

        for r in range(B):
            mine = [perm.pop() for _ in range(counts[r])]
            self.tables[r, :counts[r]] = torch.tensor(mine, dtype=torch.int32)
            skip = None if unseen is None else (lambda j, r=r: unseen(r, j))
            k, v = place(mine, lens[r], skip)
            self.keys.append(k)
            self.values.append(v)
        mine = [perm.pop() for _ in range(ppages)]
        self.prefix_table = torch.tensor(mine, dtype=torch.int32)
        self.prefix_k, self.prefix_v = place(mine, prefix, None)
        self.pool = pool.to(dtype)
        N = sum(added)
        self.q = (scale_q * torch.randn(N + extra_rows, Hq, D, generator=g)).to(dtype)
        self.starts = [0]
        for a in added:
            self.starts.append(self.starts[-1] + a)

    def oracle(self, window=0, sinks=0, scale=None):
        """(out, lse, tolerance) in 64 bits.  The tolerance of an element counts
        the roundings of the definition's steps: half a step of the output's
        type; half a step of the type for each softmax weight in the product
        with V (and 2^-25 absolute for an fp16 weight below its normal range);
        fp32 sums of D products in the scores, twice, since an error of the
        exponent also moves the sum; and 2^-20 for the 32-bit softmax steps."""
        D, G = self.D, self.Hq // self.H
        scale = 1 / math.sqrt(D) if scale is None else scale
        u = half_step(self.dtype)
        tiny = 2.0 ** -25 if self.dtype == torch.float16 else 0.0
        out = torch.zeros(sum(self.added), self.Hq, D, dtype=torch.float64)
        lse = torch.full((sum(self.added), self.Hq), -math.inf, dtype=torch.float64)
        tol = torch.zeros_like(out)
        for r, (n, kv) in enumerate(zip(self.added, self.lens)):
            k = torch.cat([self.prefix_k, self.keys[r]]).double()
            v = torch.cat([self.prefix_v, self.values[r]]).double()
            P = self.prefix
            for i in range(n):
                p = kv - n + i
                j = torch.arange(max(0, p + 1))
                if window:
                    j = j[(j > p - window) | (j < sinks)]
                j = torch.cat([torch.arange(P), j + P])
                if j.numel() == 0:
                    continue
                t = self.starts[r] + i
                for h in range(self.Hq):
                    q = self.q[t, h].double()
                    kk, vv = k[j, h // G], v[j, h // G]
                    s = kk @ q * scale
                    m = s.max()
                    e = torch.exp(s - m)
                    w = e / e.sum()
                    o = w @ vv
                    out[t, h] = o
                    lse[t, h] = m + torch.log(e.sum())
                    mass = w @ vv.abs()
                    score = (D + 4) * 2.0 ** -24 * float((kk.abs() @ q.abs()).max()) * abs(scale)
                    tol[t, h] = u * o.abs() + (u + 2 * score + 2.0 ** -20) * mass \
                        + tiny * vv.abs().sum(0) / e.sum()
        return out, lse, tol * 1.01 + 1e-7

    def device(self):
        """q, pool, q_starts, kv_lens, tables, prefix table on the GPU."""
        c = lambda x: x.cuda()  # noqa: E731
        return (c(self.q), c(self.pool), c(torch.tensor(self.starts, dtype=torch.int32)),
                c(torch.tensor(self.lens, dtype=torch.int32)), c(self.tables),
                c(self.prefix_table))


def check_close(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    bad = (got - want).abs() > tol
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{got[tuple(at)]} against {want[tuple(at)]} "
                             f"(tolerance {tol[tuple(at)]})")
