"""Sequences under a sliding window for the tests of the windowed calls: pools in which only rows
that some token attends to hold numbers, and the attention in numpy, 64 bits."""
import numpy as np
import torch

import step_model

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# fp32 outputs.  A score is a sum of D <= 128 products, each addition good to 2^-23 of the sum of
# magnitudes, which is below 13 in log2 units for normal values: 128 * 2^-23 * 13 = 2e-4 in the
# exponent, 1.4e-4 of a weight.  Weights held in two 16-bit parts add 2^-17, exp2 2^-22, the sums
# of n <= 2^13 terms 2^-10 at worst and 2^-16 as they come.  Twice the weights' error (numerator
# and denominator) times values below 5 (or below the spikes, of which a row's weights take a
# few hundredths) is below 2e-3.  f32 pools: sums of 4 to 8 at a time and fused multiply-adds,
# 16 * 2^-24 * 13 in a score, so 1e-5 and below.
TOL = {"f32": 1e-5, "f16": 2e-3, "bf16": 2e-3}


class Case:
    """Sequences of `lens` tokens of which the last new[s] (default 1) ask: queries, pools, tables.

    Rows that none of a sequence's new tokens attends to are NaN in K and V, blocks without such
    a row have the table entry -1.  Rows at the masks' borders, the oldest token of the first
    and the last new token's window, the last sink, the newest token, hold values of `spike`:
    one row too few shows."""

    def __init__(self, seed, lens, window, sinks, hq, hkv, d, bs, dtype, new=None, spike=20.0, extra_width=0):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.window, self.sinks, self.bs, self.d, self.dtype = lens, window, sinks, bs, d, dtype
        self.new = new or [min(n, 1) for n in lens]
        self.hq, self.hkv, self.scale, self.max_len = hq, hkv, d ** -0.5, max(lens + [0])
        width = max(1, -(-self.max_len // bs)) + extra_width
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.seen, places = [], []
        for s, (n, m) in enumerate(zip(lens, self.new)):
            rows = np.unique(np.concatenate([np.zeros(0, np.int64)] + [step_model.seen(p, window, sinks) for p in range(n - m, n)]))
            self.seen.append(rows)
            places += [(s, int(b)) for b in np.unique(rows // bs)]
        self.blocks = max(2, int(len(places) * 1.25))
        perm = torch.randperm(self.blocks, generator=gen)
        for i, (s, b) in enumerate(places):
            self.tables[s, b] = perm[i]
        self.k, self.v = (torch.full((self.blocks, hkv, bs, d), float("nan")) for _ in range(2))
        for s, rows in enumerate(self.seen):
            n, m = lens[s], self.new[s]
            at = torch.from_numpy(rows)
            k, v = (torch.randn(len(rows), hkv, d, generator=gen) for _ in range(2))
            border = np.isin(rows, [n - m - window + 1, n - window, sinks - 1, n - 1, n - m])
            v[torch.from_numpy(border)] *= spike
            block = self.tables[s].long()[at // bs]
            self.k[block, :, at % bs], self.v[block, :, at % bs] = k, v
        self.k, self.v = self.k.to(DT[dtype]), self.v.to(DT[dtype])
        tokens = sum(self.new) if new else len(lens)
        self.q = torch.randn(tokens, hq, d, generator=gen).to(DT[dtype])
        self.start = torch.tensor([0] + np.cumsum(self.new).tolist(), dtype=torch.int32) if new else None

    def reference(self):
        """[tokens, hq, d]; rows of empty sequences are zeros."""
        out = np.zeros(self.q.shape)
        group = self.hq // self.hkv
        for s, rows in enumerate(self.seen):
            if self.lens[s] == 0:
                continue
            at = torch.from_numpy(rows)
            block = self.tables[s].long()[at // self.bs]
            k, v = (x[block, :, at % self.bs].double().numpy() for x in (self.k, self.v))   # [rows, hkv, d]
            first = int(self.start[s]) if self.start is not None else s
            for i in range(self.new[s]):
                p = self.lens[s] - self.new[s] + i
                mine = (rows <= p) & ((rows > p - self.window) | (rows < self.sinks))
                q = self.q[first + i].double().numpy().reshape(self.hkv, group, self.d)
                x = np.einsum("hgd,nhd->hgn", q, k[mine]) * self.scale
                e = np.exp(x - x.max(-1, keepdims=True))
                out[first + i] = np.einsum("hgn,nhd->hgd", e / e.sum(-1, keepdims=True), v[mine]).reshape(self.hq, self.d)
        return out

    def cuda(self):
        for name in ("k", "v", "q", "tables", "start"):
            x = getattr(self, name)
            setattr(self, "g_" + name, None if x is None else x.cuda())
        self.g_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self

    def check(self, out, ref=None):
        """Whether the outputs are within TOL, and the rounding of their own type."""
        ref = self.reference() if ref is None else ref
        got = out.double().cpu().numpy()
        tol = TOL[self.dtype] * max(1.0, np.abs(ref).max() / 5)
        half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[out.dtype]
        bad = ~(np.abs(got - ref) <= tol + half * (np.abs(ref) + tol))
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[0][:4], float(np.nanmax(np.abs(got - ref))))
