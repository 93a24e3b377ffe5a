"""A small paged 4-bit cache for the tests: sequences of random keys and values, quantised by the oracle and
laid out in the library's tiles; every byte that holds no token is random (infinite and NaN scales among them)."""
from __future__ import annotations

import numpy as np

from oracle import hadamard as Hd
from oracle import kv4 as O


def signs_of(D: int, seed: int = 0) -> np.ndarray:
    return (1 - 2 * np.random.default_rng(seed + 77).integers(0, 2, D)).astype(np.int8)


class Scene:
    def __init__(self, lens, new, *, heads=2, D=64, G=32, page=32, rotate=True, seed=0, k_scale=1.0, v_scale=1.0,
                 spare=2, outliers=True):
        g = np.random.default_rng(seed)
        self.lens, self.new = np.asarray(lens, np.int32), np.asarray(new, np.int32)
        self.heads, self.D, self.G, self.page, self.rotate = heads, D, G, page, rotate
        self.signs = signs_of(D, seed) if rotate else None
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1])
        per = [-(-int(n) // page) for n in self.lens]
        self.cols = max(per + [1])
        self.pages = sum(per) + spare
        order = g.permutation(self.pages).astype(np.int32)
        self.table = g.integers(-5, self.pages + 9, (len(self.lens), self.cols)).astype(np.int32)  # never read
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.tb = O.tile_bytes(D, G)
        self.stale = g.integers(0, 256, (self.pages, heads, page // 32, self.tb), dtype=np.uint8)
        hot = np.where(g.random(D) < 0.05, 15.0, 1.0) if outliers else np.ones(D)
        # fp32 values that bf16 holds exactly, so that either input type sees the same rows
        self.k = [self.bf16(g.standard_normal((n, heads, D)) * hot * k_scale) for n in self.lens]
        self.v = [self.bf16((g.standard_normal((n, heads, D)) + 0.25) * v_scale) for n in self.lens]
        self._quantise()

    @staticmethod
    def bf16(x):
        import torch
        return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()

    def _quantise(self):
        """Codes, scales and the values that they stand for, in the cache's basis, sequence by sequence."""
        D, G = self.D, self.G
        self.codes = []
        for k, v in zip(self.k, self.v):
            both = []
            for x in (k, v):
                c, s = O.quantise_rows(x.reshape(-1, D), G, self.signs, self.rotate) if x.size else (
                    np.zeros((0, D), np.int8), np.zeros((0, D // G), np.float16))
                both += [c.reshape(x.shape), s.reshape(*x.shape[:2], D // G)]
            self.codes.append(both)
        self.keys = [O.dequantise(c[0], c[1], G) for c in self.codes]
        self.values = [O.dequantise(c[2], c[3], G) for c in self.codes]

    def data(self, held=None) -> np.ndarray:
        """The cache's bytes with the first held[b] tokens of each sequence in place (default: all)."""
        out = self.stale.copy()
        held = self.lens if held is None else held
        for b, n in enumerate(held):
            for t0 in range(0, int(n), 32):
                page, tile = self.table[b, t0 // self.page], t0 % self.page // 32
                m = min(32, int(n) - t0)
                for h in range(self.heads):
                    parts = list(O.unpack_tile(out[page, h, tile], self.D, self.G))
                    for i, x in enumerate(self.codes[b]):
                        parts[i][:m] = x[t0:t0 + m, h]
                    out[page, h, tile] = O.pack_tile(*parts, self.G)
        return out

    def before(self):
        """Tokens of each sequence that are not new."""
        return self.lens - self.new

    def rows(self, which):
        """The new tokens' rows [T, heads, D] of self.k or self.v, packed."""
        return np.concatenate([x[len(x) - n:] if n else x[:0] for x, n in zip(which, self.new)])

    def queries(self, share, seed=1, std=1.0):
        g = np.random.default_rng(seed)
        return self.bf16(g.standard_normal((self.T, self.heads * share, self.D)) * std)

    def rotated(self, x):
        return np.asarray(x, np.float64) if not self.rotate else Hd.rht_apply(
            np.asarray(x, np.float64).reshape(-1, self.D), self.signs).reshape(x.shape)

    def back(self, x):
        return x if not self.rotate else Hd.rht_apply(x.reshape(-1, self.D), self.signs, inverse=True).reshape(x.shape)

    # ---- on the device
    def cache(self, lib, held=None):
        import torch
        self.plan = lib.Plan.rht(self.D, self.signs) if self.rotate else None
        return lib.KV4Cache(torch.from_numpy(self.data(held)).cuda(), self.D, self.G, k_plan=self.plan, v_plan=self.plan)

    def where(self):
        import torch
        return tuple(torch.from_numpy(x).cuda() for x in (self.table, self.lens, self.cu))

    # ---- what the attention has to give
    def check_attention(self, got, q, *, scale=None, causal=True, window=0, absent=None, what=""):
        """got [T, Hq, D] (bf16, as float64) against the oracle, element by element."""
        scale = self.D ** -0.5 if scale is None else scale
        kw = dict(scale=scale, causal=causal, window=window, absent=absent)
        qr = self.rotated(q)
        with np.errstate(invalid="ignore"):
            ref = self.back(O.attention(qr, self.keys, self.values, self.lens, self.cu, **kw))
            bound = O.attention_bound(qr, self.keys, self.values, self.lens, self.cu, unrotate=self.rotate, **kw)
        bound = bound + (np.abs(ref) + bound) * 2.0 ** -8 + 1e-30
        off = np.abs(got - ref)
        # (a group whose scale overflowed stands for NaN, in the rows that see it)
        bad = ~(off <= bound) & ~(np.isnan(got) & np.isnan(ref))
        assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(off / bound)), np.argwhere(bad)[:3].tolist())
        # The bound above is a worst case. Over all elements the roundings are random: the output's alone are
        # 2^-8 / sqrt(3) of a value at most, and those inside (2^-11 steps, averaged) stay below as much again.
        fine = np.isfinite(ref)
        norm = np.linalg.norm(ref[fine])
        assert np.linalg.norm((got - ref)[fine]) <= 2.0 ** -8 * norm + 1e-30, (what, np.linalg.norm((got - ref)[fine]) / norm)
        return ref, bound
