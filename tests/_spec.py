"""Caches of quantized pages and 64-bit results for the tests of speculative decoding.

Tolerance of attention outputs, from the arithmetic alone: a logit is a sum of 128 products
accumulated in fp32, at most one rounding of 2^-23 (truncation) of the partial sums for each
product and for each of the few parts the operands are split into, so it is off by at most
2^-16 S with S = sm_scale * sum_c |q_c k_c| (the fp16 high and low parts carry 22 bits, which
the same bound covers).  A probability is then off by a factor within exp(+-2^-16 S) and the
2^-21 of the exponential and the carried parts; the weighted mean of the values moves by at most twice
the relative error of the weights times the largest distance between values, and its own fp32
sums of n terms add n 2^-24 of the same (n 2^-24 <= 2^-10 for the n <= 16384 tokens used here,
but blockwise sums leave it below 2^-17)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from bit_mixed_precision_channel_b200 import binding as kb
from bit_mixed_precision_channel_b200 import synthetic as syn

from _kv import ocfg, to_dev

D = 128


class Cache:
    """Pages of random keys and values quantized by the oracle, with a window, on the device."""

    def __init__(self, cfg: kb.Config, pages, window, seed: int, distinct: int | None = None, garbage: bool = True,
                 device="cuda", boosts=None):
        """boosts: boosted channels of each head (num_boost of all)."""
        self.cfg, self.rng = cfg, np.random.default_rng(seed)
        rng, H, P, dt = self.rng, cfg.num_kv_heads, cfg.page_tokens, cfg.dtype
        self.B, self.pages, self.window = len(pages), list(pages), list(window)
        self.oc = ocfg(cfg)
        n_used = sum(pages)
        pool_pages = (n_used if distinct is None else min(distinct, max(n_used, 1))) + 2
        self.sigma = np.exp(0.5 * rng.standard_normal((H, D))).astype(np.float32)
        self.pool = np.zeros((pool_pages, H, self.oc.record_bytes), np.uint8)
        for i in range(pool_pages):
            K, V = self.tokens(P), syn.to_bits(rng.standard_normal((P, H, D)).astype(np.float32), dt)
            for h in range(H):
                self.pool[i, h] = oracle.quantize_page_ex(K[:, h], V[:, h], self.oc, boosts and boosts[h])
        if distinct is None:
            order = rng.permutation(pool_pages)
        else:
            order = rng.integers(0, pool_pages, size=n_used)
        self.max_pages = max(max(pages), 1) + 1
        self.table = np.full((self.B, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.res_k = syn.to_bits(rng.standard_normal((self.B, H, P, D)).astype(np.float32), dt)
        self.res_v = syn.to_bits(rng.standard_normal((self.B, H, P, D)).astype(np.float32), dt)
        if garbage:  # window rows behind res_len hold NaN and infinities
            for b, r in enumerate(window):
                self.res_k[b, :, r:] = 0x7fff
                self.res_v[b, :, r:] = 0x7c00 if dt == kb.F16 else 0xff80
        self.dev = device
        self.d = dict(pool=torch.from_numpy(self.pool.reshape(-1)).to(device), page_table=self.ints(self.table),
                      num_pages=self.ints(pages), res_k=to_dev(self.res_k, dt, device),
                      res_v=to_dev(self.res_v, dt, device), res_len=self.ints(window))
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def ints(self, x):
        return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=self.dev)

    def tokens(self, n):
        x = self.rng.standard_normal((n, self.cfg.num_kv_heads, D)).astype(np.float32) * self.sigma
        return syn.to_bits(x, self.cfg.dtype)

    def values(self, n):
        return syn.to_bits(self.rng.standard_normal((n, self.cfg.num_kv_heads, D)).astype(np.float32), self.cfg.dtype)

    def queries(self, *lead, scale=1.0):
        x = scale * self.rng.standard_normal((*lead, self.cfg.num_q_heads, D)).astype(np.float32)
        return syn.to_bits(x, self.cfg.dtype)

    def rows(self, b, h, slots=None):
        """K and V of sequence b, kv head h in 64 bits: the pages in `slots` (all), then the window."""
        ks, vs = [np.zeros((0, D))], [np.zeros((0, D))]
        for s in range(self.pages[b]) if slots is None else slots:
            K, V = oracle.dequantize_page(self.pool[self.table[b, s], h], self.oc)
            ks.append(K)
            vs.append(V)
        r = self.window[b]
        ks.append(syn.from_bits(self.res_k[b, h, :r], self.cfg.dtype).astype(np.float64))
        vs.append(syn.from_bits(self.res_v[b, h, :r], self.cfg.dtype).astype(np.float64))
        return np.concatenate(ks), np.concatenate(vs)


def attend(q, K, V, sees=None, sm_scale=1.0 / math.sqrt(D)):
    """softmax(sm_scale q K^T) V in 64 bits for one row, and the tolerance derived above."""
    if sees is not None:
        K, V = K[sees], V[sees]
    if not len(K):
        return np.zeros(D), 0.0
    z = K @ q * sm_scale
    p = np.exp(z - z.max())
    o = p @ V / p.sum()
    S = abs(sm_scale) * (np.abs(K) @ np.abs(q)).max()
    return o, (2 * (2.0 ** -16 * S + 2.0 ** -20) + 2.0 ** -17) * (V.max() - V.min() + np.abs(V).max())


def assert_row(got, want, tol, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got.astype(np.float64) - want).max()
    assert off <= tol, f"{what}: off by {off:.3e}, at most {tol:.3e} by arithmetic"


def tree_mask(rng, B, T, chain=False):
    """sees [B][T][T]: a node sees itself and its ancestors."""
    sees = np.zeros((B, T, T), bool)
    for i in range(T):
        for b in range(B):
            if i:
                sees[b, i] = sees[b, i - 1 if chain else int(rng.integers(max(0, i - 5), i))]
            sees[b, i, i] = True
    return sees


def pack_mask(sees):
    B, T, n = sees.shape
    words = np.zeros((B, T, (T + 31) // 32), np.uint32)
    for j in range(n):
        words[:, :, j // 32] |= sees[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return words.view(np.int32)
