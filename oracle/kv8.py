"""fp64 model of the 8-bit K/V cache (TEST INFRASTRUCTURE ONLY).

E4M3 values with a power-of-two scale for each block of 64 tokens of a (layer, slot, K/V
head), K and V apart; softmax attention over what is stored. Written from the definition in
include/vla.h, token by token and row by row.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
MIN_EXP = -60


def e4m3_round(x):
    """Nearest E4M3 value, ties to even, of |x| <= 448 (sign, 4 exponent bits with bias 7, 3
    mantissa bits; steps of 2^-9 below 2^-6)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)                       # |x| = m 2^e, m in [0.5, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(x / step) * step          # rint: ties to even


def block_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-60 with amax / s <= 448."""
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Kv8Model:
    def __init__(self, n_layers, n_kv_heads, head_dim, capacity, n_slots):
        self.L, self.kv, self.D, self.cap, self.S = n_layers, n_kv_heads, head_dim, capacity, n_slots
        nb = -(-capacity // BLOCK)
        # quantised values (before the scale) and scales, index 0: K, 1: V
        self.q = np.zeros((2, n_layers, n_slots, n_kv_heads, nb * BLOCK, head_dim))
        self.s = np.full((2, n_layers, n_slots, n_kv_heads, nb), 2.0 ** MIN_EXP)

    def write(self, K, V, pos=None, count=None, slots=None, layer=0):
        """K, V: float64 [n, batch, n_tokens, kv * D] of bf16 values."""
        n, B, T = K.shape[:3]
        for b in range(B):
            slot = b if slots is None else int(slots[b])
            p = 0 if pos is None else int(pos[b])
            c = T if count is None else int(count[b])
            for l in range(n):
                for h in range(self.kv):
                    x = np.stack([a[l, b, :c, h * self.D:(h + 1) * self.D] for a in (K, V)])
                    self._write_row(layer + l, slot, h, p, x)

    def _write_row(self, l, slot, h, pos, x):
        n = x.shape[1]
        bad = ~np.isfinite(x).all(axis=(0, 2))           # tokens stored as K = NaN, V = 0
        for j in range(pos // BLOCK, -(-(pos + n) // BLOCK)):
            lo, hi = max(pos, j * BLOCK), min(pos + n, (j + 1) * BLOCK)
            if lo >= hi:
                continue
            new, nb = x[:, lo - pos:hi - pos], bad[lo - pos:hi - pos]
            for w in range(2):
                good = new[w][~nb]
                s = block_scale(np.abs(good).max() if good.size else 0.0)
                if lo > j * BLOCK:                       # kept tokens: the scale can only grow
                    s = max(s, self.s[w, l, slot, h, j])
                    kept = self.q[w, l, slot, h, j * BLOCK:lo]
                    kept[:] = e4m3_round(kept * (self.s[w, l, slot, h, j] / s))
                self.s[w, l, slot, h, j] = s
                rows = np.where(nb[:, None], 0.0, new[w])
                out = e4m3_round(rows / s)
                out[nb] = np.nan if w == 0 else 0.0
                self.q[w, l, slot, h, lo:hi] = out

    def values(self, w, l, slot, h):
        """Stored values [tokens, D] of K (w = 0) or V (1)."""
        return self.q[w, l, slot, h] * np.repeat(self.s[w, l, slot, h], BLOCK)[:, None]

    def read(self, w, n_tokens, pos=None, count=None, slots=None, layer=0, n_layers=None, batch=None, fill=0.0):
        n = self.L - layer if n_layers is None else n_layers
        B = batch if batch is not None else len(next(a for a in (slots, pos, count) if a is not None))
        out = np.full((n, B, n_tokens, self.kv * self.D), fill)
        for b in range(B):
            p = 0 if pos is None else int(pos[b])
            c = n_tokens if count is None else int(count[b])
            for l in range(n):
                for h in range(self.kv):
                    x = self.values(w, layer + l, b if slots is None else int(slots[b]), h)
                    out[l, b, :c, h * self.D:(h + 1) * self.D] = x[p:p + c]
        return out

    def attend(self, q, kv_len, layer=0, slots=None, q_pos=None, q_count=None, causal=False, window=0, scale=None,
               fill=0.0):
        """q: float64 [batch, n_q, H, D]. Returns out (rows behind q_count: `fill`), the natural
        log of the softmax sums and, for error bounds, the weighted mean of |v|, the largest sum
        of |q_d k_d| of a visible key (mag[0]) and of max |q| |k_d| (mag[1]), and n * the largest
        softmax weight * V scale of n keys."""
        B, nq, H, D = q.shape
        scale = 1.0 / np.sqrt(D) if scale is None else scale
        out = np.full((B, nq, H, D), fill)
        mean_v = np.zeros((B, nq, H, D))
        mag = np.zeros((2, B, nq, H))
        lse = np.full((B, nq, H), -np.inf)
        top = np.zeros((B, nq, H))
        for b in range(B):
            slot = b if slots is None else int(slots[b])
            n = int(kv_len[b])
            cnt = nq if q_count is None else int(q_count[b])
            p0 = n - cnt if q_pos is None else int(q_pos[b])
            for h in range(H):
                g = h // (H // self.kv)
                sv = np.repeat(self.s[1, layer, slot, g], BLOCK)[:n]
                k, v = self.values(0, layer, slot, g)[:n], self.values(1, layer, slot, g)[:n]
                for i in range(cnt):
                    hi = min(n, p0 + i + 1) if causal else n
                    lo = max(0, p0 + i - window + 1) if window else 0
                    if lo >= hi:
                        out[b, i, h] = 0.0
                        continue
                    x = scale * (k[lo:hi] @ q[b, i, h])
                    m = x.max()
                    e = np.exp(x - m)
                    out[b, i, h] = e @ v[lo:hi] / e.sum()
                    mean_v[b, i, h] = e @ np.abs(v[lo:hi]) / e.sum()
                    mag[0, b, i, h] = (np.abs(k[lo:hi]) @ np.abs(q[b, i, h])).max()
                    mag[1, b, i, h] = np.abs(k[lo:hi]).sum(1).max() * np.abs(q[b, i, h]).max()
                    lse[b, i, h] = m + np.log(e.sum())
                    top[b, i, h] = (hi - lo) * (e * sv[lo:hi]).max() / e.sum()
        return out, lse, mean_v, mag, top
