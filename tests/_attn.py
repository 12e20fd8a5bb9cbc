"""Seeded inputs of the attention-side tests and their tolerances."""
import numpy as np

import synth
from oracle import attn as A
from oracle import formats as F

U_BF16 = 2.0 ** -8       # half a step, relative, of bf16 and fp16
U_F16 = 2.0 ** -11
U_F32 = 2.0 ** -24


def rng(*key):
    return np.random.default_rng(list(key))


def bits(x):
    """bf16 bits of float64 values."""
    return synth.bf16_bits(x)


def val(b):
    return F.bf16_to_f64(b)


class CacheCase:
    """Random cache contents: every byte of the arrays random (so slots that
    nobody wrote hold anything, NaN scales included), then `lens` tokens of
    each stream written through the oracle."""

    def __init__(self, seed, B, H, D, page, lens, spare=2, extra_pages=1, bad=()):
        g = rng(seed, B, H, D, page)
        self.B, self.H, self.D, self.page, self.lens = B, H, D, page, list(lens)
        per = max(-(-n // page) for n in lens) + extra_pages
        self.pages = B * per + spare
        perm = g.permutation(self.pages)[:B * per].reshape(B, per).astype(np.int32)
        parts = [g.integers(0, 256, (self.pages, H, page, d), dtype=np.uint8)
                 for d in (D // 2, D // 16, D // 2, D // 16)]
        self.ts = np.array([4.5 / 2688, 5.25 / 2688], np.float32)
        self.cache = A.Cache(parts, perm, self.ts, page)
        n = max(lens)
        k, v = bits(g.standard_normal((B, n, H, D))), bits(g.standard_normal((B, n, H, D)))
        self.cache.append(k, v, [0] * B, lens)
        for b, p, entry in bad:                 # entries that name no page
            perm[b, p] = entry

    def device(self, dev):
        c = self.cache
        return [dev(c.k_q), dev(c.k_s), dev(c.v_q), dev(c.v_s), dev(self.ts[:1]), dev(self.ts[1:]),
                dev(c.table)]

    def expect(self, q, q_lens, causal, scale):
        """q bf16 bits [B, Lq, Hq, D] -> (o, spread, |q||k| scale bound) float64, rows behind q_lens zero."""
        o, spread = np.zeros(q.shape), np.zeros(q.shape)
        logit = 0.0
        for b in range(self.B):
            nq, n = q_lens[b], min(self.lens[b], self.cache.table.shape[1] * self.page)
            if nq == 0:
                continue
            k, v, has = self.cache.values(b, n)
            upto = n - (nq - 1 - np.arange(nq)) if causal else np.full(nq, n)
            seen = (np.arange(n)[None] < upto[:, None]) & has[None]
            qv = val(q[b, :nq])
            o[b, :nq], spread[b, :nq] = A.attention(qv, k, v, seen, scale)
            if n:
                logit = max(logit, np.abs(qv).sum(-1).max() * np.abs(k).max() * scale)
        return o, spread, logit


def attn_tol(o, spread, logit, D, L, u_p, vmax):
    """|error| of an output: its own rounding to bf16; the weights' rounding
    (u_p relative, or half a step of fp16's smallest where they are below its
    normal range) and exp's argument (a float32 dot product of D terms, the
    scale and the running maximum: (D + 4) half steps of |logit|; 2^-22 for
    exp2 itself), once in the numerator and once in the sum; float32 sums of
    L terms."""
    rel = u_p + 2 * ((D + 4) * U_F32 * logit + 2.0 ** -22) + 2 * (L + 64) * U_F32
    return U_BF16 * np.abs(o) + rel * spread * (1 + U_BF16) + L * 2.0 ** -25 * vmax * (u_p == U_F16) + 1e-30
