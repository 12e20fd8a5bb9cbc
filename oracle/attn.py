"""Linear of bf16 rows, head norm with rotation, the NVFP4 key/value cache
and attention, in float64 from their definitions.

Test infrastructure (see the package docstring).  The pages name none of
these; they stand around the quantized linears of a transformer block, and
each is written here as its plain definition.
"""
import numpy as np

from .formats import bf16_to_f64, e2m1_decode, e4m3_decode, f64_to_bf16_rne
from .quant import nvfp4_encode, nvfp4_unpack


def unscaled(codes, scales):
    """E2M1 element times E4M3 group scale, float64, without the tensor scale."""
    v = e2m1_decode(nvfp4_unpack(codes))
    return v * np.repeat(e4m3_decode(scales), 16, axis=-1)


def norm_rope(x, norm, w, b, eps, rope, cos, sin, pos):
    """x float64 [M, H, D]; norm 0 none, 1 RMS, 2 layer; rope 0 none, 1 pairs,
    2 halves; cos, sin [P, D/2]; pos [M] (outside 0..P-1: not turned)."""
    y = np.asarray(x, np.float64)
    if norm == 2:
        y = y - y.mean(-1, keepdims=True)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * w
        if b is not None:
            y = y + b
    if not rope:
        return y
    out = y.copy()
    for m in range(y.shape[0]):
        if not 0 <= pos[m] < len(cos):
            continue
        z = cos[pos[m]].astype(np.float64) + 1j * sin[pos[m]].astype(np.float64)
        if rope == 1:
            t = (y[m, :, 0::2] + 1j * y[m, :, 1::2]) * z
            out[m, :, 0::2], out[m, :, 1::2] = t.real, t.imag
        else:
            h = y.shape[-1] // 2
            t = (y[m, :, :h] + 1j * y[m, :, h:]) * z
            out[m, :, :h], out[m, :, h:] = t.real, t.imag
    return out


class Cache:
    """An NVFP4 key/value cache, token by token: pages of [H][page][D]."""

    def __init__(self, parts, table, ts, page):
        self.k_q, self.k_s, self.v_q, self.v_s = (p.copy() for p in parts)
        self.table, self.ts, self.page = table, ts, page
        self.pages = len(self.k_q)

    def slot(self, b, pos):
        """(page, slot) of a position, or None."""
        if not 0 <= pos < self.table.shape[1] * self.page:
            return None
        p = self.table[b, pos // self.page]
        return (p, pos % self.page) if 0 <= p < self.pages else None

    def append(self, k, v, start, count):
        """k, v bf16 bits [B, T, H, D]."""
        for b in range(len(k)):
            for t in range(count[b]):
                at = self.slot(b, start[b] + t)
                if at is None:
                    continue
                p, s = at
                for x, q, sc, ts in ((k, self.k_q, self.k_s, self.ts[0]), (v, self.v_q, self.v_s, self.ts[1])):
                    code, scale, _ = nvfp4_encode(x[b, t], tscale=ts)
                    q[p, :, s], sc[p, :, s] = code, scale

    def read(self, b, pos):
        """(k, v) float32 [H, D] as the library decodes them before the last rounding."""
        p, s = self.slot(b, pos)
        return [(unscaled(q[p, :, s], sc[p, :, s]).astype(np.float32) * np.float32(ts)).astype(np.float32)
                for q, sc, ts in ((self.k_q, self.k_s, self.ts[0]), (self.v_q, self.v_s, self.ts[1]))]

    def values(self, b, n):
        """(k, v float64 [n, H, D], has [n]): the first n positions, zeros without a slot."""
        H, D = self.k_q.shape[1], self.k_q.shape[3] * 2
        k, v, has = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros(n, bool)
        for j in range(n):
            at = self.slot(b, j)
            if at is None:
                continue
            p, s = at
            has[j] = True
            k[j] = unscaled(self.k_q[p, :, s], self.k_s[p, :, s]) * float(self.ts[0])
            v[j] = unscaled(self.v_q[p, :, s], self.v_s[p, :, s]) * float(self.ts[1])
        return k, v, has


def attention(q, k, v, seen, scale):
    """softmax(scale q k^T) v per query head; q [Lq, Hq, D], k and v [L, Hkv, D],
    seen [Lq, L]; a row that sees nothing gives zeros.  Returns (o [Lq, Hq,
    D], spread): spread = sum p |v| / sum p, what a relative error of the
    weights can move each output by."""
    Lq, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, spread = np.zeros_like(q), np.zeros_like(q)
    for h in range(Hq):
        vh = np.where(seen.any(0)[:, None], v[:, h // G], 0.0)
        kh = np.where(seen.any(0)[:, None], k[:, h // G], 0.0)
        s = np.where(seen, (q[:, h] @ kh.T) * scale, -np.inf)
        m = s.max(-1, keepdims=True, initial=-np.inf)
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        n = p.sum(-1, keepdims=True)
        p = p / np.where(n > 0, n, 1.0)
        o[:, h], spread[:, h] = p @ vh, p @ np.abs(vh)
    return o, spread


__all__ = ["Cache", "attention", "norm_rope", "unscaled", "bf16_to_f64", "f64_to_bf16_rne"]
