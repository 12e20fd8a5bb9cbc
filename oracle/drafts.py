"""A checked step of drafted tokens in float64 and whole numbers, from the
definitions: the linear of 8-bit codes, the rotation by positions, what a
tree's rows see and which tokens of the cache are kept.

Test infrastructure (see the package docstring).
"""
import numpy as np


def int8_sums(a, w):
    """Exact sums of int8 codes, int64 [M, N] (blocks whose float64 products are whole)."""
    return np.rint(np.asarray(a, np.float64) @ np.asarray(w, np.float64).T).astype(np.int64)


def turn(x, R, rope, freq, scale, pos):
    """x float64 [M, H, D]: the first R elements of every head turned by pos
    freq (rope 1: pairs, 2: halves) and times scale; a negative position: not."""
    out = np.array(x, np.float64)
    u, v = (slice(0, R, 2), slice(1, R, 2)) if rope == 1 else (slice(0, R // 2), slice(R // 2, R))
    for m, p in enumerate(np.asarray(pos, np.int64)):
        if p < 0:
            continue
        a = float(p) * np.asarray(freq, np.float64)
        z = (out[m][:, u] + 1j * out[m][:, v]) * (scale * np.exp(1j * a))
        out[m][:, u], out[m][:, v] = z.real, z.imag
    return out


def frequencies(R, base, stretch, factor, original=0.0, fast=32.0, slow=1.0):
    """(f64 [R / 2], scale): stretch 0 none, 1 linear, 2 of the base, 3 a ramp
    between pairs that turn `fast` and `slow` times over the original context."""
    if stretch == 2:
        base = base * factor ** (R / (R - 2))
    f = np.array([base ** (-2.0 * i / R) for i in range(R // 2)])
    if stretch == 1:
        return f / factor, 1.0
    if stretch != 3:
        return f, 1.0
    at = lambda turns: R * np.log(original / (turns * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
    low, high = max(np.floor(at(fast)), 0.0), min(np.ceil(at(slow)), R - 1.0)
    high = max(high, low + 0.001)
    share = np.clip((np.arange(R // 2) - low) / (high - low), 0.0, 1.0)
    return f * (1 - share) + f / factor * share, (0.1 * np.log(factor) + 1.0 if factor > 1 else 1.0)


def ancestors(parent):
    """bool [T, T]: j is i or an ancestor of i; parent[i] < i, or negative: none."""
    T = len(parent)
    seen = np.zeros((T, T), bool)
    for i, p in enumerate(parent):
        seen[i, i] = True
        if p >= 0:
            seen[i] |= seen[p]
    return seen


def words(seen):
    """bool [..., T, T] -> int64 [..., T, ceil(T / 64)], bit j % 64 of word j / 64."""
    T = seen.shape[-1]
    W = -(-T // 64)
    bits = np.zeros(seen.shape[:-1] + (W * 64,), np.uint64)
    bits[..., :T] = seen
    at = np.uint64(1) << np.arange(64, dtype=np.uint64)
    return (bits.reshape(seen.shape[:-1] + (W, 64)) * at).sum(-1, dtype=np.uint64).view(np.int64)


def tree_sees(seen, nodes, n):
    """bool [nodes, n]: what the rows of a stream of n positions see, the last
    `nodes` of them being their own (positions below zero do not exist)."""
    first = n - nodes
    out = np.zeros((nodes, n), bool)
    for t in range(nodes):
        for p in range(n):
            out[t, p] = p < first or seen[t, p - first]
    return out


def keep(cache, start, path, count):
    """Move the tokens of cache (oracle.attn.Cache), all read before any is written."""
    parts = (cache.k_q, cache.k_s, cache.v_q, cache.v_s)
    for b in range(len(start)):
        held = []
        for i in range(count[b]):
            src, dst = cache.slot(b, start[b] + path[b][i]), cache.slot(b, start[b] + i)
            if src is not None and dst is not None:
                held.append((dst, [p[src[0], :, src[1]].copy() for p in parts]))
        for dst, token in held:
            for p, x in zip(parts, token):
                p[dst[0], :, dst[1]] = x


__all__ = ["ancestors", "frequencies", "int8_sums", "keep", "tree_sees", "turn", "words"]
