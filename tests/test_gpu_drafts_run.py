"""Checked steps of drafted tokens as they are used: quantize, project, turn, cache, attend, keep, and the next step on
what was kept.  Every stage against its definition on the stage's own inputs; then the whole step on another stream and
captured, bit by bit."""
import numpy as np
import pytest

from oracle import attn as A
from oracle import drafts as O
from tests._attn import U_BF16, U_F16, U_F32, CacheCase, attn_tol, bits, rng, val
from tests._gpu import dev, host, torch
from tests.test_gpu_qk_rope import _tol as rope_tol

pytestmark = pytest.mark.gpu


def _qa():
    import mixed_precision_quantized_act_amd as qa
    return qa


class Step:
    """Weights, cache and buffers of B streams that check at most T tokens."""

    def __init__(self, seed, B, T, Hq, H, D, R, K, lens, page=32):
        qa, t = _qa(), torch()
        g = rng(731, seed, B, T, Hq, H, D)
        self.B, self.T, self.Hq, self.H, self.D, self.R, self.K, self.g = B, T, Hq, H, D, R, K, g
        self.N = (Hq + 2 * H) * D
        self.case = CacheCase(seed, B, H, D, page, [max(1, n) for n in lens], extra_pages=2 + 3 * T // page)
        self.cache = self.case.device(dev)
        self.w = dev(bits(g.standard_normal((self.N, K)) * 0.08)).view(t.bfloat16)
        self.bias = dev(bits(g.standard_normal(self.N) * 0.1)).view(t.bfloat16)
        self.w_q = t.empty((self.N, K), dtype=t.int8, device="cuda")
        self.w_s = t.empty(self.N, dtype=t.float32, device="cuda")
        qa.act_quant(qa.INT8, self.w, self.w_q, self.w_s)
        self.freq, self.attention = qa.rope_freqs(R, 10000.0, qa.STRETCH_RAMP, factor=8.0, original=4096)
        self.freq = dev(np.asarray(self.freq))

    def inputs(self, lens, q_lens, T, kind="tree"):
        """x, the streams' positions, their tree, the path that is kept and how many of it."""
        t, g, B = torch(), self.g, self.B
        parent = [[-1] + [int(g.integers(-1, i)) for i in range(1, T)] for _ in range(B)]
        depth = np.zeros((B, T), np.int64)
        for b in range(B):
            for i in range(1, T):
                p = parent[b][i]
                depth[b, i] = depth[b, p] + 1 if p >= 0 else 0
        seen = np.stack([O.ancestors(p) for p in parent])
        path, count = np.zeros((B, T), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            at = int(g.integers(0, max(1, q_lens[b])))
            line = [j for j in range(T) if seen[b, at, j]] if q_lens[b] else []
            path[b, :len(line)], count[b] = line, len(line)
        h = dict(T=T, lens=np.asarray(lens, np.int32), q_lens=np.asarray(q_lens, np.int32), seen=seen, path=path, count=count,
                 pos=(np.asarray(lens)[:, None] + depth).astype(np.int32))
        h["x"] = dev(bits(g.standard_normal((B * T, self.K)))).view(t.bfloat16)
        h["d"] = [h["x"]] + [dev(v) for v in (h["pos"].reshape(-1), h["lens"], h["lens"] + h["q_lens"], h["q_lens"],
                                              O.words(seen), path, count)]
        return h

    def buffers(self, T):
        t, M = torch(), self.B * T
        n = _qa().attn_kv4_tree_workspace(self.B, T, self.Hq, self.H, self.D, self.cache[6].shape[1] * self.case.page)
        m = _qa().qlinear_w8a8_workspace(M, self.N, self.K)
        z = lambda *s, dtype=t.bfloat16: t.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        return dict(a_q=z(M, self.K, dtype=t.int8), a_s=z(M, dtype=t.float32), y=z(M, self.N), o=z(M, self.Hq * self.D),
                    ws=t.full((max(n, m, 16),), 0xFF, dtype=t.uint8, device="cuda"))

    def run(self, T, d, f, cache, after=lambda stage: None):
        qa, B = _qa(), self.B
        x, pos, start, lens, q_lens, word, path, count = d
        nq, nk = self.Hq * self.D, self.H * self.D
        y = f["y"]
        q, k, v = y[:, :nq], y[:, nq:nq + nk], y[:, nq + nk:]
        qa.act_quant(qa.INT8, x, f["a_q"], f["a_s"])
        qa.qlinear_w8a8(f["a_q"], f["a_s"], self.w_q, self.w_s, y, B * T, self.N, self.K, bias=self.bias, ws=f["ws"])
        after("linear")
        qa.qk_rope(q, k, q, k, B * T, self.Hq, self.H, self.D, self.R, self.freq, rope=qa.ROPE_HALVES,
                   scale=self.attention, pos=pos)
        after("rope")
        qa.kv4_append(k, v, *cache, start, B, T, count=q_lens)
        after("append")
        qa.attn_kv4_tree(q, *cache, lens, word, f["o"], B, T, self.Hq, q_lens=q_lens, ws=f["ws"])
        after("attention")
        qa.kv4_keep(*cache[:4], cache[6], start, path, B, T, count=count)
        after("keep")

    def checked(self, h):
        """One step, every stage compared."""
        t, T, B, D, Hq, H = torch(), h["T"], self.B, self.D, self.Hq, self.H
        f, c = self.buffers(T), self.case.cache
        M, nq, nk = B * T, Hq * D, H * D
        prior = {}

        def after(stage):
            t.cuda.synchronize()
            y = host(f["y"])
            if stage == "linear":
                a_s, w_s = host(f["a_s"]).astype(np.float64), host(self.w_s).astype(np.float64)
                p = O.int8_sums(host(f["a_q"]), host(self.w_q)) * a_s[:, None] * w_s
                b = val(host(self.bias))
                # the sum rounded to float32, two products, the bias (4 half steps in all), then bf16
                tol = U_BF16 * np.abs(p + b) + 4 * U_F32 * (np.abs(p) + np.abs(b)) * (1 + U_BF16) + 1e-37
                assert np.all(np.abs(val(y) - (p + b)) <= tol)
                prior["y"] = y.copy()
            elif stage == "rope":
                freq, pos = host(self.freq), h["pos"].reshape(-1)
                for n, lo in ((Hq, 0), (H, nq)):
                    x = val(prior["y"][:, lo:lo + n * D].reshape(M, n, D))
                    want = O.turn(x, self.R, 2, freq, np.float64(np.float32(self.attention)), pos)
                    turns = (np.abs(pos) * np.abs(freq).max() / (2 * np.pi) + 1)[:, None, None]
                    got = val(y[:, lo:lo + n * D].reshape(M, n, D))
                    assert np.all(np.abs(got - want) <= rope_tol(want, x, self.attention, turns))
                assert np.array_equal(y[:, nq + nk:], prior["y"][:, nq + nk:])
            elif stage == "append":
                k, v = (np.ascontiguousarray(y[:, lo:lo + nk]).reshape(B, T, H, D) for lo in (nq, nq + nk))
                c.append(k, v, list(h["lens"]), list(h["q_lens"]))
            elif stage == "attention":
                o = val(host(f["o"])).reshape(B, T, Hq, D)
                q = val(np.ascontiguousarray(y[:, :nq])).reshape(B, T, Hq, D)
                for b in range(B):
                    m, n = h["q_lens"][b], h["lens"][b] + h["q_lens"][b]
                    assert np.all(o[b, m:] == 0)                       # as they were
                    if not m:
                        continue
                    k, v, has = c.values(b, n)
                    want, spread = A.attention(q[b, :m], k, v, O.tree_sees(h["seen"][b], m, n) & has[None], D ** -0.5)
                    logit = np.abs(q[b, :m]).sum(-1).max() * np.abs(k).max() * D ** -0.5
                    tol = attn_tol(want, spread, logit, D, n, U_F16, 6 * 448 * float(self.case.ts[1]))
                    assert np.all(np.abs(o[b, :m] - want) <= tol)
            else:
                O.keep(c, h["lens"], h["path"], h["count"])
            for got, want in zip(self.cache, (c.k_q, c.k_s, c.v_q, c.v_s)) if stage in ("append", "keep") else ():
                np.testing.assert_array_equal(host(got), want)

        self.run(T, h["d"], f, self.cache, after)


@pytest.mark.parametrize("B,T,Hq,H,D,R,K", [(3, 9, 6, 2, 64, 32, 320), (2, 33, 4, 4, 128, 128, 208), (2, 70, 8, 2, 64, 64, 128)])
def test_steps(B, T, Hq, H, D, R, K):
    lens = [0, 37, 230][:B]
    s = Step(1, B, T, Hq, H, D, R, K, lens)
    for nodes in (T, T // 2, 1):                       # the last: a single token
        q_lens = [nodes, max(1, nodes - 1), 0][:B]
        h = s.inputs(lens, q_lens, nodes)
        s.checked(h)
        lens = [int(a + b) for a, b in zip(lens, h["count"])]


@pytest.mark.parametrize("B,T,Hq,H,D", [(2, 12, 6, 2, 64), (2, 40, 8, 2, 128)])
def test_a_step_on_another_stream_and_captured(B, T, Hq, H, D):
    """(Where a set's positions were never written their slots hold NaN's scales: bits are compared.)"""
    t = torch()

    def same(o, cache, want):
        pairs = zip([o, *cache], [want[0], *want[1]])
        return all(t.equal(a.contiguous().view(t.uint8), b.contiguous().view(t.uint8)) for a, b in pairs)

    s = Step(2, B, T, Hq, H, D, 32, 192, [300, 41])
    sets = [s.inputs(ln, m, T) for ln, m in (([300, 41], [T, T]), ([0, 200], [T, 3]), ([77, 78], [1, T]), ([150, 20], [T, T - 1]))]
    before = [c.clone() for c in s.cache]
    want = []
    for h in sets:
        cache, f = [c.clone() for c in before], s.buffers(T)
        s.run(T, h["d"], f, cache)
        want.append((f["o"], cache[:4]))
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        cache, f = [c.clone() for c in before], s.buffers(T)
        s.run(T, sets[0]["d"], f, cache)
    side.synchronize()
    assert same(f["o"], cache, want[0])

    held, cache, f = [x.clone() for x in sets[0]["d"]], [c.clone() for c in before], s.buffers(T)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        s.run(T, held, f, cache)
    for i in (0, 1, 2, 3, 1, 0):
        for a, b in zip(held, sets[i]["d"]):
            a.copy_(b)
        for a, b in zip(cache, before):
            a.copy_(b)
        f["o"].zero_()
        graph.replay()
        j = (i + 1) % 4
        other, g = [c.clone() for c in before], s.buffers(T)
        s.run(T, sets[j]["d"], g, other)                               # eager work between the replays
        t.cuda.synchronize()
        assert same(f["o"], cache, want[i]) and same(g["o"], other, want[j])
