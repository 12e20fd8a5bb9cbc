"""Cases that measure the attention-side operators of the library.

Five operators: the linear of a few bf16 rows against an NVFP4 weight
("linear"), the norm of query and key heads with their position rotation
("rope"), new keys and values written into a paged NVFP4 cache and read back
("cache"), attention over such a cache ("attend") and cross attention to an
encoder's states ("cross").

`run` computes each in elementary torch operations in float32, or, where
`own` is true, through the library's calls.  `exact` computes the same
results in float64 from the operators' definitions.
"""
import math

import torch

own = False

PAIRS, HALVES = 1, 2           # position rotation: elements (2i, 2i+1), or (i, i + D/2)
RMS, LAYER = 1, 2              # norm of a head


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the scale and shift rows that a conditioning vector of two prompts (guided and not)
        # gives to one block: 512 -> 6 x 1920, the smallest linear a step calls
        dict(name="linear 2 rows 512-11520", op="linear", M=2, K=512, N=11520, bias=True,
             gelu=False, f32=True),
        # one token through the widest linear, where the weight's bytes are the time
        dict(name="linear 1 row 8192-16384", op="linear", M=1, K=8192, N=16384, bias=False,
             gelu=False, f32=False),
        # sixteen streams decoded together through the down projection of a 2B block
        dict(name="linear 16 rows 7680-1920", op="linear", M=16, K=7680, N=1920, bias=True,
             gelu=False, f32=False),
        # all tokens of a 2B video block: 17776 tokens, 226 of text left unrotated
        dict(name="rope 17776 tokens 30 heads", op="rope", M=17776, Hq=30, Hk=30, D=64,
             norm=LAYER, rope=PAIRS, text=226),
        # nine streams, one token each, grouped heads of 128, root mean square norm
        dict(name="rope 9 tokens 32+8 heads", op="rope", M=9, Hq=32, Hk=8, D=128, norm=RMS,
             rope=HALVES, text=0),
        # one latent frame of a 2B video (1350 tokens) entering the cache of a rollout
        dict(name="cache 1350 tokens 30 heads", op="cache", B=1, T=1350, H=30, D=64, page=64,
             start=12376),
        # one token of each of 37 streams, all at other lengths
        dict(name="cache 37 streams 1 token", op="cache", B=37, T=1, H=8, D=128, page=16,
             start=4000),
        # sixteen long streams, one token each, grouped heads: the cache's bytes are the time
        dict(name="attend 16 x 1 token to 32768", op="attend", B=16, Lq=1, Hq=32, Hkv=8, D=128,
             page=64, len=32768, low=0.5, causal=True),
        # a latent frame of 1350 tokens against the text and nine frames (its own last)
        dict(name="attend 1350 tokens to 12376", op="attend", B=1, Lq=1350, Hq=30, Hkv=30, D=64,
             page=64, len=12376, low=1.0, causal=False),
        # five short ragged streams with seven tokens each (drafted tokens being checked)
        dict(name="attend 5 x 7 tokens to 4099", op="attend", B=5, Lq=7, Hq=24, Hkv=8, D=64,
             page=16, len=4099, low=0.01, causal=True),
        # every video token against the text encoder's 226 states
        dict(name="cross 17550 tokens to 226", op="cross", B=1, Lq=17550, Lk=226, Hq=30, Hkv=30,
             D=64, low=1.0),
        # one decoder token of each of 24 requests against encoder states of ragged lengths
        dict(name="cross 24 x 1 token to 1500", op="cross", B=24, Lq=1, Lk=1500, Hq=20, Hkv=20,
             D=64, low=0.2),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "rope", "cache", "attend", "cross"])
    if op == "linear":
        K = 16 * _log(rng, 4, 1024)
        N = min(_log(rng, 16, 32768), 8192 * 16384 // K)
        return dict(op=op, M=_log(rng, 1, 32), K=K, N=N, bias=rng.random() < 0.5,
                    gelu=rng.random() < 0.3, f32=rng.random() < 0.3)
    if op == "rope":
        M, D = _log(rng, 1, 17776), rng.choice([32, 64, 80, 128, 256])
        Hq = max(1, min(_log(rng, 1, 64), 17776 * 30 * 64 // (M * D)))
        return dict(op=op, M=M, Hq=Hq, Hk=max(1, Hq // rng.choice([1, 2, 4, 8])), D=D,
                    norm=rng.choice([RMS, LAYER]), rope=rng.choice([PAIRS, HALVES]),
                    text=rng.choice([0, M // 50]))
    D = rng.choice([64, 128])
    if op == "cache":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=_log(rng, 1, max(2, 1350 // B)), H=rng.randint(1, 1920 // D),
                    D=D, page=rng.choice([16, 32, 64, 128]), start=rng.randint(0, 20000))
    G = rng.choice([1, 1, 2, 3, 4, 8])
    if op == "attend":
        B, Lq = _log(rng, 1, 16), _log(rng, 1, 1350)
        H = rng.randint(1, 8)
        pairs = 32_000_000_000 // (B * H * G * D)              # query-key pairs of a head, at most
        Lq = min(Lq, math.isqrt(pairs))
        length = _log(rng, max(16, Lq), 32768)
        length = max(Lq, min(length, pairs // Lq, 4_000_000 // (B * H)))
        return dict(op=op, B=B, Lq=Lq, Hq=H * G, Hkv=H, D=D, page=rng.choice([16, 32, 64, 128]),
                    len=length, low=rng.choice([0.05, 0.5, 1.0]), causal=rng.random() < 0.5)
    B, Lk = _log(rng, 1, 32), _log(rng, 1, 2048)
    H = rng.randint(1, 30 * 64 // (D * G))
    Lq = max(1, min(_log(rng, 1, 17550), 17550 // B, 17550 * 226 * 1920 // (B * Lk * H * G * D)))
    return dict(op=op, B=B, Lq=Lq, Lk=Lk, Hq=H * G, Hkv=H, D=D, low=rng.choice([0.2, 0.7, 1.0]))


# ------------------------------------------------- NVFP4 in torch operations --

def _e2m1(a):
    """E2M1 magnitude codes of a >= 0: nearest, ties to the even code, saturating at 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)).to(torch.uint8)


def _encode(x, ts):
    """NVFP4 codes [..., D/2] and scales [..., D/16] of float32 x [..., D], tensor scale ts."""
    g = x.unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1)
    r = torch.where(ts == 0, ts, 1.0 / (6.0 * ts))
    s = (amax * r).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = s.float() * ts
    inv = torch.where(t == 0, t, 1.0 / t)
    v = g * inv[..., None]
    code = _e2m1(v.abs()) + (v.signbit().to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(codes, scales):
    """Element times group scale (float32, exact), without the tensor scale."""
    table = torch.tensor(_MAGS + tuple(-m for m in _MAGS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = scales.view(torch.float8_e4m3fn).float()
    return (table[c].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------- prepare --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lens(g, B, longest, low):
    """Lengths between low x longest and longest, the longest among them (int32)."""
    n = torch.rand(B, generator=g, device="cuda")
    n = ((low + (1.0 - low) * n) * longest).round().clamp(1, longest).to(torch.int32)
    n[0] = longest
    return n


def prepare(case, seed):
    g, dev, c = _gen(seed), "cuda", dict(case)
    normal = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        x = normal(M, K)
        x[:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]] *= 30.0  # outlier columns
        w = (normal(N, K) * 0.02).bfloat16().float()
        c["w_ts"] = (w.abs().amax() / 2688.0).reshape(1)
        c["w_q"], c["w_s"] = _encode(w, c["w_ts"])
        c["x"] = x.bfloat16()
        c["b"] = (normal(N) * 0.1).bfloat16() if c["bias"] else None
        c["y"] = torch.empty((M, N), device=dev, dtype=torch.float32 if c["f32"] else torch.bfloat16)
    elif c["op"] == "rope":
        M, D = c["M"], c["D"]
        nq, nk = c["Hq"] * D, c["Hk"] * D
        qkv = (normal(M, nq + 2 * nk) * 2.0).bfloat16()     # one projection: queries, keys, values
        c["q"], c["k"] = qkv[:, :nq], qkv[:, nq:nq + nk]
        for n in ("q_w", "k_w"):
            c[n] = (1.0 + 0.2 * normal(D)).bfloat16()
        for n in ("q_b", "k_b"):
            c[n] = (0.1 * normal(D)).bfloat16() if c["norm"] == LAYER else None
        # a program's tables: the angles of every position, in 64 bits, rounded to float32
        freq = 10000.0 ** (-torch.arange(D // 2, device=dev, dtype=torch.float64) / (D // 2))
        first = int(torch.randint(0, 4096, (1,), generator=g, device=dev))
        a = (first + torch.arange(M, device=dev, dtype=torch.float64))[:, None] * freq
        c["cos"], c["sin"] = a.cos().float(), a.sin().float()
        pos = torch.arange(M, device=dev, dtype=torch.int32) - c["text"]
        c["pos"] = torch.where(pos < 0, torch.full_like(pos, -1), pos)
        c["q_out"] = torch.empty((M, c["Hq"] * D), device=dev, dtype=torch.bfloat16)
        c["k_out"] = torch.empty((M, c["Hk"] * D), device=dev, dtype=torch.bfloat16)
    elif c["op"] in ("cache", "attend"):
        B, D, page = c["B"], c["D"], c["page"]
        H = c["H"] if c["op"] == "cache" else c["Hkv"]
        if c["op"] == "cache":
            c["start_at"] = (c["start"] + torch.randint(0, 3 * page, (B,), generator=g, device=dev)).to(torch.int32)
            longest = c["start"] + 3 * page + c["T"]
        else:
            longest = c["len"]
            c["lens"] = _lens(g, B, longest, c["low"]).clamp(min=min(c["Lq"], longest))
        per = -(-longest // page)
        c["pages"] = B * per + 3
        c["table"] = torch.randperm(c["pages"], generator=g, device=dev)[:B * per].reshape(B, per).to(torch.int32)
        ts = torch.tensor([5.0 / 2688.0], device=dev)      # calibrated: a largest value of about 5
        c["k_ts"], c["v_ts"] = ts, ts.clone()
        if c["op"] == "cache":
            # slots that nobody has written hold any bytes
            for n, d in (("kq", D // 2), ("ks", D // 16), ("vq", D // 2), ("vs", D // 16)):
                c[n] = torch.randint(0, 256, (c["pages"], H, page, d), generator=g, device=dev, dtype=torch.uint8)
            n = H * D
            qkv = normal(B * c["T"], 3 * n).bfloat16()
            c["k"], c["v"] = qkv[:, n:2 * n], qkv[:, 2 * n:]
            c["k_out"] = torch.empty((B * c["T"], H * D), device=dev, dtype=torch.bfloat16)
            c["v_out"] = torch.empty_like(c["k_out"])
        else:
            for n in ("k", "v"):
                c[n + "q"], c[n + "s"] = _encode(normal(c["pages"], H, page, D).bfloat16().float(), ts)
            c["q"] = normal(B * c["Lq"], c["Hq"] * D).bfloat16()
            c["o"] = torch.empty_like(c["q"])
            c["ws"] = torch.empty(32 << 20, device=dev, dtype=torch.uint8)
    else:
        B, Lq, Lk, D = c["B"], c["Lq"], c["Lk"], c["D"]
        c["q"] = normal(B * Lq, c["Hq"] * D).bfloat16()
        kv = normal(B * Lk, 2 * c["Hkv"] * D).bfloat16()        # keys and values of one projection
        c["k"], c["v"] = kv[:, :c["Hkv"] * D], kv[:, c["Hkv"] * D:]
        c["k_lens"] = _lens(g, B, Lk, c["low"])
        c["o"] = torch.empty_like(c["q"])
        c["ws"] = torch.empty(32 << 20, device=dev, dtype=torch.uint8)
    return c


# -------------------------------------------------------------- plain forms --

def _plain_linear(c):
    w = _decode(c["w_q"], c["w_s"])
    y = (c["x"].float() @ w.t()) * c["w_ts"]
    if c["b"] is not None:
        y = y + c["b"].float()
    if c["gelu"]:
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(c["y"].dtype)


def _plain_norm_rope(c, x, w, b):
    """x: bf16 [M, H, D] -> bf16 [M, H * D]"""
    x = x.float()
    if c["norm"] == LAYER:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    if b is not None:
        x = x + b.float()
    at = c["pos"].clamp(min=0).long()
    turned = (c["pos"] >= 0)[:, None, None]
    cos = torch.where(turned, c["cos"][at][:, None], torch.ones((), device=x.device))
    sin = torch.where(turned, c["sin"][at][:, None], torch.zeros((), device=x.device))
    if c["rope"] == PAIRS:
        u, v = x[..., 0::2], x[..., 1::2]
        y = torch.stack((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = x.chunk(2, -1)
        y = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return y.reshape(x.shape[0], -1).bfloat16()


def _heads(c):
    return c["q"].unflatten(-1, (-1, c["D"])), c["k"].unflatten(-1, (-1, c["D"]))


def _plain_rope(c):
    q, k = _heads(c)
    return _plain_norm_rope(c, q, c["q_w"], c["q_b"]), _plain_norm_rope(c, k, c["k_w"], c["k_b"])


def _slots(c, B, T):
    """Page and slot of each stream's tokens start .. start + T - 1, [B, T] each."""
    at = c["start_at"].long()[:, None] + torch.arange(T, device="cuda")
    return torch.gather(c["table"].long(), 1, at // c["page"]), at % c["page"]


def _plain_cache(c):
    B, T, H, D = c["B"], c["T"], c["H"], c["D"]
    page, slot = _slots(c, B, T)
    out = []
    for n in "kv":
        ts = c[n + "_ts"]
        code, s = _encode(c[n].float().reshape(B, T, H, D), ts)
        c[n + "q"][page, :, slot] = code
        c[n + "s"][page, :, slot] = s
        back = _decode(c[n + "q"][page, :, slot], c[n + "s"][page, :, slot]) * ts
        out.append(back.reshape(B * T, H * D).bfloat16())
    return out


def _cached(c, q, s, table):
    """float32 [B, H, tokens, D] of a cache part, without the tensor scale."""
    x = _decode(q[table], s[table])                     # [B, pages, H, page, D]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_softmax_av(q, k, v, seen, scale):
    """q [B, Hkv, G, Lq, D], k and v [B, Hkv, L, D], seen [B, 1, 1, Lq or 1, L]; float32 or 64"""
    B, H, G, Lq, D = q.shape
    s = (q.reshape(B, H, G * Lq, D) @ k.transpose(-1, -2)).reshape(B, H, G, Lq, -1) * scale
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return (p.reshape(B, H, G * Lq, -1) @ v).reshape(B, H, G, Lq, D)


def _split(x, B, L, H, G, D):
    return x.reshape(B, L, H, G, D).permute(0, 2, 3, 1, 4)


def _joined(o, B, L):
    return o.permute(0, 3, 1, 2, 4).reshape(B * L, -1)


def _plain_attend(c):
    B, Lq, H, D = c["B"], c["Lq"], c["Hkv"], c["D"]
    table = c["table"].long()
    k, v = _cached(c, c["kq"], c["ks"], table), _cached(c, c["vq"], c["vs"], table)
    at = torch.arange(k.shape[2], device=k.device)
    upto = c["lens"].long()[:, None] - (Lq - 1 - torch.arange(Lq, device=k.device) if c["causal"]
                                        else torch.zeros(Lq, device=k.device, dtype=torch.long))
    seen = (at < upto[..., None])[:, None, None]
    v = torch.where((at < c["lens"].long()[:, None])[:, None, :, None], v, torch.zeros((), device=v.device))
    q = _split(c["q"].float(), B, Lq, H, c["Hq"] // H, D)
    o = _plain_softmax_av(q, k, v, seen, c["k_ts"] / math.sqrt(D)) * c["v_ts"]
    return _joined(o, B, Lq).bfloat16()


def _plain_cross(c):
    B, Lq, Lk, H, D = c["B"], c["Lq"], c["Lk"], c["Hkv"], c["D"]
    k, v = (c[n].float().reshape(B, Lk, H, D).transpose(1, 2) for n in "kv")
    seen = (torch.arange(Lk, device=k.device) < c["k_lens"].long()[:, None])[:, None, None, None]
    q = _split(c["q"].float(), B, Lq, H, c["Hq"] // H, D)
    return _joined(_plain_softmax_av(q, k, v, seen, 1.0 / math.sqrt(D)), B, Lq).bfloat16()


# ---------------------------------------------------------------------- run --

def _own(c):
    import mixed_precision_quantized_act_amd as qa
    if c["op"] == "linear":
        qa.qlinear_bf16(c["x"], c["w_q"], c["w_s"], c["w_ts"], c["y"], c["M"], c["N"], c["K"], bias=c["b"],
                        out=qa.OUT_F32 if c["f32"] else qa.OUT_BF16,
                        epi=qa.EPI_GELU_TANH if c["gelu"] else qa.EPI_NONE)
        return c["y"]
    if c["op"] == "rope":
        qa.qk_norm_rope(c["q"], c["k"], c["q_out"], c["k_out"], c["M"], c["Hq"], c["Hk"], c["D"], norm=c["norm"],
                        q_w=c["q_w"], q_b=c["q_b"], k_w=c["k_w"], k_b=c["k_b"], eps=1e-6, rope=c["rope"],
                        cos=c["cos"], sin=c["sin"], pos=c["pos"])
        return c["q_out"], c["k_out"]
    if c["op"] == "cache":
        kv4 = (c["kq"], c["ks"], c["vq"], c["vs"], c["k_ts"], c["v_ts"])
        qa.kv4_append(c["k"], c["v"], *kv4, c["table"], c["start_at"], c["B"], c["T"])
        qa.kv4_read(c["k_out"], c["v_out"], *kv4, c["table"], c["start_at"], c["B"], c["T"])
        return [c["k_out"], c["v_out"]]
    if c["op"] == "attend":
        qa.attn_kv4(c["q"], c["kq"], c["ks"], c["vq"], c["vs"], c["k_ts"], c["v_ts"], c["table"], c["lens"],
                    c["o"], c["B"], c["Lq"], c["Hq"], causal=c["causal"], ws=c["ws"])
        return c["o"]
    qa.attn_cross(c["q"], c["k"], c["v"], c["o"], c["B"], c["Lq"], c["Lk"], c["Hq"], c["Hkv"], c["D"],
                  k_lens=c["k_lens"], ws=c["ws"])
    return c["o"]


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "rope": _plain_rope, "cache": _plain_cache, "attend": _plain_attend,
            "cross": _plain_cross}[state["op"]](state)


# --------------------------------------------------------------------- work --

def _mean_len(longest, low, B):
    """The expected length of _lens: one stream at the longest, the others spread evenly."""
    return (longest + (B - 1) * longest * (1.0 + low) / 2.0) / B


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * 9 / 16 + 2 * M * K + M * N * (4 if c["f32"] else 2) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "rope":
        n = c["M"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 4 * n + (c["M"] - c["text"]) * c["D"] * 4 + 4 * c["M"], "flops": 10 * n}
    if c["op"] == "cache":
        n = 2 * c["B"] * c["T"] * c["H"] * c["D"]
        return {"bytes": n * (2 + 9 / 16 + 2), "flops": 6 * n}
    if c["op"] == "attend":
        B, Lq, D = c["B"], c["Lq"], c["D"]
        mean = _mean_len(c["len"], c["low"], B)
        seen = mean - (Lq - 1) / 2 if c["causal"] else mean
        return {"bytes": B * mean * c["Hkv"] * D * 2 * 9 / 16 + 4 * B * Lq * c["Hq"] * D,
                "flops": 4 * B * Lq * max(seen, 1) * c["Hq"] * D}
    B, Lq, D = c["B"], c["Lq"], c["D"]
    mean = _mean_len(c["Lk"], c["low"], B)
    return {"bytes": 4 * B * mean * c["Hkv"] * D + 4 * B * Lq * c["Hq"] * D,
            "flops": 4 * B * Lq * mean * c["Hq"] * D}


# -------------------------------------------------------------------- exact --

def _value64(codes, scales):
    """NVFP4 values in float64 from the bit fields: E2M1 is sign, two exponent bits and one
    mantissa bit (bias 1), E4M3 four exponent and three mantissa bits (bias 7)."""
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    e, m = (n // 2) % 4, (n % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    mag = torch.where(n >= 8, -mag, mag)
    f = scales.to(torch.int64)
    fe, fm = (f // 8) % 16, (f % 8).double()
    s = torch.where(fe == 0, fm / 8 * 2.0 ** -6, (1.0 + fm / 8) * torch.exp2((fe - 7).double()))
    return mag * s.repeat_interleave(16, -1)


def _nearest(a, table):
    """Index of the entry of a rising table nearest to a, the even one of two as near."""
    table = torch.tensor(table, dtype=torch.float64, device=a.device)
    hi = torch.searchsorted(table, a.contiguous()).clamp(1, len(table) - 1)
    below, above = a - table[hi - 1], table[hi] - a
    return torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


_SCALES = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16)
                                                  for m in range(8)][:-1]


def _stored64(x, ts):
    """What the cache holds of x, as values: each float32 step of the encoding is computed in
    float64 and rounded once, as its definition says."""
    ts = ts.double()
    r = (1.0 / (6.0 * ts).float().double()).float().double()
    g = x.double().unflatten(-1, (-1, 16))
    a = (g.abs().amax(-1) * r).float().double()
    s = torch.tensor(_SCALES, dtype=torch.float64, device=x.device)[_nearest(a, _SCALES)]
    t = (s * ts).float().double()
    inv = torch.where(t == 0, t, 1.0 / t).float().double()
    v = (g * inv[..., None]).float().double()
    mag = torch.tensor(_MAGS, dtype=torch.float64, device=x.device)[_nearest(v.abs(), _MAGS)]
    return (torch.copysign(mag, v) * s[..., None]).flatten(-2) * ts


def _attention64(q, k, v, upto, scale):
    """One softmax per row over the keys before `upto` ([B, Lq]); q [B, Lq, H, G, D], k and v
    [B, L, H, D], float64; one stream at a time."""
    out = torch.zeros_like(q)
    at = torch.arange(k.shape[1], device=k.device)
    for b in range(q.shape[0]):
        logits = torch.einsum("qhgd,khd->hgqk", q[b], k[b]) * scale
        logits = torch.where(at < upto[b][:, None], logits, -math.inf)
        e = torch.exp(logits - logits.amax(-1, keepdim=True).clamp(min=-1e300))
        n = e.sum(-1, keepdim=True)
        out[b] = torch.einsum("hgqk,khd->qhgd", e / torch.where(n > 0, n, 1.0), v[b])
    return out


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "linear":
        y = torch.matmul(c["x"].double(), _value64(c["w_q"], c["w_s"]).t()) * c["w_ts"].double()
        if c["b"] is not None:
            y += c["b"].double()
        if c["gelu"]:
            y = y * 0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
        return y
    if c["op"] == "rope":
        out = []
        for x, n in zip(_heads(c), "qk"):
            x = x.double()
            if c["norm"] == LAYER:
                x = x - x.sum(-1, keepdim=True) / c["D"]
            x = x / ((x ** 2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * c[n + "_w"].double()
            if c["norm"] == LAYER:
                x = x + c[n + "_b"].double()
            at = c["pos"].long().clamp(min=0)
            z = torch.complex(c["cos"].double()[at], c["sin"].double()[at])
            z = torch.where((c["pos"] < 0)[:, None], torch.ones_like(z), z)[:, None]
            if c["rope"] == PAIRS:
                y = torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * z)
            else:
                h = c["D"] // 2
                y = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * z
                y = torch.cat((y.real, y.imag), -1)
            out.append(y.reshape(c["M"], -1))
        return tuple(out)
    if c["op"] == "cache":
        return [_stored64(c["k"], c["k_ts"]), _stored64(c["v"], c["v_ts"])]
    B, Lq, H, D = c["B"], c["Lq"], c["Hkv"], c["D"]
    q = c["q"].double().reshape(B, Lq, H, c["Hq"] // H, D)
    if c["op"] == "cross":
        k, v = (c[n].double().reshape(B, c["Lk"], H, D) for n in "kv")
        upto = c["k_lens"].long()[:, None].expand(B, Lq)
        return _attention64(q, k, v, upto, D ** -0.5).reshape(B * Lq, -1)
    t = c["table"].long()
    k, v = ((_value64(c[n + "q"], c[n + "s"])[t] * c[n + "_ts"].double()).transpose(2, 3).flatten(1, 2) for n in "kv")
    back = torch.arange(Lq - 1, -1, -1, device="cuda") if c["causal"] else torch.zeros(Lq, device="cuda", dtype=torch.long)
    upto = c["lens"].long()[:, None] - back
    return _attention64(q, k, v, upto, D ** -0.5).reshape(B * Lq, -1)
