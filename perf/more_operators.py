"""Cases that measure the operators of a checked step of drafted tokens.

Four operators: the linear of INT8 activations and INT8 weights with a scale
for each token and channel ("w8a8"), the rotation of query and key heads by
positions whose angles are formed in the call ("rope"), attention of a tree of
drafted tokens over a paged NVFP4 cache ("tree") and the move of the accepted
tokens to the front of the drafted ones in that cache ("keep").

`run` computes each in elementary torch operations in float32 (or float64
where float32 loses what matters), or, where `own` is true, through the
library's calls.  `exact` computes the same results in float64 from the
operators' definitions.
"""
import math

import torch

own = False

PAIRS, HALVES = 1, 2           # rotated pairs: elements (2i, 2i+1), or (i, i + R/2)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # every token of a 2B video block through the QKV linear: matrix work alone
        dict(name="w8a8 17776 rows 1920-5760", op="w8a8", M=17776, K=1920, N=5760, bias=True,
             gelu=False, f32=False),
        # the down projection of the same block: long sums, few columns
        dict(name="w8a8 17776 rows 7680-1920", op="w8a8", M=17776, K=7680, N=1920, bias=True,
             gelu=False, f32=False),
        # one latent frame with its activation function, sizes that end inside every tile
        dict(name="w8a8 1350 rows 2000-7777", op="w8a8", M=1350, K=2000, N=7777, bias=True,
             gelu=True, f32=True),
        # a tree of 64 drafted tokens through the up projection, where latency counts
        dict(name="w8a8 64 rows 1920-7680", op="w8a8", M=64, K=1920, N=7680, bias=True, gelu=True,
             f32=False),
        # one token through the widest linear, where the weight's bytes are the time
        dict(name="w8a8 1 row 8192-16384", op="w8a8", M=1, K=8192, N=16384, bias=False, gelu=False,
             f32=False),
        # all tokens of a 2B video block, half of each head turned, 226 of text not
        dict(name="rope 17776 tokens 30+30 heads", op="rope", M=17776, Hq=30, Hk=30, D=64, R=32,
             rope=PAIRS, text=226, far=4096, factor=1.0),
        # nine streams of seven drafted tokens far into a stretched context, grouped heads
        dict(name="rope 63 tokens 32+8 heads", op="rope", M=63, Hq=32, Hk=8, D=128, R=64,
             rope=HALVES, text=0, far=1 << 20, factor=32.0),
        # sixteen long streams, 32 drafted tokens each, grouped heads
        dict(name="tree 16 x 32 tokens to 32768", op="tree", B=16, T=32, Hq=32, Hkv=8, D=128,
             page=64, len=32768, low=0.5, nodes=1.0),
        # five short ragged streams with up to 13 drafted tokens, where latency counts
        dict(name="tree 5 x 13 tokens to 4099", op="tree", B=5, T=13, Hq=24, Hkv=8, D=64, page=16,
             len=4099, low=0.01, nodes=0.5),
        # three streams with wide trees, where the products are the time
        dict(name="tree 3 x 250 tokens to 8191", op="tree", B=3, T=250, Hq=30, Hkv=30, D=64,
             page=32, len=8191, low=0.7, nodes=0.8),
        # the accepted tokens of sixteen checked trees of 32
        dict(name="keep 16 x 32 tokens", op="keep", B=16, T=32, H=8, D=128, page=64, start=2000,
             kept=0.3),
        # one stream whose tree of 250 leaves a long path, many heads
        dict(name="keep 1 x 250 tokens", op="keep", B=1, T=250, H=30, D=64, page=16, start=12376,
             kept=0.4),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["w8a8", "rope", "tree", "keep"])
    if op == "w8a8":
        M, K = _log(rng, 1, 17776), 16 * _log(rng, 4, 512)
        most = 17776 * 1920 * 5760 // (M * K)
        return dict(op=op, M=M, K=K, N=max(1, min(_log(rng, 16, 16384), most)),
                    bias=rng.random() < 0.5, gelu=rng.random() < 0.3, f32=rng.random() < 0.3)
    if op == "rope":
        M, D = _log(rng, 1, 17776), rng.choice([32, 64, 80, 96, 128, 256])
        Hq = max(1, min(_log(rng, 1, 64), 17776 * 30 * 64 // (M * D)))
        return dict(op=op, M=M, Hq=Hq, Hk=max(1, Hq // rng.choice([1, 2, 4, 8])), D=D,
                    R=16 * rng.randint(1, D // 16), rope=rng.choice([PAIRS, HALVES]),
                    text=rng.choice([0, M // 50]), far=_log(rng, 16, 1 << 24),
                    factor=rng.choice([1.0, 1.0, 4.0, 32.0]))
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "keep":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=_log(rng, 1, max(2, min(512, 1350 // B))), H=rng.randint(1, 1920 // D),
                    D=D, page=page, start=rng.randint(0, 2000), kept=rng.choice([0.1, 0.5, 1.0]))
    B, T, H, G = _log(rng, 1, 16), _log(rng, 1, 512), rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4, 8])
    T = min(T, 16384 // (B * G))
    pairs = 16 * 32 * 32 * 128 * 24576
    length = max(T, min(_log(rng, 16, 32768), pairs // (B * H * G * D * T), 4_000_000 // (B * H)))
    return dict(op=op, B=B, T=T, Hq=H * G, Hkv=H, D=D, page=page, len=length,
                low=rng.choice([0.05, 0.5, 1.0]), nodes=rng.choice([0.3, 1.0, 1.0]))


# --------------------------------------------------- formats in torch operations --

def _int8_rows(x):
    """INT8 codes and float32 scales of the rows of x: 127 steps to a row's largest value."""
    s = x.abs().amax(-1) / 127.0
    inv = torch.where(s == 0, s, 1.0 / s)
    return (x * inv[:, None]).round().clamp(-127, 127).to(torch.int8), s


def _e2m1(a):
    """E2M1 magnitude codes of a >= 0: nearest, ties to the even code, saturating at 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)).to(torch.uint8)


def _encode(x, ts):
    """NVFP4 codes [..., D/2] and scales [..., D/16] of float32 x [..., D], tensor scale ts."""
    g = x.unflatten(-1, (-1, 16))
    s = (g.abs().amax(-1) / (6.0 * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
    t = s.float() * ts
    v = g * torch.where(t == 0, t, 1.0 / t)[..., None]
    code = (_e2m1(v.abs()) + (v.signbit().to(torch.uint8) << 3)).flatten(-2)
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


def _between(g, B, most, low, dev="cuda"):
    """B whole numbers between low x most and most, most among them (int32)."""
    n = torch.rand(B, generator=g, device=dev)
    n = ((low + (1.0 - low) * n) * most).round().clamp(1, most).to(torch.int32)
    n[0] = most
    return n


def _ancestors(g, T):
    """[T, T] truth values: node j is i or one of its ancestors, in a random tree whose nodes
    come after their parents (a drafter's: most hang on one of the last few levels)."""
    back = torch.rand(T, generator=g, device="cuda") ** 2 * torch.arange(T, device="cuda") * 0.5
    parent = torch.arange(T, device="cuda") - 1 - back.long()
    seen = torch.eye(T, device="cuda")
    has = parent >= 0
    step = torch.zeros((T, T), device="cuda")
    step[has, parent[has]] = 1.0
    step += seen
    for _ in range(max(1, T.bit_length())):
        step = ((step @ step) > 0).float()
    return step > 0


def _words(seen):
    """Truth values [T, T] as bits of int64 words [T, ceil(T / 64)]."""
    T = seen.shape[0]
    bits = torch.zeros((T, -(-T // 64) * 64), device=seen.device, dtype=torch.int64)
    bits[:, :T] = seen.long()
    at = torch.ones((), device=seen.device, dtype=torch.int64) << torch.arange(64, device=seen.device)
    return (bits.unflatten(-1, (-1, 64)) * at).sum(-1)


def _frequencies(R, factor):
    """Angles per position of the R/2 pairs (float64) and the factor of the turned values: the
    slow half is stretched by `factor`, the fast quarter is not, a ramp between them."""
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    f = 10000.0 ** (-i / (R // 2))
    ramp = ((i / (R // 2) - 0.25) / 0.25).clamp(0, 1)
    return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    g, dev, c = _gen(seed), "cuda", dict(case)
    normal = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    if c["op"] == "w8a8":
        M, N, K = c["M"], c["N"], c["K"]
        x = normal(M, K)
        x[:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]] *= 30.0  # outlier columns
        c["a_q"], c["a_s"] = _int8_rows(x.bfloat16().float())
        c["w_q"], c["w_s"] = _int8_rows((normal(N, K) * 0.02).bfloat16().float())
        c["b"] = (normal(N) * 0.1).bfloat16() if c["bias"] else None
        c["y"] = torch.empty((M, N), device=dev, dtype=torch.float32 if c["f32"] else torch.bfloat16)
        c["ws"] = torch.empty(64 << 20, device=dev, dtype=torch.uint8)
        return c
    if c["op"] == "rope":
        M, D, nq, nk = c["M"], c["D"], c["Hq"] * c["D"], c["Hk"] * c["D"]
        qkv = (normal(M, nq + 2 * nk) * 2.0).bfloat16()     # one projection: queries, keys, values
        c["q"], c["k"] = qkv[:, :nq], qkv[:, nq:nq + nk]
        c["freq"], c["scale"] = _frequencies(c["R"], c["factor"])
        pos = torch.randint(0, c["far"], (M,), generator=g, device=dev, dtype=torch.int32)
        pos[:c["text"]] = -1
        c["pos"] = pos
        c["q_out"] = torch.empty((M, nq), device=dev, dtype=torch.bfloat16)
        c["k_out"] = torch.empty((M, nk), device=dev, dtype=torch.bfloat16)
        return c
    B, T, D, page = c["B"], c["T"], c["D"], c["page"]
    H = c["H"] if c["op"] == "keep" else c["Hkv"]
    if c["op"] == "keep":
        c["start_at"] = (c["start"] + torch.randint(0, 3 * page, (B,), generator=g, device=dev)).to(torch.int32)
        longest = c["start"] + 3 * page + T
    else:
        longest = c["len"]
        c["q_lens"] = _between(g, B, T, c["nodes"])
        c["lens"] = _between(g, B, longest, c["low"]).clamp(min=min(T, longest))
    per = -(-longest // page)
    pages = B * per + 3
    c["table"] = torch.randperm(pages, generator=g, device=dev)[:B * per].reshape(B, per).to(torch.int32)
    ts = torch.tensor([5.0 / 2688.0], device=dev)      # calibrated: a largest value of about 5
    c["k_ts"], c["v_ts"] = ts, ts.clone()
    for n in ("k", "v"):
        c[n + "q"], c[n + "s"] = _encode(normal(pages, H, page, D).bfloat16().float(), ts)
    if c["op"] == "keep":
        # a path: some first nodes in a row, then later ones, none of them among the places it fills
        kept = _between(g, B, max(1, int(c["kept"] * T)), 0.1)
        c["count"] = kept
        at, n = torch.arange(T, device=dev), kept.long()[:, None]
        first = torch.randint(0, 3, (B, 1), generator=g, device=dev)      # (in place already)
        later = n + (torch.rand((B, T), generator=g, device=dev).sort(-1).values * (T - n)).long()
        c["path"] = torch.where((at < first) | (later >= T), at, later).to(torch.int32)
        c["k_out"] = torch.empty((B * T, H * D), device=dev, dtype=torch.bfloat16)
        c["v_out"] = torch.empty_like(c["k_out"])
    else:
        c["tree"] = torch.stack([_words(_ancestors(g, T)) for _ in range(B)])
        c["q"] = normal(B * T, c["Hq"] * D).bfloat16()
        c["o"] = torch.zeros_like(c["q"])              # (rows behind q_lens stay zeros)
        c["ws"] = torch.empty(32 << 20, device=dev, dtype=torch.uint8)
    return c


# -------------------------------------------------------------- plain forms --

def _plain_w8a8(c):
    t = torch.float64 if c["f32"] else torch.float32       # (sums that a float32 output would show)
    y = (c["a_q"].to(t) @ c["w_q"].to(t).t()) * c["w_s"].to(t) * c["a_s"].to(t)[:, None]
    if c["b"] is not None:
        y = y + c["b"].to(t)
    if c["gelu"]:
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(c["y"].dtype)


def _plain_turn(c, x):
    """x: bf16 [M, H D] -> bf16 [M, H D]"""
    R = c["R"]
    x = x.float().unflatten(-1, (-1, c["D"]))
    turned = (c["pos"] >= 0)[:, None, None]
    a = c["pos"].double()[:, None] * c["freq"]             # angles of far positions: 64 bits
    cos, sin = (f(a).float()[:, None] * c["scale"] for f in (torch.cos, torch.sin))
    p = x[..., :R]
    if c["rope"] == PAIRS:
        u, v = p[..., 0::2], p[..., 1::2]
        y = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = p.chunk(2, -1)
        y = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((torch.where(turned, y, p), x[..., R:]), -1).flatten(1).bfloat16()


def _plain_rope(c):
    return _plain_turn(c, c["q"]), _plain_turn(c, c["k"])


def _bits(words, T):
    """Truth values [..., T] of int64 words [..., ceil(T / 64)]."""
    at = torch.arange(64, device=words.device)
    return (((words[..., None] >> at) & 1) != 0).flatten(-2)[..., :T]


def _tree_seen(c, L):
    """[B, T, L] truth values: what each drafted token sees of the cached positions."""
    B, T = c["B"], c["T"]
    first = (c["lens"] - c["q_lens"]).long()[:, None, None]          # position of node 0
    node = torch.arange(L, device="cuda")[None, None] - first        # [B, 1, L]
    bits = _bits(c["tree"], T)
    own_node = (node >= 0) & (node < c["q_lens"].long()[:, None, None])
    at = node.clamp(0, T - 1).expand(B, T, L)
    return (node < 0) | (own_node & torch.gather(bits, 2, at))


def _plain_tree(c):
    B, T, H, D = c["B"], c["T"], c["Hkv"], c["D"]
    G, table = c["Hq"] // H, c["table"].long()
    k, v = (_decode(c[n + "q"][table], c[n + "s"][table]).transpose(1, 2).flatten(2, 3) for n in "kv")
    seen = _tree_seen(c, k.shape[2])[:, None, None]
    q = c["q"].float().reshape(B, T, H, G, D).permute(0, 2, 3, 1, 4)
    s = (q.reshape(B, H, G * T, D) @ k.transpose(-1, -2)).reshape(B, H, G, T, -1)
    s = (s * (c["k_ts"] / math.sqrt(D))).masked_fill(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))                      # (a node sees itself)
    p = p / p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, G * T, -1) @ v).reshape(B, H, G, T, D) * c["v_ts"]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, -1)
    there = torch.arange(T, device="cuda") < c["q_lens"].long()[:, None]
    return torch.where(there[..., None], o, torch.zeros((), device="cuda")).reshape(B * T, -1).bfloat16()


def _slots(c):
    """Page and slot of each stream's positions start .. start + T - 1, [B, T] each."""
    at = c["start_at"].long()[:, None] + torch.arange(c["T"], device="cuda")
    return torch.gather(c["table"].long(), 1, at // c["page"]), at % c["page"]


def _plain_keep(c):
    page, slot = _slots(c)
    moves = torch.arange(c["T"], device="cuda") < c["count"].long()[:, None]
    src = torch.where(moves, c["path"].long(), torch.arange(c["T"], device="cuda"))
    from_page, from_slot = (torch.gather(x, 1, src) for x in (page, slot))
    out = []
    for n in "kv":
        for part in ("q", "s"):
            c[n + part][page, :, slot] = c[n + part][from_page, :, from_slot]
        back = _decode(c[n + "q"][page, :, slot], c[n + "s"][page, :, slot]) * c[n + "_ts"]
        out.append(back.reshape(c["B"] * c["T"], -1).bfloat16())
    return out


# ---------------------------------------------------------------------- run --

def _own(c):
    import mixed_precision_quantized_act_amd as qa
    if c["op"] == "w8a8":
        qa.qlinear_w8a8(c["a_q"], c["a_s"], c["w_q"], c["w_s"], c["y"], c["M"], c["N"], c["K"],
                        bias=c["b"], out=qa.OUT_F32 if c["f32"] else qa.OUT_BF16,
                        epi=qa.EPI_GELU_TANH if c["gelu"] else qa.EPI_NONE, ws=c["ws"])
        return c["y"]
    if c["op"] == "rope":
        qa.qk_rope(c["q"], c["k"], c["q_out"], c["k_out"], c["M"], c["Hq"], c["Hk"], c["D"], c["R"],
                   c["freq"], rope=c["rope"], scale=c["scale"], pos=c["pos"])
        return c["q_out"], c["k_out"]
    kv = (c["kq"], c["ks"], c["vq"], c["vs"])
    if c["op"] == "tree":
        qa.attn_kv4_tree(c["q"], *kv, c["k_ts"], c["v_ts"], c["table"], c["lens"], c["tree"], c["o"],
                         c["B"], c["T"], c["Hq"], q_lens=c["q_lens"], ws=c["ws"])
        return c["o"]
    qa.kv4_keep(*kv, c["table"], c["start_at"], c["path"], c["B"], c["T"], count=c["count"])
    # all drafted positions, moved and not
    qa.kv4_read(c["k_out"], c["v_out"], *kv, c["k_ts"], c["v_ts"], c["table"], c["start_at"], c["B"], c["T"])
    return [c["k_out"], c["v_out"]]


def run(state):
    if own:
        return _own(state)
    return {"w8a8": _plain_w8a8, "rope": _plain_rope, "tree": _plain_tree, "keep": _plain_keep}[state["op"]](state)


# --------------------------------------------------------------------- work --

def _mean(most, low, B):
    """The expected value of _between: the first at the most, the others spread evenly."""
    return (most + (B - 1) * most * (1.0 + low) / 2.0) / B


def work(case):
    c = case
    if c["op"] == "w8a8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * (4 if c["f32"] else 2) + (2 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "rope":
        n = c["M"] * (c["Hq"] + c["Hk"])
        return {"bytes": 4 * n * c["D"] + 4 * c["M"] + 4 * c["R"], "flops": 3 * n * c["R"]}
    if c["op"] == "keep":
        token = 2 * c["H"] * c["D"] * 9 // 16                    # bytes of a cached token
        moved = c["B"] * _mean(max(1, int(c["kept"] * c["T"])), 0.1, c["B"])
        return {"bytes": token * (2 * moved + c["B"] * c["T"]) + 4 * c["B"] * c["T"] * c["H"] * c["D"],
                "flops": 2 * c["B"] * c["T"] * c["H"] * c["D"]}
    B, D = c["B"], c["D"]
    mean, rows = _mean(c["len"], c["low"], B), B * _mean(c["T"], c["nodes"], B)
    return {"bytes": B * mean * c["Hkv"] * D * 2 * 9 / 16 + 4 * rows * c["Hq"] * D + 8 * rows * -(-c["T"] // 64),
            "flops": 4 * rows * max(1.0, mean - c["T"] / 2) * c["Hq"] * D}


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


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "w8a8":
        y = torch.matmul(c["a_q"].double(), c["w_q"].double().t())      # whole numbers below 2^53
        y *= c["a_s"].double()[:, None]
        y *= c["w_s"].double()
        if c["bias"]:
            y += c["b"].double()
        if c["gelu"]:
            y = y * 0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
        return y
    if c["op"] == "rope":
        out, h = [], c["R"] // 2
        z = torch.polar(torch.full((c["M"], h), float(c["scale"]), device="cuda", dtype=torch.float64),
                        c["pos"].double()[:, None] * c["freq"])
        z = torch.where((c["pos"] < 0)[:, None], torch.ones_like(z), z)[:, None]
        for n in ("q", "k"):
            x = c[n].double().unflatten(-1, (-1, c["D"])).clone()
            first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if c["rope"] == PAIRS else \
                (slice(0, h), slice(h, 2 * h))
            y = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
            x[..., first], x[..., second] = y.real, y.imag
            out.append(x.flatten(1))
        return tuple(out)
    B, T, D, page = c["B"], c["T"], c["D"], c["page"]
    table = c["table"].long()
    if c["op"] == "keep":
        H, out = c["H"], []
        for n in "kv":
            x = torch.zeros((B, T, H, D), device="cuda", dtype=torch.float64)
            for b in range(B):
                # the stream's drafted tokens as they lay, then the kept ones in front
                at = int(c["start_at"][b]) + torch.arange(T, device="cuda")
                q, s = (c[n + p][table[b, at // page], :, at % page] for p in "qs")
                was = _value64(q, s) * c[n + "_ts"].double()
                m = int(c["count"][b])
                x[b] = was
                x[b, :m] = was[c["path"][b, :m].long()]
            out.append(x.reshape(B * T, -1))
        return out
    H = c["Hkv"]
    o = torch.zeros((B, T, H, c["Hq"] // H, D), device="cuda", dtype=torch.float64)
    q = c["q"].double().reshape(o.shape)
    for b in range(B):
        n, m = int(c["lens"][b]), int(c["q_lens"][b])
        at = torch.arange(n, device="cuda")
        k, v = (_value64(*(c[x + p][table[b, at // page], :, at % page] for p in "qs")) * c[x + "_ts"].double()
                for x in "kv")                                          # [n, H, D]
        seen = torch.ones((m, n), device="cuda", dtype=torch.bool)
        words = c["tree"][b, :m]
        for j in range(m):
            seen[:, n - m + j] = (words[:, j // 64] >> (j % 64)) & 1 != 0
        for h in range(H):
            logits = torch.einsum("tgd,nd->gtn", q[b, :m, h], k[:, h]) * D ** -0.5
            logits = torch.where(seen, logits, -math.inf)
            e = torch.exp(logits - logits.amax(-1, keepdim=True))
            o[b, :m, h] = torch.einsum("gtn,nd->tgd", e / e.sum(-1, keepdim=True), v[:, h])
    return o.reshape(B * T, -1)
