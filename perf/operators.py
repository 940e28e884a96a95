"""Timed cases of the decoder-block operators: the residual stream's norms, the rotary split of
the q/k/v product, attention over packed prompts, and the cache held in 4 bits (written, read
back, and attended by single tokens).

``run`` computes one pass: with ``own`` false in plain torch operations (fp32, rounded once at
the end), with ``own`` true through the package's public calls.  ``exact`` gives the same outputs
from the definitions in fp64.

The operators (T tokens, D features per head):

add_norm       Xn = X + alpha . gate * N(Y; post) ; h = N(Xn; weight), N the RMS norm, or the layer
               norm with ``center``; Xn is rounded to X's type before h is taken from it.
rope_qkv       the fp32 product [T, (hq + 2 hk) D] plus bias, q and k rotated by their token's
               angles, split and rounded into q, k, v.
attention      softmax(scale q k^T) v per sequence of a packed batch, hq / hk query heads per k/v
               head; causal: the last query sees the last key.
kv4            tokens' k and v as 4-bit codes with an fp16 scale and zero point per group of a
               head's features (asymmetric, the range holding 0), written into pages and read back.
kv4_attention  one query token per sequence against its tokens in such a cache.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------- #
# Cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one decoded token of a block of width 4096: launch latency
        {"name": "norm_token", "op": "add_norm", "tokens": 1, "d": 4096, "x": "bf16", "y": "f32", "post": False,
         "gate": "none", "alpha": 1.0, "center": False, "bias": False},
        # the residual stream of a calibration batch after a block's output product
        {"name": "norm_calibration", "op": "add_norm", "tokens": 32768, "d": 4096, "x": "bf16", "y": "f32",
         "post": False, "gate": "none", "alpha": 1.0, "center": False, "bias": False},
        # norms on both sides of the block, a gate per feature, a residual scale, odd sizes, fp16
        {"name": "norm_sandwich_odd", "op": "add_norm", "tokens": 2039, "d": 5125, "x": "f16", "y": "f16",
         "post": True, "gate": "feature", "alpha": 0.5, "center": True, "bias": True},
        # sixteen decoded tokens, 64 query and 8 k/v heads, far positions
        {"name": "rope_tokens", "op": "rope_qkv", "tokens": 16, "hq": 64, "hk": 8, "d": 128, "rot": 128,
         "x": "f32", "out": "bf16", "interleaved": False, "bias": False, "maxpos": 131072},
        # a prompt through the q/k/v product of a 4096-wide block with as many k/v heads
        {"name": "rope_prompt", "op": "rope_qkv", "tokens": 8192, "hq": 32, "hk": 32, "d": 128, "rot": 128,
         "x": "f32", "out": "bf16", "interleaved": False, "bias": True, "maxpos": 8192},
        # a calibration batch: equal sequences of 2048 tokens, 32 heads
        {"name": "attention_calibration", "op": "attention", "lens_q": ",".join(["2048"] * 16), "past": "0",
         "hq": 32, "hk": 32, "d": 128, "x": "bf16", "causal": True},
        # packed prompts of different lengths, eight query heads per k/v head
        {"name": "attention_packed", "op": "attention", "lens_q": "4099,1,777,2500,63,1024,129,6007", "past": "0",
         "hq": 64, "hk": 8, "d": 128, "x": "bf16", "causal": True},
        # a short chunk of a prompt after 2011 tokens that are there already: latency
        {"name": "attention_chunk", "op": "attention", "lens_q": "37", "past": "2011", "hq": 16, "hk": 4, "d": 64,
         "x": "f16", "causal": True},
        # sixteen sequences, one decoded token each, into the cache
        {"name": "kv4_tokens", "op": "kv4", "lens": ",".join(["1"] * 16), "past": 1000, "hk": 8, "d": 128,
         "group": 64, "page": 64, "x": "bf16"},
        # packed prompts into the cache
        {"name": "kv4_prompts", "op": "kv4", "lens": "8192,4099,1,3333", "past": 5, "hk": 32, "d": 128, "group": 128,
         "page": 64, "x": "bf16"},
        # one long sequence, eight query heads per k/v head
        {"name": "kv4_attention_long", "op": "kv4_attention", "lens": "131071", "hq": 64, "hk": 8, "d": 128,
         "group": 128, "page": 64, "x": "bf16"},
        # sixteen sequences of different lengths, as many k/v heads as query heads, small groups and pages
        {"name": "kv4_attention_batch", "op": "kv4_attention",
         "lens": "4096,3001,17,2048,1,3500,999,4000,2777,0,1500,3900,64,2222,3131,4095", "hq": 32, "hk": 32,
         "d": 128, "group": 32, "page": 16, "x": "f16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["add_norm", "rope_qkv", "attention", "attention", "kv4", "kv4_attention", "kv4_attention"])
    if op == "add_norm":
        d = _spread(rng, 64, 16384)
        if rng.random() < 0.5:
            d = max(64, d // 64 * 64)
        tokens = _spread(rng, 1, max(1, 120_000_000 // d // (2 if d > 4096 else 1)))
        post = rng.random() < 0.4
        return {"op": op, "tokens": tokens, "d": d, "x": rng.choice(["bf16", "f16", "f32"]),
                "y": rng.choice(["f32", "bf16", "f16"]), "post": post,
                "gate": rng.choice(["none", "feature", "token"]), "alpha": rng.choice([1.0, 0.5, 0.22]),
                "center": rng.random() < 0.4, "bias": rng.random() < 0.4}
    if op == "rope_qkv":
        hk = rng.choice([1, 2, 4, 8, 32])
        hq = hk * rng.choice([1, 2, 4, 8] if hk <= 8 else [1, 2])
        d = rng.choice([64, 80, 128])
        tokens = _spread(rng, 1, 70_000_000 // ((hq + 2 * hk) * d))
        return {"op": op, "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rng.choice([d, d, d // 2]),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["bf16", "f16"]),
                "interleaved": rng.random() < 0.4, "bias": rng.random() < 0.5, "maxpos": _spread(rng, 64, 131072)}
    if op == "attention":
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4, 5, 8])
        n = rng.randint(1, 8)
        top = _spread(rng, 8, 6000)
        lens = [_spread(rng, 1, top) for _ in range(n)]
        past = [rng.choice([0, 0, _spread(rng, 1, 2000)]) for _ in range(n)]
        while sum(q * (q + 2 * p) for q, p in zip(lens, past)) * hq > 16 * 32 * 2048 * 2048:
            lens = [max(1, q * 2 // 3) for q in lens]
            past = [p * 2 // 3 for p in past]
        return {"op": op, "lens_q": ",".join(map(str, lens)), "past": ",".join(map(str, past)), "hq": hq, "hk": hk,
                "d": rng.choice([64, 128]), "x": rng.choice(["bf16", "f16"]), "causal": rng.random() < 0.8}
    d = rng.choice([64, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    page = rng.choice([16, 64, 256])
    n = _spread(rng, 1, 64)
    if op == "kv4":
        hk = rng.choice([1, 2, 8, 32])
        top = _spread(rng, 1, max(1, 500_000 // (hk * n)))
        return {"op": op, "lens": ",".join(str(_spread(rng, 1, top)) for _ in range(n)), "past": rng.randint(0, 300),
                "hk": hk, "d": d, "group": group, "page": page, "x": rng.choice(["bf16", "f16"])}
    hk = rng.choice([1, 2, 4, 8, 32])
    hq = hk * rng.choice([1, 2, 4, 5, 8] if hk <= 8 else [1, 2])
    top = _spread(rng, 1, max(1, 1_000_000 // (hk * n)))
    lens = [0 if rng.random() < 0.05 else _spread(rng, 1, top) for _ in range(n)]
    return {"op": op, "lens": ",".join(map(str, lens)), "hq": hq, "hk": hk, "d": d, "group": group, "page": page,
            "x": rng.choice(["bf16", "f16"])}


def _ints(text, n=None):
    v = [int(t) for t in text.split(",")]
    return v * n if n is not None and len(v) == 1 else v


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# --------------------------------------------------------------------------- #
# Inputs
# --------------------------------------------------------------------------- #
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(g, tokens, heads, d, dtype):
    """k or v of a prompt: normal values, a few features of a head larger than the others."""
    x = _randn(g, tokens, heads, d)
    big = (torch.rand(heads, d, generator=g, device="cuda") < 0.03).float() * 4 + 1
    return (x * big).to(dtype)


def _tables(g, lens, page):
    """Pages in shuffled order: a table [sequences, pages of the longest] and their number."""
    per = [(n + page - 1) // page for n in lens]
    width = max(1, max(per))
    order = torch.randperm(max(1, sum(per)), generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, max(1, at)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "status": torch.zeros(4, dtype=torch.int32, device="cuda")}
    op = case["op"]
    if op == "add_norm":
        t, d, xt = case["tokens"], case["d"], _DT[case["x"]]
        s["X"] = (_randn(g, t, d) * (1 + 4 * (torch.rand(d, generator=g, device="cuda") < 0.01).float())).to(xt)
        s["Y"] = (0.5 * _randn(g, t, d)).to(_DT[case["y"]])
        par = (lambda scale, mid: (mid + scale * _randn(g, d)).to(xt))
        s["weight"] = par(0.1, 1.0)
        s["bias"] = par(0.1, 0.0) if case["bias"] else None
        s["post"] = par(0.1, 1.0) if case["post"] else None
        s["post_bias"] = par(0.1, 0.0) if case["post"] and case["bias"] else None
        s["gate"] = {"none": lambda: None, "feature": lambda: par(0.3, 0.7),
                     "token": lambda: torch.rand(t, d, generator=g, device="cuda").to(xt)}[case["gate"]]()
    elif op == "rope_qkv":
        w = (case["hq"] + 2 * case["hk"]) * case["d"]
        s["QKV"] = _randn(g, case["tokens"], w).to(_DT[case["x"]])
        s["bias"] = 0.2 * _randn(g, w) if case["bias"] else None
        # angles of far positions are taken in fp64 and the tables kept in fp32
        rate = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        ang = torch.arange(case["maxpos"], device="cuda", dtype=torch.float64)[:, None] * rate
        s["cos"], s["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
        if case["tokens"] <= 64:
            pos = torch.randint(0, case["maxpos"], (case["tokens"],), generator=g, device="cuda")
        else:
            pos = torch.arange(case["tokens"], device="cuda") % case["maxpos"]
        s["positions"] = pos.to(torch.int32)
    elif op == "attention":
        lq = _ints(case["lens_q"])
        lk = [a + b for a, b in zip(lq, _ints(case["past"], len(lq)))]
        xt = _DT[case["x"]]
        s["q"] = _heads(g, sum(lq), case["hq"], case["d"], xt)
        s["k"] = _heads(g, sum(lk), case["hk"], case["d"], xt)
        s["v"] = _heads(g, sum(lk), case["hk"], case["d"], xt)
        s["lq"], s["lk"] = lq, lk
        s["cu_q"] = torch.tensor(_starts(lq), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(_starts(lk), dtype=torch.int32, device="cuda")
    else:
        lens = _ints(case["lens"])
        hk, d, grp, page = case["hk"], case["d"], case["group"], case["page"]
        xt = _DT[case["x"]]
        past = case["past"] if op == "kv4" else 0
        table, pages = _tables(g, [n + past for n in lens], page)
        s["table"], s["lens"], s["past"] = table, lens, past
        s["start"] = torch.full((len(lens),), past, dtype=torch.int32, device="cuda")
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(_starts(lens), dtype=torch.int32, device="cuda")
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros(pages, hk, page, d // 8, dtype=torch.int32, device="cuda")
            s[n + "_params"] = torch.zeros(pages, hk, page, d // grp, 2, dtype=torch.float16, device="cuda")
        if op == "kv4":
            s["k"] = _heads(g, sum(lens), hk, d, xt)
            s["v"] = _heads(g, sum(lens), hk, d, xt)
        else:
            # what the cache holds: quantized keys and values (every page, also behind the sequences' ends)
            for n in ("k", "v"):
                for p0 in range(0, pages, 4096):
                    x = _heads(g, min(4096, pages - p0) * page, hk, d, xt)
                    c, sc, z = _codes(x.float().view(-1, page, hk, d).transpose(1, 2), grp)
                    s[n + "_codes"][p0:p0 + 4096] = _packed(c)
                    s[n + "_params"][p0:p0 + 4096] = torch.stack([sc, z], -1)
            s["q"] = _heads(g, len(lens), case["hq"], d, xt)
    return s


# --------------------------------------------------------------------------- #
# The plain forms
# --------------------------------------------------------------------------- #
def _norm(x, w, b, center, eps):
    if center:
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    return y if b is None else y + b.float()


def _plain_add_norm(s):
    c = s["case"]
    y = s["Y"].float()
    if s["post"] is not None:
        y = _norm(y, s["post"], s["post_bias"], c["center"], 1e-6)
    if s["gate"] is not None:
        y = y * s["gate"].float()
    xn = (s["X"].float() + c["alpha"] * y).to(s["X"].dtype)
    h = _norm(xn.float(), s["weight"], s["bias"], c["center"], 1e-6)
    return xn, h.to(xn.dtype)


def _plain_rope(s):
    c = s["case"]
    hq, hk, d, r = c["hq"], c["hk"], c["d"], c["rot"]
    x = s["QKV"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    x = x.view(-1, hq + 2 * hk, d)
    pos = s["positions"].long()
    cs, sn = s["cos"][pos][:, None], s["sin"][pos][:, None]
    qk = x[:, :hq + hk]
    if c["interleaved"]:
        a, b = qk[..., 0:r:2], qk[..., 1:r:2]
        rot = torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)
    else:
        a, b = qk[..., :r // 2], qk[..., r // 2:r]
        rot = torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
    qk = torch.cat([rot, qk[..., r:]], -1).to(_DT[c["out"]])
    return qk[:, :hq].contiguous(), qk[:, hq:].contiguous(), x[:, hq + hk:].to(_DT[c["out"]]).contiguous()


def _plain_attend(q, k, v, causal, scale):
    """q [heads, Lq, D], k and v [heads, Lk, D] in fp32; rows that see no key give 0."""
    lq, lk = q.shape[1], k.shape[1]
    if lk == 0:
        return torch.zeros_like(q)
    sc = torch.bmm(q, k.transpose(1, 2)) * scale
    if causal:
        seen = torch.arange(lk, device=q.device)[None] <= torch.arange(lq, device=q.device)[:, None] + (lk - lq)
        sc = sc.masked_fill(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    den = p.sum(-1, keepdim=True)
    o = torch.bmm(p, v)
    return torch.where(den > 0, o / den, torch.zeros_like(o))


def _plain_attention(s):
    c = s["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    o = torch.empty_like(s["q"])
    cq, ck = _starts(s["lq"]), _starts(s["lk"])
    for b, (lq, lk) in enumerate(zip(s["lq"], s["lk"])):
        step = max(1, min(hk, 200_000_000 // max(1, lq * lk * (hq // hk))))
        for h0 in range(0, hk, step):
            h1 = min(hk, h0 + step)
            n = hq // hk
            q = s["q"][cq[b]:cq[b + 1], h0 * n:h1 * n].float().transpose(0, 1)
            k = s["k"][ck[b]:ck[b + 1], h0:h1].float().transpose(0, 1).repeat_interleave(n, 0)
            v = s["v"][ck[b]:ck[b + 1], h0:h1].float().transpose(0, 1).repeat_interleave(n, 0)
            r = _plain_attend(q, k, v, c["causal"], d ** -0.5)
            o[cq[b]:cq[b + 1], h0 * n:h1 * n] = r.transpose(0, 1).to(o.dtype)
    return o


def _codes(x, grp):
    """fp32 [..., D] -> codes [..., D] in 0..15, scales and zero points fp16 [..., D / grp]."""
    g = x.unflatten(-1, (-1, grp))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    flat = lo == hi
    lo, hi = torch.where(flat, -torch.ones_like(lo), lo), torch.where(flat, torch.ones_like(hi), hi)
    sc = ((hi - lo) / 15).clamp(2.0 ** -24, 65504.0).half().float()
    z = torch.round(-lo / sc).clamp(0, 15)
    c = (torch.round(g / sc[..., None]) + z[..., None]).clamp(0, 15)
    return c.flatten(-2).to(torch.int32), sc.half(), z.half()


def _packed(c):
    """codes [..., D] -> int32 words [..., D / 8], code i of a word in its bits 4 i .. 4 i + 3."""
    sh = torch.arange(0, 32, 4, device=c.device)
    w = (c.to(torch.int64).unflatten(-1, (-1, 8)) << sh).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _values(words, params):
    """int32 words [..., D / 8] and (scale, zero) [..., G, 2] -> fp32 values [..., D]."""
    sh = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    c = ((words[..., None] >> sh) & 15).flatten(-2).float()
    p = params.float()
    g = c.unflatten(-1, (p.shape[-2], -1))
    return (p[..., :1] * (g - p[..., 1:])).flatten(-2)


def _places(s):
    """The page and the row inside it of every token of the batch."""
    page = s["case"]["page"]
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"), s["lengths"].long(),
                                  output_size=sum(s["lens"]))
    pos = torch.arange(sum(s["lens"]), device="cuda") - s["cu"].long()[seq] + s["past"]
    return s["table"][seq, pos // page].long(), pos % page


def _plain_kv4(s):
    pg, row = _places(s)
    out = []
    for n in ("k", "v"):
        c, sc, z = _codes(s[n].float(), s["case"]["group"])
        s[n + "_codes"][pg, :, row] = _packed(c)
        s[n + "_params"][pg, :, row] = torch.stack([sc, z], -1)
        out.append(_values(s[n + "_codes"][pg, :, row], s[n + "_params"][pg, :, row]).to(s[n].dtype))
    return tuple(out)


def _gathered(s, b, n):
    """The fp32 keys or values [hk, length, D] of sequence b."""
    c = s["case"]
    length = s["lens"][b]
    pg = s["table"][b, :(length + c["page"] - 1) // c["page"]].long()
    x = _values(s[n + "_codes"][pg], s[n + "_params"][pg])
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def _plain_kv4_attention(s):
    c = s["case"]
    n = c["hq"] // c["hk"]
    o = torch.empty_like(s["q"])
    for b in range(len(s["lens"])):
        q = s["q"][b].float().view(c["hk"], n, c["d"])
        o[b] = _plain_attend(q, _gathered(s, b, "k"), _gathered(s, b, "v"), False, c["d"] ** -0.5).flatten(0, 1) \
            .to(o.dtype)
    return o


# --------------------------------------------------------------------------- #
# One pass
# --------------------------------------------------------------------------- #
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"add_norm": _plain_add_norm, "rope_qkv": _plain_rope, "attention": _plain_attention,
                "kv4": _plain_kv4, "kv4_attention": _plain_kv4_attention}[op](s)
    import post_weight_quantization_15_b200 as G
    st = s["status"]
    if op == "add_norm":
        return G.add_norm(s["X"], s["weight"], Y=s["Y"], post_weight=s["post"], gate=s["gate"], alpha=c["alpha"],
                          eps=1e-6, center=c["center"], bias=s["bias"], post_bias=s["post_bias"], status=st)
    if op == "rope_qkv":
        return G.rope_qkv(s["QKV"], s["cos"], s["sin"], c["hq"], c["hk"], c["d"], positions=s["positions"],
                          bias=s["bias"], interleaved=c["interleaved"], dtype=_DT[c["out"]], status=st)
    if op == "attention":
        return G.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], status=st)
    cache = G.KV4Cache(s["k_codes"], s["k_params"], s["v_codes"], s["v_params"], c["group"])
    if op == "kv4":
        G.kv4_append(cache, s["k"], s["v"], s["table"], s["cu"], s["start"], status=st)
        return G.kv4_read(cache, s["table"], s["cu"], sum(s["lens"]), start=s["start"], dtype=s["k"].dtype, status=st)
    return G.kv4_attention(s["q"], cache, s["table"], s["lengths"], status=st)


def _pairs(lq, lk, causal):
    """Query-key pairs that count."""
    if not causal:
        return lq * lk
    seen = max(0, min(lq, lk))              # queries that see a key: the last ones
    return seen * lk - seen * (seen - 1) // 2


def work(case):
    op = case["op"]
    if op == "add_norm":
        n = case["tokens"] * case["d"]
        b, y = _BYTES[case["x"]], _BYTES[case["y"]]
        vec = 1 + case["bias"] + case["post"] * (1 + case["bias"]) + (case["gate"] == "feature")
        return {"bytes": n * (3 * b + y + (b if case["gate"] == "token" else 0)) + vec * case["d"] * b,
                "flops": n * (6 + 4 * case["post"])}
    if op == "rope_qkv":
        w = (case["hq"] + 2 * case["hk"]) * case["d"]
        rows = min(case["tokens"], case["maxpos"])
        return {"bytes": case["tokens"] * w * (_BYTES[case["x"]] + _BYTES[case["out"]]) + rows * case["rot"] * 4,
                "flops": case["tokens"] * (case["hq"] + case["hk"]) * case["rot"] * 3}
    if op == "attention":
        lq = _ints(case["lens_q"])
        lk = [a + b for a, b in zip(lq, _ints(case["past"], len(lq)))]
        n = sum(_pairs(a, b, case["causal"]) for a, b in zip(lq, lk))
        return {"bytes": 2 * case["d"] * 2 * (sum(lq) * case["hq"] + sum(lk) * case["hk"]),
                "flops": 4 * case["d"] * case["hq"] * n}
    lens = _ints(case["lens"])
    row = 2 * (case["d"] // 2 + 4 * (case["d"] // case["group"])) * case["hk"]     # a token's bytes in the cache
    if op == "kv4":
        return {"bytes": sum(lens) * (2 * row + 2 * 2 * 2 * case["d"] * case["hk"]),
                "flops": sum(lens) * case["hk"] * case["d"] * 2 * 8}
    return {"bytes": sum(lens) * row + 4 * len(lens) * case["hq"] * case["d"],
            "flops": 4 * case["d"] * case["hq"] * sum(lens)}


# --------------------------------------------------------------------------- #
# The same outputs from the definitions, in fp64
# --------------------------------------------------------------------------- #
def _norm64(x, w, b, center):
    n = x.shape[-1]
    if center:
        x = x - x.sum(-1, keepdim=True) / n
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / n + 1e-6) * w.double()
    return x if b is None else x + b.double()


def _exact_add_norm(s):
    c = s["case"]
    xs, hs = [], []
    for t0 in range(0, c["tokens"], 8192):
        rows = slice(t0, t0 + 8192)
        y = s["Y"][rows].double()
        if s["post"] is not None:
            y = _norm64(y, s["post"], s["post_bias"], c["center"])
        if s["gate"] is not None:
            y = y * (s["gate"][rows] if s["gate"].dim() == 2 else s["gate"]).double()
        x = s["X"][rows].double() + c["alpha"] * y
        xs.append(x)
        hs.append(_norm64(x.to(s["X"].dtype).double(), s["weight"], s["bias"], c["center"]))
    return torch.cat(xs), torch.cat(hs)


def _exact_rope(s):
    c = s["case"]
    hq, hk, d, r = c["hq"], c["hk"], c["d"], c["rot"]
    x = s["QKV"].double() + (0 if s["bias"] is None else s["bias"].double())
    x = x.view(-1, hq + 2 * hk, d)
    ang = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None]
    i = torch.arange(r // 2, device="cuda")
    i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    t = torch.complex(x[:, :hq + hk, i0], x[:, :hq + hk, i1]) * ang
    y = x.clone()
    y[:, :hq + hk, i0] = t.real
    y[:, :hq + hk, i1] = t.imag
    return y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:]


def _exact_row_block(q, k, v, first):
    """q [n, Lq, D] against k, v [Lk, D] in fp64; query i sees the keys up to first + i (None: all)."""
    lg = (q @ k.T) / math.sqrt(q.shape[-1])
    if first is not None:
        i = torch.arange(q.shape[1], device=q.device)[:, None]
        lg[:, torch.arange(k.shape[0], device=q.device)[None] > first + i] = -math.inf
    w = torch.exp(lg - torch.logsumexp(lg, -1, keepdim=True))
    return torch.nan_to_num(w, nan=0.0) @ v


def _exact_attention(s):
    c = s["case"]
    n = c["hq"] // c["hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        for h in range(c["hk"]):
            k, v = s["k"][k0:k0 + lk, h].double(), s["v"][k0:k0 + lk, h].double()
            for r in range(0, lq, 2048):
                q = s["q"][q0 + r:q0 + min(lq, r + 2048), h * n:(h + 1) * n].double().transpose(0, 1)
                first = lk - lq + r if c["causal"] else None
                o[q0 + r:q0 + min(lq, r + 2048), h * n:(h + 1) * n] = \
                    _exact_row_block(q, k, v, first).transpose(0, 1)
        q0 += lq
        k0 += lk
    return o


def _exact_kv4(s):
    out = []
    for n in ("k", "v"):
        x = s[n].double().unflatten(-1, (-1, s["case"]["group"]))
        lo, hi = torch.clamp(x.min(-1).values, max=0), torch.clamp(x.max(-1).values, min=0)
        same = hi == lo
        lo[same], hi[same] = -1, 1
        sc = torch.clamp((hi - lo) / 15, 2.0 ** -24, 65504).to(torch.float16).double()
        z = torch.clamp(torch.round(-lo / sc), 0, 15)
        c = torch.clamp(torch.round(x / sc[..., None]) + z[..., None], 0, 15)
        out.append(((c - z[..., None]) * sc[..., None]).flatten(-2))
    return tuple(out)


def _exact_kv4_attention(s):
    c = s["case"]
    n = c["hq"] // c["hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"]):
        if length == 0:
            continue
        pos = torch.arange(length, device="cuda")
        pg, row = s["table"][b].long()[pos // c["page"]], pos % c["page"]
        for h in range(c["hk"]):
            kv = []
            for name in ("k", "v"):
                w = s[name + "_codes"][pg, h, row].long()
                code = torch.stack([(w >> (4 * i)) % 16 for i in range(8)], -1).flatten(1).double()
                par = s[name + "_params"][pg, h, row].double().repeat_interleave(c["group"], 1)
                kv.append((code - par[..., 1]) * par[..., 0])
            o[b, h * n:(h + 1) * n] = _exact_row_block(s["q"][b, h * n:(h + 1) * n].double()[:, None], *kv, None)[:, 0]
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"add_norm": _exact_add_norm, "rope_qkv": _exact_rope, "attention": _exact_attention, "kv4": _exact_kv4,
            "kv4_attention": _exact_kv4_attention}[case["op"]](s)
