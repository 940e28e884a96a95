"""A decoder block's attention half on the GPU against its fp64 oracle.

Bounds (u = the output type's eps / 2, one rounding to nearest; w = 2^-24):
  norms     a row's mean of squares is a sum of d <= 32768 terms taken as 32 per thread, then trees:
            below 64 roundings, half of them through the square root; the products add a few: each
            normed value is within 64 w of itself.  A layer norm's mean is off by at most 64 w mean|v|,
            which shifts every value by that times |w| / std.
  rope      a + bias, two products and a sum: below 4 roundings of |a| + |b|.
  scores    sums of d products with fp32 accumulation that may truncate (a unit of 2w per step and 16
            of slack): ds = scale (d + 16) 2w sum|q k|.  The weights exp(s - max): relative ds on top
            and below, plus 2^-21 + |s - max| 2w for the exponential and its argument; rounded to
            16 bits for the product with v (up); the normaliser has the same relative errors bar up.
  values    sums over n keys: (n + 16) 2w of sum p|v|.
  small weights in fp16: the largest weight of a row is at least 1 (the kept maximum is never above
            the row's), so the sum of weights is too.  In attention a weight below 2^-14 is off by up to
            2^-25: n 2^-25 max|v| in all.  In the 4-bit cache a weight times its scale s is held as
            p s 2^(10 - e), 2^e <= the group's largest scale S: off by up to 2^-25 of that unit,
            2^(e - 35) <= 2^-35 S, times |c - z| <= 15.  A group with scale S spans 15 S, so one of its
            values is at least 7 S: 15 S <= 2.2 max|v|, and n tokens give less than n 2^-33 max|v|.
"""
import numpy as np
import pytest

from oracle import block_oracle as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_15_b200 as G

W = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _np(t):
    return t.detach().to("cpu").double().numpy()


def _rand(rng, shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(dtype).to(_dev())


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def _close(got, ref, tol, what):
    got = _np(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


# --------------------------------------------------------------------------- #
# add_norm
# --------------------------------------------------------------------------- #
def _norm_tol(v, w, b, eps, center, dtype):
    """Bound of N(v; w, b) rounded to dtype."""
    ref = B.norm(v, w, b, eps, center)
    c = v - v.mean(-1, keepdims=True) if center else v
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    shift = 64 * W * np.abs(v).mean(-1, keepdims=True) * r * np.abs(w) if center else 0.0
    mag = 64 * W * (np.abs(c) * r * np.abs(w) + (np.abs(b) if b is not None else 0.0)) + shift
    return ref, mag, mag * (1 + U[dtype]) + U[dtype] * np.abs(ref) + TINY[dtype]


NORM_CASES = [
    # tokens, d, X, Y, params, post, gate, center, bias, alpha
    (1, 4096, BF, FF, BF, False, None, False, False, 1.0),
    (3, 1, FF, FF, FF, True, "feature", False, True, 0.5),
    (9, 7, HF, HF, HF, False, "token", True, True, 0.25),
    (17, 1000, BF, BF, FF, True, "feature", True, False, 1.0),
    (8, 1024, FF, BF, HF, False, None, False, True, -1.0),
    (5, 1025, BF, FF, BF, True, "token", False, False, 0.5),
    (4, 5125, HF, HF, HF, True, "feature", True, True, 0.5),
    (2, 16384, BF, HF, BF, False, "feature", True, False, 1.0),
    (2, 16392, HF, FF, FF, True, None, False, False, 1.0),
    (2, 32768, BF, FF, BF, True, "token", True, True, 0.125),
    (33, 512, FF, FF, FF, True, "token", True, True, 2.0),
]


@pytest.mark.parametrize("tokens,d,xt,yt,pt,post,gate,center,bias,alpha", NORM_CASES)
def test_add_norm(tokens, d, xt, yt, pt, post, gate, center, bias, alpha):
    rng = np.random.default_rng(tokens * 100003 + d)
    X, Y = _rand(rng, (tokens, d), xt, 2.0) + 0.5, _rand(rng, (tokens, d), yt)
    vec = [_rand(rng, (d,), pt) for _ in range(5)]
    w, b = vec[0], vec[1] if bias else None
    pw, pb = (vec[2], vec[3] if bias else None) if post else (None, None)
    g = {None: None, "feature": vec[4], "token": _rand(rng, (tokens, d), pt)}[gate]
    eps = 1e-5
    Xc = X.clone()
    xn, h = G.add_norm(X, w, Y=Y, post_weight=pw, gate=g, alpha=alpha, eps=eps, center=center, bias=b, post_bias=pb)
    assert torch.equal(X, Xc) and xn.dtype == h.dtype == xt
    n = (lambda t: None if t is None else _np(t))
    x64, y64 = _np(X), _np(Y)
    mag = 0.0
    if post:
        _, mag, _ = _norm_tol(y64, n(pw), n(pb), eps, center, FF)
    ref = B.add(x64, y64, n(g), alpha, n(pw), n(pb), eps, center)
    scale = abs(alpha) * (np.abs(n(g)) if g is not None else 1.0)
    inner = np.abs(B.norm(y64, n(pw), n(pb), eps, center)) if post else np.abs(y64)
    tol = scale * mag + 4 * W * (np.abs(x64) + scale * inner)
    _close(xn, ref, tol * (1 + U[xt]) + U[xt] * np.abs(ref) + TINY[xt], "Xn")
    hr, _, ht = _norm_tol(_np(xn), n(w), n(b), eps, center, xt)
    _close(h, hr, ht, "h")
    # the same h from the stored stream, without a branch; the stream updated in place
    same, h2 = G.add_norm(xn, w, eps=eps, center=center, bias=b)
    assert same is xn and torch.equal(h2, h)
    xi, h3 = G.add_norm(X, w, Y=Y, post_weight=pw, gate=g, alpha=alpha, eps=eps, center=center, bias=b, post_bias=pb,
                        x_out=X)
    assert xi is X and torch.equal(X, xn) and torch.equal(h3, h)


@pytest.mark.parametrize("d,xt,yt,post,gate,center", [
    (64, BF, FF, False, "token", False), (96, HF, HF, True, "feature", True), (520, HF, BF, False, "token", False),
    (776, BF, BF, True, "feature", True), (1024, FF, HF, True, None, False), (1536, BF, FF, True, "token", True),
    (4096, HF, FF, False, None, False), (12008, BF, HF, True, "feature", True), (20000, FF, FF, False, "token", False),
    (700, FF, BF, True, "feature", True), (701, HF, FF, True, "token", True)])
def test_add_norm_many_rows(d, xt, yt, post, gate, center):
    test_add_norm(310, d, xt, yt, xt, post, gate, center, post, 0.5)


def test_add_norm_strided_rows_and_neighbours():
    rng = np.random.default_rng(5)
    for pad in (8, 3):                    # rows on 16-byte boundaries, and not
        big = _rand(rng, (6, 256 + pad), BF)
        Yb = _rand(rng, (6, 256 + 2 * pad), FF)
        w = _rand(rng, (256,), BF)
        out = torch.full((6, 256 + pad), 7.0, dtype=BF, device=big.device)
        xo = torch.full((6, 256 + pad), 7.0, dtype=BF, device=big.device)
        X, Y = big[:, :256], Yb[:, :256]
        xn, h = G.add_norm(X, w, Y=Y, out=out[:, :256], x_out=xo[:, :256])
        rx, rh = G.add_norm(X.contiguous(), w, Y=Y.contiguous())
        assert torch.equal(xn, rx) and torch.equal(h, rh)
        assert (out[:, 256:] == 7).all() and (xo[:, 256:] == 7).all()


@pytest.mark.parametrize("xt,yt", [(BF, HF), (HF, FF), (FF, BF)])
@pytest.mark.parametrize("d", [1, 3, 8, 61, 64, 100, 129, 256, 260, 513, 4099])
def test_add_norm_from_any_address(d, xt, yt):
    """Rows that start on every element of a 16-byte piece give what aligned rows give, and write nothing else."""
    rng = np.random.default_rng(d)
    t = 11
    X, Y, w = _rand(rng, (t, d), xt), _rand(rng, (t, d), yt), _rand(rng, (d + 3,), xt)[3:]
    want, _ = G.add_norm(X, w.clone(), Y=Y, post_weight=w.clone(), center=d > 1, eps=1e-3)
    for shift in (1, 2, 5, 7):
        def at(src):
            flat = torch.full((t * d + 16,), 7.0, dtype=src.dtype, device=src.device)
            flat[shift:shift + t * d] = src.flatten()
            return flat, flat[shift:shift + t * d].view(t, d)
        (_, Xs), (_, Ys), (fx, xo), (fo, ho) = at(X), at(Y), at(torch.zeros_like(X)), at(torch.zeros_like(X))
        G.add_norm(Xs, w, Y=Ys, post_weight=w, center=d > 1, eps=1e-3, x_out=xo, out=ho)
        for f in (fx, fo):
            assert (f[:shift] == 7).all() and (f[shift + t * d:] == 7).all()
        # either side's normed Y is within the bound of itself and rounded once with X; h likewise, from the same Xn
        _, mag, _ = _norm_tol(_np(Y), _np(w), None, 1e-3, d > 1, FF)
        r = _np(want)
        _close(xo, r, 2 * (mag + 4 * W * (np.abs(_np(X)) + np.abs(r)) + U[xt] * np.abs(r) + TINY[xt]) * (1 + U[xt]), shift)
        hr, _, ht = _norm_tol(_np(xo), _np(w), None, 1e-3, d > 1, xt)
        _close(ho, hr, ht, shift)


def test_add_norm_extreme_rows():
    """A row of zeros gives the bias; a large common mean costs the layer norm no digits; NaN stays in its row."""
    d = 640
    X = torch.zeros(4, d, dtype=FF, device=_dev())
    X[1] = 4096 + torch.arange(d, device=X.device) % 2       # centred values exactly +-0.5
    X[2, 5] = float("nan")
    w, b = torch.ones(d, device=X.device), torch.full((d,), 0.25, device=X.device)
    _, h = G.add_norm(X, w, center=True, bias=b, eps=0.0)
    assert torch.isnan(h[0]).all() and torch.isnan(h[2]).all() and torch.isnan(h[3]).all()   # 0 / 0 with eps 0
    assert torch.equal(h[1], (X[1] - 4096.5) * 2 + 0.25)
    _, h = G.add_norm(X, w, bias=b)
    assert torch.equal(h[0], b) and torch.isnan(h[2]).all()
    st = G.new_status(X.device)
    e, f = G.add_norm(X[:0], w, Y=X[:0], status=st)
    assert e.shape == f.shape == (0, d)


# --------------------------------------------------------------------------- #
# rope_qkv
# --------------------------------------------------------------------------- #
ROPE_CASES = [
    # tokens, hq, hk, d, rot, X, out, interleaved, bias, positions
    (1, 1, 1, 2, 2, FF, BF, False, False, True),
    (5, 4, 2, 64, 64, FF, BF, False, True, True),
    (3, 8, 1, 128, 64, FF, HF, True, False, True),
    (7, 3, 3, 80, 40, BF, BF, False, True, False),
    (4, 2, 1, 80, 80, HF, HF, True, True, True),
    (2, 5, 1, 36, 12, FF, HF, True, True, True),
    (2, 5, 1, 36, 36, FF, BF, False, False, True),
    (2, 40, 8, 128, 0, FF, BF, False, True, False),
    (6401, 4, 1, 128, 128, FF, BF, False, True, True),       # several tokens per block
    (15203, 2, 1, 80, 40, BF, HF, True, True, True),
    (2, 1, 1, 4096, 4096, FF, BF, False, True, True),        # a head wider than a block
]


@pytest.mark.parametrize("tokens,hq,hk,d,rot,xt,ot,inter,bias,posn", ROPE_CASES)
def test_rope_qkv(tokens, hq, hk, d, rot, xt, ot, inter, bias, posn):
    rng = np.random.default_rng(tokens + 7 * d + rot)
    cols = (hq + 2 * hk) * d
    big = _rand(rng, (tokens, cols + 16), xt, 3.0)
    X = big[:, :cols]
    bs = _rand(rng, (cols,), FF) if bias else None
    cs = sn = None
    if rot:
        ang = np.arange(100003)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        cs, sn = (torch.from_numpy(f(ang)).float().to(_dev()) for f in (np.cos, np.sin))
    pos = rng.integers(0, 100003, tokens)
    pos[-1] = 100002
    st = G.new_status(_dev())
    out = G.rope_qkv(X, cs, sn, hq, hk, d, positions=_int(pos.tolist()) if posn else None, bias=bs, interleaved=inter,
                     dtype=ot, status=st)
    G.raise_on_status(st, "rope_qkv")
    n = (lambda t: None if t is None else _np(t))
    at = pos if posn else np.arange(tokens)
    ref = B.rope_qkv(_np(X), n(cs), n(sn), hq, hk, d, at, n(bs), inter)
    mag = B.rope_qkv(np.abs(_np(X)), n(cs), n(sn), hq, hk, d, at, None if bs is None else np.abs(n(bs)), inter)
    for got, r, m, x in zip(out, ref, mag, "qkv"):
        assert got.is_contiguous() and got.dtype == ot
        # |a| + |b| of a pair is at most sqrt(2) of the pair's length, which turning keeps
        size = 4 * W * 2 * np.abs(m).max() if x != "v" else 4 * W * np.abs(m)
        _close(got, r, size + U[ot] * np.abs(r) + TINY[ot], x)


def test_rope_qkv_records_a_position_outside_the_tables():
    X, t = torch.ones(3, 4 * 8, device=_dev()), torch.ones(4, 4, device=_dev())
    for bad in (4, -1):
        st = G.new_status(_dev())
        G.rope_qkv(X, t, t, 2, 1, 8, positions=_int([0, bad, 3]), status=st)
        assert G.status_read(st) == (G.gptq.ERR_INVALID_ARG, 1)


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #
def _attn_tol(q, k, v, cu_q, cu_k, scale, causal, dtype, up, dq=0.0, small=None):
    """(oracle, bound): dq = what q's own rounding inside the kernel adds to a score, per sum|k|;
    small = what a weight below its 16-bit type's normal range is off by, per max|v|."""
    if small is None:
        small = 2.0 ** -25 if dtype == HF else 0.0
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    ref, mag = B.attention(q, k, v, cu_q, cu_k, scale, causal)
    tol = np.zeros(q.shape)
    for b in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        n = cu_k[b + 1] - cu_k[b]
        if n == 0:
            continue
        for h in range(hq):
            g = h // (hq // hk)
            ka = np.nan_to_num(np.abs(k[ks, g]), nan=0.0, posinf=0.0)
            qa = np.abs(q[qs, h])
            s = abs(scale) * (qa @ ka.T).max(1)                  # the largest sum of |terms|
            ds = s * (d + 16) * 2 * W + abs(scale) * dq * qa.max(1) * ka.sum(1).max()
            rel = 2 * (ds + 2.0 ** -21 + 2 * s * 2 * W) + up + (n + 16) * 2 * W
            vmax = np.nan_to_num(np.abs(v[ks, g]), nan=0.0, posinf=0.0).max()
            tol[qs, h] = rel[:, None] * mag[qs, h] + small * n * vmax
    return ref, tol * (1 + U[dtype]) + U[dtype] * np.abs(np.nan_to_num(ref)) + TINY[dtype]


def _cu(lens):
    return [0] + np.cumsum(lens).tolist()


ATTN_CASES = [
    # query lengths, keys before them, hq, hk, d, type, causal
    ([1], [0], 1, 1, 64, BF, True),
    ([1], [0], 2, 1, 128, HF, False),
    ([5, 1, 0, 130], [0, 3, 4, 0], 4, 2, 64, BF, True),
    ([128, 127, 129], [0, 1, 127], 2, 2, 128, BF, True),
    ([256, 257], [0, 0], 2, 1, 128, HF, True),
    ([300], [711], 8, 1, 128, BF, True),
    ([37], [1011], 4, 4, 64, HF, True),
    ([100, 60], [-40, -60], 4, 2, 64, HF, True),           # more queries than keys: the first see none
    ([100, 60], [-40, -60], 4, 2, 128, BF, False),         # a sequence without keys
    ([200, 50], [19, 333], 5, 1, 128, BF, False),
    ([70, 3], [0, 90], 6, 3, 80, BF, True),
    ([33, 140], [5, 0], 2, 1, 8, HF, True),
    ([150], [0], 3, 1, 120, HF, False),
    ([1] * 40 + [90], [17] * 41, 2, 2, 64, BF, True),
    ([513], [700], 2, 1, 64, BF, True),
]


def _attn_inputs(lens, past, hq, hk, d, dt, seed=0, tail=3):
    rng = np.random.default_rng(seed + sum(lens) * 31 + d)
    lk = [a + b for a, b in zip(lens, past)]
    q = _rand(rng, (sum(lens) + tail, hq, d), dt, 1.5)
    k = _rand(rng, (sum(lk) + tail, hk, d), dt, 1.5)
    v = _rand(rng, (sum(lk) + tail, hk, d), dt) + 0.25
    return q, k, v, _cu(lens), _cu(lk)


@pytest.mark.parametrize("lens,past,hq,hk,d,dt,causal", ATTN_CASES)
def test_attention(lens, past, hq, hk, d, dt, causal):
    q, k, v, cq, ck = _attn_inputs(lens, past, hq, hk, d, dt)
    out = torch.full(q.shape, 7.0, dtype=dt, device=q.device)
    st = G.new_status(q.device)
    o = G.attention(q, k, v, _int(cq), _int(ck), causal=causal, out=out, status=st)
    G.raise_on_status(st, "attention")
    assert o is out and (o[cq[-1]:] == 7).all()              # rows behind the last sequence
    ref, tol = _attn_tol(_np(q), _np(k), _np(v), cq, ck, d ** -0.5, causal, dt, U[dt])
    _close(o[:cq[-1]], ref[:cq[-1]], tol[:cq[-1]], "o")
    again = G.attention(q, k, v, _int(cq), _int(ck), causal=causal)
    assert torch.equal(again[:cq[-1]], o[:cq[-1]])


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64)])
def test_attention_masked_rows_take_no_part(dt, d):
    """NaN and infinities in keys and values behind a sequence's end, in the other sequence, and
    behind a causal query leave the queries that do not see them exactly as they were."""
    q, k, v, cq, ck = _attn_inputs([150, 90], [20, 0], 4, 2, d, dt)
    clean = G.attention(q, k, v, _int(cq), _int(ck))
    k2, v2 = k.clone(), v.clone()
    v2[ck[-1]:] = float("nan")
    k2[ck[-1]:] = float("inf")
    bad = 20 + 100                                           # a key of sequence 0 that queries 0 .. 99 do not see
    v2[bad, 0] = float("nan")
    v2[bad + 3, 1, 5] = float("inf")
    k2[bad + 2, 0] = float("nan")
    got = G.attention(q, k2, v2, _int(cq), _int(ck))
    ref, tol = _attn_tol(_np(q), _np(k), _np(v), cq, ck, d ** -0.5, True, dt, U[dt])
    rows = list(range(100)) + list(range(cq[1], cq[2]))      # queries that see none of it
    _close(got[rows], ref[rows], tol[rows], "rows that see none")
    assert torch.equal(got[cq[1]:cq[2]], clean[cq[1]:cq[2]])
    assert torch.isnan(got[100:150, :2]).all()               # heads of k/v head 0: a NaN value, then a NaN key
    assert torch.isfinite(got[100:103, 2:]).all()
    assert torch.isinf(got[103:150, 2:, 5]).all() and torch.isfinite(got[103:150, 2:, :5]).all()


# few queries over many keys: blocks that share a pair of query tiles
SPLIT_CASES = [
    ([1], [3000], 2, 1, 128, BF, True),
    ([130], [2500], 3, 3, 64, HF, True),
    ([257], [1800], 1, 1, 128, BF, False),
    ([5, 0, 40], [4000, 0, 900], 2, 2, 64, BF, True),      # a sequence with far fewer keys than the average
    ([1200], [-600], 1, 1, 128, HF, True),                 # the first queries see no key
    ([3, 2], [1500, -2], 4, 4, 72, BF, True),              # a sequence without keys
    ([300], [1749], 1, 1, 128, BF, True),                  # the last tile of keys reaches past the end by one
]


@pytest.mark.parametrize("lens,past,hq,hk,d,dt,causal", SPLIT_CASES)
def test_attention_few_queries_over_many_keys(lens, past, hq, hk, d, dt, causal):
    test_attention(lens, past, hq, hk, d, dt, causal)


@pytest.mark.parametrize("dt,d", [(BF, 128), (HF, 64)])
def test_attention_few_queries_masked_rows_take_no_part(dt, d):
    """The same as above where several blocks share the keys."""
    q, k, v, cq, ck = _attn_inputs([40], [2000], 4, 2, d, dt)
    k2, v2 = k.clone(), v.clone()
    v2[ck[-1]:] = float("nan")
    k2[ck[-1]:] = float("inf")
    v2[2020, 0] = float("nan")                               # queries 0 .. 19 do not see it
    k2[2025, 1] = float("nan")
    got = G.attention(q, k2, v2, _int(cq), _int(ck))
    ref, tol = _attn_tol(_np(q), _np(k), _np(v), cq, ck, d ** -0.5, True, dt, U[dt])
    _close(got[:20], ref[:20], tol[:20], "rows that see none")
    _close(got[:25, 2:], ref[:25, 2:], tol[:25, 2:], "heads that see none")
    assert torch.isnan(got[20:40, :2]).all() and torch.isnan(got[25:40, 2:]).all()


# heads that share tiles: 2 of 6, 16 of 32, 16 of 16, 4 of 4, 8 of 8 per k/v head
PACKED_CASES = [
    ([2, 61], [1500, 3], 12, 2, 64, HF, True),
    ([3, 9, 0, 1], [200, 0, 4, 7], 32, 1, 128, BF, True),
    ([17], [130], 16, 1, 72, BF, True),
    ([40, 33], [-39, 100], 8, 2, 128, HF, True),
    ([1] * 9, [255, 0, 1, 128, 127, 126, 300, 64, 5], 16, 2, 128, BF, True),
    ([100, 30], [0, 0], 4, 1, 64, BF, False),
]


@pytest.mark.parametrize("lens,past,hq,hk,d,dt,causal", PACKED_CASES)
def test_attention_heads_that_share_tiles(lens, past, hq, hk, d, dt, causal):
    test_attention(lens, past, hq, hk, d, dt, causal)


def test_attention_heads_that_share_tiles_masked_rows():
    q, k, v, cq, ck = _attn_inputs([20, 9], [30, 0], 8, 1, 128, BF)
    v2 = v.clone()
    v2[35] = float("nan")                                    # queries 0 .. 4 of sequence 0 do not see it
    got = G.attention(q, k, v2, _int(cq), _int(ck))
    ref, tol = _attn_tol(_np(q), _np(k), _np(v), cq, ck, 128 ** -0.5, True, BF, U[BF])
    rows = list(range(5)) + list(range(20, 29))
    _close(got[rows], ref[rows], tol[rows], "rows that see none")
    assert torch.isnan(got[5:20]).all()


@pytest.mark.parametrize("hq,hk,d,dt,causal", [(8, 2, 128, BF, True), (6, 6, 64, HF, True), (9, 3, 80, BF, False)])
def test_attention_many_pairs_per_block(hq, hk, d, dt, causal):
    """Far more pairs of tiles than SMs, of every size, empty sequences among them: blocks go from pair to pair."""
    rng = np.random.default_rng(hq)
    lens = [int(n) for n in rng.integers(0, 700, 70)]
    past = [int(n) for n in rng.integers(-100, 300, 70)]
    lens[3] = lens[41] = 0
    past = [max(p, -n) for p, n in zip(past, lens)]
    past[10] = -lens[10]                                     # a sequence without keys
    test_attention(lens, past, hq, hk, d, dt, causal)


def test_attention_very_many_sequences():
    rng = np.random.default_rng(77)
    lens = [int(n) for n in rng.integers(0, 4, 3000)]
    test_attention(lens, [int(n) for n in rng.integers(0, 3, 3000)], 2, 1, 64, HF, True)
    q, k, v, cq, ck = _attn_inputs([1] * 2000, [0] * 2000, 3, 1, 64, HF)
    cq[1500] = -5                                            # sequences 1499 and 1500 have bad bounds
    st = G.new_status(q.device)
    G.attention(q, k, v, _int(cq), _int(ck), status=st)
    code, at = G.status_read(st)
    assert code == G.gptq.ERR_INVALID_ARG and at in (1499, 1500)


def test_attention_large_scores_and_scale():
    """Scores in the thousands (weights 0 and 1), a negative and a zero scale."""
    q, k, v, cq, ck = _attn_inputs([140], [0], 2, 1, 128, HF)
    for scale in (25.0, -3.0, 0.0):
        o = G.attention(q, k, v, _int(cq), _int(ck), scale=scale)
        ref, tol = _attn_tol(_np(q), _np(k), _np(v), cq, ck, scale, True, HF, U[HF])
        _close(o[:140], ref[:140], tol[:140], scale)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_strided_heads(d):
    """q, k and v as slices of one product [tokens, (hq + 2 hk) d], o into a wider tensor; heads before tokens."""
    rng = np.random.default_rng(3)
    hq, hk, n = 6, 2, 141
    qkv = _rand(rng, (n, hq + 2 * hk, d), BF)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wide = torch.full((n, hq + 1, d), 7.0, dtype=BF, device=q.device)
    cu = _int([0, 60, n])
    o = G.attention(q, k, v, cu, out=wide[:, :hq])
    ref = G.attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    assert torch.equal(o, ref) and (wide[:, hq:] == 7).all()
    t = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    assert torch.equal(G.attention(*t, cu), ref)
    with pytest.raises(ValueError, match="overlaps"):
        G.attention(q, k, v, cu, out=q)
    with pytest.raises(G.GptqError):                         # heads that do not start on 16 bytes
        G.attention(qkv[..., 4:d - 4], k[..., :d - 8], v[..., :d - 8], cu)


def test_attention_records_bad_bounds():
    q, k, v, _, _ = _attn_inputs([20, 20], [0, 0], 2, 1, 64, BF, tail=0)
    good = G.attention(q, k, v, _int([0, 20, 40]))
    for cq, ck, b in (([0, 20, 41], [0, 20, 40], 1), ([0, 20, 40], [0, 20, 41], 1), ([0, 20, 40], [0, 21, 20], 1),
                      ([0, 20, 40], [-1, 20, 40], 0)):
        st = G.new_status(q.device)
        out = torch.full(q.shape, 7.0, dtype=BF, device=q.device)
        G.attention(q, k, v, _int(cq), _int(ck), out=out, status=st)
        assert G.status_read(st) == (G.gptq.ERR_INVALID_ARG, b)
        assert (out[20 * b:20 * b + 20] == 7).all()
    st = G.new_status(q.device)
    assert torch.equal(G.attention(q, k, v, _int([0, 20, 40]), status=st), good)


def test_attention_no_keys_at_all_and_no_queries():
    q = torch.ones(5, 2, 64, dtype=BF, device=_dev())
    z = torch.ones(0, 1, 64, dtype=BF, device=_dev())
    assert (G.attention(q, z, z, _int([0, 2, 5]), _int([0, 0, 0])) == 0).all()
    assert G.attention(q[:0], z, z, _int([0])).shape == (0, 2, 64)


# --------------------------------------------------------------------------- #
# The 4-bit cache
# --------------------------------------------------------------------------- #
def _pages(rng, lens, page, spare=2):
    """A shuffled table for sequences of these lengths, and the number of pages."""
    per = [-(-n // page) for n in lens]
    order = rng.permutation(sum(per) + spare)
    table = np.full((len(lens), max(1, max(per))), -1, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return _int(table.tolist()), sum(per) + spare


KV_CASES = [
    # new tokens, already there, heads, d, group, page, type
    ([1], [0], 1, 64, 32, 16, BF),
    ([1, 1, 1], [15, 16, 0], 2, 128, 128, 16, HF),
    ([40, 0, 7], [3, 5, 9], 8, 128, 64, 32, BF),
    ([33, 65], [31, 100], 3, 64, 64, 64, HF),
    ([130], [0], 5, 128, 32, 1024, BF),
]


def _special(x, dt):
    """Groups that are constant, zero, tiny, one-signed, and of mixed magnitude."""
    x[0, 0] = 0.0
    if x.shape[0] > 1:
        x[1, 0] = 3.0
        x[1, -1] = -2.5
    if x.shape[0] > 6:
        x[2] = x[2].abs()
        x[3] = -x[3].abs()
        x[4] = x[4] * 1e-7
        x[5, :, 0] = 60000.0 if dt == HF else 3e30           # beyond fp16's scale in bf16: saturates
        x[6, :, ::2] *= 1e-3
    return x


@pytest.mark.parametrize("lens,past,heads,d,group,page,dt", KV_CASES)
def test_kv4_append_and_read(lens, past, heads, d, group, page, dt):
    rng = np.random.default_rng(sum(lens) + d + group)
    total = sum(lens)
    table, pages = _pages(rng, [a + b for a, b in zip(lens, past)], page)
    cache = G.kv4_alloc(pages, page, heads, d, group, device=_dev())
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x5A5A5A5A)
    big = _rand(rng, (total + 2, 2 * heads + 1, d), dt, 2.0)     # rows behind the last sequence, strided heads
    big[:, :heads] = _special(big[:, :heads], dt)
    k, v = big[:, :heads], big[:, heads:2 * heads]
    st = G.new_status(_dev())
    cu = _cu(lens)
    before = cache.k_codes.clone()
    G.kv4_append(cache, k, v, table, _int(cu), _int(past), status=st)
    G.raise_on_status(st, "kv4_append")
    tb = table.cpu().numpy()
    written = np.zeros((pages, page), bool)
    outs = {}
    for x, codes, par, name in ((k, cache.k_codes, cache.k_params, "k"), (v, cache.v_codes, cache.v_params, "v")):
        c, s, z = B.kv4_quantize(x[:total].float().cpu().numpy(), group)
        words, par = codes.cpu().numpy().view(np.uint32), _np(par)
        rw = B.kv4_words(c)
        outs[name] = B.kv4_values(c, s, z)
        for b in range(len(lens)):
            for i in range(lens[b]):
                p = past[b] + i
                pg, r = tb[b, p // page], p % page
                written[pg, r] = True
                assert np.array_equal(words[pg, :, r], rw[cu[b] + i]), (name, b, i)
                assert np.array_equal(par[pg, :, r, :, 0], s[cu[b] + i]) and np.array_equal(par[pg, :, r, :, 1], z[cu[b] + i])
    keep = torch.from_numpy(~written).to(_dev())[:, None, :, None].expand_as(before)
    assert torch.equal(cache.k_codes[keep], before[keep])        # everything else untouched
    for dtype in (FF, BF, HF):
        rk, rv = G.kv4_read(cache, table, _int(cu), total, start=_int(past), dtype=dtype, status=st)
        for got, n in ((rk, "k"), (rv, "v")):
            want = torch.from_numpy(outs[n]).to(dtype)           # one rounding of an exact value
            assert torch.equal(got.cpu(), want), (n, dtype)
    G.raise_on_status(st, "kv4_read")


def test_kv4_records_what_does_not_fit():
    dev = _dev()
    k = torch.ones(3, 1, 64, dtype=HF, device=dev)
    cache = G.kv4_alloc(2, 16, 1, 64, 32, device=dev)
    inv, nonf = G.gptq.ERR_INVALID_ARG, G.gptq.ERR_NONFINITE
    for table, start, cu, info in (([[0]], [14], [0, 3], 2), ([[0]], [-1], [0, 3], 0), ([[0, 2]], [15], [0, 3], 1),
                                   ([[-1]], [0], [0, 3], 0)):
        st = G.new_status(dev)
        G.kv4_append(cache, k, k, _int(table), _int(cu), _int(start), status=st)
        code, at = G.status_read(st)
        assert code == inv and at >= info
        st = G.new_status(dev)
        G.kv4_read(cache, _int(table), _int(cu), 3, start=_int(start), status=st)
        assert G.status_read(st)[0] == inv
    assert (cache.k_codes[1] == 0).all()
    k[1, 0, 3] = float("inf")
    st = G.new_status(dev)
    G.kv4_append(cache, k, torch.ones_like(k), _int([[1]]), _int([0, 3]), _int([0]), status=st)
    assert G.status_read(st) == (nonf, 1)
    rk, rv = G.kv4_read(cache, _int([[1]]), _int([0, 3]), 3, dtype=HF)
    assert torch.isnan(rk[1, 0, :32]).all() and torch.isfinite(rk[1, 0, 32:]).all()
    assert torch.isfinite(rk[[0, 2]]).all() and torch.isfinite(rv).all()


# --------------------------------------------------------------------------- #
# kv4_attention
# --------------------------------------------------------------------------- #
KVA_CASES = [
    # lengths, hq, hk, d, group, page, type
    ([1], 1, 1, 64, 32, 16, BF),
    ([0, 1, 2, 15, 16, 17], 4, 2, 64, 64, 16, HF),
    ([63, 64, 65, 127, 128, 129], 8, 1, 128, 128, 32, BF),
    ([300, 0, 1000], 12, 2, 128, 64, 64, HF),
    ([777, 31], 16, 1, 128, 32, 16, BF),
    ([5000], 8, 8, 128, 128, 64, BF),
    ([2049, 100, 1], 24, 1, 64, 32, 256, HF),
    ([4097], 40, 2, 128, 64, 1024, BF),
    ([9000, 3], 5, 5, 64, 64, 128, HF),
    ([200] * 30, 4, 4, 128, 32, 32, BF),
]


def _kv_cache(rng, lens, hk, d, group, page, dt, scale=1.5):
    """A filled cache, its table, and the keys and values it stands for, per sequence, fp64."""
    table, pages = _pages(rng, lens, page)
    cache = G.kv4_alloc(pages, page, hk, d, group, device=_dev())
    total = sum(lens)
    k, v = _rand(rng, (total, hk, d), dt, scale), _rand(rng, (total, hk, d), dt) + 0.25
    cu = _int(_cu(lens))
    if total:
        G.kv4_append(cache, k, v, table, cu, _int([0] * len(lens)))
    rk, rv = G.kv4_read(cache, table, cu, total, dtype=FF)
    return cache, table, _np(rk), _np(rv)


@pytest.mark.parametrize("lens,hq,hk,d,group,page,dt", KVA_CASES)
def test_kv4_attention(lens, hq, hk, d, group, page, dt):
    rng = np.random.default_rng(sum(lens) + hq)
    cache, table, k64, v64 = _kv_cache(rng, lens, hk, d, group, page, dt)
    q = _rand(rng, (len(lens), hq, d), dt, 1.5)
    st = G.new_status(_dev())
    o = G.kv4_attention(q, cache, table, _int(lens), status=st)
    G.raise_on_status(st, "kv4_attention")
    # inside the kernel q may be held in fp16 under a power of two: 2^-25 of its largest value;
    # the weights in fp16 (2^-11)
    ref, tol = _attn_tol(_np(q), k64, v64, list(range(len(lens) + 1)), _cu(lens), d ** -0.5, False, dt, 2.0 ** -11,
                         dq=2.0 ** -25, small=2.0 ** -33)
    _close(o, ref, tol, "o")
    assert torch.equal(o, G.kv4_attention(q, cache, table, _int(lens)))


def test_kv4_attention_rows_behind_the_end_and_extremes():
    """Rows of a page behind a sequence's end hold NaN; scores in the hundreds; q of every magnitude."""
    rng = np.random.default_rng(9)
    lens = [100, 37]
    cache, table, k64, v64 = _kv_cache(rng, lens, 2, 128, 64, 32, BF, scale=10.0)
    tb = table.cpu().numpy()
    for b, n in enumerate(lens):
        pg, r = int(tb[b, n // 32]), n % 32
        for t in (cache.k_params, cache.v_params):
            t[pg, :, r:] = float("nan")
        cache.k_codes[pg, :, r:] = -1
    for mul in (1.0, 2.0 ** 100, 2.0 ** -60, 2.0 ** -133):
        q = (_rand(rng, (2, 4, 128), FF) * mul).to(BF)
        q[0, 0] = 0.0
        scale = 0.5 / mul if mul > 2.0 ** -100 else 1.0
        o = G.kv4_attention(q, cache, table, _int(lens), scale=scale)
        ref, tol = _attn_tol(_np(q), k64, v64, [0, 1, 2], _cu(lens), scale, False, BF, 2.0 ** -11, dq=2.0 ** -25, small=2.0 ** -33)
        _close(o, ref, tol, mul)


@pytest.mark.parametrize("n", [100, 5000, 40000])
def test_kv4_attention_nan_stays_in_its_rows(n):
    """A NaN in a query makes that head's result NaN, one in a group of values that group's features,
    whatever blocks the tokens fall to; every other result stays as it was."""
    rng = np.random.default_rng(n)
    cache, table, k64, v64 = _kv_cache(rng, [n, 64], 2, 128, 64, 32, HF)
    q = _rand(rng, (2, 8, 128), HF)
    clean = G.kv4_attention(q, cache, table, _int([n, 64]))
    ref, tol = _attn_tol(_np(q), k64, v64, [0, 1, 2], _cu([n, 64]), 128 ** -0.5, False, HF, 2.0 ** -11, dq=2.0 ** -25,
                         small=2.0 ** -33)
    q2 = q.clone()
    q2[0, 3, 5] = float("nan")
    got = G.kv4_attention(q2, cache, table, _int([n, 64]))
    assert torch.isnan(got[0, 3]).all()
    got[0, 3] = clean[0, 3]
    # the heads of one k/v head move their kept maxima together: head 3's no longer moves the others'
    _close(got, ref, tol, "other heads")
    assert torch.equal(got[0, 4:], clean[0, 4:]) and torch.equal(got[1], clean[1])
    pg, r = int(table[0, (n - 3) // 32]), (n - 3) % 32
    cache.v_params[pg, 1, r, 1, 0] = float("nan")
    got = G.kv4_attention(q, cache, table, _int([n, 64]))
    assert torch.isnan(got[0, 4:, 64:]).all()
    got[0, 4:, 64:] = clean[0, 4:, 64:]
    assert torch.equal(got, clean)


def test_kv4_attention_very_many_sequences():
    rng = np.random.default_rng(12)
    lens = [int(n) for n in rng.integers(0, 4, 3000)]
    cache, table, k64, v64 = _kv_cache(rng, lens, 1, 64, 32, 16, HF)
    q = _rand(rng, (3000, 2, 64), HF)
    o = G.kv4_attention(q, cache, table, _int(lens))
    ref, tol = _attn_tol(_np(q), k64, v64, list(range(3001)), _cu(lens), 0.125, False, HF, 2.0 ** -11, dq=2.0 ** -25,
                         small=2.0 ** -33)
    _close(o, ref, tol, "o")


def test_two_calls_at_once_on_two_streams():
    """Long calls of every operator on two streams at the same time give what they give alone."""
    rng = np.random.default_rng(13)
    lens = [[20000, 300], [15000, 7000]]
    made = [_kv_cache(rng, ln, 4, 128, 64, 64, BF)[:2] for ln in lens]
    qs = [_rand(rng, (2, 16, 128), BF) for _ in lens]
    qkv = [[_rand(rng, (1500, h, 128), BF) for h in (16, 4, 4)] for _ in lens]
    cu = _int([0, 400, 1500])
    X = [_rand(rng, (3000, 1000), HF) for _ in lens]
    w = _rand(rng, (1000,), HF)

    def go(i):
        return (G.kv4_attention(qs[i], made[i][0], made[i][1], _int(lens[i])), G.attention(*qkv[i], cu),
                *G.add_norm(X[i], w, Y=X[1 - i]))
    want = [go(0), go(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lens]
    for _ in range(5):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(go(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_kv4_attention_records_bad_lengths_and_pages():
    rng = np.random.default_rng(10)
    lens = [40, 20, 30]
    cache, table, _, _ = _kv_cache(rng, lens, 1, 64, 32, 16, HF)
    q = _rand(rng, (3, 2, 64), HF)
    good = G.kv4_attention(q, cache, table, _int(lens))
    inv = G.gptq.ERR_INVALID_ARG
    for bad in (-1, 49):
        st = G.new_status(_dev())
        out = torch.full(q.shape, 7.0, dtype=HF, device=q.device)
        G.kv4_attention(q, cache, table, _int([40, bad, 30]), out=out, status=st)
        assert G.status_read(st) == (inv, 1)
        assert (out[1] == 7).all()
    for bad in (-1, 10 ** 6):
        t2 = table.clone()
        t2[2, 1] = bad
        st = G.new_status(_dev())
        G.kv4_attention(q, cache, t2, _int(lens), status=st)
        assert G.status_read(st) == (inv, 2)
    assert torch.equal(G.kv4_attention(q, cache, table, _int(lens)), good)


# --------------------------------------------------------------------------- #
# Streams and graphs
# --------------------------------------------------------------------------- #
def _step(q, k, v, cache, table, cu, start, lengths, x, w, tabs, pos, stream=None):
    """The operators of one decoded token after another, as a block calls them."""
    xn, h = G.add_norm(x, w, Y=x, stream=stream)
    rq, rk, rv = G.rope_qkv(torch.cat([h.float()] * 1, 1), *tabs, 4, 2, 64, positions=pos, dtype=HF, stream=stream)
    G.kv4_append(cache, rk, rv, table, cu, start, stream=stream)
    return xn, G.kv4_attention(rq, cache, table, lengths, stream=stream), G.attention(q, k, v, cu, stream=stream)


def _step_inputs(seed):
    rng = np.random.default_rng(seed)
    lens = [50, 33]
    cache, table, _, _ = _kv_cache(rng, lens, 2, 64, 32, 32, HF)
    q, k, v = (_rand(rng, (2, h, 64), HF) for h in (4, 2, 2))
    ang = np.arange(128)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    tabs = [torch.from_numpy(f(ang)).float().to(_dev()) for f in (np.cos, np.sin)]
    return dict(q=q, k=k, v=v, cache=cache, table=table, cu=_int([0, 1, 2]), start=_int([50, 33]),
                lengths=_int([51, 34]), x=_rand(rng, (2, 512), FF), w=_rand(rng, (512,), FF), tabs=tabs,
                pos=_int([50, 33]))


def test_graph_replay_on_changed_inputs_and_side_stream():
    a, b = _step_inputs(1), _step_inputs(2)
    want_a = [t.clone() for t in _step(**a)]
    want_b = [t.clone() for t in _step(**b)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = None
    with torch.cuda.stream(s):
        got = _step(**a)
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want_a):
        assert torch.equal(x, y)
    got = [t for t in _step(**{**a, "stream": s})[1:]]       # the stream passed instead of made current
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for x, y in zip(got, want_a[1:]):
        assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _step(**a)
    for src, want in ((b, want_b), (a, want_a)):
        src = _step_inputs(2 if src is b else 1)
        for n in ("q", "k", "v", "table", "cu", "start", "lengths", "x", "w", "pos"):
            a[n].copy_(src[n])
        for n in ("k_codes", "k_params", "v_codes", "v_params"):
            getattr(a["cache"], n).copy_(getattr(src["cache"], n))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_an_error_in_the_status_block_skips_later_calls():
    a = _step_inputs(3)
    st = G.new_status(_dev())
    st[0] = G.gptq.ERR_NONFINITE
    out = torch.full(a["q"].shape, 7.0, dtype=HF, device=_dev())
    G.attention(a["q"], a["k"], a["v"], a["cu"], out=out, status=st)
    assert (out == 7).all()
    G.kv4_attention(a["q"], a["cache"], a["table"], a["lengths"], out=out, status=st)
    assert (out == 7).all()
    before = a["cache"].k_codes.clone()
    G.kv4_append(a["cache"], a["k"], a["v"], a["table"], a["cu"], a["start"], status=st)
    assert torch.equal(before, a["cache"].k_codes)
    x = torch.full((2, 512), 7.0, device=_dev())
    G.add_norm(a["x"], a["w"], out=x, status=st)
    assert (x == 7).all()
