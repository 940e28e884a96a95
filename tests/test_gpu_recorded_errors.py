"""What a call records about one token or sequence leaves the rest of that call alone: the other results are
those of a call without the bad one, however many blocks start after the error is recorded; calls after it,
in a replayed graph too, stop."""
import numpy as np
import pytest

from tests.test_gpu_block import BF, FF, HF, _cu, _dev, _int, _pages, _rand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_15_b200 as G

INVALID, NONFINITE = -1, -4
TENSORS = ("k_codes", "k_params", "v_codes", "v_params")


def _same_bits(a, b):
    """Equal, NaNs included."""
    as_int = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(as_int), b.view(as_int))


# --------------------------------------------------------------------------- #
# The cache: 8000 tokens are 2000 blocks of kv4_append and as many of kv4_read
# --------------------------------------------------------------------------- #
HEADS, D, GROUP, PAGE = 8, 128, 32, 64


def _kv4_inputs(seed, dt=BF):
    rng = np.random.default_rng(seed)
    lens = [5, 4000, 995, 3000]
    table, pages = _pages(rng, lens, PAGE)
    k, v = (_rand(rng, (sum(lens), HEADS, D), dt) for _ in range(2))
    return lens, table, pages, k, v


def _filled(pages):
    cache = G.kv4_alloc(pages, PAGE, HEADS, D, GROUP, device=_dev())
    for n in TENSORS:
        getattr(cache, n).view(torch.int16).fill_(0x2A2A)
    return cache


def _row(table, b, pos):
    """The page and the row in it of a sequence's position."""
    return int(table[b, pos // PAGE]), pos % PAGE


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_kv4_append_of_one_bad_group(dt, value):
    """Token 2's group reads back as NaN, all that is written besides is as without it."""
    lens, table, pages, k, v = _kv4_inputs(1, dt)
    cu, zero = _int(_cu(lens)), _int([0] * len(lens))
    want, got = _filled(pages), _filled(pages)
    G.kv4_append(want, k, v, table, cu, zero)
    k[2, 3, 40] = value
    st = G.new_status(_dev())
    G.kv4_append(got, k, v, table, cu, zero, status=st)
    assert G.status_read(st) == (NONFINITE, 2)
    page, r = _row(table, 0, 2)
    rk, _ = G.kv4_read(got, table, cu, sum(lens), dtype=FF)
    assert torch.isnan(rk[2, 3, 32:64]).all() and torch.isfinite(rk[2, 3, :32]).all()
    got.k_codes[page, 3, r, 4:8] = want.k_codes[page, 3, r, 4:8]
    got.k_params[page, 3, r, 1] = want.k_params[page, 3, r, 1]
    for n in TENSORS:
        assert _same_bits(getattr(got, n), getattr(want, n)), n


@pytest.mark.parametrize("bad", ["start", "beyond", "page", "no page"])
def test_kv4_positions_that_the_table_does_not_hold(bad):
    """Sequence 0's tokens are left out, those of the others are written and read as without it."""
    lens, table, pages, k, v = _kv4_inputs(2)
    cu, zero = _int(_cu(lens)), _int([0] * len(lens))
    want, got = _filled(pages), _filled(pages)
    G.kv4_append(want, k, v, table, cu, zero)
    rk, rv = G.kv4_read(want, table, cu, sum(lens))
    start, t2 = zero.clone(), table.clone()
    if bad == "start":
        start[0] = -100
    elif bad == "beyond":
        start[0] = table.shape[1] * PAGE
    else:
        t2[0, 0] = pages if bad == "page" else -1
    st = G.new_status(_dev())
    G.kv4_append(got, k, v, t2, cu, start, status=st)
    code, token = G.status_read(st)
    assert code == INVALID and 0 <= token < 5
    page, _ = _row(table, 0, 0)
    for n in TENSORS:
        x, y, old = getattr(got, n), getattr(want, n), getattr(_filled(pages), n)
        assert _same_bits(x[page], old[page]), n              # (sequence 0 lies in one page)
        y[page] = old[page]
        assert _same_bits(x, y), n
    G.status_reset(st)
    ok, ov = G.kv4_read(got, t2, cu, sum(lens), start=start, status=st)
    assert G.status_read(st)[0] == INVALID
    assert torch.equal(ok[5:], rk[5:]) and torch.equal(ov[5:], rv[5:])


def test_kv4_calls_after_the_error_stop():
    lens, table, pages, k, v = _kv4_inputs(3)
    cu, zero = _int(_cu(lens)), _int([0] * len(lens))
    bad = k.clone()
    bad[0, 0, 0] = float("nan")
    st, cache = G.new_status(_dev()), _filled(pages)
    G.kv4_append(cache, bad, v, table, cu, zero, status=st)
    kept = [getattr(cache, n).clone() for n in TENSORS]
    for _ in range(2):
        G.kv4_append(cache, v, k, table, cu, zero, status=st)
        for n, x in zip(TENSORS, kept):
            assert _same_bits(getattr(cache, n), x), n
    assert G.status_read(st) == (NONFINITE, 0)


def test_a_replayed_graph_stops_at_its_own_error():
    lens, table, pages, k, v = _kv4_inputs(4)
    cu, zero = _int(_cu(lens)), _int([0] * len(lens))
    st, cache = G.new_status(_dev()), _filled(pages)
    G.kv4_append(cache, k, v, table, cu, zero, status=st)     # (and a warm-up)
    G.kv4_read(cache, table, cu, sum(lens), status=st)
    want = [getattr(cache, n).clone() for n in TENSORS]
    k_in = k.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.kv4_append(cache, k_in, v, table, cu, zero, status=st)
        rk, _ = G.kv4_read(cache, table, cu, sum(lens), status=st)
    g.replay()
    assert G.status_read(st)[0] == 0
    good = rk.clone()
    k_in[1, 1, 1] = float("inf")
    g.replay()                                               # the append goes on, the read stops
    assert G.status_read(st) == (NONFINITE, 1)
    page, r = _row(table, 0, 1)
    kept = [getattr(cache, n).clone() for n in TENSORS]
    for n, x, y in zip(TENSORS, kept, want):
        same = x == y                                        # (nothing of `want` is NaN)
        same[page, 1, r] = True
        assert same.all(), n
    assert torch.equal(rk, good)
    k_in.copy_(v)
    g.replay()                                               # both stop
    for n, x in zip(TENSORS, kept):
        assert _same_bits(getattr(cache, n), x), n
    G.status_reset(st)
    k_in.copy_(k)
    g.replay()
    assert G.status_read(st)[0] == 0 and torch.equal(rk, good)
    for n, x in zip(TENSORS, want):
        assert _same_bits(getattr(cache, n), x), n


# --------------------------------------------------------------------------- #
# kv4_attention: 300 sequences, some of one warp's run, some of many, 8 heads
# --------------------------------------------------------------------------- #
def _attention_inputs(seed, hq=16, dt=BF):
    rng = np.random.default_rng(seed)
    lens = [int(n) for n in rng.integers(1, 90, 300)]
    lens[100], lens[101], lens[200], lens[250] = 5000, 0, 3000, 0
    table, pages = _pages(rng, lens, PAGE)
    cache = G.kv4_alloc(pages, PAGE, HEADS, D, GROUP, device=_dev())
    k, v = (_rand(rng, (sum(lens), HEADS, D), dt) for _ in range(2))
    G.kv4_append(cache, k, v, table, _int(_cu(lens)), _int([0] * len(lens)))
    q = _rand(rng, (len(lens), hq, D), dt)
    return lens, cache, table, q, k, v


# one bad sequence at a time: its cut of the work is that of a batch where it is empty
@pytest.mark.parametrize("seq", [0, 100, 299])
@pytest.mark.parametrize("length", [-1, 10 ** 6])
def test_kv4_attention_beside_a_bad_length(seq, length):
    lens, cache, table, q, _, _ = _attention_inputs(5)
    without = list(lens)
    without[seq] = 0
    want = G.kv4_attention(q, cache, table, _int(without))
    lens[seq] = length
    for _ in range(3):
        st, out = G.new_status(_dev()), torch.full_like(q, 7.0)
        G.kv4_attention(q, cache, table, _int(lens), out=out, status=st)
        assert G.status_read(st) == (INVALID, seq)
        assert (out[seq] == 7).all()
        out[seq] = want[seq]
        assert torch.equal(out, want)
    assert (want[[101, 250]] == 0).all()


@pytest.mark.parametrize("seq", [0, 100, 299])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_kv4_attention_beside_a_bad_page(seq, entry):
    """The bad page's tokens take no part, in that sequence alone: the result is that of a sequence with the
    other tokens."""
    lens, cache, table, q, k, v = _attention_inputs(6)
    want = G.kv4_attention(q, cache, table, _int(lens))
    t2 = table.clone()
    last = (lens[seq] - 1) // PAGE
    t2[seq, last] = entry
    for _ in range(3):
        st, out = G.new_status(_dev()), torch.full_like(q, 7.0)
        G.kv4_attention(q, cache, t2, _int(lens), out=out, status=st)
        assert G.status_read(st) == (INVALID, seq)
        got = out[seq].clone()
        out[seq] = want[seq]
        assert torch.equal(out, want)
        # the sequence cut before that page, taken in other runs: each side's weights are off by 2^-11 of
        # sum p|v| <= max|v| (a cached v may be half a step larger) and its result is rounded once (2^-8)
        ref = G.kv4_attention(q[seq:seq + 1], cache, table[seq:seq + 1], _int([last * PAGE]))[0]
        assert torch.allclose(got.float(), ref.float(), rtol=2.0 ** -6, atol=2.0 ** -9 * float(v.abs().max()))
    assert torch.equal(G.kv4_attention(q, cache, table, _int(lens)), want)


def test_kv4_attention_after_the_error_stops():
    lens, cache, table, q, _, _ = _attention_inputs(7)
    st, out = G.new_status(_dev()), torch.full_like(q, 7.0)
    bad = list(lens)
    bad[3] = -5
    G.kv4_attention(q, cache, table, _int(bad), status=st)
    for _ in range(2):
        G.kv4_attention(q, cache, table, _int(lens), out=out, status=st)
        assert (out == 7).all()
    assert G.status_read(st) == (INVALID, 3)


# --------------------------------------------------------------------------- #
# attention: pairs of tiles for every SM several times over, and shared ones
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("which", ["queries", "keys"])
@pytest.mark.parametrize("lens,past,hq,hk,at", [([150] * 300, 10, 8, 2, 1), ([600] * 40, 0, 4, 4, 20),
                                                 ([1, 3, 2, 1], 4000, 4, 1, 2)])
def test_attention_beside_bad_bounds(lens, past, hq, hk, at, which):
    """A bound that is out of range takes the two sequences beside it, and no other."""
    rng = np.random.default_rng(8)
    cu_q, cu_k = _cu(lens), _cu([n + past for n in lens])
    q = _rand(rng, (cu_q[-1], hq, 64), HF)
    k, v = (_rand(rng, (cu_k[-1], hk, 64), HF) for _ in range(2))
    want = G.attention(q, k, v, _int(cu_q), _int(cu_k))
    rows = slice(cu_q[at - 1], cu_q[at + 1])
    (cu_q if which == "queries" else cu_k)[at] = -3
    for _ in range(3):
        st, out = G.new_status(_dev()), torch.full_like(q, 7.0)
        G.attention(q, k, v, _int(cu_q), _int(cu_k), out=out, status=st)
        code, seq = G.status_read(st)
        assert code == INVALID and seq in (at - 1, at)
        assert (out[rows] == 7).all()
        out[rows] = want[rows]
        assert torch.equal(out, want)
    G.attention(q, k, v, _int(cu_q), _int(cu_k), out=out.fill_(5.0), status=st)      # the error is an earlier call's
    assert (out == 5).all()


# --------------------------------------------------------------------------- #
# rope_qkv
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("tokens,hq,hk,d,dt", [(20000, 4, 1, 64, FF), (3000, 32, 8, 128, BF), (9001, 2, 2, 20, HF),
                                               (2000, 1, 1, 600, FF)])
@pytest.mark.parametrize("bad", [-1, 500])
def test_rope_qkv_beside_a_bad_position(tokens, hq, hk, d, dt, bad):
    """A position outside the tables is read as 0, in blocks that start after it was recorded too."""
    rng = np.random.default_rng(9)
    X = _rand(rng, (tokens, (hq + 2 * hk) * d), dt)
    cos, sin = (_rand(rng, (500, d // 2), FF) for _ in range(2))
    pos = torch.arange(tokens, dtype=torch.int32, device=_dev()) % 500
    pos[1] = pos[tokens - 2] = 0
    want = G.rope_qkv(X, cos, sin, hq, hk, d, positions=pos)
    pos[1] = pos[tokens - 2] = bad
    for _ in range(3):
        st = G.new_status(_dev())
        got = G.rope_qkv(X, cos, sin, hq, hk, d, positions=pos, status=st)
        code, token = G.status_read(st)
        assert code == INVALID and token in (1, tokens - 2)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


# --------------------------------------------------------------------------- #
# qmatvec: 512 blocks that all find the bad group index while others start
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("rows", [1, 4])
def test_qmatvec_records_a_bad_group_index(rows):
    rng = np.random.default_rng(10)
    out, n, groups = 65536, 1024, 8
    q = G.QuantizedLayer(torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (n // 8, out), dtype=np.int32)).to(_dev()),
                         (_rand(rng, (groups, out), FF).abs() + 0.5).to(HF), torch.full((groups, out), 8.0, dtype=HF,
                                                                                      device=_dev()),
                         torch.arange(n, dtype=torch.int32, device=_dev()) // 128, None, None, 4, 128, False)
    X = _rand(rng, (rows, n), BF)
    want = G.qmatvec(q, X)
    good = q.g_idx.clone()
    for bad in (groups, -1, 2 ** 31 - 1):
        q.g_idx[5] = bad
        st = G.new_status(_dev())
        for _ in range(5):
            G.status_reset(st)
            G.qmatvec(q, X, st)
            assert G.status_read(st) == (INVALID, 5)
    q.g_idx.copy_(good)
    G.status_reset(st)
    assert torch.equal(G.qmatvec(q, X, st), want)
    assert G.status_read(st)[0] == 0
