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
