"""Attention where scores are not finite: whole rows of NaN, at once, and nothing else."""
import numpy as np
import pytest

from tests.test_gpu_block import BF, HF, _cu, _dev, _int, _rand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_15_b200 as G


@pytest.mark.parametrize("lens,past,hq,hk,d,dt", [([300, 7], 0, 4, 2, 64, BF), ([130, 400], 50, 3, 1, 128, HF),
                                                  ([37], 4000, 4, 1, 64, HF), ([1, 2], 2500, 2, 2, 128, BF)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_scores_that_are_not_finite(lens, past, hq, hk, d, dt, value):
    """A query that is not finite gives a row of NaN (with inf: the score of some key is +inf, or NaN), a key the
    rows of the queries that see it; the others' bits stay."""
    rng = np.random.default_rng(len(lens) + d)
    cu_q, cu_k = _cu(lens), _cu([n + past for n in lens])
    q = _rand(rng, (cu_q[-1], hq, d), dt)
    k, v = (_rand(rng, (cu_k[-1], hk, d), dt) for _ in range(2))
    clean = G.attention(q, k, v, _int(cu_q), _int(cu_k))
    st = G.new_status(_dev())
    at, h = cu_q[1] - 1, hq - 1
    bad = q.clone()
    bad[at, h, 3] = value
    k3 = k.clone()
    k3[:, :, 3] = k3[:, :, 3].abs() + 1                          # (every score +inf, or NaN)
    ref = G.attention(q, k3, v, _int(cu_q), _int(cu_k))
    got = G.attention(bad, k3, v, _int(cu_q), _int(cu_k), status=st)
    assert torch.isnan(got[at, h]).all()
    got[at, h] = ref[at, h]
    assert torch.equal(got, ref)
    # a key in the middle: the queries at or behind it
    j = lens[0] // 2
    k2 = k.clone()
    k2[past + j, 0, 1] = float("nan")
    got = G.attention(q, k2, v, _int(cu_q), _int(cu_k), status=st)
    heads = slice(0, hq // hk)
    assert torch.isnan(got[j:cu_q[1], heads]).all()
    got[j:cu_q[1], heads] = clean[j:cu_q[1], heads]
    assert torch.equal(got, clean)
    G.raise_on_status(st, "attention")


def test_a_key_that_is_not_finite_before_a_long_prompt():
    """60,000 queries that all see it: one pass, well inside the bounded waits."""
    rng = np.random.default_rng(3)
    n = 60000
    q, k, v = (_rand(rng, (n, 1, 64), BF) for _ in range(3))
    k[0, 0, 0] = float("nan")
    st = G.new_status(_dev())
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    o = G.attention(q, k, v, _int([0, n]), status=st)
    b.record()
    G.raise_on_status(st, "attention")
    assert torch.isnan(o).all()
    # 1.8e9 pairs: a few ms by tiles; one key at a time and one row after another it is seconds
    assert a.elapsed_time(b) < 500
