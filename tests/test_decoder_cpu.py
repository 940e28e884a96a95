"""Host-side planning of the decoder path, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
from post_weight_quantization_15_b200 import decoder as D  # noqa: E402


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


TABLE = torch.zeros(3, 4, dtype=torch.int32)


def test_keys_of_a_continued_batch():
    p = D._past(_i(0, 2, 3, 5), _i(3, 0, 1), TABLE, 128, 5)
    # sequence 0: three cached and two new, 1: one new, 2: one cached and two new
    assert p.cu_k.tolist() == [0, 5, 6, 9] and p.total == 9
    assert p.new.tolist() == [3, 4, 5, 7, 8] and (p.first, p.last) == (0, 5)
    p = D._past(_i(2, 2, 4, 5), _i(9, 1, 0), TABLE, 128, 8)       # no new token: nothing of it is needed
    assert p.cu_k.tolist() == [0, 0, 3, 4] and p.new.tolist() == [1, 2, 3] and (p.first, p.last) == (2, 5)
    assert D._past(_i(0, 2, 2, 5), _i(0, 7, 0), TABLE, 128, 5) is None
    assert D._past(_i(0), _i(), TABLE[:0], 128, 5) is None


@pytest.mark.parametrize("cu,start,what", [
    ((0, 2, 1, 5), (0, 0, 1), "cu"), ((-1, 2, 3, 5), (0, 0, 1), "cu"), ((0, 2, 3, 6), (0, 0, 1), "cu"),
    ((0, 2, 3, 5), (0, -1, 0), "positions"), ((0, 2, 3, 5), (0, 0, 127), "positions"),
    ((0, 2, 3, 5), (0, 0), "start"), ((0, 5), (0, 0, 1), "start")])
def test_continued_batches_that_are_refused(cu, start, what):
    with pytest.raises(ValueError, match=what):
        D._past(_i(*cu), _i(*start), TABLE, 128, 5)


def test_types_of_a_continued_batch():
    for cu, start in ((_i(0, 2, 3, 5).long(), _i(0, 0, 1)), (_i(0, 2, 3, 5), _i(0, 0, 1).long())):
        with pytest.raises(ValueError, match="int32"):
            D._past(cu, start, TABLE, 128, 5)
    with pytest.raises(ValueError, match="table"):
        D._past(_i(0, 2, 3, 5), _i(0, 0, 1), TABLE[:2], 128, 5)


def test_positions_inside_the_sequences():
    cu = _i(0, 3, 3, 5)
    assert D._positions(cu, None, 7).tolist() == [0, 1, 2, 0, 1, 0, 0]       # (rows 5 and 6 have no sequence)
    assert D._positions(cu, _i(10, 5, 1), 5).tolist() == [10, 11, 12, 1, 2]
    assert D._positions(_i(2, 4), _i(7), 6).tolist() == [0, 0, 7, 8, 0, 0]
    assert D._positions(cu, None, 7).dtype == torch.int32 and D._positions(_i(0), None, 2).tolist() == [0, 0]
    assert D._positions(_i(0, 0, 0), _i(3, 4), 0).shape == (0,)


def test_rows_of_no_sequence_are_cleared():
    x = torch.full((6, 2), float("nan"))
    x[1:4] = torch.tensor([[1.0, -0.0], [2.0, 3.0], [float("inf"), 4.0]])
    y = D._without_strays(x, _i(1, 3, 4))
    assert torch.equal(y[1:4], x[1:4]) and (y[[0, 4, 5]] == 0).all()
    assert torch.equal(D._without_strays(x[1:4], _i(0, 3)), x[1:4])
    assert (D._without_strays(x, _i(0)) == 0).all() and (D._without_strays(x, _i(2, 2)) == 0).all()
    with pytest.raises(ValueError, match="cu"):
        D._without_strays(x, _i(0, 3).long())


def test_positions_refuse_a_start_of_another_length():
    """Also where no block is there to check it: rows would be looked up past its end."""
    for start in (_i(0, 0, 0), _i(0), _i(0, 0).long()):
        with pytest.raises(ValueError, match="start"):
            D._positions(_i(0, 3, 5), start, 5)
    with pytest.raises(ValueError, match="cu"):
        D._positions(_i(0, 3, 5).long(), None, 5)
