"""What the decoder-block operators refuse before anything is launched: outputs and workspaces that do not
have a place of their own for every value, and sizes that do not fit the arithmetic of the kernels."""
import pytest

import post_weight_quantization_15_b200 as G

torch = pytest.importorskip("torch")


def _cpu(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


def _i(*v):
    return torch.tensor(v, dtype=torch.int32)


CACHE = G.KV4Cache(*(_cpu(1, 2, 16, *w, dtype=t) for _ in range(2) for w, t in (((8,), torch.int32),
                                                                               ((2, 2), torch.float16))), group=32)


def _attention(q, out):
    return G.attention(q, _cpu(3, 2, 64), _cpu(3, 2, 64), _i(0, 3), out=out)


def _kv4_attention(q, out):
    return G.kv4_attention(q, CACHE, _i(0, 0, 0).view(3, 1), _i(1, 1, 1), out=out)


@pytest.mark.parametrize("call", [_attention, _kv4_attention])
def test_outputs_whose_rows_overlap(call):
    q = _cpu(3, 4, 64)
    for out in (_cpu(1, 4, 64).expand(3, 4, 64), _cpu(3, 1, 64).expand(3, 4, 64), _cpu(64).expand(3, 4, 64),
                _cpu(1024).as_strided((3, 4, 64), (256, 32, 1)), _cpu(1024).as_strided((3, 4, 64), (192, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            call(q, out)
    with pytest.raises(ValueError, match="shape"):
        call(q, _cpu(3, 5, 64))
    # tokens before heads, heads before tokens, slices of something wider: only the device is missing
    for out in (_cpu(3, 4, 64), _cpu(4, 3, 64).transpose(0, 1), _cpu(3, 9, 64)[:, 2:6], _cpu(3, 4, 80)[..., :64]):
        with pytest.raises(ValueError, match="CUDA"):
            call(q, out)


def test_workspaces_that_are_not_as_long_as_they_say():
    q = _cpu(3, 4, 64)
    for ws in (_cpu(1).expand(10 ** 9), _cpu(100, 2)[:, 0]):
        with pytest.raises(ValueError, match="ws"):
            G.kv4_attention(q, CACHE, _i(0, 0, 0).view(3, 1), _i(1, 1, 1), ws=ws)
