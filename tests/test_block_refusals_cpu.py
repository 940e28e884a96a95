"""What the decoder-block operators refuse before anything is launched: outputs and workspaces that do not
have a place of their own for every value, and sizes that do not fit the arithmetic of the kernels."""
import ctypes

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


# --------------------------------------------------------------------------- #
# The C ABI near 2^31 (pointers that are never used: without a GPU nothing is launched)
# --------------------------------------------------------------------------- #
FAKE = ctypes.c_void_p(256)
LIMIT = 2 ** 31 - 2048                                           # the first size that is refused
UNSUPPORTED = -2


def test_rows_of_attention_near_the_end_of_32_bits():
    """Tiles reach past the last row: 128 rows, times the eight blocks that may share them."""
    def call(total_q, total_k):
        return G.lib().gptq_attention(FAKE, 64, 64, FAKE, 64, 64, FAKE, 64, 64, 2, FAKE, FAKE, 1, total_q, total_k, 1, 1,
                                      64, 0.1, 1, FAKE, 64, 64, None, None)
    for n in (LIMIT, 2 ** 31 - 1):
        assert call(n, 5) == UNSUPPORTED and call(5, n) == UNSUPPORTED


def test_tokens_of_rope_near_the_end_of_32_bits():
    """Blocks of up to 256 tokens count past the last one."""
    def call(tokens):
        return G.lib().gptq_rope_qkv(FAKE, 0, 512, None, FAKE, FAKE, 8, 64, 0, None, tokens, 4, 2, 64, 2, FAKE, FAKE,
                                     FAKE, None, None)
    assert call(LIMIT) == UNSUPPORTED and call(2 ** 31 - 1) == UNSUPPORTED


def test_positions_of_kv4_attention_near_the_end_of_32_bits():
    """A length's tiles of 32 are counted from length + 31."""
    desc = G.gptq._KV4(256, 256, 256, 256, 4, 16, 2, 64, 32)

    def call(width):
        return G.lib().gptq_kv4_attention(ctypes.byref(desc), FAKE, 64, 64, 2, 1, 4, FAKE, width, FAKE, 0.1, FAKE, 64, 64,
                                          FAKE, 1 << 40, None, None)
    assert call(LIMIT // 16) == UNSUPPORTED and call((2 ** 31 - 1) // 16) == UNSUPPORTED


# --------------------------------------------------------------------------- #
# Sizes that the ABI's ints would cut off (2^32 + 5 would become 5)
# --------------------------------------------------------------------------- #
BIG = 2 ** 32 + 5


def _meta(*shape, dtype=torch.float16):
    return torch.empty(*shape, dtype=dtype, device="meta")


I32 = torch.int32


@pytest.mark.parametrize("call", [
    lambda: G.add_norm(_meta(BIG, 8), _meta(8)),
    lambda: G.add_norm(_meta(1, BIG), _meta(BIG)),
    lambda: G.rope_qkv(_meta(BIG, 24), None, None, 1, 1, 8),
    lambda: G.rope_qkv(_meta(1, (BIG + 2) * 2), None, None, BIG, 1, 2),
    lambda: G.attention(_meta(BIG, 1, 8), _meta(4, 1, 8), _meta(4, 1, 8), _meta(2, dtype=I32)),
    lambda: G.attention(_meta(4, 1, 8), _meta(BIG, 1, 8), _meta(BIG, 1, 8), _meta(2, dtype=I32)),
    lambda: G.attention(_meta(4, 1, 8), _meta(4, 1, 8), _meta(4, 1, 8), _meta(BIG, dtype=I32)),
    lambda: G.kv4_append(CACHE, _meta(BIG, 2, 64), _meta(BIG, 2, 64), _meta(1, 1, dtype=I32), _meta(2, dtype=I32),
                         _meta(1, dtype=I32)),
    lambda: G.kv4_append(CACHE, _meta(4, 2, 64), _meta(4, 2, 64), _meta(1, BIG, dtype=I32), _meta(2, dtype=I32),
                         _meta(1, dtype=I32)),
    lambda: G.kv4_read(CACHE, _meta(1, 1, dtype=I32), _meta(2, dtype=I32), BIG),
    lambda: G.kv4_attention(_meta(BIG, 2, 64), CACHE, _meta(BIG, 1, dtype=I32), _meta(BIG, dtype=I32)),
    lambda: G.kv4_attention(_meta(1, 2, 64), CACHE, _meta(1, BIG, dtype=I32), _meta(1, dtype=I32)),
])
def test_sizes_beyond_the_abi(call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()
