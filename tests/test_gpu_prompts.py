"""Prompts through quantized blocks into the 4-bit cache where the call's defaults and the batch's shape
matter: continued prompts, positions, what is reported, rows that no sequence has."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests.test_gpu_block import BF, U, _attn_tol, _close, _cu, _dev, _int, _np
from tests.test_gpu_decoder import (  # noqa: F401
    EPS, HD, HK, HQ, TABLE, _caches, _positions, _rotary, _stream_of, _weights, quantized)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_15_b200 as G
    from post_weight_quantization_15_b200 import decoder as D

TENSORS = ("k_codes", "k_params", "v_codes", "v_params")


def _rows(n, seed):
    return _stream_of(-(-n // 8) * 8, seed)[:n].contiguous()


def _forward(q, X):
    return G.linear_bf16(X, G.dequantize(q, BF))


def _mlp(b, h):
    w = G.dequantize(b.gate_up, BF)
    f = w.shape[0] // 2
    return _forward(b.down, G.silu_mul(G.linear_bf16(h, w[:f].contiguous()), G.linear_bf16(h, w[f:].contiguous())))


def _explicit(x, lens, start, blocks, rot, caches, table):
    """The operators one by one, the keys put together sequence by sequence; the attention against the oracle."""
    cu, after = _cu(lens), [s + n if n else 0 for s, n in zip(start, lens)]
    before, cu_k = [s if n else 0 for s, n in zip(start, lens)], _cu(after)
    pos = _int(np.concatenate([s + np.arange(n) for s, n in zip(start, lens)]).tolist())
    y = None
    for b, c in zip(blocks, caches):
        x, h = G.add_norm(x, b.norm_attn, Y=y, eps=EPS)
        q, k, v = G.rope_qkv(_forward(b.qkv, h), rot.cos, rot.sin, HQ, HK, HD, positions=pos)
        old = G.kv4_read(c, table, _int(_cu(before)), sum(before))
        cb = _cu(before)
        both = [torch.cat([t for i in range(len(lens)) for t in (o[cb[i]:cb[i + 1]], z[cu[i]:cu[i + 1]])])
                for o, z in zip(old, (k, v))]
        G.kv4_append(c, k, v, table, _int(cu), _int(start))
        a = G.attention(q, *both, _int(cu), _int(cu_k))
        ref, tol = _attn_tol(_np(q), *(_np(t) for t in both), cu, cu_k, HD ** -0.5, True, BF, U[BF])
        _close(a, ref, tol, "a")
        x, h = G.add_norm(x, b.norm_mlp, Y=_forward(b.o, a.flatten(1)), eps=EPS)
        y = _mlp(b, h)
    return G.residual_add(x, y)


@pytest.mark.parametrize("lens,start", [([20, 33, 1], [37, 0, 90]), ([5, 0, 38], [0, 64, 90]), ([1, 1, 1], [31, 32, 95]),
                                        ([0, 0, 9], [10, 20, 30])])
def test_a_prompt_goes_on_behind_what_the_cache_holds(quantized, lens, start):  # noqa: F811
    blocks, rot, _ = quantized
    table = _int(TABLE)
    caches, kept = _caches(2), _caches(2)
    first = _rows(sum(start), 31)
    for c in (caches, kept):
        D.prompt_blocks(first, _int(_cu(start)), blocks, rot, positions=_positions(start), caches=c, table=table)
    x = _rows(sum(lens), 32)
    pos = _int(np.concatenate([s + np.arange(n) for s, n in zip(start, lens)]).tolist())
    got = D.prompt_blocks(x, _int(_cu(lens)), blocks, rot, positions=pos, caches=caches, table=table, start=_int(start))
    want = _explicit(x, lens, start, blocks, rot, kept, table)
    assert torch.equal(got, want)
    for a, b in zip(caches, kept):
        for n in TENSORS:
            assert torch.equal(getattr(a, n), getattr(b, n)), n


def test_a_start_of_zero_is_no_start(quantized):  # noqa: F811
    blocks, rot, _ = quantized
    lens, table = [37, 0, 90], _int(TABLE)
    x, pos = _rows(127, 33), _positions([37, 0, 90])
    outs, caches = [], []
    for start in (None, _int([0, 0, 0]), _int([0, 55, 0])):      # (a sequence without new tokens has nothing to see)
        caches.append(_caches(2))
        outs.append(D.prompt_blocks(x, _int(_cu(lens)), blocks, rot, positions=pos, caches=caches[-1], table=table,
                                    start=start))
    for o, c in zip(outs[1:], caches[1:]):
        assert torch.equal(o, outs[0])
        for a, b in zip(c, caches[0]):
            assert all(torch.equal(getattr(a, n), getattr(b, n)) for n in TENSORS)


def test_continued_prompt_refusals(quantized):  # noqa: F811
    blocks, rot, _ = quantized
    x, table = _rows(6, 34), _int(TABLE)
    cu, pos = _int([0, 2, 4, 6]), _int([0, 1] * 3)
    for start in ([0, -1, 0], [0, 127, 0]):                      # (TABLE: 128 positions)
        caches = _caches(2)
        with pytest.raises(ValueError, match="positions"):
            D.prompt_blocks(x, cu, blocks, rot, pos, caches, table, _int(start))
        assert not any(c.k_codes.any() for c in caches)
    with pytest.raises(ValueError, match="start"):
        D.prompt_blocks(x, cu, blocks, rot, pos, start=_int([0, 0, 0]))
    with pytest.raises(ValueError, match="start"):
        D.prompt_blocks(x, cu, blocks, rot, pos, _caches(2), table, _int([0, 0]))
    with pytest.raises(ValueError, match="cu"):
        D.prompt_blocks(x, _int([0, 2, 4, 7]), blocks, rot, pos, _caches(2), table, _int([0, 0, 1]))


@pytest.mark.parametrize("lens,start", [([37, 0, 90], None), ([20, 33, 1], [37, 0, 90])])
def test_positions_follow_from_the_sequences(quantized, lens, start):  # noqa: F811
    """Without positions a token is at its place in its own sequence, in the cache too."""
    blocks, rot, _ = quantized
    table, x = _int(TABLE), _rows(sum(lens), 35)
    pos = _int(np.concatenate([s + np.arange(n) for s, n in zip(start or [0] * 3, lens)]).tolist())
    results = []
    for p in (pos, None):
        caches = _caches(2)
        if start:
            D.prompt_blocks(_rows(sum(start), 36), _int(_cu(start)), blocks, rot, positions=_positions(start),
                            caches=caches, table=table)
        results.append((D.prompt_blocks(x, _int(_cu(lens)), blocks, rot, p, caches, table,
                                        _int(start) if start else None), caches))
    (a, ca), (b, cb) = results
    assert torch.equal(a, b)
    for c, d in zip(ca, cb):
        assert all(torch.equal(getattr(c, n), getattr(d, n)) for n in TENSORS)


def test_errors_on_the_device_are_raised(quantized):  # noqa: F811
    """Without a status block of the caller's nothing goes wrong in silence; with one it is recorded there."""
    blocks, rot, _ = quantized
    x, table, short = _rows(3, 39), _int(TABLE), _int([t[:1] for t in TABLE])
    nan = x.clone()
    nan[1, 5] = float("nan")
    far = _int([0, 5000, 0])                                     # (the tables end at 2048)

    def step(x, lengths, table, **kw):
        return D.decode_blocks(x, _int(lengths), blocks, rot, _caches(2), table, **kw)

    def prompt(x, table, positions=None, **kw):
        return D.prompt_blocks(x, _int([0, 1, 2, 3]), blocks, rot, positions, _caches(2), table, **kw)

    inv, nonf = G.gptq.ERR_INVALID_ARG, G.gptq.ERR_NONFINITE
    for code, call in ((inv, lambda **kw: step(x, [0, 32, 0], short, **kw)),      # no page for the new token
                       (inv, lambda **kw: step(x, [0, 5000, 0], table, **kw)),
                       (nonf, lambda **kw: step(nan, [0, 0, 0], table, **kw)),
                       (inv, lambda **kw: prompt(x, table, far, **kw)),
                       (inv, lambda **kw: prompt(x, _int([[0], [-1], [1]]), **kw)),
                       (nonf, lambda **kw: prompt(nan, table, **kw))):
        with pytest.raises(G.GptqError) as e:
            call()
        assert e.value.code == code
        st = G.new_status(_dev())
        call(status=st)
        assert G.status_read(st) == (code, 1)
    assert torch.isfinite(step(x, [0, 1, 2], table)).all() and torch.isfinite(prompt(x, table)).all()


def test_rows_of_no_sequence_take_no_part_in_the_calibration():
    """A batch padded to a multiple of 8: whatever the padding holds, the layers are those of zeros there, and
    every product's input is 0 in those rows (so the Hessians are the sequences' alone)."""
    cu, pos = _int([0, 600, 997]), _positions([600, 397, 27])
    results = []
    for pad in (0.0, 3.0, float("nan")):
        x = _stream_of(1024, 40)
        x[997:] = pad
        blocks, out = D.quantize_decoder_blocks(x, cu, [_weights(5), _weights(6)], _rotary(), positions=pos, eps=EPS,
                                                record=True)
        assert (out[997:] == 0).all() and torch.isfinite(out).all()
        for b in blocks:
            for n in ("h", "a", "h_mlp", "m"):
                assert (b.stages[n][997:] == 0).all() and b.stages[n][:997].any(), n
        results.append((blocks, out))
    for blocks, out in results[1:]:
        assert torch.equal(out, results[0][1])
        for a, b in zip(blocks, results[0][0]):
            for layer in ("qkv", "o", "gate_up", "down"):
                for n in ("qweight", "scales", "zeros", "g_idx"):
                    assert torch.equal(getattr(getattr(a, layer), n), getattr(getattr(b, layer), n)), (layer, n)


def test_rows_of_no_sequence_leave_a_prompt_alone(quantized):  # noqa: F811
    blocks, rot, _ = quantized
    table, cu = _int(TABLE), _int([2, 39, 39, 120])
    outs, caches = [], []
    for pad in (0.0, float("inf")):
        x = _stream_of(128, 41)
        x[:2], x[120:] = 1.0, pad
        st = G.new_status(_dev())
        caches.append(_caches(2))
        outs.append(D.prompt_blocks(x, cu, blocks, rot, caches=caches[-1], table=table, status=st))
        G.raise_on_status(st, "prompt_blocks")
    assert torch.equal(outs[0][:120], outs[1][:120]) and torch.isfinite(outs[0]).all()
    for a, b in zip(*caches):
        assert all(torch.equal(getattr(a, n), getattr(b, n)) for n in TENSORS)


def test_a_captured_prompt(quantized):  # noqa: F811
    """Defaults for start, positions and status, replayed on another batch of the same shape."""
    blocks, rot, _ = quantized
    table, cu = _int(TABLE), _int([0, 37, 37, 127])
    xs = [_rows(127, 42), _rows(127, 43)]
    want, kept = [], []
    for x in xs:
        kept.append(_caches(2))
        want.append(D.prompt_blocks(x, cu, blocks, rot, caches=kept[-1], table=table))
    caches, x_in = _caches(2), xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = D.prompt_blocks(x_in, cu, blocks, rot, caches=caches, table=table)
    for x, w, k in zip(xs, want, kept):
        x_in.copy_(x)
        g.replay()
        assert torch.equal(out, w)
        for a, b in zip(caches, k):
            assert all(torch.equal(getattr(a, n), getattr(b, n)) for n in TENSORS)
