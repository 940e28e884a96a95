"""Whole decoder blocks on the GPU: every stage of the calibration against the oracle, given the GPU's own
inputs to that stage (so that each stage is measured, not roundings compounded through earlier ones); prompts
and single tokens over the 4-bit cache against the stages called one by one, the attention over the cache
against the oracle on what the cache holds."""
import numpy as np
import pytest

import synthetic as S
from oracle import block_oracle as B
from oracle import gptq_oracle as O
from tests.parity import compare_layer
from tests.test_gpu_block import BF, TINY, U, W, _attn_tol, _close, _dev, _int, _norm_tol, _np
from tests.test_gpu_pipeline import _as_bf16, _bits, _linear_bound

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import post_weight_quantization_15_b200 as G
    from post_weight_quantization_15_b200 import decoder as D

WIDTH, HQ, HK, HD, FF_ = 256, 4, 2, 64, 512
EPS = 1e-6


def _weights(seed):
    def layer(out, n, i):
        return torch.from_numpy(S.make_w(S.WSpec(out, n, 0.04, "f16", 3, 100 * seed + i))).to(_dev())

    rng = np.random.default_rng(seed)
    norms = [torch.from_numpy(1 + 0.1 * rng.standard_normal(WIDTH)).to(BF).to(_dev()) for _ in range(2)]
    return D.DecoderWeights(layer(HQ * HD, WIDTH, 1), layer(HK * HD, WIDTH, 2), layer(HK * HD, WIDTH, 3),
                            layer(WIDTH, HQ * HD, 4), layer(FF_, WIDTH, 5), layer(FF_, WIDTH, 6),
                            layer(WIDTH, FF_, 7), *norms)


def _rotary(n=2048):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, HD, 2) / HD)
    return D.Rotary(HQ, HK, HD, *(torch.from_numpy(f(ang)).float().to(_dev()) for f in (np.cos, np.sin)))


def _stream_of(tokens, seed):
    x = S.make_x(S.XSpec(WIDTH, tokens, 16, 0.01, 20.0, 3, seed))
    return torch.from_numpy(x.view(np.int16)).to(_dev()).view(BF).t().contiguous()


def _positions(lens):
    return _int(np.concatenate([np.arange(n) for n in lens]).tolist())


def _what(q, n):
    """The dequantized weights in bf16, as the forward uses them, in fp64."""
    return _as_bf16(O.dequantize(q.qweight.cpu().numpy(), q.scales.cpu().numpy(), q.zeros.cpu().numpy(),
                                 q.g_idx.cpu().numpy(), 4, n))


def _layer_ok(Ws, q, perm, x, n, what):
    Wn = np.concatenate([w.cpu().numpy() for w in Ws], axis=0)
    H64 = O.hessian(_bits(x.t()))
    ora = O.gptq_layer(Wn, None, 4, 128, True, True, H=H64)
    qw = q.qweight.cpu().numpy()
    c = compare_layer(Wn, H64, ora, qw, q.scales.cpu().numpy(), q.zeros.cpu().numpy(), q.g_idx.cpu().numpy(),
                      O.unpack(qw, 4, n).astype(np.uint8), perm.cpu().numpy(), 4, 128)
    assert c.ok(), (what, c)


def _product(x, Wh):
    """(x . Wh^T, its bound) for the tensor-core product."""
    return x @ Wh.T, _linear_bound(x.shape[1], np.abs(x) @ np.abs(Wh).T)


def _added(x, y, E, u):
    """(x + y, bound) where y is off by E, the sum rounded once."""
    ref = x + y
    return ref, E * (1 + u) + 4 * W * (np.abs(x) + np.abs(y)) + u * np.abs(ref) + TINY[BF]


def test_calibration_stage_by_stage():
    lens = [400, 113, 511]
    cu = [0, 400, 513, 1024]
    ws, rot = [_weights(1), _weights(2)], _rotary()
    X0 = _stream_of(1024, 1)
    pos = _positions(lens)
    blocks, X_out = D.quantize_decoder_blocks(X0, _int(cu), ws, rot, positions=pos, eps=EPS, record=True)
    u, cos, sin = U[BF], _np(rot.cos), _np(rot.sin)
    before = None
    for w, b in zip(ws, blocks):
        t = b.stages
        s = {n: _np(t[n]) for n in ("x_in", "h", "q", "k", "v", "a", "x_mid", "h_mlp", "m", "y")}
        if before is None:
            assert torch.equal(t["x_in"], X0)
        else:
            ref, tol = _added(before["x_mid"], before["y"], 0.0, u)
            _close(t["x_in"], ref, tol, "the block's input")
        ref, _, tol = _norm_tol(s["x_in"], _np(w.norm_attn), None, EPS, False, BF)
        _close(t["h"], ref, tol, "h")
        _layer_ok((w.wq, w.wk, w.wv), b.qkv, t["perm_qkv"], t["h"], WIDTH, "qkv")
        prod, E = _product(s["h"], _what(b.qkv, WIDTH))
        for n, r, e, x in zip("qkv", B.rope_qkv(prod, cos, sin, HQ, HK, HD, pos.cpu().numpy()),
                              *(B.rope_qkv(z, None, None, HQ, HK, HD, None) for z in (E, np.abs(prod)))):
            # a turned pair is off by at most what both of its features are; four roundings of its own
            off = 2 * (e + 4 * W * x).max(-1, keepdims=True) if n != "v" else e + 4 * W * x
            _close(t[n], r, off * (1 + u) + u * np.abs(r) + TINY[BF], n)
        ref, tol = _attn_tol(s["q"], s["k"], s["v"], cu, cu, HD ** -0.5, True, BF, u)
        _close(t["a"], ref.reshape(s["a"].shape), tol.reshape(s["a"].shape), "a")
        _layer_ok((w.wo,), b.o, t["perm_o"], t["a"], HQ * HD, "o")
        ref, tol = _added(s["x_in"], *_product(s["a"], _what(b.o, HQ * HD)), u)
        _close(t["x_mid"], ref, tol, "x_mid")
        ref, _, tol = _norm_tol(s["x_mid"], _np(w.norm_mlp), None, EPS, False, BF)
        _close(t["h_mlp"], ref, tol, "h_mlp")
        _layer_ok((w.w_gate, w.w_up), b.gate_up, t["perm_gate_up"], t["h_mlp"], WIDTH, "gate_up")
        Wgu = _what(b.gate_up, WIDTH)
        (g, Eg), (p, Ep) = _product(s["h_mlp"], Wgu[:FF_]), _product(s["h_mlp"], Wgu[FF_:])
        ref = O.silu(g) * p
        # silu' is within [-0.1, 1.1]; fp32 silu a few ulps; one bf16 rounding
        tol = np.abs(O.silu(g)) * Ep + 1.1 * Eg * (np.abs(p) + Ep) + (2.0 ** -20 + u) * np.abs(ref)
        _close(t["m"], ref, tol * (1 + u) + TINY[BF], "m")
        _layer_ok((w.w_down,), b.down, t["perm_down"], t["m"], FF_, "down")
        ref, tol = _product(s["m"], _what(b.down, FF_))
        _close(t["y"], ref, tol + TINY[BF], "y")
        before = s
    ref, tol = _added(before["x_mid"], before["y"], 0.0, u)
    _close(X_out, ref, tol, "the output")


@pytest.fixture(scope="module")
def quantized():
    rot = _rotary()
    blocks, X = D.quantize_decoder_blocks(_stream_of(1024, 3), _int([0, 600, 1024]), [_weights(3), _weights(4)], rot,
                                          positions=_positions([600, 424]), eps=EPS, desc_act=False)
    return blocks, rot, X


def test_prompts_give_what_the_calibration_gave(quantized):
    blocks, rot, X = quantized
    st = G.new_status(_dev())
    got = D.prompt_blocks(_stream_of(1024, 3), _int([0, 600, 1024]), blocks, rot, positions=_positions([600, 424]),
                          status=st)
    G.raise_on_status(st, "prompt_blocks")
    assert torch.equal(got, X)


def _caches(n):
    return [G.kv4_alloc(16, 32, HK, HD, 64, device=_dev()) for _ in range(n)]


TABLE = [[5, 2, 9, 0], [7, 1, 4, 3], [11, 6, 8, 10]]


def test_decoding_over_the_cache(quantized):
    blocks, rot, _ = quantized
    lens = [37, 0, 90]
    st = G.new_status(_dev())
    table = _int(TABLE)
    caches = _caches(2)
    D.prompt_blocks(_stream_of(128, 5)[:127].contiguous(), _int([0, 37, 37, 127]), blocks, rot,
                    positions=_positions(lens), caches=caches, table=table, status=st)
    kept = [(c.k_codes.clone(), c.v_params.clone()) for c in caches]
    x0 = _stream_of(8, 6)[:3].contiguous()
    lengths = _int(lens)
    got = D.decode_blocks(x0, lengths, blocks, rot, caches, table, status=st)
    G.raise_on_status(st, "decode_blocks")
    for c, (kc, vp) in zip(caches, kept):                    # only the new tokens' rows changed
        changed = (c.k_codes != kc).any(-1).any(1) | (c.v_params != vp).flatten(3).any(-1).any(1)
        new = torch.zeros_like(changed)
        for b, n in enumerate(lens):
            new[TABLE[b][n // 32], n % 32] = True
        assert torch.equal(changed, new)
    # the stages one by one; the attention against the oracle on what the cache holds
    x, y = x0, None
    for b, c in zip(blocks, caches):
        x, h = G.add_norm(x, b.norm_attn, Y=y, eps=EPS)
        q, k, v = G.rope_qkv(G.qmatvec(b.qkv, h), rot.cos, rot.sin, HQ, HK, HD, lengths)
        after = [n + 1 for n in lens]
        cu = [0, 38, 39, 130]
        rk, rv = (_np(z) for z in G.kv4_read(c, table, _int(cu), 130, dtype=torch.float32))
        for z, r in ((k, rk), (v, rv)):
            codes, sc, zp = B.kv4_quantize(z.float().cpu().numpy(), 64)
            assert np.array_equal(B.kv4_values(codes, sc, zp), r[[37, 38, 129]])
        a = G.kv4_attention(q, c, table, _int(after))
        ref, tol = _attn_tol(_np(q), rk, rv, [0, 1, 2, 3], cu, HD ** -0.5, False, BF, 2.0 ** -11, dq=2.0 ** -25,
                             small=2.0 ** -33)
        _close(a, ref, tol, "a")
        x, h = G.add_norm(x, b.norm_mlp, Y=G.qmatvec(b.o, a.flatten(1)), eps=EPS)
        gu = G.qmatvec(b.gate_up, h)
        y = G.qmatvec(b.down, G.silu_mul(gu[:, :FF_].contiguous(), gu[:, FF_:].contiguous()))
    assert torch.equal(got, G.residual_add(x, y))


def test_a_captured_step_decodes_token_after_token(quantized):
    """One graph replayed for successive tokens gives what eager steps give."""
    blocks, rot, _ = quantized
    table = _int(TABLE)
    xs = [_stream_of(8, 20 + i)[:3].contiguous() for i in range(4)]
    want, caches, lengths = [], _caches(2), _int([0, 0, 0])
    for x in xs:
        want.append(D.decode_blocks(x, lengths, blocks, rot, caches, table))
        lengths += 1
    caches2, lengths2, x_in = _caches(2), _int([0, 0, 0]), xs[0].clone()
    ws = G.workspace(G.kv4_attention_workspace_size(3, HQ, HK, HD, 4, 32), _dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                            # warm-up on caches of its own
        D.decode_blocks(x_in, lengths2, blocks, rot, _caches(2), table, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = D.decode_blocks(x_in, lengths2, blocks, rot, caches2, table, ws=ws)
        lengths2 += 1
    for c in caches2:                                        # nothing ran during the capture
        assert not c.k_codes.any()
    for x, w in zip(xs, want):
        x_in.copy_(x)
        g.replay()
        assert torch.equal(out, w)
    for a, b in zip(caches, caches2):
        assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_params, b.v_params)


def test_decoder_refusals(quantized):
    blocks, rot, _ = quantized
    x = torch.zeros(17, WIDTH, dtype=BF, device=_dev())
    table, ln = _int(TABLE), _int([0, 0, 0])
    for args in ((x, _int([0] * 17), blocks, rot, _caches(2), table), (x[:3], ln, blocks, rot, _caches(1), table),
                 (x[:3], ln.long(), blocks, rot, _caches(2), table), (x[:3].float(), ln, blocks, rot, _caches(2), table)):
        with pytest.raises(ValueError):
            D.decode_blocks(*args)
    with pytest.raises(ValueError):
        D.prompt_blocks(x, _int([0, 17]), blocks, rot, caches=_caches(2))
    with pytest.raises(ValueError, match="CUDA"):
        D.prompt_blocks(x.cpu(), _int([0, 17]), blocks, rot)
