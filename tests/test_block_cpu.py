"""The decoder block's operators without a GPU: refusals of the C ABI and of the binding, and
hand-worked values of their oracle."""
import ctypes

import numpy as np
import pytest

import post_weight_quantization_15_b200 as G
from oracle import block_oracle as B

torch = pytest.importorskip("torch")
P = ctypes.c_void_p
fake = P(256)        # never dereferenced: every call below fails its argument checks first


@pytest.fixture(scope="module")
def L():
    return G.lib()


def _norm(L, **kw):
    a = dict(X=fake, xt=2, ldx=64, Y=fake, yt=0, ldy=64, w=fake, b=None, pw=None, pb=None, gate=None, ldg=0, pt=2,
             tokens=4, d=64, alpha=1.0, eps=1e-6, center=0, xn=fake, ldxn=64, h=fake, ldh=64)
    a.update(kw)
    v = list(a.values())
    v[15], v[16] = ctypes.c_float(a["alpha"]), ctypes.c_float(a["eps"])
    return L.gptq_add_norm(*v, None, None)


def test_add_norm_refusals(L):
    assert _norm(L, X=None) == -1 and _norm(L, w=None) == -1 and _norm(L, h=None) == -1
    assert _norm(L, xn=None) == -1 and _norm(L, ldx=63) == -1 and _norm(L, ldy=63) == -1
    assert _norm(L, xt=3) == -1 and _norm(L, yt=-1) == -1 and _norm(L, pt=9) == -1
    assert _norm(L, d=0) == -1 and _norm(L, tokens=-1) == -1 and _norm(L, eps=-1.0) == -1
    assert _norm(L, eps=float("nan")) == -1
    assert _norm(L, Y=None, gate=fake) == -1 and _norm(L, Y=None, pw=fake) == -1 and _norm(L, pb=fake) == -1
    assert _norm(L, gate=fake, ldg=63) == -1
    assert _norm(L, d=32769, ldx=40000, ldy=40000, ldxn=40000, ldh=40000) == -2
    assert _norm(L, tokens=0) == 0


def _rope(L, **kw):
    a = dict(X=fake, xt=0, ld=512, bias=None, cos=fake, sin=fake, maxpos=8, rot=64, il=0, pos=None, tokens=4, hq=4,
             hk=2, d=64, ot=2, q=fake, k=fake, v=fake)
    a.update(kw)
    return L.gptq_rope_qkv(*a.values(), None, None)


def test_rope_qkv_refusals(L):
    assert _rope(L, ld=511) == -1 and _rope(L, rot=63) == -1 and _rope(L, rot=66) == -1 and _rope(L, rot=-2) == -1
    assert _rope(L, cos=None) == -1 and _rope(L, maxpos=0) == -1 and _rope(L, ot=0) == -1 and _rope(L, xt=4) == -1
    assert _rope(L, q=None) == -1 and _rope(L, hk=0) == -1 and _rope(L, d=63) == -1 and _rope(L, tokens=-1) == -1
    assert _rope(L, tokens=0) == 0
    assert _rope(L, hq=1 << 20, d=2048, ld=1 << 40, rot=64) == -2


def _attn(L, **kw):
    a = dict(q=fake, qt=256, qh=64, k=fake, kt=128, kh=64, v=fake, vt=128, vh=64, dt=2, cuq=fake, cuk=fake, n=2,
             tq=8, tk=8, hq=4, hk=2, d=64, scale=0.1, causal=1, o=fake, ot=256, oh=64)
    a.update(kw)
    a["scale"] = ctypes.c_float(a["scale"])
    return L.gptq_attention(*a.values(), None, None)


def test_attention_refusals(L):
    assert _attn(L, q=None) == -1 and _attn(L, o=None) == -1 and _attn(L, k=None) == -1 and _attn(L, cuk=None) == -1
    assert _attn(L, q=P(264)) == -1 and _attn(L, vt=132) == -1 and _attn(L, oh=4) == -1 and _attn(L, kt=-128) == -1
    assert _attn(L, dt=0) == -1 and _attn(L, hk=3) == -1 and _attn(L, hk=0) == -1 and _attn(L, n=-1) == -1
    assert _attn(L, scale=float("nan")) == -1
    assert _attn(L, d=60) == -2 and _attn(L, d=136) == -2 and _attn(L, hq=65536, hk=1) == -2
    assert _attn(L, n=0) == 0 and _attn(L, tq=0) == 0


def _desc(**kw):
    a = dict(kc=256, kp=256, vc=256, vp=256, pages=4, page=16, heads=2, d=64, group=32)
    a.update(kw)
    return G.gptq._KV4(*a.values())


def test_kv4_refusals(L):
    ok = _desc()

    def append(c=ok, k=fake, kt=128, kh=64, v=fake, vt=128, vh=64, dt=2, tokens=4, table=fake, width=2, cu=fake,
               start=fake, n=2):
        return L.gptq_kv4_append(ctypes.byref(c), k, kt, kh, v, vt, vh, dt, tokens, table, width, cu, start, n, None,
                                 None)

    for bad, code in ((_desc(kc=0), -1), (_desc(vp=264), -1), (_desc(pages=0), -1), (_desc(d=96), -2),
                      (_desc(group=16), -2), (_desc(group=128), -2), (_desc(page=24), -2), (_desc(page=8), -2),
                      (_desc(page=2048), -2), (_desc(heads=65536), -2)):
        assert append(bad) == code
        assert L.gptq_kv4_read(ctypes.byref(bad), fake, 2, fake, None, 2, 4, 2, fake, fake, None, None) == code
        assert L.gptq_kv4_attention(ctypes.byref(bad), fake, 256, 64, 2, 2, 4, fake, 2, fake, ctypes.c_float(0.1),
                                    fake, 256, 64, fake, 1 << 30, None, None) == code
    assert append(k=None) == -1 and append(kt=100) == -1 and append(v=P(260)) == -1 and append(dt=0) == -1
    assert append(table=None) == -1 and append(width=0) == -1 and append(start=None) == -1 and append(tokens=-1) == -1
    assert append(tokens=0) == 0 and append(n=0) == 0

    def read(table=fake, width=2, cu=fake, n=2, tokens=4, dt=0, k=fake, v=fake):
        return L.gptq_kv4_read(ctypes.byref(ok), table, width, cu, None, n, tokens, dt, k, v, None, None)

    assert read(table=None) == -1 and read(cu=None) == -1 and read(dt=3) == -1 and read(k=P(260)) == -1
    assert read(tokens=0) == 0

    def attend(q=fake, qt=256, qh=64, dt=2, n=2, hq=4, table=fake, width=2, lengths=fake, scale=0.1, o=fake, ws=fake,
               wsb=1 << 30):
        return L.gptq_kv4_attention(ctypes.byref(ok), q, qt, qh, dt, n, hq, table, width, lengths,
                                    ctypes.c_float(scale), o, 256, 64, ws, wsb, None, None)

    assert attend(q=None) == -1 and attend(qt=100) == -1 and attend(dt=0) == -1 and attend(hq=3) == -1
    assert attend(lengths=None) == -1 and attend(scale=float("nan")) == -1 and attend(n=65536) == -2
    assert attend(hq=65536) == -2 and attend(width=1 << 28) == -2
    need = G.kv4_attention_workspace_size(2, 4, 2, 64, 2, 16)
    assert need > 0 and attend(wsb=need - 1) == -7 and attend(ws=None) == -7 and attend(ws=P(264)) == -7
    assert attend(n=0) == 0


def test_binding_refuses_before_the_library():
    """Shapes, types and overlaps raise ValueError on host tensors (nothing reaches the library)."""
    X, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for kw in (dict(Y=torch.zeros(4, 63)), dict(gate=w), dict(x_out=X), dict(post_weight=w),
               dict(Y=X, post_bias=w), dict(Y=X, gate=torch.ones(4, 63, dtype=torch.bfloat16)),
               dict(Y=X, gate=torch.ones(64)), dict(bias=torch.ones(63, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            G.add_norm(X, w, **kw)
    with pytest.raises(ValueError):
        G.add_norm(X.t(), w)
    with pytest.raises(ValueError, match="CUDA"):
        G.add_norm(X, w)
    qkv, cs = torch.zeros(3, 8 * 64), torch.zeros(8, 32)
    for a, kw in (((qkv, cs, None, 4, 2, 64), {}), ((qkv, cs, cs, 4, 1, 64), {}),
                  ((qkv, cs.double(), cs.double(), 4, 2, 64), {}), ((qkv, cs, cs, 4, 2, 64), {"dtype": torch.float32}),
                  ((qkv, cs, cs, 4, 2, 64), {"positions": torch.zeros(3, dtype=torch.int64)}),
                  ((qkv, cs, cs, 4, 2, 64), {"bias": torch.zeros(3)})):
        with pytest.raises(ValueError):
            G.rope_qkv(*a, **kw)
    h = dict(dtype=torch.float16)
    q, k = torch.zeros(8, 4, 64, **h), torch.zeros(8, 2, 64, **h)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for a in ((q, k, k[:7], cu), (q, k, k.bfloat16(), cu), (q, torch.zeros(8, 3, 64, **h), torch.zeros(8, 3, 64, **h), cu),
              (q, k, k, cu.long()), (q.float(), k.float(), k.float(), cu), (q, k, k, cu, torch.zeros(3, dtype=torch.int32)),
              (q.transpose(1, 2), k, k, cu)):
        with pytest.raises(ValueError):
            G.attention(*a)
    with pytest.raises(ValueError, match="CUDA"):
        G.attention(q, k, k, cu)
    c = G.kv4_alloc(3, 16, 2, 64, 32, device="cpu")
    assert c.k_codes.shape == (3, 2, 16, 8) and c.v_params.shape == (3, 2, 16, 2, 2)
    table = torch.zeros(1, 3, dtype=torch.int32)
    st, ln = torch.zeros(1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for a in ((k[:, :1], k[:, :1], table, cu, st), (k, k, table[0], cu, st), (k, k, table, cu, st.long()),
              (k, k.bfloat16(), table, cu, st), (k, k, table, torch.zeros(3, dtype=torch.int32), st)):
        with pytest.raises(ValueError):
            G.kv4_append(c, *a)
    with pytest.raises(ValueError, match="CUDA"):
        G.kv4_append(c, k, k, table, cu, st)
    for a in ((q[:1, :3], table, ln), (q[:2], table, ln), (q[:1].float(), table, ln), (q[:1], table, ln.long())):
        with pytest.raises(ValueError):
            G.kv4_attention(a[0], c, *a[1:])
    bad = G.KV4Cache(c.k_codes, c.k_params, c.v_codes[:2], c.v_params, 32)
    with pytest.raises(ValueError):
        G.kv4_read(bad, table, cu, 8)
    with pytest.raises(ValueError):
        G.kv4_read(G.KV4Cache(c.k_codes, c.k_params, c.v_codes, c.v_params, 64), table, cu, 8)


def test_overlap_check():
    from post_weight_quantization_15_b200.block import _apart
    t = torch.zeros(64)
    _apart(t[:32], t[32:], None)
    _apart(t[:0], t)
    with pytest.raises(ValueError):
        _apart(t[:33], t[32:])


def test_oracle_by_hand():
    # RMS norm of (3, 4): mean square 12.5; layer norm of (1, 3): centred (-1, 1), mean square 1
    assert np.allclose(B.norm([[3.0, 4.0]], [1, 2], None, 0.0, False), [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    assert np.allclose(B.norm([[1.0, 3.0]], [1, 2], [1, 1], 0.0, True), [[0.0, 3.0]])
    # a quarter turn: (a, b) -> (-b, a), pairs (0, 2), (1, 3) or (0, 1), (2, 3)
    x = np.array([[1.0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12]])
    c, s = np.zeros((1, 2)), np.ones((1, 2))
    q, k, v = B.rope_qkv(x, c, s, 1, 1, 4, [0])
    assert q.ravel().tolist() == [-3, -4, 1, 2] and k.ravel().tolist() == [-7, -8, 5, 6]
    assert v.ravel().tolist() == [9, 10, 11, 12]
    q, _, _ = B.rope_qkv(x, c, s, 1, 1, 4, [0], interleaved=True)
    assert q.ravel().tolist() == [-2, 1, -4, 3]
    # two equal scores weigh a half each; an unseen NaN key takes no part; a row without keys is 0
    o, _ = B.attend([[1.0], [1.0], [1.0]], [[2.0], [2.0], [np.nan]], [[1.0], [3.0], [np.inf]], 1.0, [2, 1, 0])
    assert o.ravel().tolist() == [2.0, 1.0, 0.0]
    # 0 .. 15: scale 1, zero point 0; -5 .. 10: zero point 5
    c, s, z = B.kv4_quantize(np.stack([np.arange(16.0), np.arange(-5.0, 11)]).repeat(2, 1), 32)
    assert s.ravel().tolist() == [1, 1] and z.ravel().tolist() == [0, 5]
    assert c[0].tolist() == np.arange(16).repeat(2).tolist() == c[1].tolist()
    assert B.kv4_values(c, s, z)[1].tolist() == np.arange(-5.0, 11).repeat(2).tolist()
    assert B.kv4_words(np.array([[1, 2, 3, 4, 5, 6, 7, 8]])).tolist() == [[0x87654321]]
