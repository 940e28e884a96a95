"""The attention half of a decoder block: argument marshalling only, as in gptq.py.

    add_norm(X, weight, Y, ...)                  -> (Xn, h)    norms around a block, residual, gate
    rope_qkv(QKV, cos, sin, heads_q, heads_kv, head_dim, ...)  -> (q, k, v)
    attention(q, k, v, cu_q, cu_k, causal)       -> o          packed prompts, grouped heads
    kv4_alloc(pages, page_size, heads, head_dim, group) -> KV4Cache   keys and values in 4 bits
    kv4_append(cache, k, v, table, cu, start)    tokens into the cache
    kv4_read(cache, table, cu, tokens, start)    -> (k, v)     and back
    kv4_attention(q, cache, table, lengths)      -> o          one token per sequence

include/gptq.h holds the formulas, the layouts and what is recorded in the status block.
All tensors of a call are on one device, which need not be the current one.  stream: the
stream to launch on (default: that device's current stream); the caller orders it with the
streams that made the inputs.  What a call allocates belongs to the stream it launches on.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from .gptq import _DTYPE_CODE, _KV4, OK, GptqError, _check, _require_cuda, lib, workspace

_16BIT = (torch.float16, torch.bfloat16)
_INT_MAX = 2 ** 31 - 1        # the C ABI's counts; ctypes would cut a larger one off without a word


def _too_large(what: str):
    return ValueError(f"{what}: sizes from 2^31 on are not supported")


class _Launching:
    """With the call's device and stream current (allocations go to that stream): the stream's pointer.

    A call on the current device's current stream, the usual one, changes and restores nothing."""
    __slots__ = ("ptr", "cm")

    def __init__(self, stream, first: torch.Tensor, *ts: Optional[torch.Tensor]):
        dev = first.get_device()
        if dev < 0:
            _require_cuda(first)
        for t in ts:
            if t is not None and t.get_device() != dev:
                _require_cuda(t)
                raise ValueError("all tensors must be on one device")
        self.cm = None
        if stream is not None:
            if stream.device.index != dev:
                raise ValueError("stream must be on the tensors' device")
            self.ptr = stream.cuda_stream
            self.cm = torch.cuda.stream(stream)
        else:
            self.ptr = torch._C._cuda_getCurrentRawStream(dev)
            if dev != torch.cuda.current_device():
                self.cm = torch.cuda.device(dev)

    def __enter__(self):
        if self.cm is not None:
            self.cm.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        if self.cm is not None:
            self.cm.__exit__(*exc)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _status_ok(status: Optional[torch.Tensor]):
    if status is not None and (status.numel() != 4 or status.dtype != torch.int32 or not status.is_contiguous()):
        raise ValueError("status must be a contiguous int32 [4] tensor")


def _span(t: torch.Tensor):
    """First and last byte of a tensor's elements (end exclusive)."""
    if t.numel() == 0:
        return t.data_ptr(), t.data_ptr()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(out: Optional[torch.Tensor], *ins: Optional[torch.Tensor]):
    """Raise if out's memory overlaps an input's."""
    if out is None or out.numel() == 0:
        return
    a0, a1 = _span(out)
    for t in ins:
        if t is not None and t.numel() > 0 and t.device == out.device:
            b0, b1 = _span(t)
            if a0 < b1 and b0 < a1:
                raise ValueError("an output overlaps an input")


def _rows(t: torch.Tensor, tokens: int, d: int, what: str):
    if t.dtype in _DTYPE_CODE and t.shape == (tokens, d):
        if t.is_contiguous() or ((d == 1 or t.stride(1) == 1) and (tokens == 1 or t.stride(0) >= d)):
            if tokens > _INT_MAX or d > _INT_MAX:
                raise _too_large(what)
            return
    raise ValueError(f"{what} must be an fp32/fp16/bf16 [{tokens}, {d}] tensor with contiguous rows")


def _vector(t: torch.Tensor, dtype, d: int):
    if t.dtype != dtype or t.dim() != 1 or t.numel() != d or not t.is_contiguous():
        raise ValueError(f"weight, bias, post_weight and post_bias must be contiguous [{d}] tensors of one type")


def _ld(t: Optional[torch.Tensor], d: int) -> int:
    """Row stride; that of a single row is not used (torch may report any)."""
    return d if t is None or t.shape[0] <= 1 else t.stride(0)


def _ints(t: torch.Tensor, shape, what: str):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)}")
    if shape[0] > _INT_MAX:
        raise _too_large(what)


# --------------------------------------------------------------------------- #
# The residual stream
# --------------------------------------------------------------------------- #
def add_norm(X: torch.Tensor, weight: torch.Tensor, Y: Optional[torch.Tensor] = None,
             post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
             eps: float = 1e-6, center: bool = False, bias: Optional[torch.Tensor] = None,
             post_bias: Optional[torch.Tensor] = None, x_out: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(Xn, h): Xn = X + alpha . gate . N(Y; post_weight, post_bias), h = N(Xn; weight, bias).

    N is the RMS norm, or with center the layer norm; without post_weight N(Y) is Y, without Y
    Xn is X itself.  X [tokens, d] and Y [tokens, d] fp32/fp16/bf16; weights, biases [d] and
    gate [d] or [tokens, d] of one of those types.  x_out may be X (the stream updated in place).
    """
    if X.dim() != 2:
        raise ValueError("X must be a [tokens, d] tensor")
    tokens, d = X.shape
    _rows(X, tokens, d, "X")
    if Y is None and (post_weight is not None or gate is not None or x_out is not None):
        raise ValueError("post_weight, gate and x_out belong to Y")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias belongs to post_weight")
    if Y is not None:
        _rows(Y, tokens, d, "Y")
    pt = weight.dtype
    if pt not in _DTYPE_CODE:
        raise ValueError("weight must be fp32/fp16/bf16")
    _vector(weight, pt, d)
    if bias is not None:
        _vector(bias, pt, d)
    if post_weight is not None:
        _vector(post_weight, pt, d)
        if post_bias is not None:
            _vector(post_bias, pt, d)
    ld_gate = 0
    if gate is not None:
        if gate.dtype != pt:
            raise ValueError("gate must have weight's type")
        if gate.dim() == 2:
            _rows(gate, tokens, d, "gate")
            ld_gate = _ld(gate, d)
        elif tuple(gate.shape) != (d,) or not gate.is_contiguous():
            raise ValueError(f"gate must be a contiguous [{d}] or a [{tokens}, {d}] tensor")
    _status_ok(status)
    with _Launching(stream, X, weight, Y, post_weight, gate, bias, post_bias, x_out, out, status) as s:
        given = [t for t in (out, x_out) if t is not None] if out is not None or x_out is not None else ()
        if out is None:
            out = torch.empty_like(X, memory_format=torch.contiguous_format)
        if Y is not None and x_out is None:
            x_out = torch.empty_like(X, memory_format=torch.contiguous_format)
        if given:                         # what was allocated here fits and lies apart
            for t in given:
                _rows(t, tokens, d, "out" if t is out else "x_out")
                if t.dtype != X.dtype:
                    raise ValueError("out and x_out must have X's type")
            par = (weight, bias, post_weight, post_bias, gate)
            _apart(out, X, Y, x_out, *par)
            same = x_out is not None and x_out.data_ptr() == X.data_ptr() and _ld(x_out, d) == _ld(X, d)
            _apart(x_out, None if same else X, Y, *par)
        code = _DTYPE_CODE[X.dtype]
        rc = lib().gptq_add_norm(X.data_ptr(), code, d if tokens <= 1 else X.stride(0), _at(Y),
                                 code if Y is None else _DTYPE_CODE[Y.dtype], _ld(Y, d), weight.data_ptr(), _at(bias),
                                 _at(post_weight), _at(post_bias), _at(gate), ld_gate, _DTYPE_CODE[pt], tokens, d,
                                 float(alpha), float(eps), bool(center), _at(x_out), _ld(x_out, d) if given else d,
                                 out.data_ptr(), _ld(out, d) if given else d, _at(status), s)
    if rc != OK:
        raise GptqError(rc, "gptq_add_norm")
    return (X if Y is None else x_out), out


def rope_qkv(QKV: torch.Tensor, cos: Optional[torch.Tensor], sin: Optional[torch.Tensor], heads_q: int, heads_kv: int,
             head_dim: int, positions: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
             interleaved: bool = False, dtype=torch.bfloat16, status: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(q, k, v) from the product of the stacked q, k and v layers, q and k rotated by position.

    QKV [tokens, (heads_q + 2 heads_kv) head_dim] fp32/fp16/bf16; bias fp32; cos, sin fp32
    [positions, rot / 2] (None: no rotation); positions int32 [tokens] (None: 0, 1, ...).
    """
    heads_q, heads_kv, head_dim = int(heads_q), int(heads_kv), int(head_dim)
    cols = (heads_q + 2 * heads_kv) * head_dim
    if heads_q < 1 or heads_kv < 1 or head_dim < 2 or QKV.dim() != 2:
        raise ValueError("QKV must be a [tokens, (heads_q + 2 heads_kv) head_dim] tensor")
    tokens = QKV.shape[0]
    _rows(QKV, tokens, cols, "QKV")
    if dtype not in _16BIT:
        raise ValueError("dtype must be float16 or bfloat16")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    rot = max_pos = 0
    if cos is not None:
        if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.dim() != 2 or sin.shape != cos.shape \
                or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous fp32 [positions, rot / 2] tensors of one shape")
        max_pos, half = cos.shape
        rot = 2 * half
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (cols,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous fp32 [{cols}] tensor")
    if positions is not None:
        _ints(positions, (tokens,), "positions")
    _status_ok(status)
    with _Launching(stream, QKV, cos, sin, positions, bias, status) as s:
        q = QKV.new_empty((tokens, heads_q, head_dim), dtype=dtype)
        k = QKV.new_empty((tokens, heads_kv, head_dim), dtype=dtype)
        v = torch.empty_like(k)
        rc = lib().gptq_rope_qkv(QKV.data_ptr(), _DTYPE_CODE[QKV.dtype], cols if tokens <= 1 else QKV.stride(0),
                                 _at(bias), _at(cos), _at(sin), max_pos, rot, bool(interleaved), _at(positions),
                                 tokens, heads_q, heads_kv, head_dim, _DTYPE_CODE[dtype], q.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), _at(status), s)
    if rc != OK:
        raise GptqError(rc, "gptq_rope_qkv")
    return q, k, v


# --------------------------------------------------------------------------- #
# Attention over packed prompts
# --------------------------------------------------------------------------- #
def _heads(t: torch.Tensor, dtype, what: str):
    """(tokens, heads, head_dim, token stride, head stride); strides of a single token or head are not used."""
    if t.dim() == 3 and t.dtype == dtype:
        n, h, d = t.shape
        ts, hs, fs = t.stride()
        if h > 0 and (fs == 1 or d <= 1):
            if n > _INT_MAX or h > _INT_MAX or d > _INT_MAX:
                raise _too_large(what)
            if h == 1:
                hs = d
            return n, h, d, ts if n > 1 else h * hs, hs
    raise ValueError(f"{what} must be a [tokens, heads, head_dim] tensor of type {dtype} with contiguous features")


def _written(out: torch.Tensor, like: torch.Tensor, *ins: torch.Tensor):
    """(token stride, head stride) of a given output: every row has a place of its own, apart from the inputs."""
    n, h, d, ts, hs = _heads(out, like.dtype, "out")
    if out.shape != like.shape:
        raise ValueError("out must have q's shape")
    if (h > 1 and hs < d) or (n > 1 and ts < d) or \
            (n > 1 and h > 1 and ts < (h - 1) * hs + d and hs < (n - 1) * ts + d):
        raise ValueError("out's rows must not overlap")
    _apart(out, *ins)
    return ts, hs


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
              cu_k: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
              out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """o = softmax(scale q k^T) v over the sequences of a packed batch.

    q [total_q, heads_q, head_dim], k and v [total_k, heads_kv, head_dim], fp16 or bf16; cu_q and
    cu_k int32 [sequences + 1], the first row of each sequence and the end (cu_k None: cu_q).
    causal: the last query of a sequence sees its last key.  scale None: 1 / sqrt(head_dim).
    Rows of o that belong to no sequence are not written.
    """
    dt = q.dtype
    if dt not in _16BIT:
        raise ValueError("q must be fp16 or bf16")
    nq, hq, d, qt, qh = _heads(q, dt, "q")
    nk, hk, dk, kt, kh = _heads(k, dt, "k")
    nv, hv, dv, vt, vh = _heads(v, dt, "v")
    if nk != nv or hk != hv or dk != d or dv != d or hq % hk != 0:
        raise ValueError("k and v must have one shape, q's head size, and a number of heads that divides q's")
    if cu_k is None:
        cu_k = cu_q
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be int32 [sequences + 1]")
    _ints(cu_q, cu_q.shape, "cu_q")
    if cu_k is not cu_q:
        _ints(cu_k, cu_q.shape, "cu_k")
    ot, oh = (hq * d, d) if out is None else _written(out, q, q, k, v)
    _status_ok(status)
    with _Launching(stream, q, k, v, cu_q, cu_k, out, status) as s:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        rc = lib().gptq_attention(q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _DTYPE_CODE[dt],
                                  cu_q.data_ptr(), cu_k.data_ptr(), cu_q.numel() - 1, nq, nk, hq, hk, d,
                                  d ** -0.5 if scale is None else float(scale), bool(causal), out.data_ptr(), ot, oh,
                                  _at(status), s)
    if rc != OK:
        raise GptqError(rc, "gptq_attention")
    return out


# --------------------------------------------------------------------------- #
# The cache in 4 bits
# --------------------------------------------------------------------------- #
@dataclasses.dataclass
class KV4Cache:
    k_codes: torch.Tensor    # int32 [pages, heads, page_size, head_dim / 8]
    k_params: torch.Tensor   # fp16 [pages, heads, page_size, head_dim / group, 2]: scale, zero point
    v_codes: torch.Tensor
    v_params: torch.Tensor
    group: int


def kv4_alloc(pages: int, page_size: int, heads: int, head_dim: int, group: int = 128, device="cuda") -> KV4Cache:
    """An empty cache (every value 0)."""
    t = [torch.zeros(*s, dtype=dt, device=device)
         for _ in range(2) for s, dt in (((pages, heads, page_size, head_dim // 8), torch.int32),
                                         ((pages, heads, page_size, head_dim // group, 2), torch.float16))]
    return KV4Cache(*t, group=int(group))


def _cache(c: KV4Cache) -> _KV4:
    kc, kp, vc, vp, group = c.k_codes, c.k_params, c.v_codes, c.v_params, c.group
    if kc.dim() != 4:
        raise ValueError("k_codes must be int32 [pages, heads, page_size, head_dim / 8]")
    shape = kc.shape
    pages, heads, page, words = shape
    if pages > _INT_MAX or heads > _INT_MAX or page > _INT_MAX:
        raise _too_large("k_codes")
    d = words * 8
    if group < 1 or d % group:
        raise ValueError("group must divide head_dim")
    i32, f16 = torch.int32, torch.float16
    if kc.dtype != i32 or vc.dtype != i32 or vc.shape != shape or not kc.is_contiguous() or not vc.is_contiguous():
        raise ValueError("codes must be contiguous int32 tensors of one shape")
    if kp.dtype != f16 or vp.dtype != f16 or kp.shape != (pages, heads, page, d // group, 2) or vp.shape != kp.shape \
            or not kp.is_contiguous() or not vp.is_contiguous():
        raise ValueError("params must be contiguous fp16 [pages, heads, page_size, head_dim / group, 2] tensors")
    return _KV4(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), pages, page, heads, d, int(group))


def _table(table: torch.Tensor, count: int):
    if table.dim() != 2 or table.dtype != torch.int32 or table.shape[0] != count or not table.is_contiguous():
        raise ValueError("table must be a contiguous int32 tensor [sequences, pages of a sequence]")
    if table.shape[1] > _INT_MAX:
        raise _too_large("table")


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, cu: torch.Tensor,
               start: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> KV4Cache:
    """Tokens' keys and values into the cache: row t of k and v, cu[b] <= t < cu[b + 1], goes to
    position start[b] + t - cu[b] of sequence b, which lies in page table[b][position / page_size].

    k, v [tokens, heads, head_dim] fp16 or bf16; table int32 [sequences, width], cu int32
    [sequences + 1], start int32 [sequences].  A position must be written by one token only.
    """
    desc = _cache(cache)
    dt = k.dtype
    if dt not in _16BIT:
        raise ValueError("k must be fp16 or bf16")
    n, h, d, kt, kh = _heads(k, dt, "k")
    nv, hv, dv, vt, vh = _heads(v, dt, "v")
    if n != nv or h != hv or d != dv or h != desc.heads or d != desc.head_dim:
        raise ValueError("k and v must be [tokens, heads, head_dim] with the cache's heads and head_dim")
    count = start.numel()
    _ints(start, (count,), "start")
    _ints(cu, (count + 1,), "cu")
    _table(table, count)
    _status_ok(status)
    with _Launching(stream, cache.k_codes, cache.k_params, cache.v_codes, cache.v_params, k, v, table, cu, start,
                    status) as s:
        rc = lib().gptq_kv4_append(ctypes.byref(desc), k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _DTYPE_CODE[dt], n,
                                   table.data_ptr(), table.shape[1], cu.data_ptr(), start.data_ptr(), count,
                                   _at(status), s)
    if rc != OK:
        raise GptqError(rc, "gptq_kv4_append")
    return cache


def kv4_read(cache: KV4Cache, table: torch.Tensor, cu: torch.Tensor, tokens: int, start: Optional[torch.Tensor] = None,
             dtype=torch.bfloat16, status: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [tokens, heads, head_dim] as the cache holds them: row t, cu[b] <= t < cu[b + 1], is
    position start[b] + t - cu[b] of sequence b (start None: 0).  Rows of no sequence are not written."""
    desc = _cache(cache)
    if dtype not in _DTYPE_CODE:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    count = cu.numel() - 1
    if count < 0 or tokens < 0:
        raise ValueError("cu must be int32 [sequences + 1] and tokens not negative")
    if tokens > _INT_MAX:
        raise _too_large("tokens")
    _ints(cu, (count + 1,), "cu")
    if start is not None:
        _ints(start, (count,), "start")
    _table(table, count)
    _status_ok(status)
    with _Launching(stream, cache.k_codes, cache.k_params, cache.v_codes, cache.v_params, table, cu, start,
                    status) as s:
        k = cache.k_codes.new_empty((int(tokens), desc.heads, desc.head_dim), dtype=dtype)
        v = torch.empty_like(k)
        _check(lib().gptq_kv4_read(ctypes.byref(desc), _at(table), table.shape[1], _at(cu), _at(start), count,
                                   int(tokens), _DTYPE_CODE[dtype], _at(k), _at(v), _at(status), s),
               "gptq_kv4_read")
    return k, v


def kv4_attention_workspace_size(count: int, heads_q: int, heads_kv: int, head_dim: int, width: int,
                                 page_size: int) -> int:
    return int(lib().gptq_kv4_attention_workspace_size(count, heads_q, heads_kv, head_dim, width, page_size))


def kv4_attention(q: torch.Tensor, cache: KV4Cache, table: torch.Tensor, lengths: torch.Tensor,
                  scale: Optional[float] = None, ws: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """o [sequences, heads_q, head_dim]: one query token per sequence against positions
    0 .. lengths[b] - 1 of its cache (lengths int32 [sequences]; 0 gives a row of 0).

    ws: at least kv4_attention_workspace_size(...) bytes (None: allocated for the call); calls that
    may run at the same time need one each."""
    desc = _cache(cache)
    dt = q.dtype
    if dt not in _16BIT:
        raise ValueError("q must be fp16 or bf16")
    count, hq, d, qt, qh = _heads(q, dt, "q")
    if d != desc.head_dim or hq % desc.heads != 0:
        raise ValueError("q must have the cache's head size and a multiple of its heads")
    _ints(lengths, (count,), "lengths")
    _table(table, count)
    ot, oh = (hq * d, d) if out is None else _written(out, q, q)
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _status_ok(status)
    width = table.shape[1]
    with _Launching(stream, cache.k_codes, cache.k_params, cache.v_codes, cache.v_params, q, table, lengths, ws, out,
                    status) as s:
        if ws is None:
            ws = workspace(lib().gptq_kv4_attention_workspace_size(count, hq, desc.heads, d, width, desc.page_size),
                           q.device)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        rc = lib().gptq_kv4_attention(ctypes.byref(desc), q.data_ptr(), qt, qh, _DTYPE_CODE[dt], count, hq,
                                      table.data_ptr(), width, lengths.data_ptr(),
                                      d ** -0.5 if scale is None else float(scale), out.data_ptr(), ot, oh,
                                      ws.data_ptr(), ws.numel() * ws.element_size(), _at(status), s)
    if rc != OK:
        raise GptqError(rc, "gptq_kv4_attention")
    return out
