"""Whole decoder blocks: calibration through both halves, prompts into a 4-bit cache, single tokens.

pipeline.py chains the solver over the MLP half of a block; here the attention half comes before it,
with the operators of block.py between the quantized layers.  Activations are token-major,
[tokens, features] bf16; a block of width d with hq query and hk k/v heads of D features is

    h  = N(x; norm_attn)                         add_norm (RMS)
    q, k, v = rotary(h . [Wq; Wk; Wv]^T)         linear_bf16 or qmatvec, rope_qkv
    a  = softmax(q k^T / sqrt(D)) v              attention; kv4_attention over the cache
    x' = x + a . Wo^T,  h' = N(x'; norm_mlp)     add_norm, one pass
    x'' = x' + (silu(h' Wgate^T) * (h' Wup^T)) . Wdown^T

    quantize_decoder_blocks   each layer calibrated on what the layers before it, quantized, produce
    prompt_blocks             a packed batch of prompts through quantized blocks, into their caches
    decode_blocks             one token of each of up to 16 sequences, against the caches

Products with the dequantized weights run on the tensor cores (prompts), with the stored codes in
qmatvec (single tokens).
"""
from __future__ import annotations

import dataclasses
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import block as B
from . import gptq as G


@dataclasses.dataclass
class DecoderWeights:
    """One block's weights: layers [out, in] fp16/bf16/fp32, norms [d] (bf16, fp16 or fp32)."""
    wq: torch.Tensor
    wk: torch.Tensor
    wv: torch.Tensor
    wo: torch.Tensor
    w_gate: torch.Tensor
    w_up: torch.Tensor
    w_down: torch.Tensor
    norm_attn: torch.Tensor
    norm_mlp: torch.Tensor


@dataclasses.dataclass
class Rotary:
    """Heads of a block and its rotary tables, cos and sin fp32 [positions, rot / 2]."""
    heads_q: int
    heads_kv: int
    head_dim: int
    cos: Optional[torch.Tensor]
    sin: Optional[torch.Tensor]
    interleaved: bool = False


@dataclasses.dataclass
class QuantizedBlock:
    qkv: G.QuantizedLayer          # q, k and v stacked along the outputs
    o: G.QuantizedLayer
    gate_up: G.QuantizedLayer      # gate's rows first
    down: G.QuantizedLayer
    norm_attn: torch.Tensor
    norm_mlp: torch.Tensor
    eps: float
    stages: Optional[Dict[str, torch.Tensor]] = None   # what each stage gave (record=True)


def _quantize(ws: Sequence[torch.Tensor], X: torch.Tensor, bits, group_size, sym, desc_act, damp, st):
    """The layers ws quantized together on the token-major calibration input X; their processing order."""
    n = X.shape[1]
    H = torch.zeros((n, n), dtype=torch.float32, device=X.device)
    hd = torch.zeros(n, dtype=torch.float64, device=X.device) if desc_act else None
    G.hessian_accumulate(H, G.transpose_bf16(X, st), hd, st)
    prep = G.prepare(H, damp, desc_act, hd, st)
    if len(ws) == 1:
        return G.quantize_layer(ws[0], prep, bits, group_size, sym), prep.perm
    return G.quantize_layers(ws, prep, bits, group_size, sym)[0], prep.perm


def _forward(q: G.QuantizedLayer, X: torch.Tensor, st) -> torch.Tensor:
    """fp32 [tokens, out] = X . What^T, the weights dequantized to bf16."""
    return G.linear_bf16(X, G.dequantize(q, torch.bfloat16, st), st)


def _mlp_hidden(gate_up: G.QuantizedLayer, h: torch.Tensor, st) -> torch.Tensor:
    What = G.dequantize(gate_up, torch.bfloat16, st)
    f = What.shape[0] // 2
    return G.silu_mul(G.linear_bf16(h, What[:f], st), G.linear_bf16(h, What[f:], st), st)


def _without_strays(X: torch.Tensor, cu: torch.Tensor) -> torch.Tensor:
    """X with the rows of no sequence (before cu[0], from cu[-1] on) as 0."""
    B._ints(cu, (cu.numel(),), "cu")
    if cu.numel() < 2:
        return torch.zeros_like(X)
    t = torch.arange(X.shape[0], dtype=torch.int32, device=X.device)
    return torch.where(((t >= cu[0]) & (t < cu[-1]))[:, None], X, 0)


def _watched(status: Optional[torch.Tensor], X: torch.Tensor):
    """(status block, whether the call made it and has to read it); none inside a stream capture, where nothing
    can be read back."""
    if status is not None or torch.cuda.is_current_stream_capturing():
        return status, False
    return G.new_status(X.device), True


def _check_stream(X: torch.Tensor):
    if X.dim() != 2 or X.dtype != torch.bfloat16 or not X.is_contiguous():
        raise ValueError("X must be a contiguous bf16 [tokens, d] tensor")
    if not X.is_cuda:
        raise ValueError("X must be a CUDA tensor")


def quantize_decoder_blocks(X0: torch.Tensor, cu: torch.Tensor, blocks: Sequence[DecoderWeights], rotary: Rotary,
                            positions: Optional[torch.Tensor] = None, eps: float = 1e-6, bits: int = 4,
                            group_size: int = 128, sym: bool = True, desc_act: bool = True,
                            damp_percent: float = 0.01, record: bool = False,
                            status: Optional[torch.Tensor] = None) -> Tuple[List[QuantizedBlock], torch.Tensor]:
    """Quantize decoder blocks in sequence; returns (the blocks, the last block's output).

    X0 bf16 [tokens, d] (tokens a multiple of 8), the packed calibration sequences; cu int32
    [sequences + 1] their first rows and the end (rows of no sequence, such as those that pad the batch to a
    multiple of 8, take no part in the calibration and come out as 0); positions int32 [tokens] for the rotary tables
    (None: row t is at position t).  decode_blocks takes desc_act blocks too, more slowly (qmatvec
    reads their groups column by column).
    """
    _check_stream(X0)
    st = status if status is not None else G.new_status(X0.device)
    how = (bits, group_size, sym, desc_act, damp_percent, st)
    r = rotary
    x, y = _without_strays(X0, cu), None   # the stream, and what is still to be added to it
    out: List[QuantizedBlock] = []
    for w in blocks:
        x, h = B.add_norm(x, w.norm_attn, Y=y, eps=eps, status=st)
        x_in = x
        qkv, perm_qkv = _quantize([w.wq, w.wk, w.wv], h, *how)
        q, k, v = B.rope_qkv(_forward(qkv, h, st), r.cos, r.sin, r.heads_q, r.heads_kv, r.head_dim, positions,
                             interleaved=r.interleaved, status=st)
        # (attention leaves rows of no sequence as they are: 0, where the Hessian of o must not see them)
        a = B.attention(q, k, v, cu, out=torch.zeros_like(q), status=st).flatten(1)
        o, perm_o = _quantize([w.wo], a, *how)
        x_mid, h2 = B.add_norm(x, w.norm_mlp, Y=_forward(o, a, st), eps=eps, status=st)
        gate_up, perm_gate_up = _quantize([w.w_gate, w.w_up], h2, *how)
        m = _mlp_hidden(gate_up, h2, st)
        down, perm_down = _quantize([w.w_down], m, *how)
        x, y = x_mid, _forward(down, m, st)
        out.append(QuantizedBlock(qkv, o, gate_up, down, w.norm_attn, w.norm_mlp, eps, dict(
            x_in=x_in, h=h, q=q, k=k, v=v, a=a, x_mid=x_mid, h_mlp=h2, m=m, y=y, perm_qkv=perm_qkv, perm_o=perm_o,
            perm_gate_up=perm_gate_up, perm_down=perm_down) if record else None))
    X = x if y is None else G.residual_add(x, y, st)
    G.raise_on_status(st, "quantize_decoder_blocks")
    return out, X


def _positions(cu: torch.Tensor, start: Optional[torch.Tensor], tokens: int) -> torch.Tensor:
    """Each row's position inside its sequence, behind start[b]; 0 for a row of no sequence."""
    B._ints(cu, (cu.numel(),), "cu")
    if start is not None:
        B._ints(start, (max(0, cu.numel() - 1),), "start")
    if cu.numel() < 2:
        return torch.zeros(tokens, dtype=torch.int32, device=cu.device)
    t = torch.arange(tokens, dtype=torch.int32, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1                     # the last sequence that begins by row t
    inside = (b >= 0) & (b < cu.numel() - 1)
    b = b.clamp(0, cu.numel() - 2)
    pos = t - cu[b] if start is None else t - cu[b] + start[b]
    return torch.where(inside, pos, 0)


@dataclasses.dataclass
class _Past:
    """Where a continued batch's keys lie when the cached ones come before them."""
    cu_k: torch.Tensor             # int32 [sequences + 1]: cached and new keys of each sequence
    total: int
    new: torch.Tensor              # the new tokens' rows among them
    first: int                     # the first and last + 1 of the batch's tokens that a sequence has
    last: int


def _past(cu: torch.Tensor, start: torch.Tensor, table: torch.Tensor, capacity: int, tokens: int) -> Optional[_Past]:
    """None if no sequence has anything before its new tokens.  Reads cu and start back."""
    n = cu.numel() - 1
    B._ints(cu, (n + 1,), "cu")
    B._ints(start, (n,), "start")
    B._table(table, n)
    c0, c1, s0 = torch.stack([cu[:-1], cu[1:], start]).tolist()
    if any(a < 0 or b < a or b > tokens for a, b in zip(c0, c1)):
        raise ValueError("cu must be non-decreasing rows of X")
    if any(s < 0 or s + b - a > capacity for a, b, s in zip(c0, c1, s0)):
        raise ValueError("a sequence's positions do not fit its row of the table")
    s0 = [s if b > a else 0 for a, b, s in zip(c0, c1, s0)]           # (without a query nothing is read)
    if not any(s0):
        return None
    ends = [0]
    for a, b, s in zip(c0, c1, s0):
        ends.append(ends[-1] + s + b - a)
    if ends[-1] > 2 ** 31 - 1:
        raise ValueError("the sequences and what precedes them have more than 2^31 - 1 tokens")
    lens = torch.tensor([b - a for a, b in zip(c0, c1)], device=cu.device)
    shift = torch.tensor([e + s - a for e, s, a in zip(ends, s0, c0)], device=cu.device)
    new = torch.arange(c0[0], c1[-1], device=cu.device) + shift.repeat_interleave(lens, output_size=c1[-1] - c0[0])
    return _Past(torch.tensor(ends, dtype=torch.int32, device=cu.device), ends[-1], new, c0[0], c1[-1])


def _attend(q, k, v, cu, cache, table, past: Optional[_Past], status) -> torch.Tensor:
    """Attention of the new tokens over themselves, and over what the cache holds before them."""
    o = torch.zeros_like(q)                        # rows of no sequence attend to nothing
    if past is None:
        return B.attention(q, k, v, cu, out=o, status=status)
    held = B.kv4_read(cache, table, past.cu_k, past.total, dtype=k.dtype, status=status)
    for h, x in zip(held, (k, v)):                 # the new ones as they are, as in a prompt from position 0
        h[past.new] = x[past.first:past.last]
    return B.attention(q, *held, cu, past.cu_k, out=o, status=status)


def prompt_blocks(X: torch.Tensor, cu: torch.Tensor, blocks: Sequence[QuantizedBlock], rotary: Rotary,
                  positions: Optional[torch.Tensor] = None, caches: Optional[Sequence[B.KV4Cache]] = None,
                  table: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A packed batch of prompts, bf16 [tokens, d], through the blocks; returns the stream after them.

    positions int32 [tokens] for the rotary tables; None: those inside the sequences, row cu[b] + i at
    start[b] + i, as decode_blocks counts on.
    caches (one per block): the prompts' keys and values are appended at positions start[b] ...
    (int32 [sequences]; None: 0) of sequence b, in the pages that table names, and the tokens attend
    to the cached positions before them too (a prompt in chunks, the next turn of a conversation).
    With start given, cu and start are read back: not inside a stream capture.

    status: the caller's status block, read by the caller.  None: errors found on the device (a position outside
    the tables, a group that is not finite, ...) are waited for and raised, except inside a stream capture.
    """
    _check_stream(X)
    if caches is not None and (table is None or len(caches) != len(blocks)):
        raise ValueError("caches need a table, and one cache per block")
    status, own = _watched(status, X)
    if start is not None and caches is None:
        raise ValueError("start belongs to caches")
    r, y, past = rotary, None, None
    if start is not None and blocks:
        past = _past(cu, start, table, table.shape[1] * caches[0].k_codes.shape[2], X.shape[0])
    if caches is not None and start is None:
        start = torch.zeros(cu.numel() - 1, dtype=torch.int32, device=X.device)
    if positions is None and r.cos is not None:
        positions = _positions(cu, start, X.shape[0])
    for i, b in enumerate(blocks):
        X, h = B.add_norm(X, b.norm_attn, Y=y, eps=b.eps, status=status)
        q, k, v = B.rope_qkv(_forward(b.qkv, h, status), r.cos, r.sin, r.heads_q, r.heads_kv, r.head_dim, positions,
                             interleaved=r.interleaved, status=status)
        if caches is not None:
            B.kv4_append(caches[i], k, v, table, cu, start, status=status)
        a = _attend(q, k, v, cu, caches[i] if past else None, table, past, status).flatten(1)
        X, h = B.add_norm(X, b.norm_mlp, Y=_forward(b.o, a, status), eps=b.eps, status=status)
        y = _forward(b.down, _mlp_hidden(b.gate_up, h, status), status)
    out = X if y is None else G.residual_add(X, y, status)
    if own:
        G.raise_on_status(status, "prompt_blocks")
    return out


def decode_blocks(X: torch.Tensor, lengths: torch.Tensor, blocks: Sequence[QuantizedBlock], rotary: Rotary,
                  caches: Sequence[B.KV4Cache], table: torch.Tensor, ws: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of each sequence, bf16 [sequences, d], through the blocks; returns the stream after them.

    lengths int32 [sequences]: tokens of each sequence in the caches before this one, which is the
    new token's position too; it is appended and attended to.  lengths itself is not advanced.
    At most 16 sequences (qmatvec's rows).  ws: kv4_attention's workspace (a captured step needs its own).
    status: as prompt_blocks's; steps that should not be waited for one by one, and captured ones, take one.
    """
    _check_stream(X)
    n = X.shape[0]
    if n < 1 or n > 16:
        raise ValueError("decode_blocks takes 1 to 16 sequences")
    if len(caches) != len(blocks):
        raise ValueError("decode_blocks needs one cache per block")
    if lengths.dtype != torch.int32 or tuple(lengths.shape) != (n,):
        raise ValueError("lengths must be int32 [sequences]")
    status, own = _watched(status, X)
    r, y = rotary, None
    cu = torch.arange(n + 1, dtype=torch.int32, device=X.device)
    after = lengths + 1
    for b, cache in zip(blocks, caches):
        X, h = B.add_norm(X, b.norm_attn, Y=y, eps=b.eps, status=status)
        q, k, v = B.rope_qkv(G.qmatvec(b.qkv, h, status), r.cos, r.sin, r.heads_q, r.heads_kv, r.head_dim, lengths,
                             interleaved=r.interleaved, status=status)
        B.kv4_append(cache, k, v, table, cu, lengths, status=status)
        a = B.kv4_attention(q, cache, table, after, ws=ws, status=status).flatten(1)
        X, h = B.add_norm(X, b.norm_mlp, Y=G.qmatvec(b.o, a, status), eps=b.eps, status=status)
        gu = G.qmatvec(b.gate_up, h, status)
        f = gu.shape[1] // 2
        y = G.qmatvec(b.down, G.silu_mul(gu[:, :f].contiguous(), gu[:, f:].contiguous(), status), status)
    out = X if y is None else G.residual_add(X, y, status)
    if own:
        G.raise_on_status(status, "decode_blocks")
    return out
