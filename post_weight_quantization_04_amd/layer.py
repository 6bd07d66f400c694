"""Per-layer driver over the three C-ABI entry points.

Allocates device buffers with torch (memory and streams only) and enqueues
the library calls; it performs no arithmetic of its own.
"""
from __future__ import annotations

import dataclasses
from typing import Iterable, Optional

from . import _lib


@dataclasses.dataclass
class Factor:
    U: "torch.Tensor"        # [d_in, d_in] float32, upper
    dead: "torch.Tensor"     # [d_in] uint8
    info: "torch.Tensor"     # [1] int32 (0 = ok)
    lam: "torch.Tensor"      # [1] float64


@dataclasses.dataclass
class Quantized:
    codes: "torch.Tensor"    # [d_out, d_in] uint8
    scales: "torch.Tensor"   # [d_out, n_groups] float32
    zeros: "torch.Tensor"    # [d_out, n_groups] int32
    err_row: "torch.Tensor"  # [d_out] float32
    minmax: "torch.Tensor"   # [d_out, n_groups, 2] float32


class Workspace:
    """Grow-only device scratch buffer shared by the calls of one stream.

    A buffer that a captured graph uses is kept when the workspace grows: the
    graph goes on writing to it whenever it is replayed, so the workspace has
    to live as long as the graph.  Replays and calls that share a workspace
    have to run one after the other."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None
        self._captured = False  # handed out while a graph was being captured
        self._kept = []

    def get(self, nbytes: int):
        import torch
        if self.buf is None or self.buf.numel() < nbytes:
            if self._captured:
                self._kept.append(self.buf)
                self._captured = False
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        if self.buf.is_cuda and torch.cuda.is_current_stream_capturing():
            self._captured = True
        return self.buf


def hessian(X, chunk: Optional[int] = None, H=None, stream=None):
    """``H = 2 X X^T`` (lower triangle) from a device ``X [d_in, N]``,
    streamed in token chunks of ``chunk`` (whole X if None): the first chunk
    sets the lower triangle, the others accumulate into it.  A new H has a
    zero upper triangle; that of a given H is left as it is."""
    import torch
    d_in, n = X.shape
    if H is None:
        H = torch.zeros((d_in, d_in), dtype=torch.float32, device=X.device)
    step = chunk or max(n, 1)
    full = [X[:, t0:t0 + step] for t0 in range(0, n - step + 1, step)]
    if len(full) > 1:
        # whole chunks in one call (summed before each add into H), then
        # the ragged last chunk
        _lib.hessian_chunks(H, full, set_first=True, stream=stream)
        t0 = len(full) * step
        if t0 < n:
            _lib.hessian_accumulate(H, X[:, t0:], stream=stream)
        return H
    _lib.hessian_set(H, X[:, 0:min(step, n)], stream=stream)
    for t0 in range(step, n, step):
        _lib.hessian_accumulate(H, X[:, t0:t0 + step], stream=stream)
    return H


def hessian_chunks(chunks: Iterable, d_in: int, device="cuda", H=None, stream=None):
    import torch
    if H is None:
        H = torch.zeros((d_in, d_in), dtype=torch.float32, device=device)
    for xc in chunks:
        _lib.hessian_accumulate(H, xc, stream=stream)
    return H


def prepare(H, damp_frac: float = 0.01, ws: Optional[Workspace] = None, out: Optional[Factor] = None,
            stream=None, fp32: bool = False) -> Factor:
    import torch
    d_in = H.shape[0]
    dev = H.device
    if out is None:
        out = Factor(torch.empty((d_in, d_in), dtype=torch.float32, device=dev),
                     torch.empty((d_in,), dtype=torch.uint8, device=dev),
                     torch.empty((1,), dtype=torch.int32, device=dev),
                     torch.empty((1,), dtype=torch.float64, device=dev))
    ws = ws or Workspace(dev)
    buf = ws.get(_lib.prepare_hinv_workspace(d_in, fp32=fp32))
    _lib.prepare_hinv(H, damp_frac, out.U, out.dead, out.info, out.lam, buf, stream=stream, fp32=fp32)
    return out


def quantize(W, factor: Factor, bits: int, group_size: int, block_size: int, ws: Optional[Workspace] = None,
             out: Optional[Quantized] = None, use_dead: bool = True, stream=None, split: bool = False) -> Quantized:
    import torch
    d_out, d_in = W.shape
    dev = W.device
    ng = 1 if group_size == 0 else d_in // group_size
    if out is None:
        out = Quantized(torch.empty((d_out, d_in), dtype=torch.uint8, device=dev),
                        torch.empty((d_out, ng), dtype=torch.float32, device=dev),
                        torch.empty((d_out, ng), dtype=torch.int32, device=dev),
                        torch.empty((d_out,), dtype=torch.float32, device=dev),
                        torch.empty((d_out, ng, 2), dtype=torch.float32, device=dev))
    ws = ws or Workspace(dev)
    buf = ws.get(_lib.quantize_layer_workspace(d_out, d_in, block_size, split=split))
    _lib.quantize_layer(W, factor.U, factor.dead if use_dead else None, bits, group_size, block_size, out.codes,
                        out.scales, out.zeros, out.err_row, out.minmax, buf, stream=stream, split=split)
    return out


def pack(codes, bits: int, stream=None):
    """Few-bit storage of ``codes [d_out, d_in]`` (uint32 words, see
    ``gptq_pack_codes``)."""
    import torch
    d_out, d_in = codes.shape
    packed = _empty(d_out, max(_lib.packed_words(d_in, bits), 1), torch.int32, codes.device, stream)
    _lib.pack_codes(codes, bits, packed, stream=stream)
    return packed


def dequantize(packed, bits: int, d_in: int, scales, zeros, group_size: int, dtype=None, stream=None):
    """``What = s (q - z)`` from packed codes, as ``dtype`` (float16 or float32)."""
    import torch
    out = torch.empty((packed.shape[0], d_in), dtype=dtype or torch.float32, device=packed.device)
    _lib.dequantize(packed, bits, d_in, scales, zeros, group_size, out, stream=stream)
    return out


def propagate(W_hat, X, relu: bool = False, out=None, stream=None):
    """The next layer's input from a quantized layer: ``Y = act(W_hat X)``
    in f16 (``gptq_propagate``); ``W_hat`` is the f16 dequantized layer."""
    import torch
    if out is None:
        out = torch.empty((W_hat.shape[0], X.shape[1]), dtype=torch.float16, device=X.device)
    _lib.propagate(W_hat, X, out, 1 if relu else 0, stream=stream)
    return out


def output_error(W, factor: Factor, q: Quantized, packed, bits: int, group_size: int, stream=None):
    """Per-row ``||dw X||^2`` from the loss identity (``gptq_output_error``)."""
    import torch
    out = torch.empty((W.shape[0],), dtype=torch.float32, device=W.device)
    _lib.output_error(W, factor.dead, packed, bits, q.scales, q.zeros, group_size, q.err_row, factor.lam, out,
                      stream=stream)
    return out


@dataclasses.dataclass
class GreedyQuantized:
    codes: "torch.Tensor"    # [d_out, d_in] uint8
    scales: "torch.Tensor"   # [d_out] float32
    zeros: "torch.Tensor"    # [d_out] int32
    order: "torch.Tensor"    # [d_out, d_in] int32: the column quantized at each step
    loss: "torch.Tensor"     # [d_out] float64: dw H_damped dw^T


def quantize_greedy(W, factor: Factor, bits: int, ws: Optional[Workspace] = None, use_dead: bool = True,
                    stream=None) -> GreedyQuantized:
    """Greedy-order (OBQ) quantization of a small layer (``d_in <= 128``,
    ``gptq_obq_quantize``)."""
    import torch
    d_out, d_in = W.shape
    dev = W.device
    out = GreedyQuantized(torch.empty((d_out, d_in), dtype=torch.uint8, device=dev),
                          torch.empty((d_out,), dtype=torch.float32, device=dev),
                          torch.empty((d_out,), dtype=torch.int32, device=dev),
                          torch.empty((d_out, d_in), dtype=torch.int32, device=dev),
                          torch.empty((d_out,), dtype=torch.float64, device=dev))
    ws = ws or Workspace(dev)
    buf = ws.get(_lib.obq_workspace(d_in))
    _lib.obq_quantize(W, factor.U, factor.dead if use_dead else None, bits, out.codes, out.scales, out.zeros,
                      out.order, out.loss, buf, stream=stream)
    return out


# ---------------------------------------------------------------------------
# 8-bit operands (e4m3 values, a float32 scale per block of 128)
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Fp8:
    """An 8-bit matrix of ``cols`` columns.  Activations hold a row per token
    and ``scales [ceil(cols/128), rows]``; weights a row per output channel
    and ``scales [ceil(rows/128), ceil(cols/128)]``."""
    data: "torch.Tensor"     # [rows, ld] float8_e4m3fn, ld >= cols rounded up to 128, zeros behind cols
    scales: "torch.Tensor"   # float32
    cols: int

    @property
    def values(self):
        """``[rows, cols]`` view of the e4m3 values (without their scales)."""
        return self.data[:, :self.cols]


def _empty(rows: int, cols: int, dtype, device, stream):
    """Memory of the stream that the call runs on.  (Sizes one by one: torch
    takes 0.35 us longer over a tuple.)"""
    import torch
    if stream is None:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(rows, cols, dtype=dtype, device=device)


def _scratch(need: int, ws: Optional[Workspace], device, stream):
    """``need`` bytes of ``ws``, or of the call's own; None for 0."""
    if not need:
        return None
    import torch
    if ws is None:
        return _empty(1, need, torch.uint8, device, stream)
    if stream is None:
        return ws.get(need)
    with torch.cuda.stream(stream):
        return ws.get(need)


def _fp8_out(rows: int, cols: int, lead: int, along: int, device, stream) -> Fp8:
    """An 8-bit matrix with scales ``[lead, along]``."""
    import torch
    return Fp8(_empty(rows, (cols + 127) // 128 * 128, torch.float8_e4m3fn, device, stream),
               _empty(lead, along, torch.float32, device, stream), cols)


def _fp8_cols(out: Fp8, cols: int) -> Fp8:
    if out.cols != cols:
        raise ValueError(f"out holds {out.cols} columns, the result has {cols}")
    return out


def fp8_weight(W, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """``W [d_out, d_in]`` (float16, bfloat16 or float32) in 8 bits, one scale
    per 128 x 128 block (``gptq_fp8_weight``)."""
    d_out, d_in = W.shape
    out = (_fp8_cols(out, d_in) if out is not None else
           _fp8_out(d_out, d_in, (d_out + 127) // 128, (d_in + 127) // 128, W.device, stream))
    _lib.fp8_weight(W, out.data, out.scales, stream=stream)
    return out


def fp8_activations(X, channel_major: bool = False, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """Activations ``X [n, d]``, or ``[d, n]`` with ``channel_major`` (the
    layout of the calibration inputs), in 8 bits, one scale per token and 128
    channels (``gptq_fp8_activations``)."""
    n, d = (X.shape[1], X.shape[0]) if channel_major else X.shape
    made = out is None
    out = _fp8_out(n, d, (d + 127) // 128, n, X.device, stream) if made else _fp8_cols(out, d)
    _lib.fp8_activations(X, out.data, out.scales, channel_major, stream, made)
    return out


def fp8_rms_norm(x, gain, eps: float = 1e-6, residual=None, out: Optional[Fp8] = None, sum_out=None, stream=None):
    """``h = x + residual`` and ``h / sqrt(mean(h^2) + eps) * gain`` in 8 bits
    (``gptq_fp8_rms_norm``): returns the 8-bit activations and ``h`` in x's
    type (None without a residual).  ``sum_out`` may be ``x`` or ``residual``."""
    n, d = x.shape
    made, sum_made = out is None, residual is not None and sum_out is None
    out = _fp8_out(n, d, (d + 127) // 128, n, x.device, stream) if made else _fp8_cols(out, d)
    if sum_made:
        sum_out = _empty(n, d, x.dtype, x.device, stream)
    _lib.fp8_rms_norm(x, gain, eps, out.data, out.scales, residual, sum_out, stream, made, sum_made)
    return out, sum_out


def fp8_matmul(w: Fp8, x: Fp8, dtype=None, relu: bool = False, channel_major: bool = False, out=None, stream=None):
    """``act(X W^T)`` of an 8-bit weight and 8-bit activations
    (``gptq_fp8_matmul``): ``[n, d_out]``, or ``[d_out, n]`` with
    ``channel_major``, as ``dtype`` (float16 by default).  float32 results are
    summed in float32; 16-bit ones of more than 32 tokens may lose what lies 13
    bits below the largest of eight neighbouring products."""
    if w.cols != x.cols:
        raise ValueError(f"weights of {w.cols} columns, activations of {x.cols}")
    if out is None:
        import torch
        n, d_out = x.data.shape[0], w.data.shape[0]
        rows, cols = (d_out, n) if channel_major else (n, d_out)
        out = _empty(rows, cols, dtype or torch.float16, x.data.device, stream)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError(f"out is {out.dtype}, not {dtype}")
    _lib.fp8_matmul(w.data, w.scales, x.data, x.scales, w.cols, out, channel_major=channel_major,
                    activation=1 if relu else 0, stream=stream)
    return out


def fp8_gated(gate: Fp8, up: Fp8, x: Fp8, ws: Optional[Workspace] = None, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """``silu(X G^T) * (X U^T)`` in 8 bits (``gptq_fp8_gated``): the input of
    the down projection.  Small calls need scratch memory: that of ``ws``, or
    memory of the call's own."""
    if gate.cols != x.cols or up.cols != x.cols:
        raise ValueError(f"weights of {gate.cols} and {up.cols} columns, activations of {x.cols}")
    n, d_ff = x.data.shape[0], gate.data.shape[0]
    made = out is None
    out = _fp8_out(n, d_ff, (d_ff + 127) // 128, n, x.data.device, stream) if made else _fp8_cols(out, d_ff)
    buf = _scratch(_lib.fp8_gated_workspace(n, d_ff), ws, x.data.device, stream)
    _lib.fp8_gated(gate.data, gate.scales, up.data, up.scales, x.data, x.scales, gate.cols, out.data, out.scales, buf,
                   stream, made)
    return out


def propagate_fp8(w: Fp8, X, relu: bool = False, out=None, stream=None):
    """``propagate`` through a layer kept in 8 bits: the activations ``X [d_in,
    n]`` go to 8 bits, and ``act(W X)`` comes back as ``[d_out, n]``, the next
    layer's input: in X's type, or float32 for bfloat16 X, since ``hessian``
    takes float16 and float32.  A given ``out`` has the type that its owner
    chose."""
    x = fp8_activations(X, channel_major=True, stream=stream)
    dtype = None
    if out is None:
        import torch
        dtype = torch.float32 if X.dtype == torch.bfloat16 else X.dtype
    return fp8_matmul(w, x, dtype=dtype, relu=relu, channel_major=True, out=out, stream=stream)


# ---------------------------------------------------------------------------
# A block of quantized layers: products with packed weights, attention over
# prompts, and the paged cache with the attention over it
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Packed:
    """A few-bit weight as it is stored: ``cols`` codes a row, packed, and the
    grids of its groups (``group_size`` 0: one a row)."""
    codes: "torch.Tensor"    # [d_out, words] int32
    scales: "torch.Tensor"   # [d_out, n_groups] float32
    zeros: "torch.Tensor"    # [d_out, n_groups] int32
    bits: int
    cols: int
    group_size: int


def packed(q: Quantized, bits: int, group_size: int, stream=None) -> Packed:
    """A quantized layer in packed form (``gptq_pack_codes``)."""
    return Packed(pack(q.codes, bits, stream=stream), q.scales, q.zeros, bits, q.codes.shape[1], group_size)


def packed_matmul(w: Packed, x, bias=None, activation: Optional[str] = None, residual=None, dtype=None, out=None,
                  stream=None):
    """``act(x W^T + bias) + residual`` of packed weights and activations ``x
    [n, d_in]`` in float16 or bfloat16 (``gptq_packed_matmul``): ``[n, d_out]``
    in x's type, or float32 by ``dtype`` or ``out``.  ``activation``: None,
    "relu", "silu" or "gelu".  ``residual`` may be ``out``."""
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if out is None:
        out = _empty(x.shape[0], w.codes.shape[0], dtype or x.dtype, x.device, stream)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError(f"out is {out.dtype}, not {dtype}")
    _lib.packed_matmul(w.codes, w.bits, w.cols, w.scales, w.zeros, w.group_size, x, out, bias, residual,
                       _lib.ACTIVATIONS[activation], stream)
    return out


def _like(q, stream):
    """Memory of q's shape and type, contiguous."""
    import torch
    if stream is None:
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    with torch.cuda.stream(stream):
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)


def attention(q, k, v, starts=None, causal: bool = True, scale: Optional[float] = None, out=None, stream=None):
    """Attention over whole prompts (``gptq_attention``): ``q [n, heads, d]``,
    ``k`` and ``v [n, kv_heads, d]``, float16 or bfloat16, views of a fused
    projection among them.  ``starts`` (int32, one value per sequence and one
    more) packs several sequences one behind the other; None: one sequence.
    ``scale``: 1 / sqrt(d) by default."""
    if out is None:
        out = _like(q, stream)
    _lib.attention(q, k, v, starts, out, causal, max(q.shape[-1], 1) ** -0.5 if scale is None else scale, stream)
    return out


@dataclasses.dataclass
class KVCache:
    """Pages of keys and values, each ``[pages, kv_heads, page_size, d]``; a
    token's slot is ``page * page_size + row``.  Which page belongs to which
    sequence is the caller's to keep."""
    keys: "torch.Tensor"
    values: "torch.Tensor"


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=None, device="cuda") -> KVCache:
    """An empty cache (float16 by default)."""
    import torch
    shape = (pages, kv_heads, page_size, head_dim)
    return KVCache(torch.empty(shape, dtype=dtype or torch.float16, device=device),
                   torch.empty(shape, dtype=dtype or torch.float16, device=device))


def cache_store(cache: KVCache, k, v, slots, stream=None) -> None:
    """Keys and values ``[n, kv_heads, d]`` of new tokens to their ``slots``
    (int32; below 0: not stored) of a cache (``gptq_cache_store``)."""
    _lib.cache_store(k, v, slots, cache.keys, cache.values, stream)


def cached_attention(q, cache: KVCache, table, lengths, scale: Optional[float] = None, ws: Optional[Workspace] = None,
                     out=None, stream=None):
    """Attention of one new token of each sequence, ``q [n_seqs, heads, d]``,
    over its pages (``gptq_cached_attention``): sequence b's token j is on page
    ``table[b, j // page_size]``, and there are ``lengths[b]`` (both int32).
    Scratch memory is that of ``ws``, or memory of the call's own."""
    if out is None:
        out = _like(q, stream)
    n, heads, d = q.shape
    _, kv_heads, page_size, _ = cache.keys.shape
    need = _lib.cached_attention_workspace(n, heads, kv_heads, d, table.shape[1], page_size)
    buf = _scratch(need, ws, q.device, stream)
    _lib.cached_attention(q, cache.keys, cache.values, table, lengths, out, max(d, 1) ** -0.5 if scale is None else scale, buf,
                          stream)
    return out
