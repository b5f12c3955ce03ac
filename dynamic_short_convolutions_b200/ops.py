"""Torch-facing helpers over the C ABI: output and workspace allocation, and an
autograd Function.  Marshalling only; the arithmetic runs in libdynconv.so.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib as L


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return L.BF16
    if t.dtype == torch.float32:
        return L.F32
    raise TypeError(f"storage dtype must be bf16 or fp32, got {t.dtype}")


def rope_table(max_pos: int, head_dim: int, base: float = 10000.0, device=None, scaling: Optional[str] = None,
               factor: float = 1.0, original_max_pos: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
               gain: Optional[float] = None) -> torch.Tensor:
    """The RoPE table the C ABI reads: fp32 [max_pos, head_dim] with entries 2i, 2i+1 of row p
    the cosine and sine of p * base^(-2i/head_dim) (RoFormer's angles), computed once in fp64.
    For a part of the head, head_dim is the number of rotated channels.

    ``scaling`` stretches the table to contexts ``factor`` times the ``original_max_pos`` of training:
    ``"linear"`` divides every angle by factor (position interpolation); ``"ntk"`` raises the base by
    factor^(d/(d-2)), which leaves the fastest pair and slows the slowest by factor; ``"yarn"`` divides
    the angles of pairs that turn at most ``beta_slow`` times over original_max_pos by factor, leaves
    those of ``beta_fast`` turns and more, ramps in between, and multiplies cosine and sine by ``gain``
    (0.1 ln factor + 1 unless given)."""
    if head_dim < 2 or head_dim % 2:
        raise ValueError(f"the rotated channels must be even and at least 2, got {head_dim}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if factor < 1.0:
        raise ValueError(f"factor must be at least 1, got {factor}")
    p = torch.arange(max_pos, dtype=torch.float64).unsqueeze(1)
    if scaling == "ntk" and head_dim > 2:
        base = base * factor ** (head_dim / (head_dim - 2))
    theta = base ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
    scale = 1.0 if gain is None else gain
    if scaling == "linear":
        theta = theta / factor
    elif scaling == "yarn":
        # the pair that makes `turns` turns over original_max_pos positions
        at = [head_dim * math.log(original_max_pos / (turns * 2 * math.pi)) / (2 * math.log(base))
              for turns in (beta_fast, beta_slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), head_dim - 1)
        slow = ((torch.arange(head_dim // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        theta = theta * (1 - slow) + theta / factor * slow
        if gain is None:
            scale = 0.1 * math.log(factor) + 1.0
    ang = p * theta
    table = torch.stack((ang.cos(), ang.sin()), dim=-1).reshape(max_pos, head_dim)
    return (table if scale == 1.0 else scale * table).float().to(device or "cuda")


def _rows(t: torch.Tensor, name: str, rows: int, width: int, dtype: torch.dtype, stride: int,
          device: torch.device) -> None:
    """A tensor of `rows` rows of `width` contiguous elements, `stride` (0: width) elements apart, on `device`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {list(t.shape)}")
    at = t.stride()
    if (width > 1 and at[1] != 1) or (rows > 1 and at[0] != (stride or width)):
        raise ValueError(f"{name} must have contiguous channels and a row stride of {stride or width}, "
                         f"got strides {at}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: a call's tensors must be on its plan's device, {device}")


def _flat(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, device: torch.device, shape=None) -> None:
    """A contiguous tensor (or None) on `device`."""
    if t is None:
        return
    if t.dtype is not dtype or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + (f" of shape {list(shape)}" if shape else "")
                         + f", got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: a call's tensors must be on its plan's device, {device}")


def _cu(t: Optional[torch.Tensor], device: torch.device) -> None:
    if t is None:
        return
    _flat(t, "cu_seqlens", torch.int32, device)
    if t.dim() != 1 or t.numel() < 2:
        raise ValueError(f"cu_seqlens must be [documents + 1], got {list(t.shape)}")


def _table(t: torch.Tensor, name: str) -> None:
    if t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 [max_pos, rotated channels] tensor")


def _device(device) -> torch.device:
    d = torch.device(device or "cuda")
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


# The handle of a device's current stream.
_current = L._raw_stream or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check_errors(t: torch.Tensor, device: torch.device) -> None:
    """What a caller gives for the device errors of an autograd call."""
    _flat(t, "errors", torch.uint8, device)
    if t.numel() < 256 or t.data_ptr() % 16:
        raise ValueError("errors must hold 256 bytes or more, on a 16-byte boundary")


def _report(errors: torch.Tensor, ws: torch.Tensor) -> None:
    """The error bits of a plan's workspace into the caller's `errors`."""
    errors[:4].view(torch.int32).bitwise_or_(ws[:4].view(torch.int32))


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy where its rows are not dense or do not start on a 16-byte boundary (rows or columns out of the
    middle of a larger buffer, as autograd hands them back through cat or split)."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _like(t: torch.Tensor, rows: int, width: int) -> torch.Tensor:
    """An uninitialised [rows, width] tensor of t's type, on its device."""
    return torch.empty_like(t) if t.shape == (rows, width) and t.is_contiguous() else t.new_empty((rows, width))


class DynConvPlan:
    """Descriptor + workspace for one problem shape.

    Token-major (default): u [N, C] (rows may be strided, channels contiguous),
    y, g, du [N, C].  Channel-first (``layout=L.CHANNEL_FIRST``): u, y, g, du
    [batch, C, seqlen] (u's channel rows ``u_row_stride`` apart, 0 = seqlen).
    h is [N, d] in both.  For packed documents pass ``cu_seqlens`` (int32 device
    tensor [docs+1]) and batch = 1, seqlen = N.
    """

    def __init__(self, kind: int, dtype: torch.dtype, batch: int, seqlen: int, d_model: int, channels: int,
                 ksize: int, rank: int = 0, head_dim: int = 0, u_row_stride: int = 0, h_row_stride: int = 0,
                 deterministic: bool = False, algo: int = L.ALGO_AUTO, device=None, layout: int = L.TOKEN_MAJOR,
                 rope_channels: int = 0, rope_head_dim: int = 0, rope_table: Optional[torch.Tensor] = None):
        self.rope_table = rope_table            # kept alive: the descriptor holds its address
        self.desc = L.make_desc(kind, L.BF16 if dtype == torch.bfloat16 else L.F32, batch, seqlen, d_model,
                                channels, ksize, rank, head_dim, u_row_stride, h_row_stride, int(deterministic),
                                algo, layout, rope_channels, rope_head_dim, rope_table)
        nbytes = L.dynconv_workspace_bytes(self.desc)
        if nbytes == 0:
            raise L.DynConvError(1, "invalid descriptor")
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")
        self.kind, self.dtype, self.layout = kind, dtype, layout
        self.N, self.d, self.C, self.K, self.r = batch * seqlen, d_model, channels, ksize, rank
        self.batch, self.seqlen = batch, seqlen

    def _conv_shape(self):
        return (self.batch, self.C, self.seqlen) if self.layout == L.CHANNEL_FIRST else (self.N, self.C)

    def forward(self, u, h, A, B_or_W, cu_seqlens=None, y=None, z_save=None, stream=None):
        if y is None:
            y = torch.empty(self._conv_shape(), dtype=self.dtype, device=u.device)
        if cu_seqlens is None:
            L.dynconv_fwd(self.desc, u, h, A, B_or_W, y, z_save, self.ws, stream)
        else:
            L.dynconv_fwd_varlen(self.desc, cu_seqlens, u, h, A, B_or_W, y, z_save, self.ws, stream)
        return y

    def backward(self, g, u, h, A, B_or_W, cu_seqlens=None, z_saved=None, want_dh=True, out=None, stream=None):
        dev = g.device
        if out is None:
            out = {"du": torch.empty(self._conv_shape(), dtype=self.dtype, device=dev),
                   "dh": torch.empty((self.N, self.d), dtype=self.dtype, device=dev) if want_dh else None,
                   "dA": torch.empty(tuple(A.shape), dtype=torch.float32, device=dev) if A is not None else None,
                   "dBW": torch.empty(tuple(B_or_W.shape), dtype=torch.float32, device=dev)}
        L.dynconv_bwd(self.desc, cu_seqlens, g, u, h, A, B_or_W, z_saved, out["du"], out["dh"], out["dA"],
                      out["dBW"], self.ws, stream)
        return out


class DynConvDecoder:
    """Decode steps for `batch` sequences (one new token each per step) with the K-1
    previous conv inputs of every sequence kept on the device (``self.state``,
    ``[batch, K-1, C]``, zero = sequence start; call :meth:`reset` to start over)."""

    def __init__(self, kind: int, dtype: torch.dtype, batch: int, d_model: int, channels: int, ksize: int,
                 rank: int = 0, head_dim: int = 0, u_row_stride: int = 0, h_row_stride: int = 0, device=None):
        self.desc = L.make_desc(kind, L.BF16 if dtype == torch.bfloat16 else L.F32, batch, 1, d_model, channels,
                                ksize, rank, head_dim, u_row_stride, h_row_stride, 0, L.ALGO_AUTO)
        nbytes = L.dynconv_workspace_bytes(self.desc)
        if nbytes == 0:
            raise L.DynConvError(1, "invalid descriptor")
        dev = device or "cuda"
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.state = torch.zeros((batch, ksize - 1, channels), dtype=dtype, device=dev) if ksize > 1 else None
        self.dtype, self.batch, self.C = dtype, batch, channels

    def reset(self):
        if self.state is not None:
            self.state.zero_()

    def step(self, u, h, A, B_or_W, y=None, stream=None):
        if y is None:
            y = torch.empty((self.batch, self.C), dtype=self.dtype, device=u.device)
        L.dynconv_decode_step(self.desc, u, h, A, B_or_W, self.state, y, self.ws, stream)
        return y


class DynamicShortConv(torch.autograd.Function):
    """y = u + dynamic causal depthwise conv(u) with filters generated from h.

    Low-rank: pass A [d, r] and B [r, C*K].  Head-wise: A = None and B_or_W = W
    [d, (C/head_dim)*K].  Parameter gradients come back in the parameters'
    dtype (accumulated in fp32 by the kernels)."""

    @staticmethod
    def forward(ctx, u, h, A, B_or_W, ksize: int, head_dim: int, batch: int, cu_seqlens, algo: int, errors=None):
        if errors is not None:
            _check_errors(errors, u.device)
        d = h.shape[1]
        kind = L.LOWRANK if A is not None else L.HEADWISE
        rank = A.shape[1] if A is not None else 0
        if u.dim() == 3:        # channel-first [batch, C, seqlen]
            batch, C, seqlen = u.shape
            if u.stride(2) != 1 or u.stride(0) != C * u.stride(1):
                u = u.contiguous()
            N, layout, us = batch * seqlen, L.CHANNEL_FIRST, u.stride(1)
        else:
            N, C = u.shape
            seqlen, layout, us = N // batch, L.TOKEN_MAJOR, u.stride(0)
        plan = DynConvPlan(kind, u.dtype, batch, seqlen, d, C, ksize, rank, head_dim, us, h.stride(0),
                           algo=algo, device=u.device, layout=layout)
        R = rank if A is not None else (C // head_dim) * ksize
        z = torch.empty((N, R), dtype=u.dtype, device=u.device)    # generator output, reused by backward
        y = plan.forward(u, h, A, B_or_W, cu_seqlens, z_save=z)
        if errors is not None:
            _report(errors, plan.ws)
        ctx.plan, ctx.errors = plan, errors
        ctx.save_for_backward(u, h, A, B_or_W, cu_seqlens, z)
        return y

    @staticmethod
    def backward(ctx, gy):
        u, h, A, B_or_W, cu_seqlens, z = ctx.saved_tensors
        out = ctx.plan.backward(gy.contiguous(), u, h, A, B_or_W, cu_seqlens, z_saved=z)
        if ctx.errors is not None:
            _report(ctx.errors, ctx.plan.ws)
        dA = out["dA"].to(A.dtype) if A is not None else None
        return out["du"], out["dh"], dA, out["dBW"].to(B_or_W.dtype), None, None, None, None, None, None


def dynamic_short_conv(u: torch.Tensor, h: torch.Tensor, A: Optional[torch.Tensor], B_or_W: torch.Tensor,
                       ksize: int, head_dim: int = 0, batch: int = 1,
                       cu_seqlens: Optional[torch.Tensor] = None, algo: int = L.ALGO_AUTO,
                       errors: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Functional form with autograd: u [N, C] token-major (N = batch * seqlen) or
    [batch, C, seqlen] channel-first; h [N, d].  ``errors``: as in :func:`qkv_attention`."""
    return DynamicShortConv.apply(u, h, A, B_or_W, ksize, head_dim, batch, cu_seqlens, algo, errors)


class _Plan:
    """What the plans of rotary positions and attention share: the zeroed workspace on ``device``, and the order of the
    streams they are made, called and given their tensors on.

    A call runs on the current stream, or on ``stream``: there it comes behind what the current stream holds by
    then, its outputs belong to that stream, and its inputs and the plan may be dropped at once.  The first call on
    another stream than the one the plan was made on waits for that one; not so inside a capture, which cannot wait
    for anything outside it: synchronise before.  In a capture the current stream waits for ``stream`` at once.

    Calls of one plan share its workspace, so one must be over on the device before the next starts: a call that was
    given ``stream`` is waited for, the rest is the order of the streams that are current."""

    _last = None            # the last call, where it ran on a stream of its own
    _behind = None          # handles of the streams that are behind the zeroing, the first the one it ran on

    def _workspace(self, nbytes: int, one_stream: bool) -> None:
        """Last in the making of a plan; one_stream: never called on another stream than this one."""
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self._index = self.device.index
        if not one_stream and self._index is not None and not torch.cuda.is_current_stream_capturing():
            self._behind = [_current(self._index)]

    def _run(self, call, *args) -> None:
        index = self._index
        here = None if index is None else _current(index)
        if self._behind is not None and here not in self._behind:
            self._order(here)
        if self._last is not None:
            self._settle()
        if index is None or index == torch.cuda.current_device():
            call(*args, here)
        else:                                   # kernels launch on the current device
            with torch.cuda.device(index):
                call(*args, here)

    def _settle(self) -> None:
        """The current stream behind the last call, where that ran on a stream of its own."""
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).wait_event(self._last)
            self._last = None

    def _order(self, here: int) -> None:
        if torch.cuda.is_current_stream_capturing():
            return
        made = self._stream(self._behind[0])
        with torch.cuda.stream(made):
            capturing = torch.cuda.is_current_stream_capturing()
        if not capturing:                       # else the zeroing was over before the capture began
            torch.cuda.current_stream(self.device).wait_stream(made)
        self._behind.append(here)

    def _stream(self, handle: int) -> torch.cuda.Stream:
        return torch.cuda.ExternalStream(handle, self.device) if handle else torch.cuda.default_stream(self.device)

    def _other(self, stream) -> Optional[torch.cuda.Stream]:
        """`stream` (a stream, or a handle) where it is another than the current one."""
        if self._index is None:
            return None
        at = L._stream(stream, None)
        return None if at == _current(self._index) else self._stream(at)

    def _call_on(self, stream: torch.cuda.Stream, call, *args):
        """call(*args) with `stream` current, behind what the stream that is current now holds."""
        here = torch.cuda.current_stream(self.device)
        with torch.cuda.stream(here):
            captured = torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(stream):
            if captured or not torch.cuda.is_current_stream_capturing():
                stream.wait_stream(here)
            result = call(*args)
            if not torch.cuda.is_current_stream_capturing():
                self._last = stream.record_event()
                for t in (*args, *vars(self).values()):
                    for x in t.values() if isinstance(t, dict) else (t,):
                        if isinstance(x, torch.Tensor):
                            x.record_stream(stream)
        if captured:                            # a branch of the capture ends where the call does
            here.wait_stream(stream)
        return result


class RopePlan(_Plan):
    """Rotary positions for rows of ``heads`` heads of ``head_dim`` channels, the first
    ``table.shape[1]`` channels of each head rotated.

    x and y: [N, heads * head_dim], N = batch * seqlen (rows may be strided, so x may be the Q and K
    columns of a fused QKV buffer).  A token's position is its place in its sequence, its packed
    document (``cu_seqlens``, batch = 1) or ``positions`` (int32 [N]).  ``table``: fp32
    [max_pos, rotated channels], see :func:`rope_table`."""

    def __init__(self, dtype: torch.dtype, batch: int, seqlen: int, heads: int, head_dim: int, table: torch.Tensor,
                 layout: int = L.ROPE_INTERLEAVED, x_row_stride: int = 0, y_row_stride: int = 0, device=None,
                 _one_stream: bool = False):
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"storage dtype must be bf16 or fp32, got {dtype}")
        _table(table, "table")
        self.device = table.device if device is None else _device(device)
        _flat(table, "table", torch.float32, self.device)
        self.table = table                      # kept alive: the descriptors hold its address
        code = L.BF16 if dtype == torch.bfloat16 else L.F32
        self.desc = [L.make_rope_desc(code, layout, batch, seqlen, heads, head_dim, table, inv, x_row_stride,
                                      y_row_stride) for inv in (0, 1)]
        self.dtype, self.N, self.width = dtype, batch * seqlen, heads * head_dim
        self.strides = (x_row_stride, y_row_stride)
        self._workspace(256, _one_stream)

    def apply(self, x, y=None, positions=None, cu_seqlens=None, inverse: bool = False, stream=None):
        """y = R(p) x, or the transposed rotation (the backward).  ``y=x`` rotates in place."""
        if stream is not None and (other := self._other(stream)) is not None:
            return self._call_on(other, self.apply, x, y, positions, cu_seqlens, inverse)
        _rows(x, "x", self.N, self.width, self.dtype, self.strides[0], self.device)
        if y is None:
            if self.strides[1] not in (0, self.width):
                raise ValueError("a plan with a strided y needs the y to write")
            y = _like(x, self.N, self.width)
        else:
            _rows(y, "y", self.N, self.width, self.dtype, self.strides[1], self.device)
        _flat(positions, "positions", torch.int32, self.device, (self.N,))
        _cu(cu_seqlens, self.device)
        self._run(L.dynconv_rope, self.desc[int(inverse)], cu_seqlens, positions, x, y, self.ws)
        return y


class AttnPlan(_Plan):
    """Causal attention for one problem shape: q [N, heads * head_dim], k and v
    [N, kv_heads * head_dim], N = batch * seqlen, rows optionally strided (column slices of a fused
    QKV buffer).  For packed documents pass ``cu_seqlens`` (int32 device tensor [docs + 1]) and
    batch = 1, seqlen = N.  Query head i reads key/value head i // (heads // kv_heads)."""

    def __init__(self, dtype: torch.dtype, batch: int, seqlen: int, heads: int, kv_heads: int, head_dim: int,
                 scale: float = 0.0, q_row_stride: int = 0, k_row_stride: int = 0, v_row_stride: int = 0,
                 dq_row_stride: int = 0, dk_row_stride: int = 0, dv_row_stride: int = 0, algo: int = L.ALGO_AUTO,
                 device=None, _one_stream: bool = False):
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"storage dtype must be bf16 or fp32, got {dtype}")
        self.desc = L.make_attn_desc(L.BF16 if dtype == torch.bfloat16 else L.F32, batch, seqlen, heads, kv_heads,
                                     head_dim, algo, scale, q_row_stride, k_row_stride, v_row_stride, 0, 0,
                                     dq_row_stride, dk_row_stride, dv_row_stride)
        nbytes = L.dynconv_attn_workspace_bytes(self.desc)
        if nbytes == 0:
            raise L.DynConvError(1, L.dynconv_last_error() or "invalid descriptor")
        self.device = _device(device)
        self.dtype, self.N, self.heads = dtype, batch * seqlen, heads
        self.wq, self.wk = heads * head_dim, kv_heads * head_dim
        self.strides = (q_row_stride, k_row_stride, v_row_stride)
        self.grad_strides = (dq_row_stride, dk_row_stride, dv_row_stride)
        self._workspace(nbytes, _one_stream)

    def _inputs(self, q, k, v, cu_seqlens):
        _rows(q, "q", self.N, self.wq, self.dtype, self.strides[0], self.device)
        _rows(k, "k", self.N, self.wk, self.dtype, self.strides[1], self.device)
        _rows(v, "v", self.N, self.wk, self.dtype, self.strides[2], self.device)
        _cu(cu_seqlens, self.device)

    def forward(self, q, k, v, cu_seqlens=None, o=None, want_lse: bool = False, stream=None):
        """o [N, heads * head_dim]; with ``want_lse`` (o, lse), lse fp32 [heads, N] for :meth:`backward`."""
        if stream is not None and (other := self._other(stream)) is not None:
            return self._call_on(other, self.forward, q, k, v, cu_seqlens, o, want_lse)
        self._inputs(q, k, v, cu_seqlens)
        if o is None:
            o = _like(q, self.N, self.wq)
        else:
            _rows(o, "o", self.N, self.wq, self.dtype, 0, self.device)
        lse = torch.empty((self.heads, self.N), dtype=torch.float32, device=self.device) if want_lse else None
        self._run(L.dynconv_attn_fwd, self.desc, cu_seqlens, q, k, v, o, lse, self.ws)
        return (o, lse) if want_lse else o

    def backward(self, d_o, q, k, v, o, lse, cu_seqlens=None, out=None, stream=None):
        """{"dq", "dk", "dv"} from the forward's o and lse; ``out`` gives tensors to write (dq_row_stride and
        so on apart), for instance column slices of one gradient buffer."""
        if stream is not None and (other := self._other(stream)) is not None:
            return self._call_on(other, self.backward, d_o, q, k, v, o, lse, cu_seqlens, out)
        self._inputs(q, k, v, cu_seqlens)
        if out is None:
            if any(self.grad_strides):
                raise ValueError("a plan with strided gradients needs the tensors to write (out)")
            out = {"dq": _like(q, self.N, self.wq), "dk": _like(k, self.N, self.wk), "dv": _like(v, self.N, self.wk)}
        for name, t, width, stride in (("d_o", d_o, self.wq, 0), ("o", o, self.wq, 0),
                                       ("dq", out["dq"], self.wq, self.grad_strides[0]),
                                       ("dk", out["dk"], self.wk, self.grad_strides[1]),
                                       ("dv", out["dv"], self.wk, self.grad_strides[2])):
            _rows(t, name, self.N, width, self.dtype, stride, self.device)
        if lse is None:
            raise ValueError("the backward needs the forward's lse (want_lse=True)")
        _flat(lse, "lse", torch.float32, self.device, (self.heads, self.N))
        self._run(L.dynconv_attn_bwd, self.desc, cu_seqlens, d_o, q, k, v, o, lse, out["dq"], out["dk"], out["dv"],
                  self.ws)
        return out


class AttnDecoder(_Plan):
    """Serving steps of ``batch`` sequences over a key/value cache: each step takes ``tokens`` new or drafted
    tokens per sequence, rotates their q and k (``rope_table``, see :func:`rope_table`), appends k and v to the
    caches and returns their attention.

    ``k_cache``, ``v_cache`` [batch, kv_heads, max_len, head_dim] and ``lens`` (int32 [batch]: tokens cached, a
    negative entry for an idle slot) are made here, empty, or taken from the caller.  A step reads ``lens`` and
    leaves it: :meth:`advance` adds the tokens that are kept.  Behind a convolution tokens is 1, as
    :class:`DynConvDecoder` takes one token per step."""

    def __init__(self, dtype: torch.dtype, batch: int, heads: int, kv_heads: int, head_dim: int, max_len: int,
                 tokens: int = 1, scale: float = 0.0, rope_table: Optional[torch.Tensor] = None,
                 rope_layout: int = L.ROPE_INTERLEAVED, q_row_stride: int = 0, k_row_stride: int = 0,
                 v_row_stride: int = 0, k_cache=None, v_cache=None, lens=None, device=None):
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"storage dtype must be bf16 or fp32, got {dtype}")
        if rope_table is not None:
            _table(rope_table, "rope_table")
        self.table = rope_table                 # kept alive: the descriptor holds its address
        self.desc = L.make_attn_decode_desc(L.BF16 if dtype == torch.bfloat16 else L.F32, batch, tokens, heads, kv_heads,
                                            head_dim, max_len, scale, rope_table, rope_layout, q_row_stride,
                                            k_row_stride, v_row_stride)
        nbytes = L.dynconv_attn_decode_workspace_bytes(self.desc)
        if nbytes == 0:
            raise L.DynConvError(1, L.dynconv_last_error() or "invalid descriptor")
        self.device = k_cache.device if device is None and k_cache is not None else _device(device)
        shape = (batch, kv_heads, max_len, head_dim)
        self.k_cache = torch.zeros(shape, dtype=dtype, device=self.device) if k_cache is None else k_cache
        self.v_cache = torch.zeros(shape, dtype=dtype, device=self.device) if v_cache is None else v_cache
        self.lens = torch.zeros(batch, dtype=torch.int32, device=self.device) if lens is None else lens
        _flat(self.k_cache, "k_cache", dtype, self.device, shape)
        _flat(self.v_cache, "v_cache", dtype, self.device, shape)
        _flat(self.lens, "lens", torch.int32, self.device, (batch,))
        _flat(rope_table, "rope_table", torch.float32, self.device)
        self.dtype, self.batch, self.tokens = dtype, batch, tokens
        self.wq, self.wk = heads * head_dim, kv_heads * head_dim
        self.strides = (q_row_stride, k_row_stride, v_row_stride)
        self._workspace(nbytes, False)

    def step(self, q, k, v, ancestors=None, o=None, stream=None):
        """o [batch * tokens, heads * head_dim] of q [batch * tokens, heads * head_dim], k and v
        [batch * tokens, kv_heads * head_dim] (rows by sequence, then token).  ``ancestors`` (int64
        [batch, tokens]): bit j of an entry set where that token sees drafted token j, its own bit included;
        None: a chain."""
        if stream is not None and (other := self._other(stream)) is not None:
            return self._call_on(other, self.step, q, k, v, ancestors, o)
        rows = self.batch * self.tokens
        _rows(q, "q", rows, self.wq, self.dtype, self.strides[0], self.device)
        if o is None:
            o = _like(q, rows, self.wq)
        else:
            _rows(o, "o", rows, self.wq, self.dtype, 0, self.device)
        _rows(k, "k", rows, self.wk, self.dtype, self.strides[1], self.device)
        _rows(v, "v", rows, self.wk, self.dtype, self.strides[2], self.device)
        _flat(ancestors, "ancestors", torch.int64, self.device, (self.batch, self.tokens))
        self._run(L.dynconv_attn_decode, self.desc, q, k, v, self.k_cache, self.v_cache, self.lens, ancestors, o,
                  self.ws)
        return o

    def advance(self, kept=None):
        """Adds the tokens kept of the last step to ``lens``: all of them, or ``kept`` (int32 [batch]).  Idle
        slots stay idle.  Kept tokens of a tree have to lie in the cache in order (tokens 0 .. kept - 1)."""
        _flat(kept, "kept", torch.int32, self.device, (self.batch,))
        if self._last is not None:              # a step that may still read lens
            self._settle()
        self.lens.add_(torch.where(self.lens < 0, 0, self.tokens if kept is None else kept).to(torch.int32))

    def reset(self):
        if self._last is not None:              # a step that may still read lens
            self._settle()
        self.lens.zero_()


class QKVAttention(torch.autograd.Function):
    """Causal attention of a fused QKV buffer, with the rotation of Q and K where a table is given.

    qkv [N, (heads + 2 kv_heads) * head_dim] is what the QKV convolution leaves; the backward writes
    one buffer of that shape, which the convolution's backward takes as its g."""

    @staticmethod
    def forward(ctx, qkv, table, heads: int, kv_heads: int, head_dim: int, batch: int, cu_seqlens, scale: float,
                layout: int, algo: int, errors=None):
        N, C = qkv.shape
        if errors is not None:
            _check_errors(errors, qkv.device)
        wq, wk = heads * head_dim, kv_heads * head_dim
        if C != wq + 2 * wk:
            raise ValueError(f"qkv must be [N, (heads + 2 kv_heads) * head_dim] = [N, {wq + 2 * wk}], got {list(qkv.shape)}")
        if batch < 1 or N % batch:
            raise ValueError(f"{N} tokens are not {batch} sequences of one length")
        if qkv.stride(1) != 1 or (N > 1 and qkv.stride(0) < C) or qkv.data_ptr() % 16:
            qkv = qkv.clone(memory_format=torch.contiguous_format)
        row = qkv.stride(0) if N > 1 else C
        qk, rope, qk_row = qkv[:, :wq + wk], None, row
        if table is not None:
            rope = (qkv.dtype, batch, N // batch, heads + kv_heads, head_dim)
            turn = RopePlan(*rope, table, layout, x_row_stride=row, device=qkv.device, _one_stream=True)
            qk = turn.apply(qk, cu_seqlens=cu_seqlens)
            if errors is not None:
                _report(errors, turn.ws)
            qk_row = wq + wk
        q, k, v = qk[:, :wq], qk[:, wq:], qkv[:, wq + wk:]
        # columns that start off a 16-byte boundary (heads of odd widths) are copied out, and their gradients in
        apart = any(n * qkv.element_size() % 16 for n in (wq, wk))
        if apart:
            # (not contiguous(), which gives back the slices of a single row as they are)
            q, k, v = (t.clone(memory_format=torch.contiguous_format) for t in (q, k, v))
        strides = (0,) * 6 if apart else (qk_row, qk_row, row, C, C, C)
        plan = AttnPlan(qkv.dtype, batch, N // batch, heads, kv_heads, head_dim, scale, *strides, algo=algo,
                        device=qkv.device, _one_stream=True)
        train = ctx.needs_input_grad[0]
        o, lse = plan.forward(q, k, v, cu_seqlens, want_lse=True) if train else (plan.forward(q, k, v, cu_seqlens), None)
        if errors is not None:
            _report(errors, plan.ws)
        if train:
            ctx.plan, ctx.rope, ctx.layout, ctx.apart, ctx.errors = plan, rope, layout, apart, errors
            ctx.width = N, C, wq, wk
            ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, table)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, go):
        q, k, v, o, lse, cu_seqlens, table = ctx.saved_tensors
        N, C, wq, wk = ctx.width
        d = torch.empty((N, C), dtype=q.dtype, device=q.device)
        out = {"dq": d[:, :wq], "dk": d[:, wq:wq + wk], "dv": d[:, wq + wk:]}
        grads = ctx.plan.backward(_dense(go), q, k, v, o, lse, cu_seqlens, None if ctx.apart else out)
        if ctx.apart:
            for name, part in out.items():
                part.copy_(grads[name])
        if ctx.errors is not None:
            _report(ctx.errors, ctx.plan.ws)
        if ctx.rope is not None:
            turn = RopePlan(*ctx.rope, table, ctx.layout, x_row_stride=C, y_row_stride=C, device=q.device,
                            _one_stream=True)
            turn.apply(d[:, :wq + wk], y=d[:, :wq + wk], cu_seqlens=cu_seqlens, inverse=True)
            if ctx.errors is not None:
                _report(ctx.errors, turn.ws)
        return (d,) + (None,) * 10


def qkv_attention(qkv: torch.Tensor, heads: int, kv_heads: int, head_dim: int, table: Optional[torch.Tensor] = None,
                  batch: int = 1, cu_seqlens: Optional[torch.Tensor] = None, scale: float = 0.0,
                  layout: int = L.ROPE_INTERLEAVED, algo: int = L.ALGO_AUTO,
                  errors: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Functional form with autograd: rotary positions (``table``, see :func:`rope_table`) on the Q and K
    columns of qkv [N, (heads + 2 kv_heads) * head_dim], then causal attention; o [N, heads * head_dim].
    The table has a row for every position; a packed document that is longer repeats the last one.  ``errors``
    (uint8, 256 bytes, zeroed once, for the calls of one stream): what the device finds wrong in the forward or the
    backward -- such a document, a malformed cu_seqlens (undefined results), a pipeline wait that ran out (outputs not
    written) -- is kept there for ``dynconv_device_status(errors)``; without it nothing tells of them.  Calls and their
    backward may be captured into a CUDA graph; as for any autograd function, no eager graph of the same leaves may
    be alive then."""
    return QKVAttention.apply(qkv, table, heads, kv_heads, head_dim, batch, cu_seqlens, scale, layout, algo, errors)


def dynamic_conv_attention(u: torch.Tensor, h: torch.Tensor, A: Optional[torch.Tensor], B_or_W: torch.Tensor,
                           ksize: int, heads: int, kv_heads: int, head_dim: int, table: Optional[torch.Tensor] = None,
                           filter_head_dim: int = 0, batch: int = 1, cu_seqlens: Optional[torch.Tensor] = None,
                           scale: float = 0.0, layout: int = L.ROPE_INTERLEAVED, algo: int = L.ALGO_AUTO,
                           errors: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The QKV placement as a layer runs it: the dynamic short convolution of the fused QKV rows u [N, C]
    (C = (heads + 2 kv_heads) * head_dim; head-wise filters where filter_head_dim > 0), rotary positions on
    Q and K, causal attention.  With autograd; o [N, heads * head_dim].  ``errors``: as in :func:`qkv_attention`."""
    y = dynamic_short_conv(u, h, A, B_or_W, ksize, filter_head_dim, batch, cu_seqlens, algo, errors)
    return qkv_attention(y, heads, kv_heads, head_dim, table, batch, cu_seqlens, scale, layout, algo, errors)
