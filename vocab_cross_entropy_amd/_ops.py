"""The operators around the loss: logit processing, embedding, RMS norm, token log-probabilities and distillation.

Like the rest of the binding, the ``ce_*`` functions marshal torch device
tensors into the C ABI's descriptors (``include/ce.h`` defines each operator)
and run on torch's current stream of the tensors' device; those that write over
logits raise the tensor's version, as torch's in-place operations do.  ``process_logits``,
``processed_cross_entropy``, ``embedding``, ``rms_norm``,
``norm_linear_cross_entropy``, ``token_logprobs`` and ``distillation_loss`` are
their autograd forms.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from . import (CeArgumentError, _check, _device_of, _need, _need_targets, _raw_stream, _workspace,
               _is_prepared, _overwritten, ce_fwd_bwd_fused, ce_scale_grad_inplace, ce_workspace_bytes,
               ce_workspace_init, lib, linear_cross_entropy, reduction_code)

__all__ = [
    "ce_logits_process", "ce_logits_process_backward", "logits_signs", "process_logits", "processed_cross_entropy",
    "ce_embedding", "ce_embedding_backward", "ce_embedding_workspace_bytes", "embedding",
    "ce_rms_norm", "ce_rms_norm_quant", "ce_rms_norm_backward", "ce_rms_norm_workspace_bytes", "rms_norm",
    "norm_linear_cross_entropy",
    "TokenLogprobs", "ce_token_logprobs", "ce_token_logprobs_backward", "ce_token_logprobs_workspace_bytes",
    "token_logprobs",
    "ce_distill_fwd_bwd", "ce_distill_workspace_bytes", "distillation_loss",
]


# These calls are small beside the loss (one decoding step's norm takes 3 us on the device), so the checks below
# first test the common case in one expression, with devices as their index, and name what is wrong only when it
# fails.
_Tensor = torch.Tensor
_code = {torch.float32: _abi.CE_F32, torch.bfloat16: _abi.CE_BF16}.get
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _index(x, what) -> int:
    """The index of the GPU that ``x`` is on."""
    if isinstance(x, _Tensor) and x.is_cuda:
        return x.get_device()
    _device_of(x, what)  # raises


def _call(dev: int, fn, *args):
    """Run an entry point on torch's current stream of GPU ``dev``, with ``dev`` the current device (kernels are
    looked up per device)."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


def _einval(msg: str):
    raise CeArgumentError(_abi.CE_EINVAL, msg)


def _elayout(msg: str):
    raise CeArgumentError(_abi.CE_ELAYOUT, msg)


def _flat(dev, what, t, dtype, n):
    """The address of a contiguous array of at least ``n`` elements on GPU ``dev`` (None without one)."""
    if t is None:
        return None
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype and t.numel() >= n
            and t.is_contiguous()):
        _need(torch.device("cuda", dev), what, t, dtype, n)  # raises
    return t.data_ptr()


def _rows(dev, what, t, shape, dtype):
    """``t`` is a [rows, columns] matrix on GPU ``dev`` with contiguous columns (``dtype`` None: any): its row
    stride."""
    if not (isinstance(t, _Tensor) and t.shape == shape and t.get_device() == dev
            and (dtype is None or t.dtype is dtype)):
        if t is None:
            _einval(f"{what} is missing")
        _need(torch.device("cuda", dev), what, t, dtype, contiguous=False)
        if tuple(t.shape) != tuple(shape):
            _einval(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")
    ld, col = t.stride()
    if col != 1 and shape[1] > 1:
        _elayout(f"{what} needs contiguous columns")
    return ld if shape[0] > 1 else max(ld, shape[1])


# ---- logit processing ------------------------------------------------------------------------------------


def _side(dev, what, t, d0, d1, width, dtype):
    """A (d0, d1, >= width) companion of the logits, any row strides: (pointer, s0, s1)."""
    if t is None:
        return None, 0, 0
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype):
        _need(torch.device("cuda", dev), what, t, dtype, contiguous=False)  # raises
    shape = t.shape
    if len(shape) != 3 or shape[0] != d0 or shape[1] != d1 or shape[2] < width:
        _einval(f"{what} must be ({d0}, {d1}, {width}), got {tuple(shape)}")
    s0, s1, col = t.stride()
    if col != 1 and shape[2] > 1:
        _elayout(f"{what} needs a contiguous last dimension")
    return t.data_ptr(), s0, s1


def _logits(x, what, vocab_start, vocab_total):
    """logits_desc, and the dimensions."""
    if len(x.shape) != 3:
        _einval(f"{what} must be a 3-d (d0, d1, V) tensor")
    d0, d1, v = x.shape
    s0, s1, col = x.stride()
    if col != 1 and v > 1:
        _elayout(f"{what} columns must be contiguous (stride 1)")
    return _abi.CeLogits(x.data_ptr(), _code(x.dtype, -1), 0, d0, d1, s0, s1, v, vocab_start,
                         v if vocab_total is None else vocab_total), d0, d1, v


def _process(fn, x, out, vocab_start, vocab_total, history, history_len, prompt_len, repetition, presence, frequency,
             bias, mask, temperature, signs):
    dev = _index(x, "logits")
    xd, d0, d1, V = _logits(x, "logits", vocab_start, vocab_total)
    zd, N = xd, d0 * d1
    if out is not None and out is not x:
        if not (isinstance(out, _Tensor) and out.get_device() == dev and out.dtype is x.dtype):
            _need(torch.device("cuda", dev), "out", out, x.dtype, contiguous=False)  # raises
        if out.shape != x.shape:
            _einval(f"out must be {tuple(x.shape)}, got {tuple(out.shape)}")
        zd = _logits(out, "out", vocab_start, vocab_total)[0]
    f32, i32 = torch.float32, torch.int32
    hist, h0, h1 = _side(dev, "history", history, d0, d1, 0, torch.int64)
    hist_max = 0 if history is None else history.shape[2]
    hist_len, prompt = _flat(dev, "history_len", history_len, i32, N), _flat(dev, "prompt_len", prompt_len, i32, N)
    rep, freq, pres = (_flat(dev, "repetition", repetition, f32, N), _flat(dev, "frequency", frequency, f32, N),
                       _flat(dev, "presence", presence, f32, N))
    if history is not None and not hist:
        # an empty tensor (it has no address): no row has a token, and nothing is counted
        hist = hist_len = prompt = rep = freq = pres = None
        hist_max = 0
    signs_ptr, signs_ld = None, 0
    if signs is not None:
        if signs.dim() != 2 or signs.shape[1] < (V + 7) // 8:
            _einval(f"signs must be ({N}, {(V + 7) // 8}), see logits_signs")
        signs_ptr, signs_ld = signs.data_ptr(), _rows(dev, "signs", signs, (N, signs.shape[1]), torch.uint8)
    p = _abi.CeProcess(hist, h0, h1, hist_max, hist_len, prompt, rep, freq, pres,
                       _flat(dev, "temperature", temperature, f32, N), *_side(dev, "bias", bias, d0, d1, V, f32),
                       *_side(dev, "mask", mask, d0, d1, (V + 31) // 32, i32), signs_ptr, signs_ld)
    _call(dev, fn, xd, zd, p)
    # (a gradient's processing in place writes over no logits: a loss may have staged it, for its backward to return)
    if zd.data == xd.data and fn is lib.ce_logits_process:
        _overwritten(x)
    return x if out is None else out


def logits_signs(x: torch.Tensor) -> torch.Tensor:
    """An empty ``signs`` buffer for (d0, d1, V) logits: one bit per logit, [N, ceil(V / 8)] bytes."""
    return torch.empty((x.shape[0] * x.shape[1], (x.shape[2] + 7) // 8), dtype=torch.uint8, device=x.device)


def ce_logits_process(x, *, out=None, history=None, history_len=None, prompt_len=None, repetition=None,
                      presence=None, frequency=None, bias=None, mask=None, temperature=None, signs=None,
                      vocab_start=0, vocab_total=None):
    """Penalties, bias, grammar mask and temperature over (d0, d1, V) logits, in place or into ``out``.

    ``history`` (d0, d1, L) int64 tokens (rows may share storage, ``expand``), ``history_len`` and
    ``prompt_len`` [N] int32; ``repetition``, ``frequency``, ``presence`` and ``temperature`` [N] FP32;
    ``bias`` (d0, d1, V) FP32 and ``mask`` (d0, d1, ceil(V / 32)) int32 words of allowed columns, both any row
    strides.  ``signs`` (see logits_signs) is written for the gradient.  Each is optional.  Returns the
    processed logits."""
    return _process(lib.ce_logits_process, x, out, vocab_start, vocab_total, history, history_len, prompt_len,
                    repetition, presence, frequency, bias, mask, temperature, signs)


def ce_logits_process_backward(dz, *, out=None, signs=None, history=None, history_len=None, prompt_len=None,
                               repetition=None, mask=None, temperature=None, vocab_start=0, vocab_total=None):
    """The gradient of ce_logits_process with respect to the logits, in place over ``dz`` or into ``out``.
    ``signs`` are the forward's, needed with ``repetition``."""
    return _process(lib.ce_logits_process_backward, dz, out, vocab_start, vocab_total, history, history_len,
                    prompt_len, repetition, None, None, None, mask, temperature, signs)


def _constants(**steps):
    for name, t in steps.items():
        if isinstance(t, _Tensor) and t.requires_grad:
            _einval(f"{name} is a constant of the processing and gets no gradient (it requires one)")


def _own_rows(t: torch.Tensor) -> torch.Tensor:
    """``t`` as the kernels can read it: contiguous columns, rows of their own (an expanded tensor is copied)."""
    ok = t.stride(-1) == 1 and all(n <= 1 or s >= t.shape[-1] for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    return t if ok and t.shape[-1] > 0 else t.contiguous()


class ProcessLogits(torch.autograd.Function):
    """Autograd form of ce_logits_process, out of place: the logits are left as they are and not kept (the
    backward needs their signs alone, one bit each, and those only with a repetition penalty)."""

    @staticmethod
    def forward(ctx, x, history, history_len, prompt_len, repetition, presence, frequency, bias, mask, temperature):
        if x.dim() != 3:
            _einval("logits must be a 3-d (d0, d1, V) tensor")
        signs = logits_signs(x) if repetition is not None and ctx.needs_input_grad[0] else None
        x = _own_rows(x.detach())
        z = ce_logits_process(x, out=torch.empty_like(x), history=history, history_len=history_len,
                              prompt_len=prompt_len, repetition=repetition, presence=presence, frequency=frequency,
                              bias=bias, mask=mask, temperature=temperature, signs=signs)
        ctx.save_for_backward(signs, history, history_len, prompt_len, repetition, mask, temperature)
        return z

    @staticmethod
    @once_differentiable
    def backward(ctx, dz):
        signs, history, history_len, prompt_len, repetition, mask, temperature = ctx.saved_tensors
        if repetition is None:
            history = history_len = prompt_len = None
        dz = _own_rows(dz)
        dx = ce_logits_process_backward(dz, out=torch.empty_like(dz), signs=signs, history=history,
                                        history_len=history_len, prompt_len=prompt_len, repetition=repetition,
                                        mask=mask, temperature=temperature)
        return dx, None, None, None, None, None, None, None, None, None


def process_logits(logits, *, history=None, history_len=None, prompt_len=None, repetition=None, presence=None,
                   frequency=None, bias=None, mask=None, temperature=None):
    """Processed logits (a new tensor, in the logits' dtype) with the options of ce_logits_process, for whole rows of
    the vocabulary (a shard's: ce_logits_process and its backward, with ``vocab_start`` and ``vocab_total``); the
    gradient reaches ``logits``, everything else is a constant."""
    _constants(repetition=repetition, presence=presence, frequency=frequency, bias=bias, temperature=temperature)
    return ProcessLogits.apply(logits, history, history_len, prompt_len, repetition, presence, frequency, bias, mask,
                               temperature)


class ProcessedCrossEntropy(torch.autograd.Function):
    """ce_logits_process, the fused loss and the processing's gradient, all in place over the logits' storage
    (TENPU #29 section 6 stages the gradient there): the forward leaves in ``inp`` the gradient for an upstream
    gradient of 1, the backward scales it (ce_scale_grad_inplace)."""

    @staticmethod
    def forward(ctx, inp, target, label_smoothing, reduce_loss, ignore_idx, smoothing, history, history_len,
                prompt_len, repetition, presence, frequency, bias, mask, temperature):
        buf = inp.detach()
        # the loss's own checks come first: a refused call leaves the logits as they are
        if buf.dim() != 3:
            _einval("logits must be a 3-d (d0, d1, V) tensor")
        _need_targets(torch.device("cuda", _index(buf, "logits")), target, buf.shape[0], buf.shape[1])
        ws = _workspace(ce_workspace_bytes(buf, label_smoothing, reduce_loss, ignore_idx, smoothing=smoothing),
                        buf.device)
        signs = logits_signs(buf) if repetition is not None else None
        ce_logits_process(buf, history=history, history_len=history_len, prompt_len=prompt_len,
                          repetition=repetition, presence=presence, frequency=frequency, bias=bias, mask=mask,
                          temperature=temperature, signs=signs)
        loss, _ = ce_fwd_bwd_fused(buf, target, label_smoothing, reduce_loss, ignore_idx, smoothing=smoothing, ws=ws)
        if repetition is None:
            history = history_len = prompt_len = None
        if repetition is not None or mask is not None or temperature is not None:
            ce_logits_process_backward(buf, signs=signs, history=history, history_len=history_len,
                                       prompt_len=prompt_len, repetition=repetition, mask=mask,
                                       temperature=temperature)
        ctx.reduced = reduction_code(reduce_loss) != _abi.CE_REDUCE_NONE
        ctx.save_for_backward(buf)
        return loss[0] if ctx.reduced else loss.view(target.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        (buf,) = ctx.saved_tensors
        ce_scale_grad_inplace(buf, grad_loss, per_row=not ctx.reduced)
        return (buf,) + (None,) * 14


def processed_cross_entropy(inp, target, label_smoothing=0.0, reduce_loss=False, ignore_idx=-100, *, smoothing="all",
                            history=None, history_len=None, prompt_len=None, repetition=None, presence=None,
                            frequency=None, bias=None, mask=None, temperature=None):
    """Cross-entropy (the negative log-probability) under the distribution that sampling drew from:
    parallel_cross_entropy of the processed logits, whole rows of the vocabulary, with its options (reduction,
    smoothing, ignored index) and those of process_logits.  As there, the gradient is staged in place in ``inp``, and what
    was called on these logits before and keeps them has taken a copy."""
    _constants(repetition=repetition, presence=presence, frequency=frequency, bias=bias, temperature=temperature)
    return ProcessedCrossEntropy.apply(inp, target, label_smoothing, reduce_loss, ignore_idx, smoothing, history,
                                       history_len, prompt_len, repetition, presence, frequency, bias, mask,
                                       temperature)


# ---- embedding -------------------------------------------------------------------------------------------


def _embedding_desc(ids, weight_ptr, w_ld, of, D, v_local, scale, vocab_start, vocab_total):
    N = ids.shape[0]
    return _abi.CeEmbeddingDesc(ids.data_ptr(), ids.stride(0) if N > 1 else 1, N, D, weight_ptr, w_ld,
                                _code(of.dtype, -1), 0, v_local, vocab_start,
                                v_local if vocab_total is None else vocab_total, scale)


def _need_ids(dev, ids):
    if not (isinstance(ids, _Tensor) and ids.get_device() == dev and ids.dtype is torch.int64):
        _need(torch.device("cuda", dev), "ids", ids, torch.int64, contiguous=False)  # raises
    if ids is None or ids.dim() != 1:
        _einval("ids must be a 1-d int64 tensor")


def _need_padding(padding_idx):
    if padding_idx is not None and padding_idx < 0:
        _einval("padding_idx must be a vocabulary index")


def ce_embedding(ids, weight, scale=1.0, *, out=None, vocab_start=0, vocab_total=None):
    """``scale * weight[ids]`` for [N] int64 ``ids`` and a [V, D] table, or the rows from ``vocab_start`` on of a
    vocabulary of ``vocab_total`` (other shards' ids give zeros).  Returns [N, D]."""
    dev = _index(weight, "weight")
    if weight.dim() != 2:
        _einval("weight must be [V, D]")
    _need_ids(dev, ids)
    V, D = weight.shape
    m = _embedding_desc(ids, weight.data_ptr(), _rows(dev, "weight", weight, weight.shape, None), weight, D, V, scale,
                        vocab_start, vocab_total)
    if out is None:
        out, out_ld = weight.new_empty((m.N, D)), D
    else:
        out_ld = _rows(dev, "out", out, (m.N, D), weight.dtype)
    _call(dev, lib.ce_embedding, m, out.data_ptr(), out_ld)
    return out


def ce_embedding_workspace_bytes(tokens: int, D: int, v_local: int) -> int:
    n = lib.ce_embedding_workspace_bytes(int(tokens), int(D), int(v_local))
    if n == 0:
        _check(_abi.CE_EINVAL)
    return int(n)


def ce_embedding_backward(dout, ids, v_local, scale=1.0, *, padding_idx=None, dw=None, accumulate=False, ws=None,
                          vocab_start=0, vocab_total=None):
    """The table's FP32 [v_local, D] gradient from ``dout`` [N, D], written to ``dw`` or added to it
    (``accumulate``; a tied head's ce_linear_cross_entropy gradient).  Tokens equal to ``padding_idx`` add
    nothing.  Returns dw."""
    dev = _index(dout, "dout")
    if dout.dim() != 2:
        _einval("dout must be [N, D]")
    _need_ids(dev, ids)
    N, D = dout.shape
    if ids.shape[0] != N:
        _einval(f"{ids.shape[0]} ids for {N} rows of dout")
    _need_padding(padding_idx)
    v_local = int(v_local)
    m = _embedding_desc(ids, None, D, dout, D, v_local, scale, vocab_start, vocab_total)
    if dw is None:
        if accumulate:
            _einval("accumulate needs dw")
        dw = torch.empty((v_local, D), dtype=torch.float32, device=dout.device)
    if ws is None:
        ws = _workspace(ce_embedding_workspace_bytes(N, D, v_local), dout.device)
    ws_ptr = _flat(dev, "workspace", ws, torch.uint8, 0)
    _call(dev, lib.ce_embedding_backward, m, dout.data_ptr(), _rows(dev, "dout", dout, dout.shape, None),
          -1 if padding_idx is None else padding_idx, dw.data_ptr(),
          _rows(dev, "dw", dw, (v_local, D), torch.float32), 1 if accumulate else 0, ws_ptr, ws.numel())
    return dw


class Embedding(torch.autograd.Function):
    """Autograd form of ce_embedding; the gradient by ce_embedding_backward."""

    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx, grad_buffer, vocab_start, vocab_total):
        flat = ids.reshape(-1)
        out = ce_embedding(flat, weight.detach(), scale, vocab_start=vocab_start, vocab_total=vocab_total)
        ctx.args = (scale, padding_idx, vocab_start, vocab_total, weight.shape)
        ctx.grad_buffer = grad_buffer
        ctx.save_for_backward(flat)
        return out.view(*ids.shape, weight.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (flat,) = ctx.saved_tensors
        scale, padding_idx, vocab_start, vocab_total, (V, D) = ctx.args
        dw = ce_embedding_backward(dout.reshape(-1, D).contiguous(), flat, V, scale, padding_idx=padding_idx,
                                   dw=ctx.grad_buffer, accumulate=ctx.grad_buffer is not None,
                                   vocab_start=vocab_start, vocab_total=vocab_total)
        return dw if ctx.grad_buffer is None else None, None, None, None, None, None, None


def embedding(ids, weight, scale=1.0, *, padding_idx=None, grad_buffer=None, vocab_start=0, vocab_total=None):
    """``scale * weight[ids]`` for int64 ``ids`` of any shape; reaches autograd through Embedding (the FP32
    gradient, which autograd casts to the weight's dtype).  With ``grad_buffer``, an FP32 [V, D] tensor, the
    backward adds the gradient to it instead and ``weight.grad`` stays as it is: with a tied head, the buffer that
    ce_linear_cross_entropy adds its dw to.  (A weight that requires no gradient has none in either.)"""
    _need_padding(padding_idx)  # here: the forward has no use for it, and the backward is too late
    if grad_buffer is not None:
        _rows(_index(weight, "weight"), "grad_buffer", grad_buffer, weight.shape, torch.float32)
    return Embedding.apply(weight, ids, scale, padding_idx, grad_buffer, vocab_start, vocab_total)


# ---- RMS norm --------------------------------------------------------------------------------------------


def _norm_desc(dev, x, weight, residual, eps):
    if x.dim() != 2:
        _einval("x must be [N, D]")
    shape = x.shape
    N, D = shape
    if not (isinstance(weight, _Tensor) and weight.get_device() == dev and weight.shape == (D,)
            and weight.is_contiguous()):
        _need(torch.device("cuda", dev), "weight", weight, None, D)
        _einval(f"weight must be a contiguous [{D}] tensor")
    res, res_ld = None, 0
    if residual is not None:
        res, res_ld = residual.data_ptr(), _rows(dev, "residual", residual, shape, x.dtype)
    return _abi.CeNorm(x.data_ptr(), res, weight.data_ptr(), _code(x.dtype, -1), _code(weight.dtype, -1), N, D,
                       _rows(dev, "x", x, shape, None), res_ld, eps)


def _like(dev, what, t, x):
    """``t``, or a new tensor like ``x``: (tensor, address, row stride)."""
    if t is None:
        t = torch.empty_like(x)
        return t, t.data_ptr(), t.stride(0) if x.shape[0] > 1 else x.shape[1]
    return t, t.data_ptr(), _rows(dev, what, t, x.shape, x.dtype)


def _sum_out(dev, x, residual, sum_out):
    """Where the sum goes: nowhere without a residual unless a buffer is given."""
    return (None, None, 0) if residual is None and sum_out is None else _like(dev, "sum_out", sum_out, x)


def ce_rms_norm(x, weight, residual=None, eps=1e-6, *, out=None, sum_out=None):
    """RMS norm of ``x + residual`` ([N, D]); returns (y, sum), the sum None without a residual (unless
    ``sum_out`` asks for it).  ``out`` and ``sum_out`` may be x or residual themselves, not one another."""
    dev = _index(x, "x")
    n = _norm_desc(dev, x, weight, residual, eps)
    out, ptr, ld = _like(dev, "out", out, x)
    total, total_ptr, total_ld = _sum_out(dev, x, residual, sum_out)
    _call(dev, lib.ce_rms_norm, n, ptr, ld, total_ptr, total_ld)
    return out, total


def ce_rms_norm_quant(x, weight, residual=None, eps=1e-6, *, group=0, out=None, scales=None, sum_out=None):
    """ce_rms_norm with its output in e4m3 (torch.float8_e4m3fn) and FP32 scales, one for each ``group`` columns
    (32, 64 or 128; 0: one for the row).  Returns (q, scales [N, groups], sum or None)."""
    dev = _index(x, "x")
    n = _norm_desc(dev, x, weight, residual, eps)
    N, D = x.shape
    groups = -(-D // group) if group > 0 else 1
    out = torch.empty((N, D), dtype=torch.float8_e4m3fn, device=x.device) if out is None else out
    scales = torch.empty((N, groups), dtype=torch.float32, device=x.device) if scales is None else scales
    total, total_ptr, total_ld = _sum_out(dev, x, residual, sum_out)
    _call(dev, lib.ce_rms_norm_quant, n, out.data_ptr(), _rows(dev, "out", out, (N, D), torch.float8_e4m3fn),
          int(group), _flat(dev, "scales", scales, torch.float32, N * groups), total_ptr, total_ld)
    return out, scales, total


def ce_rms_norm_workspace_bytes(rows: int, D: int) -> int:
    n = lib.ce_rms_norm_workspace_bytes(int(rows), int(D))
    if n == 0:
        _check(_abi.CE_EINVAL)
    return int(n)


def ce_rms_norm_backward(dy, s, weight, eps=1e-6, *, dsum=None, dx=None, dweight=None, accumulate=False, ws=None,
                         want_dx=True, want_dweight=True):
    """The gradient from the forward's sum ``s`` ([N, D]): (dx, the gradient of x and of the residual, in s's
    dtype; dweight, FP32 [D]).  ``dsum`` is the gradient that reaches the sum by the residual stream; ``dx`` may
    be dy, dsum or s itself; ``accumulate`` adds to ``dweight``."""
    dev = _index(s, "s")
    n = _norm_desc(dev, s, weight, None, eps)
    N, D = s.shape
    dy_ptr, dy_ld = _like(dev, "dy", dy, s)[1:] if dy is not None else _einval("dy is missing")
    dsum_ptr, dsum_ld = (None, 0) if dsum is None else _like(dev, "dsum", dsum, s)[1:]
    dx_ptr, dx_ld = None, 0
    if dx is not None or want_dx:
        dx, dx_ptr, dx_ld = _like(dev, "dx", dx, s)
    if dweight is None:
        if accumulate:
            _einval("accumulate needs dweight")
        if want_dweight:
            dweight = torch.empty(D, dtype=torch.float32, device=s.device)
    dweight_ptr = ws_ptr = None
    ws_bytes = 0
    if dweight is not None:
        dweight_ptr = _flat(dev, "dweight", dweight, torch.float32, D)
        ws = _workspace(ce_rms_norm_workspace_bytes(N, D), s.device) if ws is None else ws
        ws_ptr, ws_bytes = _flat(dev, "workspace", ws, torch.uint8, 0), ws.numel()
    _call(dev, lib.ce_rms_norm_backward, n, dy_ptr, dy_ld, dsum_ptr, dsum_ld, dx_ptr, dx_ld, dweight_ptr,
          1 if accumulate else 0, ws_ptr, ws_bytes)
    return dx, dweight


class RmsNorm(torch.autograd.Function):
    """Autograd form of ce_rms_norm and ce_rms_norm_backward over (..., D) tensors.  Only the sum (or x itself)
    and the weight are kept; the backward recomputes the row's scale from them."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        D = x.shape[-1]
        flat = _own_rows(x.reshape(-1, D))
        y, total = ce_rms_norm(flat, weight, None if residual is None else _own_rows(residual.reshape(-1, D)), eps)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        if residual is None:
            ctx.save_for_backward(x, weight)
            return y.view(x.shape)
        total = total.view(x.shape)
        ctx.save_for_backward(total, weight)
        return y.view(x.shape), total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum=None):
        s, weight = ctx.saved_tensors
        if dy is None:  # only the sum was used
            return dsum, None, dsum if ctx.needs_input_grad[2] else None, None
        D = s.shape[-1]

        def flat(t):
            return None if t is None else _own_rows(t.reshape(-1, D))

        dx, dweight = ce_rms_norm_backward(flat(dy), flat(s), weight, ctx.eps, dsum=flat(dsum),
                                           want_dx=ctx.needs_input_grad[0] or ctx.needs_input_grad[2],
                                           want_dweight=ctx.needs_input_grad[1])
        dx = None if dx is None else dx.view(s.shape)
        return (dx if ctx.needs_input_grad[0] else None, dweight, dx if ctx.needs_input_grad[2] else None, None)


def rms_norm(x, weight, residual=None, eps=1e-6):
    """RMS norm over the last dimension; with ``residual`` of ``x + residual``, returning (y, sum).  Reaches
    autograd through RmsNorm: x, residual and weight (an FP32 gradient, cast to the weight's dtype)."""
    if residual is not None and residual.shape != x.shape:
        _einval(f"residual must be {tuple(x.shape)}, got {tuple(residual.shape)}")
    return RmsNorm.apply(x, weight, residual, eps)


def norm_linear_cross_entropy(h, norm_weight, weight, target, label_smoothing=0.0, reduce_loss="mean",
                              ignore_idx=-100, *, residual=None, eps=1e-6, smoothing="all", chunk_rows=0,
                              gemm="auto"):
    """The end of a language model: the final RMS norm (of ``h``, or of ``h + residual``), the head and the loss,
    by rms_norm and linear_cross_entropy.  ``h`` and ``residual`` [N, D]."""
    y = rms_norm(h, norm_weight, residual, eps)
    return linear_cross_entropy(y if residual is None else y[0], weight, target, label_smoothing, reduce_loss,
                                ignore_idx, smoothing=smoothing, chunk_rows=chunk_rows, gemm=gemm)


# ---- token log-probabilities -----------------------------------------------------------------------------


class TokenLogprobs(NamedTuple):
    """What ce_token_logprobs and token_logprobs return; None where it was not asked for."""

    logprobs: Optional[torch.Tensor]      # FP32, the shape of ids
    entropy: Optional[torch.Tensor]       # FP32 (d0, d1)
    top_ids: Optional[torch.Tensor]       # int64 (d0, d1, top_k)
    top_logprobs: Optional[torch.Tensor]  # FP32 (d0, d1, top_k)
    stats: Optional[torch.Tensor]         # FP32 [N, 4], for ce_token_logprobs_backward
    lse: Optional[torch.Tensor]           # FP32 (d0, d1)


def _too_many(what, n):
    """Counts are 32-bit in the C interface; ctypes would take this one modulo 2^32."""
    _einval(f"{what}: {n} a row is out of range")


def _listed(dev, what, t, d0, d1, dtype):
    """A (d0, d1, n) companion of the logits, (d0, d1) standing for n = 1: (pointer, s0, s1, n)."""
    if not (isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype):
        _need(torch.device("cuda", dev), what, t, dtype, contiguous=False)  # raises
        _einval(f"{what} is missing")
    shape, st = t.shape, t.stride()
    if len(shape) not in (2, 3) or shape[0] != d0 or shape[1] != d1:
        _einval(f"{what} must be ({d0}, {d1}) or ({d0}, {d1}, n), got {tuple(shape)}")
    n = shape[2] if len(shape) == 3 else 1
    if n > 1 and st[2] != 1:
        _elayout(f"{what} needs a contiguous last dimension")
    if n >> 31:
        _too_many(what, n)
    return t.data_ptr(), st[0], st[1], n


def _out_logits(dev, x, out):
    """The descriptor of a tensor like x that a gradient is written to."""
    if not (isinstance(out, _Tensor) and out.get_device() == dev and out.dtype is x.dtype):
        _need(torch.device("cuda", dev), "out", out, x.dtype, contiguous=False)  # raises
    if out.shape != x.shape:
        _einval(f"out must be {tuple(x.shape)}, got {tuple(out.shape)}")
    return _logits(out, "out", 0, None)[0]


def _prepared(dev, ws, nbytes, x):
    """A prepared workspace: the caller's, or a new one of ``nbytes`` bytes."""
    if ws is None:
        ws = _workspace(nbytes, x.device)
    elif not (isinstance(ws, _Tensor) and ws.get_device() == dev and ws.dtype is torch.uint8 and ws.is_contiguous()):
        _need(torch.device("cuda", dev), "workspace", ws, torch.uint8)  # raises
    if not _is_prepared(ws):
        ce_workspace_init(ws)
    return ws


def ce_token_logprobs_workspace_bytes(x, top_k=0) -> int:
    """Workspace bytes of ce_token_logprobs for (d0, d1, V) logits (256: it uses none)."""
    top_k = int(top_k)
    if top_k >> 31:
        _too_many("top_k", top_k)
    n = lib.ce_token_logprobs_workspace_bytes(_logits(x, "logits", 0, None)[0], top_k)
    if n == 0:
        _check(_abi.CE_EINVAL)
    return int(n)


def ce_token_logprobs(x, ids=None, *, top_k=0, entropy=False, stats=False, lse=False, ignore_idx=-100, ws=None):
    """Log-probabilities of given tokens under the softmax of (d0, d1, V) logits, which are left as they are.

    ``ids`` (d0, d1) or (d0, d1, M) int64, M up to 128, any row strides; those equal to ``ignore_idx`` get 0.
    ``top_k`` (up to 128): the columns of the largest logits, equal ones by the lower column, and their
    log-probabilities.  ``entropy``, ``lse`` and ``stats`` (what the gradient takes) on request.  ``ws`` is a
    workspace of ce_token_logprobs_workspace_bytes bytes to keep between calls.  Returns a TokenLogprobs."""
    dev = _index(x, "logits")
    xd, d0, d1, V = _logits(x, "logits", 0, None)
    top_k = int(top_k)
    if top_k >> 31:
        _too_many("top_k", top_k)
    f32, device = torch.float32, x.device
    ids_ptr, s0, s1, M = (None, 0, 0, 0) if ids is None else _listed(dev, "ids", ids, d0, d1, torch.int64)
    q = _abi.CeLogprobs(ids_ptr, s0, s1, M, top_k, int(ignore_idx))
    nbytes = lib.ce_token_logprobs_workspace_bytes(xd, top_k)
    if nbytes == 0:
        _check(_abi.CE_EINVAL)
    # (sizes by themselves: 1.3 us a tensor, 1.65 as a tuple)
    logp = None if ids is None else torch.empty(*ids.shape, dtype=f32, device=device)
    ent = torch.empty(d0, d1, dtype=f32, device=device) if entropy else None
    top_ids = top_logp = None
    if top_k:
        top_ids = torch.empty(d0, d1, top_k, dtype=torch.int64, device=device)
        top_logp = torch.empty(d0, d1, top_k, dtype=f32, device=device)
    st = torch.empty(d0 * d1, 4, dtype=f32, device=device) if stats else None
    log_sum = torch.empty(d0, d1, dtype=f32, device=device) if lse else None
    ws_ptr, ws_bytes = None, 0
    if nbytes > 256:
        ws = _prepared(dev, ws, nbytes, x)
        ws_ptr, ws_bytes = ws.data_ptr(), ws.numel()
    _call(dev, lib.ce_token_logprobs, xd, q, None if logp is None else logp.data_ptr(),
          None if ent is None else ent.data_ptr(), None if log_sum is None else log_sum.data_ptr(),
          None if top_ids is None else top_ids.data_ptr(), None if top_logp is None else top_logp.data_ptr(),
          None if st is None else st.data_ptr(), ws_ptr, ws_bytes)
    return TokenLogprobs(logp, ent, top_ids, top_logp, st, log_sum)


def ce_token_logprobs_backward(x, stats, ids=None, dlogprobs=None, *, dentropy=None, top_ids=None, dtop=None,
                               out=None, ignore_idx=-100):
    """The gradient of ce_token_logprobs with respect to the logits ``x``, from its ``stats`` and the gradients of
    its log-probabilities (``dlogprobs``, FP32, contiguous, for ``ids``), its entropy (``dentropy``; the forward was
    asked for it) and its alternatives' log-probabilities (``dtop`` for ``top_ids``).  Into ``out``, which may be
    ``x`` itself, or a new tensor."""
    dev = _index(x, "logits")
    xd, d0, d1, V = _logits(x, "logits", 0, None)
    N, f32 = d0 * d1, torch.float32
    ids_ptr, s0, s1, M, K = None, 0, 0, 0, 0
    if ids is not None:
        if dlogprobs is None:
            _einval("ids need dlogprobs")
        ids_ptr, s0, s1, M = _listed(dev, "ids", ids, d0, d1, torch.int64)
    elif dlogprobs is not None:
        _einval("dlogprobs need ids")
    if (top_ids is None) != (dtop is None):
        _einval("top_ids and dtop come together")
    if top_ids is not None:
        K = _listed(dev, "top_ids", top_ids, d0, d1, torch.int64)[3]
    if stats is None:
        _einval("stats is missing")
    out = torch.empty_like(x) if out is None else out
    od = xd if out is x else _out_logits(dev, x, out)
    q = _abi.CeLogprobs(ids_ptr, s0, s1, M, K, int(ignore_idx))
    _call(dev, lib.ce_token_logprobs_backward, xd, od, q, _flat(dev, "stats", stats, f32, 4 * N),
          _flat(dev, "dlogprobs", dlogprobs, f32, N * M), _flat(dev, "dentropy", dentropy, f32, N),
          _flat(dev, "top_ids", top_ids, torch.int64, N * K), _flat(dev, "dtop", dtop, f32, N * K))
    if od.data == xd.data:
        _overwritten(x)
    return out


class TokenLogprobsFn(torch.autograd.Function):
    """Autograd form of ce_token_logprobs: the logits, 16 bytes a row and the ids are kept."""

    @staticmethod
    def forward(ctx, x, ids, top_k, entropy, ignore_idx, ws):
        if x.dim() != 3:
            _einval("logits must be a 3-d (d0, d1, V) tensor")
        flat = _own_rows(x.detach())
        r = ce_token_logprobs(flat, ids, top_k=top_k, entropy=entropy, stats=ctx.needs_input_grad[0],
                              ignore_idx=ignore_idx, ws=ws)
        ctx.ignore_idx = ignore_idx
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, ids, r.stats, r.top_ids)
        if r.top_ids is not None:
            ctx.mark_non_differentiable(r.top_ids)
        return r.logprobs, r.entropy, r.top_ids, r.top_logprobs

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, _, dtop):
        x, ids, stats, top_ids = ctx.saved_tensors
        if dlogp is None and dentropy is None and dtop is None:
            return (None,) * 6

        def flat(t):
            return None if t is None else t.float().contiguous()

        x = _own_rows(x)
        dx = ce_token_logprobs_backward(x, stats, None if dlogp is None else ids, flat(dlogp), dentropy=flat(dentropy),
                                        top_ids=None if dtop is None else top_ids, dtop=flat(dtop),
                                        out=torch.empty_like(x), ignore_idx=ctx.ignore_idx)
        return (dx,) + (None,) * 5


def token_logprobs(logits, ids=None, *, top_k=0, entropy=False, ignore_idx=-100, ws=None):
    """Log-probabilities of ``ids``, the entropy and the ``top_k`` alternatives as ce_token_logprobs gives them, with
    a gradient: of the log-probabilities, of the entropy and of the alternatives' log-probabilities.  Returns a
    TokenLogprobs (without stats and lse).

    The logits are kept for the backward, which raises if something has written over them since.  A loss that stages its
    gradient in its logits (parallel_cross_entropy, processed_cross_entropy, sharded_cross_entropy, distillation_loss)
    therefore comes after this call and takes a copy, ``logits.clone()``; called before, it leaves its gradient to be
    read here."""
    if ids is None and not top_k and not entropy:
        _einval("nothing is asked for: ids, top_k or entropy")
    logp, ent, top_ids, top_logp = TokenLogprobsFn.apply(logits, ids, int(top_k), bool(entropy), int(ignore_idx), ws)
    return TokenLogprobs(logp, ent, top_ids, top_logp, None, None)


# ---- distillation ----------------------------------------------------------------------------------------

_TEACHERS = {"logits": _abi.CE_TEACHER_LOGITS, "logprobs": _abi.CE_TEACHER_LOGPROBS}


def ce_distill_workspace_bytes(x) -> int:
    """Workspace bytes of ce_distill_fwd_bwd for (d0, d1, V) logits."""
    n = lib.ce_distill_workspace_bytes(_logits(x, "logits", 0, None)[0])
    if n == 0:
        _check(_abi.CE_EINVAL)
    return int(n)


def ce_distill_fwd_bwd(x, teacher_ids, teacher_values, temperature=1.0, reduce_loss=False, *, teacher="logits",
                       teacher_len=None, out=None, want_grad=True, grad_out=None, loss=None, n_valid=None, ws=None):
    """Distillation of (d0, d1, V) logits from a teacher's top logits: T^2 times the Kullback-Leibler divergence of
    softmax(x / T) from the teacher's distribution, and its gradient, written over ``x`` or into ``out``.

    ``teacher_ids`` (d0, d1, K) int64 and ``teacher_values`` (d0, d1, K) FP32 or BF16, K up to 128, any row strides:
    ``teacher="logits"``, the softmax of their values at T is the whole distribution; ``"logprobs"``, they are
    log-probabilities (at T), and what they leave of 1 goes to all the other columns as one class.  ``teacher_len``
    [N] int32: how many entries of a row, the first ones, count; a row of none is left out.  ``reduce_loss`` and
    ``grad_out`` as in ce_fwd_bwd_fused; ``want_grad=False`` computes the loss alone and leaves ``x`` as it is.
    Returns (loss [N] or [1], n_valid if given or None)."""
    dev = _index(x, "logits")
    xd, d0, d1, V = _logits(x, "logits", 0, None)
    N, f32 = d0 * d1, torch.float32
    code = reduction_code(reduce_loss)
    if teacher not in _TEACHERS:
        _einval(f"teacher {teacher!r} is not one of {sorted(_TEACHERS)}")
    ids_ptr, is0, is1, K = _listed(dev, "teacher_ids", teacher_ids, d0, d1, torch.int64)
    if not isinstance(teacher_values, _Tensor):
        _einval("teacher_values must be a torch tensor")
    val_ptr, vs0, vs1, Kv = _listed(dev, "teacher_values", teacher_values, d0, d1, teacher_values.dtype)
    if K != Kv:
        _einval(f"{K} teacher_ids and {Kv} teacher_values a row")
    d = _abi.CeDistill(ids_ptr, is0, is1, val_ptr, vs0, vs1, _code(teacher_values.dtype, -1), _TEACHERS[teacher], K,
                       float(temperature), _flat(dev, "teacher_len", teacher_len, torch.int32, N))
    od = None
    if want_grad:
        od = xd if out is None or out is x else _out_logits(dev, x, out)
    elif out is not None:
        _einval("out without want_grad")
    n_loss = N if code == _abi.CE_REDUCE_NONE else 1
    loss = torch.empty(n_loss, dtype=f32, device=x.device) if loss is None else loss
    loss_ptr = _flat(dev, "loss", loss, f32, n_loss)
    g_ptr = _flat(dev, "grad_out", grad_out, f32, n_loss)
    n_ptr = _flat(dev, "n_valid", n_valid, torch.int32, 1)
    nbytes = lib.ce_distill_workspace_bytes(xd)
    if nbytes == 0:
        _check(_abi.CE_EINVAL)
    ws = _prepared(dev, ws, nbytes, x)
    _call(dev, lib.ce_distill_fwd_bwd, xd, od, d, code, g_ptr, loss_ptr, n_ptr, ws.data_ptr(), ws.numel())
    if want_grad and od.data == xd.data:
        _overwritten(x)
    return loss, n_valid


class DistillationLoss(torch.autograd.Function):
    """The loss, with the gradient staged in place in ``inp`` for an upstream gradient of 1, which the backward then
    applies (ce_scale_grad_inplace), as for the cross-entropy.  Without a gradient to give, ``inp`` is left as it is."""

    @staticmethod
    def forward(ctx, inp, teacher_ids, teacher_values, temperature, reduce_loss, teacher, teacher_len, ws, want_grad):
        buf = inp.detach()
        if buf.dim() != 3:
            _einval("logits must be a 3-d (d0, d1, V) tensor")
        loss, _ = ce_distill_fwd_bwd(buf, teacher_ids, teacher_values, temperature, reduce_loss, teacher=teacher,
                                     teacher_len=teacher_len, want_grad=want_grad, ws=ws)
        ctx.reduced = reduction_code(reduce_loss) != _abi.CE_REDUCE_NONE
        ctx.save_for_backward(buf)
        return loss[0] if ctx.reduced else loss.view(buf.shape[:2])

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        (buf,) = ctx.saved_tensors
        ce_scale_grad_inplace(buf, grad_loss, per_row=not ctx.reduced)
        return (buf,) + (None,) * 8


def distillation_loss(inp, teacher_ids, teacher_values, temperature=1.0, reduce_loss=False, *, teacher="logits",
                      teacher_len=None, ws=None):
    """ce_distill_fwd_bwd through autograd: the loss ((d0, d1), or a scalar with a reduction), whose gradient reaches
    ``inp`` and is staged in its storage, as parallel_cross_entropy's; where none is recorded (no_grad), ``inp`` is left
    as it is.  The teacher's values are constants.

    Beside another loss on the same logits all but the last take a copy: ``distillation_loss(inp.clone(), ...)``, then
    ``parallel_cross_entropy(inp, ...)``.  Without it the backward of what came before raises."""
    _constants(teacher_values=teacher_values)
    return DistillationLoss.apply(inp, teacher_ids, teacher_values, temperature, reduce_loss, teacher, teacher_len, ws,
                                  inp.requires_grad and torch.is_grad_enabled())
