"""The operators around the loss: logit processing, embedding and RMS norm.

Like the rest of the binding, the ``ce_*`` functions marshal torch device
tensors into the C ABI's descriptors (``include/ce.h`` defines each operator)
and run on torch's current stream of the tensors' device; ``process_logits``,
``processed_cross_entropy``, ``embedding``, ``rms_norm`` and
``norm_linear_cross_entropy`` are their autograd forms.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from . import (CeArgumentError, _check, _device_of, _need, _need_targets, _raw_stream, _workspace,
               ce_fwd_bwd_fused, ce_scale_grad_inplace, ce_workspace_bytes, lib, linear_cross_entropy, reduction_code)

__all__ = [
    "ce_logits_process", "ce_logits_process_backward", "logits_signs", "process_logits", "processed_cross_entropy",
    "ce_embedding", "ce_embedding_backward", "ce_embedding_workspace_bytes", "embedding",
    "ce_rms_norm", "ce_rms_norm_quant", "ce_rms_norm_backward", "ce_rms_norm_workspace_bytes", "rms_norm",
    "norm_linear_cross_entropy",
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
    smoothing, ignored index) and those of process_logits.  As there, the gradient is staged in place in ``inp``."""
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
