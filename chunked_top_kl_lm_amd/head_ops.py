"""Operators around the output head: layer norm, 8-bit activation checkpoints,
head logits and token sampling (C ABI in include/kd_head_ops.h).

As for the loss, the computation runs entirely in libkdtopk.so; this module
checks and marshals arguments.  Calls run on the current stream of their
tensors' device.
"""
from __future__ import annotations

import ctypes

__all__ = ["ACT8_BLOCK", "act8_quantize", "act8_dequantize", "layer_norm_fwd", "layer_norm_bwd", "layer_norm",
           "KdLayerNormFunction", "head_logits", "head_logits_workspace_bytes", "sample", "sample_workspace_bytes"]

ACT8_BLOCK = 128              # KD_ACT8_BLOCK

_kd = None                    # the package, for what the entry points share


def _pkg():
    global _kd
    if _kd is None:
        import chunked_top_kl_lm_amd as kd
        _kd = kd
    return _kd


def declare(L) -> None:
    """Argument types of the library's entry points."""
    i64, i32, vp, f32, f64, sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_double,
                                  ctypes.c_size_t)
    L.kd_act8_quantize.argtypes = [vp, i64, i32, i64, i64, vp, vp, vp]
    L.kd_act8_dequantize.argtypes = [vp, vp, i32, i64, i64, vp, vp]
    L.kd_layer_norm_fwd.argtypes = [vp, i64, i32, vp, vp, i32, i64, i64, f32, vp, vp, vp, vp, vp, vp]
    L.kd_layer_norm_bwd_workspace_bytes.argtypes = [i64, i64]
    L.kd_layer_norm_bwd_workspace_bytes.restype = sz
    L.kd_layer_norm_bwd.argtypes = [vp, vp, i64, vp, vp, i32, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.kd_topk_kl_bwd_act8_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32]
    L.kd_topk_kl_bwd_act8_workspace_bytes.restype = sz
    L.kd_topk_kl_bwd_act8.argtypes = [vp, vp, vp, i32, vp, vp, vp, i64, i64, i64, i64, f32, i64, vp, vp, vp, i32, vp,
                                      i32, vp, vp, sz, vp, vp]
    L.kd_head_logits_workspace_bytes.argtypes = [i64, i64, i64, i32]
    L.kd_head_logits_workspace_bytes.restype = sz
    L.kd_head_logits.argtypes = [vp, i64, vp, i32, i64, i64, i64, vp, vp, sz, vp]
    L.kd_sample_workspace_bytes.argtypes = [i64, i64]
    L.kd_sample_workspace_bytes.restype = sz
    L.kd_sample.argtypes = [vp, i64, i32, i64, i64, vp, i32, f64, i64, f64, f64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for name in ("kd_act8_quantize", "kd_act8_dequantize", "kd_layer_norm_fwd", "kd_layer_norm_bwd",
                 "kd_topk_kl_bwd_act8", "kd_head_logits", "kd_sample"):
        getattr(L, name).restype = i32


def _stream(dev):
    """Handle of the current stream of `dev`.  Small calls are bound by the
    host; where torch has it, the handle without a Stream object around it is
    taken (0.1 instead of 1.9 us)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev.index) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _call(dev, name, *args):
    """Enqueue one entry point on the current stream of `dev` (its last
    argument), with that device current."""
    import torch
    kd = _pkg()
    fn = getattr(kd.lib(), name)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    if rc != 0:
        raise kd.KdError(rc)


def _dtype_code(name, t):
    import torch
    if t.dtype == torch.bfloat16:
        return 0                # KD_BF16
    if t.dtype == torch.float32:
        return 1                # KD_F32
    raise TypeError(f"{name} must be bfloat16 or float32")


def _rows(name, t):
    """(rows, width, row stride) of a 2-d tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    n, d = t.shape
    if d > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    ld = t.stride(0) if n > 1 else d
    if ld < d:
        raise ValueError(f"{name}: rows overlap")
    return n, d, ld


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _expect(name, t, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype).replace('torch.', '')} tensor of shape {shape}")


def _workspace(dev, nbytes, workspace):
    import torch
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    kd = _pkg()
    kd._check_device(dev, workspace=workspace)
    kd._check_workspace(workspace, None)
    return workspace


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints
# ---------------------------------------------------------------------------
def act8_blocks(d: int) -> int:
    return -(-d // ACT8_BLOCK)


def check_act8(checkpoint, dev=None):
    """(q, scale, T, d) of an 8-bit checkpoint, checked."""
    import torch
    if len(checkpoint) != 2:
        raise ValueError("a checkpoint is a pair (q, scale)")
    q, scale = checkpoint
    if dev is None:
        dev = _cuda("q", q)
    _pkg()._check_device(dev, q=q, scale=scale)
    if q.dim() != 2:
        raise ValueError("q must have two dimensions")
    T, d = q.shape
    _expect("q", q, torch.int8, (T, d))
    _expect("scale", scale, torch.float32, (T, act8_blocks(d)))
    return q, scale, T, d


def act8_quantize(x):
    """8-bit checkpoint of an activation x [T, d] (bfloat16 or float32; rows
    contiguous, any row stride): (q int8 [T, d], scale float32
    [T, ceil(d / 128)]).  Each block of 128 elements of a row is kept within
    1/254 of its largest magnitude; a block with an Inf or NaN comes back as
    NaN (kd_act8_quantize)."""
    import torch
    dev = _cuda("x", x)
    dt = _dtype_code("x", x)
    T, d, ld = _rows("x", x)
    q = torch.empty((T, d), dtype=torch.int8, device=dev)
    scale = torch.empty((T, act8_blocks(d)), dtype=torch.float32, device=dev)
    _call(dev, "kd_act8_quantize", x.data_ptr(), ld, dt, T, d, q.data_ptr(), scale.data_ptr())
    return q, scale


def act8_dequantize(q, scale, dtype=None):
    """The values an 8-bit checkpoint stands for, as `dtype` (bfloat16 by
    default, or float32) [T, d]."""
    import torch
    q, scale, T, d = check_act8((q, scale))
    out = torch.empty((T, d), dtype=torch.bfloat16 if dtype is None else dtype, device=q.device)
    _call(q.device, "kd_act8_dequantize", q.data_ptr(), scale.data_ptr(), _dtype_code("dtype", out), T, d, out.data_ptr())
    return out


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def _check_weight(dev, d, dt, weight, bias):
    import torch
    _pkg()._check_device(dev, weight=weight, bias=bias)
    wdt = _dtype_code("weight", weight)
    if dt == 1 and wdt != 1:
        raise TypeError("weight must be float32 or of x's dtype")
    _expect("weight", weight, weight.dtype, (d,))
    if bias is not None:
        _expect("bias", bias, weight.dtype, (d,))
    return wdt


def _check_kind(checkpoint):
    if checkpoint not in (None, "int8"):
        raise ValueError("checkpoint must be None or 'int8'")


def layer_norm_fwd(x, weight, bias=None, eps: float = 1e-5, checkpoint=None):
    """Layer norm of the rows of x [T, d] (bfloat16 or float32; rows
    contiguous, any row stride), weight [d] and optional bias [d] in float32
    or x's dtype.  Returns (y [T, d], mean [T], rstd [T]; the statistics
    float32) and, with checkpoint="int8", also (q, scale): x's 8-bit
    checkpoint, written in the same pass, for a backward that does not keep
    x (kd_layer_norm_fwd)."""
    import torch
    dev = _cuda("x", x)
    dt = _dtype_code("x", x)
    T, d, ld = _rows("x", x)
    wdt = _check_weight(dev, d, dt, weight, bias)
    _check_kind(checkpoint)
    y = torch.empty((T, d), dtype=x.dtype, device=dev) if ld != d else torch.empty_like(x)
    mean = torch.empty(T, dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    q = scale = None
    if checkpoint is not None:
        q = torch.empty((T, d), dtype=torch.int8, device=dev)
        scale = torch.empty((T, act8_blocks(d)), dtype=torch.float32, device=dev)
    _call(dev, "kd_layer_norm_fwd", x.data_ptr(), ld, dt, weight.data_ptr(), None if bias is None else bias.data_ptr(),
          wdt, T, d, float(eps), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), None if q is None else q.data_ptr(),
          None if q is None else scale.data_ptr())
    return (y, mean, rstd) if q is None else (y, mean, rstd, q, scale)


def layer_norm_bwd(dy, x, weight, mean, rstd, need_dx: bool = True, need_dweight: bool = True, workspace=None):
    """Backward of layer_norm_fwd: (dx in dy's dtype, dweight, dbias; the last
    two float32), None for what was not asked.  `x` is the forward's input,
    or its checkpoint (q, scale), whose values then stand for it.
    `workspace`: a uint8 CUDA tensor of kd_layer_norm_bwd_workspace_bytes."""
    import torch
    kd = _pkg()
    dev = _cuda("dy", dy)
    dt = _dtype_code("dy", dy)
    T, d, ld = _rows("dy", dy)
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    q = scale = None
    if isinstance(x, (tuple, list)):
        q, scale, Tq, dq = check_act8(x, dev)
        if (Tq, dq) != (T, d):
            raise ValueError("shapes: dy and the checkpoint [T,d]")
    else:
        kd._check_device(dev, x=x)
        if x.dtype != dy.dtype:
            raise TypeError("dy must have x's dtype")
        if tuple(x.shape) != (T, d):
            raise ValueError("shapes: dy and x [T,d]")
        ld = _rows("x", x)[2]
    wdt = _check_weight(dev, d, dt, weight, None)
    kd._check_device(dev, mean=mean, rstd=rstd)
    _expect("mean", mean, torch.float32, (T,))
    _expect("rstd", rstd, torch.float32, (T,))
    dx = torch.empty_like(dy) if need_dx else None
    dw = torch.empty(d, dtype=torch.float32, device=dev) if need_dweight else None
    db = torch.empty_like(dw) if need_dweight else None
    ws = None
    if need_dweight:
        ws = _workspace(dev, int(kd.lib().kd_layer_norm_bwd_workspace_bytes(T, d)), workspace)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(dev, "kd_layer_norm_bwd", dy.data_ptr(), p(None if q is not None else x), ld, p(q), p(scale), dt, p(weight), wdt,
          T, d, p(mean), p(rstd), p(dx), p(dw), p(db), p(ws), 0 if ws is None else ws.numel())
    return dx, dw, db


def _layer_norm_function():
    import torch

    class KdLayerNormFunction(torch.autograd.Function):
        """Layer norm over the last dimension as an autograd node.

        forward(x, weight, bias, eps, checkpoint) -> y.  Saves x, or with
        checkpoint="int8" its 8-bit checkpoint instead, and two floats per
        row.  Gradients come back in their inputs' dtypes (the weight's
        summed in float32)."""

        @staticmethod
        def forward(ctx, x, weight, bias, eps, checkpoint):
            rows = x if x.dim() == 2 else (x.flatten(0, -2) if x.dim() > 2 else x[None])
            if rows.dim() == 2 and (rows.stride(1) != 1 or rows.stride(0) < rows.shape[1]):
                rows = rows.contiguous()         # transposed, or rows that share memory (a broadcast input)
            y, mean, rstd, *kept = layer_norm_fwd(rows, weight, bias, eps, checkpoint)
            ctx.save_for_backward(weight, mean, rstd, *(kept or (rows,)))
            ctx.shape, ctx.rows, ctx.bias_dtype = x.shape, rows.shape, None if bias is None else bias.dtype
            return y.view(x.shape)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            weight, mean, rstd, *kept = ctx.saved_tensors
            need_x, need_w, need_b = ctx.needs_input_grad[:3]
            if not (need_x or need_w or need_b):
                return (None,) * 5
            dx, dw, db = layer_norm_bwd(dy.reshape(ctx.rows).contiguous(), kept[0] if len(kept) == 1 else tuple(kept),
                                        weight, mean, rstd, need_dx=need_x, need_dweight=need_w or need_b)
            return (dx.view(ctx.shape) if need_x else None, dw.to(weight.dtype) if need_w else None,
                    db.to(ctx.bias_dtype) if need_b else None, None, None)

    return KdLayerNormFunction


_LN = None


def __getattr__(name):
    global _LN
    if name == "KdLayerNormFunction":
        if _LN is None:
            _LN = _layer_norm_function()
        return _LN
    raise AttributeError(name)


def layer_norm(x, weight, bias=None, eps: float = 1e-5, checkpoint=None):
    """Differentiable layer norm over the last dimension of x (the final norm
    whose output is the loss's `hidden`).  checkpoint="int8" keeps x for the
    backward pass as an 8-bit checkpoint: half of bfloat16's memory, a
    quarter of float32's, for a rounding of x of at most 1/254 of each
    block's largest magnitude in the gradients (y is not affected)."""
    return __getattr__("KdLayerNormFunction").apply(x, weight, bias, eps, checkpoint)


# ---------------------------------------------------------------------------
# head logits
# ---------------------------------------------------------------------------
def head_logits_workspace_bytes(T: int, d: int, V: int, dtype: int) -> int:
    return int(_pkg().lib().kd_head_logits_workspace_bytes(T, d, V, dtype))


def head_logits(hidden, W, out=None, workspace=None):
    """Logits of the output head, hidden [T, d] times W [V, d] transposed, as
    float32 [T, V] (kd_head_logits): the form for decoding steps (few rows,
    W read once) and for scoring (many rows).  hidden and W bfloat16 or
    float32; hidden's rows may be strided.  Not differentiable (training goes
    through kd_topk_kl_loss).  `out`: a contiguous float32 [T, V] CUDA tensor; `workspace`: a uint8 CUDA tensor of
    head_logits_workspace_bytes(...) bytes."""
    import torch
    kd = _pkg()
    dev = _cuda("hidden", hidden)
    dt = _dtype_code("hidden", hidden)
    T, d, ld = _rows("hidden", hidden)
    kd._check_device(dev, W=W, out=out)
    if W.dtype != hidden.dtype:
        raise TypeError("W must match hidden's dtype")
    if W.dim() != 2 or W.shape[1] != d or not W.is_contiguous():
        raise ValueError("shapes: hidden [T,d], W [V,d] (contiguous)")
    V = W.shape[0]
    if out is None:
        out = torch.empty((T, V), dtype=torch.float32, device=dev)
    else:
        _expect("out", out, torch.float32, (T, V))
    nbytes = head_logits_workspace_bytes(T, d, V, dt)
    ws = None
    if workspace is not None or nbytes:
        ws = _workspace(dev, nbytes, workspace)
    _call(dev, "kd_head_logits", hidden.data_ptr(), ld, W.data_ptr(), dt, T, d, V, out.data_ptr(),
          None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return out


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------
def sample_workspace_bytes(R: int, V: int) -> int:
    return int(_pkg().lib().kd_sample_workspace_bytes(R, V))


def _row_param(name, value, dtype, dev, R):
    """(scalar or None, per-row tensor or None) of one sampling parameter."""
    import torch
    if not torch.is_tensor(value):
        return value, None
    _pkg()._check_device(dev, **{name: value})
    if tuple(value.shape) != (R,):
        raise ValueError(f"{name} must be a number or a tensor of shape ({R},)")
    if value.dtype.is_complex or (dtype == torch.int32 and value.dtype.is_floating_point):
        raise TypeError(f"{name} has the wrong dtype")
    if dtype == torch.int32 and value.dtype == torch.int64:
        value = value.clamp(0, 2 ** 31 - 1)
    return None, value.to(dtype).contiguous()


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, workspace=None):
    """One token id per row of logits [R, V] (bfloat16 or float32; rows may be
    strided) from given uniform numbers u [R] in [0, 1) (float32 or float64):
    (token int32 [R], logprob float32 [R]).

    Ids are ordered by (logit descending, id ascending) under
    softmax(logits / temperature); top_k (0: off) keeps the first ids, top_p
    (1: off) the shortest prefix of these with that share of their mass,
    min_p (0: off) those of at least that share of the largest probability;
    the token is the first kept id, in id order, whose inclusive mass exceeds
    u times the kept mass, and logprob the log of the probability it was
    drawn with.  temperature 0 takes the largest logit.  Each parameter is a
    number or a tensor of one value per row.  A row with nothing to draw
    from (all logits -inf or NaN) gives token -1 and logprob -inf
    (kd_sample)."""
    import torch
    kd = _pkg()
    dev = _cuda("logits", logits)
    dt = _dtype_code("logits", logits)
    R, V, ld = _rows("logits", logits)
    kd._check_device(dev, u=u)
    if u.dtype not in (torch.float32, torch.float64) or tuple(u.shape) != (R,) or not u.is_contiguous():
        raise ValueError(f"u must be a contiguous float32 or float64 tensor of shape ({R},)")
    t, tr = _row_param("temperature", temperature, torch.float64, dev, R)
    k, kr = _row_param("top_k", top_k, torch.int32, dev, R)
    tp, tpr = _row_param("top_p", top_p, torch.float64, dev, R)
    mp, mpr = _row_param("min_p", min_p, torch.float64, dev, R)
    nbytes = sample_workspace_bytes(R, V)
    if nbytes == 0:
        raise kd.KdError(2)
    ws = _workspace(dev, nbytes, workspace)
    token = torch.empty(R, dtype=torch.int32, device=dev)
    logprob = torch.empty(R, dtype=torch.float32, device=dev)
    p = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    _call(dev, "kd_sample", logits.data_ptr(), ld, dt, R, V, u.data_ptr(), 1 if u.dtype == torch.float64 else 0,
          1.0 if t is None else float(t), 0 if k is None else int(k), 1.0 if tp is None else float(tp),
          0.0 if mp is None else float(mp), p(tr), p(kr), p(tpr), p(mpr), token.data_ptr(), logprob.data_ptr(),
          ws.data_ptr(), ws.numel())
    return token, logprob
