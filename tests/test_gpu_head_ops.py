"""The operators around the head on the GPU against the fp64 oracle
(oracle/head_ops.py): layer norm forward and backward, 8-bit checkpoints and
the backward passes that read them, head logits, sampling, and a run of them
together.

Tolerances.  A result rounded to a type is off by at most half a step of it,
finfo(t).eps / 2 relative (bf16 2^-8, fp32 2^-24).  The fp32 arithmetic
before that rounding: sums of n terms in fp32 are off by at most n 2^-24 of
the sum of the terms' magnitudes, however they are ordered; the bounds below
count the terms and scale by those magnitudes.
"""
import numpy as np
import pytest

from datagen import config_for, make_inputs, to_device
from oracle import fused_kl
from oracle import head_ops as o
from tests.gpu_util import log, rel, rel_f

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def _t():
    import torch
    return torch


def _half(dtype):
    return _t().finfo(dtype).eps / 2


def _np(t):
    return t.detach().double().cpu().numpy()


def _norm_inputs(T, d, dtype, seed, wdtype=None):
    torch = _t()
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) + 0.3).to(dtype)
    dy = torch.randn(T, d, generator=g).to(dtype)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(wdtype or dtype)
    b = (0.3 * torch.randn(d, generator=g)).to(wdtype or dtype)
    return [v.cuda() for v in (x, dy, w, b)]


def _check_norm(x, dy, w, b, got, kept=None):
    """got: (y, mean, rstd, dx, dw, db); kept: the values the backward saw for x."""
    y, mean, rstd, dx, dw, db = got
    T, d = x.shape
    X, DY, W = _np(x), _np(dy), _np(w)
    ry, rm, rr = o.layer_norm(X, W, None if b is None else _np(b), EPS)
    # mean: a sum of d terms; rstd: sums of d squares of differences with that mean, a division and a root
    n = d + 16
    scale = np.abs(X).mean(1)
    assert (np.abs(_np(mean) - rm) <= n * U * scale).all()
    em = (n * U * scale * rr)[:, None]                       # the mean's error in units of the row's deviation
    er = n * U + em[:, 0]                                    # relative error of rstd
    assert (np.abs(_np(rstd) - rr) <= rr * er).all()
    xh = np.abs((X - rm[:, None]) * rr[:, None])
    fp = (em + xh * (er[:, None] + 4 * U)) * np.abs(W) + 2 * U * (0 if b is None else np.abs(_np(b)))
    assert (np.abs(_np(y) - ry) <= _half(y.dtype) * np.abs(ry) + fp * 1.01 + 1e-37).all()
    # the backward against its formula with the statistics that it was given
    XB = X if kept is None else kept
    rdx, rdw, rdb = o.layer_norm_grads(DY, XB, W, _np(mean), _np(rstd))
    s = _np(rstd)[:, None]
    xh = np.abs((XB - _np(mean)[:, None]) * s)
    exh = 4 * U * (np.abs(XB) + np.abs(_np(mean))[:, None]) * s   # x - mean, q * scale and the product
    g = np.abs(DY * W)
    a, c = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    ec = (g * exh).mean(1, keepdims=True)
    fp = s * (4 * U * g + n * U * a + (n * U * c + ec) * xh + c * exh + 4 * U * c * xh)
    assert (np.abs(_np(dx) - rdx) <= _half(dx.dtype) * np.abs(rdx) + fp * 1.01 + 1e-37).all()
    m = T + 16
    assert (np.abs(_np(dw) - rdw) <= (m * U * np.abs(DY) * xh + np.abs(DY) * exh).sum(0) * 1.01 + 1e-37).all()
    assert (np.abs(_np(db) - rdb) <= m * U * np.abs(DY).sum(0) * 1.01 + 1e-37).all()


SHAPES = [(1, 1), (3, 2), (1, 2880), (5, 63), (9, 511), (4, 513), (130, 257), (33, 1024), (7, 1999), (300, 2880), (2, 3073),
          (17, 4096), (6, 5001), (3, 8192), (5, 9001), (2, 16384), (3, 20001), (2, 32768), (3000, 128)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
def test_layer_norm(T, d, dtype, wdtype):
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    log(f"[layer_norm] T={T} d={d} {dtype} {wdtype}")
    x, dy, w, b = _norm_inputs(T, d, getattr(torch, dtype), T + d, getattr(torch, wdtype))
    y, mean, rstd = kd.layer_norm_fwd(x, w, b, EPS)
    _check_norm(x, dy, w, b, (y, mean, rstd, *kd.layer_norm_bwd(dy, x, w, mean, rstd)))
    # from the 8-bit checkpoint that the forward writes: the same y, the checkpoint of act8_quantize
    y8, mean8, rstd8, q, s = kd.layer_norm_fwd(x, w, b, EPS, checkpoint="int8")
    assert torch.equal(y8, y) and torch.equal(mean8, mean) and torch.equal(rstd8, rstd)
    rq, rs = o.act8(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    _check_norm(x, dy, w, b, (y, mean, rstd, *kd.layer_norm_bwd(dy, (q, s), w, mean, rstd)), o.act8_values(rq, rs))


def test_layer_norm_without_bias_strided_and_partial():
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x, dy, w, _ = _norm_inputs(21, 301, torch.bfloat16, 3)
    wide = torch.full((21, 400), 7.0, dtype=torch.bfloat16, device="cuda:0")
    wide[:, 5:306] = x
    view = wide[:, 5:306]                                        # rows start at odd multiples of 2 bytes
    y, mean, rstd, q, s = kd.layer_norm_fwd(view, w, None, EPS, checkpoint="int8")
    y0, mean0, rstd0 = kd.layer_norm_fwd(x, w, None, EPS)
    assert torch.equal(y, y0) and torch.equal(rstd, rstd0)
    full = kd.layer_norm_bwd(dy, view, w, mean, rstd)
    _check_norm(x, dy, w, None, (y, mean, rstd, *full))
    a = kd.layer_norm_bwd(dy, view, w, mean, rstd, need_dweight=False)
    b = kd.layer_norm_bwd(dy, view, w, mean, rstd, need_dx=False)
    assert a[1] is a[2] is b[0] is None
    assert torch.equal(a[0], full[0]) and torch.equal(b[1], full[1]) and torch.equal(b[2], full[2])
    assert (wide[:, :5] == 7).all() and (wide[:, 306:] == 7).all()


@pytest.mark.parametrize("ckpt", [None, "int8"])
def test_layer_norm_autograd(ckpt):
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x, dy, w, b = _norm_inputs(6 * 7, 96, torch.float32, 11)
    x, dy = x.view(6, 7, 96).requires_grad_(), dy.view(6, 7, 96)
    w, b = w.requires_grad_(), b.requires_grad_()
    y = kd.layer_norm(x, w, b, EPS, checkpoint=ckpt)
    y.backward(dy.transpose(0, 1).contiguous().transpose(0, 1))  # a gradient with other strides
    X = _np(x).reshape(-1, 96)
    ry, rm, rr = o.layer_norm(X, _np(w), _np(b), EPS)
    kept = X if ckpt is None else o.act8_values(*o.act8(X.astype(np.float32)))
    rdx, rdw, rdb = o.layer_norm_grads(_np(dy).reshape(-1, 96), kept, _np(w), rm, rr)
    # fp32 throughout, rows of 96 and sums over 42 rows: about 100 roundings of order-one terms
    for got, ref in ((y, ry), (x.grad, rdx), (w.grad, rdw), (b.grad, rdb)):
        assert rel_f(_np(got).reshape(ref.shape), ref) <= 100 * U
    # against differences of y along a direction (the 8-bit rounding of x moves the gradient by a part of 1/254)
    if ckpt is None:
        e = np.random.default_rng(0).normal(size=X.shape)
        h = 1e-4
        num = ((o.layer_norm(X + h * e, _np(w), _np(b), EPS)[0] - o.layer_norm(X - h * e, _np(w), _np(b), EPS)[0])
               * _np(dy).reshape(-1, 96)).sum() / (2 * h)
        assert abs(num - (_np(x.grad).reshape(-1, 96) * e).sum()) <= 1e-4 * np.abs(_np(x.grad).reshape(-1, 96) * e).sum()


def test_layer_norm_autograd_of_broadcast_and_shared_inputs():
    """A broadcast input's gradient is the sum over its copies; a weight used
    twice gets both uses' gradients; transposed inputs are taken."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    g = torch.Generator().manual_seed(9)
    x0, w = torch.randn(1, 40, generator=g).cuda().requires_grad_(), torch.randn(40, generator=g).cuda().requires_grad_()
    dy = torch.randn(6, 40, generator=g).cuda()
    y = kd.layer_norm(kd.layer_norm(x0.expand(6, 40), w), w)
    y.backward(dy)
    xr, wr = x0.detach().cpu().double().requires_grad_(), w.detach().cpu().double().requires_grad_()
    ln = lambda v: torch.nn.functional.layer_norm(v, (40,), wr, None, 1e-5)  # noqa: E731
    ln(ln(xr.expand(6, 40))).backward(dy.cpu().double())
    # two fp32 norms of 40 columns, sums over 6 rows: about 200 roundings, and
    # the second norm's 1 / deviation (here above 0.3) on the first one's error
    assert rel_f(_np(x0.grad), xr.grad.numpy()) <= 1000 * U and rel_f(_np(w.grad), wr.grad.numpy()) <= 1000 * U
    t = torch.randn(40, 5, generator=g).cuda()
    assert torch.equal(kd.layer_norm(t.t(), w), kd.layer_norm(t.t().contiguous(), w))
    # a second derivative is refused, not silently zero
    v = torch.randn(3, 40, generator=g).cuda().requires_grad_()
    gr, = torch.autograd.grad(kd.layer_norm(v, w).sum(), v, create_graph=True)
    with pytest.raises(RuntimeError):
        gr.sum().backward()


def test_layer_norm_more_rows_than_one_launch_covers():
    import chunked_top_kl_lm_amd as kd
    T = 4 * (1 << 20) + 7
    x, dy, w, b = _norm_inputs(T, 3, _t().bfloat16, 1)
    y, mean, rstd, q, s = kd.layer_norm_fwd(x, w, b, EPS, checkpoint="int8")
    rq, rs = o.act8(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    _check_norm(x, dy, w, b, (y, mean, rstd, *kd.layer_norm_bwd(dy, x, w, mean, rstd)))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows come out as they do alone."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    T, d = 1100000, 2000
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda:0").normal_()
    w, b = torch.rand(d, device="cuda:0"), torch.rand(d, device="cuda:0")
    tail = slice(T - 37, T)
    y, mean, rstd, q, s = kd.layer_norm_fwd(x, w, b, EPS, checkpoint="int8")
    one = kd.layer_norm_fwd(x[tail], w, b, EPS, checkpoint="int8")
    for a, c in zip((y, mean, rstd, q, s), one):
        assert torch.equal(a[tail], c)
    q2, s2 = kd.act8_quantize(x)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    back = kd.act8_dequantize(q, s)
    assert torch.equal(back[tail], kd.act8_dequantize(q[tail], s[tail]))
    del back, q2, s2
    dx = kd.layer_norm_bwd(y, (q, s), w, mean, rstd, need_dweight=False)[0]
    assert torch.equal(dx[tail], kd.layer_norm_bwd(y[tail], (q[tail], s[tail]), w, mean[tail], rstd[tail], need_dweight=False)[0])
    del x, y, q, s, dx
    T, V, d = 11000, 201088, 64
    h = torch.empty(T, d, dtype=torch.bfloat16, device="cuda:0").normal_()
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda:0").normal_()
    z = kd.head_logits(h, W)
    last = kd.head_logits(h[-128:], W)
    assert torch.equal(z[-128:], last)
    u = torch.rand(T, device="cuda:0")
    for kw in (dict(), dict(top_k=50), dict(top_p=0.9)):
        tok, lp = kd.sample(z, u, **kw)
        t2, l2 = kd.sample(z[-37:], u[-37:], **kw)
        assert torch.equal(tok[-37:], t2) and torch.equal(lp[-37:], l2)


def test_layer_norm_special_rows():
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x, dy, w, b = _norm_inputs(6, 200, torch.float32, 5)
    x[1] = 3.25                                                  # no deviation: y = b
    x[2] = 0
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    y, mean, rstd = kd.layer_norm_fwd(x, w, b, EPS)
    assert torch.equal(y[1], b) and torch.equal(y[2], b)
    assert y[3].isnan().all() and y[4].isnan().any()
    ry = o.layer_norm(_np(x[[0, 5]]), _np(w), _np(b), EPS)[0]
    assert np.allclose(_np(y[[0, 5]]), ry, atol=1e-5)
    dx, dw, db = kd.layer_norm_bwd(dy, x, w, mean, rstd)
    assert dx[3].isnan().all() and dx[[0, 1, 2, 5]].isfinite().all() and db.isfinite().all()


@pytest.mark.parametrize("T,d", [(1, 1), (2, 127), (3, 128), (5, 129), (64, 2880), (7, 2047), (9, 2049), (2, 70001), (4097, 8)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_act8(T, d, dtype):
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    log(f"[act8] T={T} d={d} {dtype}")
    g = torch.Generator().manual_seed(T * d)
    x = torch.randn(T, d, generator=g) * torch.exp(3 * torch.randn(T, 1, generator=g))
    if T > 4:
        x[0], x[1], x[2, 0], x[3, d - 1] = 0, 1e-39, float("inf"), float("nan")
        x[4] = torch.finfo(torch.bfloat16).max
    x = x.to(getattr(torch, dtype)).cuda()
    q, s = kd.act8_quantize(x)
    rq, rs = o.act8(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    ref = o.act8_values(rq, rs)
    for out_t in (torch.bfloat16, torch.float32):
        v = _np(kd.act8_dequantize(q, s, out_t))
        assert np.array_equal(np.isnan(v), np.isnan(ref))
        ok = ~np.isnan(ref)
        # one rounding of the product to fp32, one to the output's type; subnormals step by the smallest one
        tol = (_half(out_t) + U) * np.abs(ref) + 2.0 ** -133
        fin = np.isfinite(v) & ok
        assert (np.abs(v - ref)[fin] <= tol[fin]).all()
        assert (fin == ok).all() or T > 4                          # (the largest bf16 may round to Inf)
    # strided rows
    wide = torch.zeros(T, d + 3, dtype=x.dtype, device="cuda:0")
    wide[:, 1:d + 1] = x
    q2, s2 = kd.act8_quantize(wide[:, 1:d + 1])
    assert torch.equal(q, q2) and torch.equal(s.nan_to_num(-1), s2.nan_to_num(-1))


@pytest.mark.parametrize("num,kw,chunk", [
    (1, dict(T=300), 128), (3, dict(T=520, d=192, V=3000), 256), (3, dict(T=300, d=257, V=2000), 128),
    (2, dict(T=1, d=64, V=500, K=7), 16)])
def test_loss_backward_from_8_bits(num, kw, chunk):
    """The gradients are those formed from the values the checkpoint stands
    for, with the forward's logsumexp: the plain backward of these values
    with the same row_lse must give the same bits."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x = make_inputs(config_for(num, **kw), seed=3)
    t = to_device(x)
    a = (t["W"], t["teacher_idx"], t["teacher_logit"], t["mask"])
    log(f"[loss act8] workload {num} {kw}")
    loss, row_lse = kd.fwd(t["hidden"], *a, tau=x["tau"], chunk=chunk)
    q, s = kd.act8_quantize(t["hidden"])
    back = kd.act8_dequantize(q, s, t["hidden"].dtype)
    got = kd.bwd((q, s), *a, row_lse, x["tau"], chunk)
    ref = kd.bwd(back, *a, row_lse, x["tau"], chunk)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    # autograd: the loss's bits unchanged, gradients near the exact ones
    h, W = t["hidden"].clone().requires_grad_(), t["W"].clone().requires_grad_()
    l8 = kd.kd_topk_kl_loss(h, W, *a[1:], tau=x["tau"], chunk=chunk, checkpoint="int8")
    l8.backward()
    assert torch.equal(l8.detach(), loss) and h.grad.dtype == h.dtype
    assert torch.equal(h.grad.float(), got[0].to(h.dtype).float())
    r = fused_kl(x["hidden"], x["W"], x["teacher_idx"], x["teacher_logit"], x["mask"], x["tau"])
    e = rel_f(_np(h.grad), r["grad_hidden"]), rel_f(_np(W.grad), r["grad_W"])
    log(f"[loss act8] dH {e[0]:.2e} dW {e[1]:.2e}")
    # each element of hidden is off by up to amax / 254, about 0.6% of its
    # row's deviation rms (amax about 2.7 deviations, a uniform error): as much
    # on G^T H, and a logit error of 0.6% |h| |w| in q: together within 5e-2
    assert max(e) <= 5e-2


LOGIT_SHAPES = [(1, 1, 1), (1, 64, 1000), (3, 40, 17), (16, 257, 333), (17, 2880, 5000), (32, 96, 4096), (33, 64, 999), (64, 200, 5001), (65, 64, 640), (128, 192, 1537), (129, 64, 700),
                (100, 65, 1031), (256, 320, 2048), (300, 128, 70001), (1, 8193, 700), (64, 1000, 258)]


@pytest.mark.parametrize("T,d,V", LOGIT_SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_head_logits(T, d, V, dtype):
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    log(f"[head_logits] T={T} d={d} V={V} {dtype}")
    g = torch.Generator().manual_seed(T + d + V)
    h = torch.randn(T, d, generator=g).to(getattr(torch, dtype)).cuda()
    W = torch.randn(V, d, generator=g).to(getattr(torch, dtype)).cuda()
    H64, W64 = h.double().cpu().numpy(), W.double().cpu().numpy()
    ref = H64 @ W64.T
    # products: exact in bf16, one rounding in fp32; fp32 sums of d terms
    tol = (d + 2) * U * (np.abs(H64) @ np.abs(W64).T)
    z = kd.head_logits(h, W)
    assert z.dtype == torch.float32 and (np.abs(_np(z) - ref) <= tol).all()
    assert torch.equal(z, kd.head_logits(h, W))
    # strided hidden rows that start anywhere, a caller's output and what lies behind it
    wide = torch.zeros(T, d + 5, dtype=h.dtype, device="cuda:0")
    wide[:, 3:3 + d] = h
    buf = torch.full((T * V + 64,), 5.0, device="cuda:0")
    out = kd.head_logits(wide[:, 3:3 + d], W, out=buf[:T * V].view(T, V))
    assert torch.equal(out, z) and (buf[T * V:] == 5).all()


def _check_sample(z, u, kw, rows=None):
    """z [R, V] device tensor; kw scalars or per-row lists."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    R = z.shape[0]
    dev = {k: torch.tensor(v, device="cuda:0") if isinstance(v, list) else v for k, v in kw.items()}
    tok, lp = kd.sample(z, u, **dev)
    tok2, lp2 = kd.sample(z, u, **dev)
    assert torch.equal(tok, tok2) and torch.equal(lp.nan_to_num(9), lp2.nan_to_num(9))
    zn, un = z.double().cpu().numpy(), u.double().cpu().numpy()
    for r in rows if rows is not None else range(R):
        a = {k: (v[r] if isinstance(v, list) else v) for k, v in kw.items()}
        if a.get("top_p", 1.0) <= 0:
            a["top_p"] = 1e-300
        t, p = o.sample(zn[r], un[r], **a)
        got, glp = int(tok[r]), float(lp[r])
        assert got == t, (r, a, got, t, float(un[r]))
        # one rounding to fp32, and the masses' own 1e-11
        assert (p == -np.inf and glp == p) or abs(glp - p) <= U * abs(p) + 1e-9, (r, a, glp, p)


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=7), dict(top_k=50, top_p=0.9), dict(top_p=0.5),
           dict(top_p=0.97, temperature=1.3), dict(min_p=0.05), dict(min_p=0.3, top_p=0.8), dict(top_k=40, top_p=0.9, min_p=0.1),
           dict(top_k=3000), dict(top_k=3000, top_p=0.99), dict(temperature=0.0), dict(temperature=50.0, top_p=0.6),
           dict(min_p=1e-6), dict(top_p=1e-9), dict(min_p=1.0), dict(temperature=1e-30), dict(temperature=1e-30, top_p=0.4),
           dict(temperature=1e-3, min_p=0.1), dict(temperature=1e4, top_p=0.3), dict(temperature=1e30, top_k=500, top_p=0.5),
           dict(temperature=1e30, min_p=0.9), dict(top_k=4096), dict(top_p=0.999999)]


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 1024, 1025, 5000, 33001])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample(V, dtype):
    torch = _t()
    g = torch.Generator().manual_seed(V)
    R = 9
    width = torch.linspace(0.2, 6, R)[:, None]
    wide = torch.full((R, V + 3), 50.0)                          # rows start anywhere; the pad is never drawn
    wide[:, 1:V + 1] = torch.randn(R, V, generator=g) * width
    if V > 3:
        wide[2, 1:1 + V // 2] = -float("inf")
        wide[3, 1:1 + V // 3] = torch.finfo(torch.bfloat16).min
        wide[4, 1 + V // 4] = float("nan")
        wide[5, 1:V + 1] = wide[5, 1:V + 1].round()              # many equal logits
    z = wide.to(getattr(torch, dtype)).cuda()[:, 1:V + 1]
    for i, kw in enumerate(FILTERS):
        log(f"[sample] V={V} {dtype} {kw}")
        u = torch.rand(R, generator=g)
        u[0], u[1] = 0.0, 1 - 2.0 ** -24
        _check_sample(z, (u.double() if i % 2 else u).cuda(), kw)


def test_sample_rows_that_have_nothing_or_infinities():
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    inf, low = float("inf"), torch.finfo(torch.float32).min
    V = 2000
    z = torch.zeros(7, V)
    z[0], z[1] = -inf, float("nan")
    z[2, 5:9] = inf
    z[3] = low
    z[4], z[4, 1999] = -inf, low
    z[5, ::2] = -0.0                                             # zeros of both signs are equal
    z[6] = -inf
    z[6, 1234] = 2.0
    u = torch.tensor([0.3, 0.3, 0.6, 0.5, 0.9, 0.25, 0.999])
    for kw in (dict(), dict(top_k=3), dict(top_p=0.5), dict(min_p=0.5), dict(temperature=0.0), dict(top_k=900, top_p=0.7)):
        log(f"[sample special] {kw}")
        _check_sample(z.cuda(), u.cuda(), kw)
    tok, lp = kd.sample(z.cuda(), u.cuda())
    assert tok.tolist()[:2] == [-1, -1] and (lp[:2] == -inf).all()
    # u outside [0, 1): the nearest end; NaN: 0
    w = torch.zeros(4, 10, device="cuda:0")
    tok, _ = kd.sample(w, torch.tensor([-1.0, 1.0, 1e30, float("nan")], device="cuda:0"))
    assert tok.tolist() == [0, 9, 9, 0]


@pytest.mark.parametrize("V,value", [(20000, 0.0), (9000, -3.5)])
def test_sample_long_ties(V, value):
    """More equal logits at the border than any list holds."""
    torch = _t()
    z = torch.full((3, V), value)
    z[1, 100] = value + 1
    z[2, ::3] = value - 0.25
    for u in (0.0, 0.123, 0.77, 0.9999):
        for kw in (dict(top_p=0.5), dict(top_k=6000), dict(top_k=6000, top_p=0.75), dict(top_p=0.9, min_p=0.9), dict(min_p=0.5)):
            log(f"[sample ties] V={V} u={u} {kw}")
            _check_sample(z.cuda(), torch.full((3,), u, device="cuda:0"), kw)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_logits_on_an_even_grid(dtype):
    """Logits whose distances from the largest are whole and half multiples of
    T/64, and their fp32 neighbours; rows long enough for every path."""
    torch = _t()
    g = torch.Generator().manual_seed(5)
    V = 40000
    z = torch.stack([torch.randint(-n, n, (V,), generator=g).float() / 128 for n in (60, 400, 1500, 3000)])
    if dtype == "float32":
        near = torch.randint(-1, 2, z.shape, generator=g)
        z = torch.where(near > 0, torch.nextafter(z, torch.full_like(z, 99.0)),
                        torch.where(near < 0, torch.nextafter(z, torch.full_like(z, -99.0)), z))
    z = z.to(getattr(torch, dtype)).cuda()
    for kw in (dict(), dict(top_p=0.3), dict(top_p=0.9), dict(min_p=0.2), dict(top_p=0.95, min_p=0.01), dict(temperature=0.5, top_p=0.8),
               dict(temperature=2.0, min_p=0.5), dict(top_k=300), dict(top_k=9000, top_p=0.5)):
        log(f"[sample grid] {dtype} {kw}")
        _check_sample(z, torch.rand(4, generator=g).cuda(), kw)


def test_sample_infinities_in_long_rows():
    torch = _t()
    V = 30000
    z = torch.randn(4, V, generator=torch.Generator().manual_seed(8))
    z[0, 77::1000] = float("inf")
    z[1] = torch.finfo(torch.float32).min
    z[1, 500:9000] = torch.linspace(-3, 3, 8500)
    z[2, 20000:] = float("nan")
    z[3, :29999] = -float("inf")
    z = z.cuda()
    for u in (0.0, 0.4, 0.95):
        for kw in (dict(), dict(top_k=2), dict(top_k=5000), dict(top_p=0.3), dict(top_p=0.9, min_p=0.1), dict(top_k=7000, top_p=0.6)):
            log(f"[sample inf] u={u} {kw}")
            _check_sample(z, torch.full((4,), u, device="cuda:0"), kw)


def test_sample_per_row_parameters_and_large_rows():
    torch = _t()
    g = torch.Generator().manual_seed(77)
    R, V = 12, 201088
    z = (torch.randn(R, V, generator=g) * torch.linspace(0.5, 4, R)[:, None]).cuda()
    u = torch.rand(R, generator=g).cuda()
    kw = dict(temperature=[1.0, 0.0, 0.7, 1.3, 1.0, -2.0, 2.0, 1.0, 0.5, 1.0, 0.9, 1.0],
              top_k=[0, 5, 50, 0, 100, 9, -3, 300000, 1, 20000, 0, 0],
              top_p=[1.0, 0.5, 0.9, 0.95, 0.99, 0.4, 1.5, 0.8, 0.9, 0.7, 0.0, 0.95],
              min_p=[0.0, 0.1, 0.0, 0.02, 0.0, 0.3, -1.0, 0.0, 0.5, 0.0, 0.1, 1e-7])
    # what the values outside the ranges mean
    want = dict(kw, temperature=[max(t, 0.0) for t in kw["temperature"]],
                top_k=[k if 0 < k < V else 0 for k in kw["top_k"]], top_p=[min(max(p, 1e-300), 1.0) for p in kw["top_p"]],
                min_p=[max(p, 0.0) for p in kw["min_p"]])
    import chunked_top_kl_lm_amd as kd
    tok, lp = kd.sample(z, u, **{k: torch.tensor(v, device="cuda:0") for k, v in kw.items()})
    zn, un = z.double().cpu().numpy(), u.double().cpu().numpy()
    for r in range(R):
        t, p = o.sample(zn[r], un[r], **{k: v[r] for k, v in want.items()})
        assert int(tok[r]) == t and abs(float(lp[r]) - p) <= U * abs(p) + 1e-9, r


def test_sample_follows_the_distribution():
    """Over an even grid of u each id is drawn as often as its probability
    says, to one draw per border."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    n, V = 4096, 11
    z = torch.randn(V, generator=torch.Generator().manual_seed(1))
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    tok, _ = kd.sample(z.cuda().expand(n, V).contiguous(), u.cuda())
    count = np.bincount(tok.cpu().numpy(), minlength=V)
    assert (np.abs(count - n * torch.softmax(z.double(), 0).numpy()) <= 1.0 + 1e-6).all()


def _loop_inputs(seed):
    torch = _t()
    x = make_inputs(config_for(3, T=96, d=192, V=3000, K=10), seed=seed)
    t = to_device(x)
    g = torch.Generator().manual_seed(seed)
    feat = (torch.randn(96, 192, generator=g) * 2).to(torch.bfloat16).cuda()
    w, b = (1 + 0.1 * torch.randn(192, generator=g)).cuda(), (0.1 * torch.randn(192, generator=g)).cuda()
    return x, t, feat, w, b, torch.rand(96, generator=g).cuda()


@pytest.mark.parametrize("ckpt", [None, "int8"])
def test_together_training_step(ckpt):
    """Final norm, loss and both backward passes as one autograd graph,
    against the oracle's chain."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x, t, feat, w, b, _ = _loop_inputs(4)
    feat, w, b, W = (v.clone().requires_grad_() for v in (feat, w, b, t["W"]))
    h = kd.layer_norm(feat, w, b, EPS, checkpoint=ckpt)
    loss = kd.kd_topk_kl_loss(h, W, t["teacher_idx"], t["teacher_logit"], t["mask"], tau=1.0, chunk=64, checkpoint=ckpt)
    loss.backward()
    hr, rm, rr = o.layer_norm(_np(feat), _np(w), _np(b), EPS)
    r = fused_kl(hr, _np(W), x["teacher_idx"], x["teacher_logit"], x["mask"], 1.0)
    rdx, rdw, rdb = o.layer_norm_grads(r["grad_hidden"], _np(feat), _np(w), rm, rr)
    e = [rel(float(loss.detach()), r["loss"]), rel_f(_np(W.grad), r["grad_W"]), rel_f(_np(feat.grad), rdx), rel_f(_np(w.grad), rdw),
         rel_f(_np(b.grad), rdb)]
    log(f"[together] {ckpt}: loss {e[0]:.1e} dW {e[1]:.1e} dx {e[2]:.1e} dw {e[3]:.1e} db {e[4]:.1e}")
    # h and the gradients between the calls are bf16 (2^-8 each, three of
    # them); with checkpoints the 8-bit bound of test_loss_backward_from_8_bits
    assert e[0] <= 1e-3 and max(e[1:]) <= (2e-2 if ckpt is None else 5e-2)


def test_together_rollout():
    """Norm, head logits and sampling of a batch, and the cache builder's ids
    of the same head: greedy sampling takes the cache's first id."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    _, t, feat, w, b, u = _loop_inputs(6)
    for T in (1, 7, 96):
        h = kd.layer_norm_fwd(feat[:T], w, b, EPS)[0]
        z = kd.head_logits(h, t["W"])
        _check_sample(z, u[:T], dict(temperature=0.9, top_k=20, top_p=0.95))
        ids, logit = kd.topk_cache(h, t["W"], K=10, chunk=64)
        # the two products sum in other orders: d roundings of order-one terms
        top = z.gather(1, ids.long())
        assert (top - logit).abs().max().item() <= 192 * U * (_np(h.float().abs()) @ _np(t["W"].float().abs()).T).max()
        greedy = kd.sample(z, u[:T], temperature=0.0)[0]
        assert torch.equal(greedy.long(), z.argmax(1))
        one = kd.sample(z, u[:T], top_k=1)[0]
        assert torch.equal(one, greedy)


def test_together_captured_and_on_another_stream():
    """A decoding step and a norm's training step captured into graphs,
    replayed on new inputs with eager work between, and the same calls on a
    side stream: the eager results, bit for bit."""
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    _, t, feat, w, b, u = _loop_inputs(8)
    dy = torch.randn(96, 192, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()

    def step(f, uu):
        h, mean, rstd, q, s = kd.layer_norm_fwd(f, w, b, EPS, checkpoint="int8")
        grads = kd.layer_norm_bwd(dy, (q, s), w, mean, rstd)
        z = kd.head_logits(h, t["W"])
        few = kd.head_logits(h[:5], t["W"])
        return (h, *grads, z, few, *kd.sample(z, uu, 0.8, 50, 0.9, 0.01), *kd.sample(z, uu, top_p=0.9), kd.act8_dequantize(q, s))

    f, uu = feat.clone(), u.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = step(f, uu)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = step(f, uu)
    for a, c in zip(warm, eager):
        assert torch.equal(a, c)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(f, uu))
        graphs.append(g)
    for i in range(4):
        f.copy_(torch.roll(feat, i, 0))
        uu.copy_(torch.roll(u, 2 * i))
        want = [v.clone() for v in step(f, uu)]
        torch.cuda.synchronize()
        for g, out in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            for a, c in zip(out, want):
                assert torch.equal(a, c), i


def test_refusals_on_device_tensors():
    import chunked_top_kl_lm_amd as kd
    torch = _t()
    x, w = torch.zeros(4, 8, device="cuda:0"), torch.ones(8, device="cuda:0")
    u = torch.zeros(4, device="cuda:0")
    q, s = kd.act8_quantize(x)
    for call, err in [
        (lambda: kd.act8_quantize(x.half()), TypeError), (lambda: kd.act8_quantize(x.t()), ValueError),
        (lambda: kd.act8_quantize(x[0]), ValueError), (lambda: kd.act8_quantize(x[:0]), kd.KdError),
        (lambda: kd.act8_quantize(x[:1].expand(4, 8)), ValueError),
        (lambda: kd.act8_dequantize(q, s[:2]), ValueError), (lambda: kd.act8_dequantize(q, s, torch.float16), TypeError),
        (lambda: kd.layer_norm_fwd(x, w[:4]), ValueError), (lambda: kd.layer_norm_fwd(x, w.bfloat16()), TypeError),
        (lambda: kd.layer_norm_fwd(x, w.cpu()), ValueError), (lambda: kd.layer_norm_fwd(x, w, eps=-1.0), kd.KdError),
        (lambda: kd.layer_norm_fwd(x, w, checkpoint="fp8"), ValueError), (lambda: kd.layer_norm(x[:, :0], w[:0]), kd.KdError),
        (lambda: kd.layer_norm_bwd(x, x.bfloat16(), w, u, u), TypeError), (lambda: kd.layer_norm_bwd(x, (q,), w, u, u), ValueError),
        (lambda: kd.layer_norm_bwd(x, x, w, u[:3], u), ValueError),
        (lambda: kd.layer_norm_bwd(x, x, w, u, u, need_dx=False, need_dweight=False), kd.KdError),
        (lambda: kd.head_logits(x, x.bfloat16()), TypeError), (lambda: kd.head_logits(x, torch.zeros(9, 7, device="cuda:0")), ValueError),
        (lambda: kd.head_logits(x, x, out=torch.zeros(4, 5, device="cuda:0")), ValueError),
        (lambda: kd.sample(x, u[:3]), ValueError), (lambda: kd.sample(x, u.half()), ValueError),
        (lambda: kd.sample(x.t(), torch.zeros(8, device="cuda:0")), ValueError), (lambda: kd.sample(x, u, temperature=-1), kd.KdError),
        (lambda: kd.sample(x, u, top_p=0.0), kd.KdError), (lambda: kd.sample(x, u, top_k=-1), kd.KdError),
        (lambda: kd.sample(x, u, min_p=2.0), kd.KdError), (lambda: kd.sample(x, u, top_k=u), TypeError),
        (lambda: kd.sample(x, u, top_p=u[:2]), ValueError), (lambda: kd.sample(x, u, top_p=u.cpu()), ValueError),
        (lambda: kd.sample(x, u, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda:0")), kd.KdError),
    ]:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
