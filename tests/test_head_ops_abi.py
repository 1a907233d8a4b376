"""C ABI of the operators around the head (include/kd_head_ops.h): exports,
workspace sizes and the refusal of bad arguments on the host, before anything
touches a GPU; and the binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

import chunked_top_kl_lm_amd as kd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000        # a pointer that no refused call follows
NAN, INF = float("nan"), float("inf")


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kd_head_ops.h")).read(), flags=re.S)


def test_library_exports_the_header():
    names = re.findall(r"^[A-Za-z_][\w\s\*]*?\b(kd_\w+)\s*\(", _header(), flags=re.M)
    assert len(names) == len(set(names)) == 11
    for n in names:
        fn = getattr(kd.lib(), n)
        assert fn.argtypes, n
        proto = re.search(r"\b%s\s*\((.*?)\)" % n, _header(), flags=re.S).group(1)
        assert len(fn.argtypes) == len(proto.split(",")), n


def test_header_constants_match_the_binding():
    h = open(os.path.join(ROOT, "include", "kd_head_ops.h")).read()
    assert int(re.search(r"#define KD_ACT8_BLOCK (\d+)", h).group(1)) == kd.ACT8_BLOCK
    assert kd.STATUS[int(re.search(r"#define KD_ERR_BAD_PARAM (\d+)", h).group(1))] == "KD_ERR_BAD_PARAM"
    assert kd.status_str(10) != "unknown status"


def _run(name, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(kd.lib(), name)(*a.values())


QUANT = dict(x=P, ldx=64, dt=0, T=4, d=64, q=P, scale=P, st=None)
DEQUANT = dict(q=P, scale=P, dt=0, T=4, d=64, out=P, st=None)
FWD = dict(x=P, ldx=64, dt=0, w=P, b=P, wdt=0, T=4, d=64, eps=1e-5, y=P, mean=P, rstd=P, q=None, scale=None, st=None)
BWD = dict(dy=P, x=P, ldx=64, q=None, scale=None, dt=0, w=P, wdt=0, T=4, d=64, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P,
           wsb=1 << 30, st=None)
LOGITS = dict(h=P, ldh=64, W=P, dt=0, T=4, d=64, V=1000, z=P, ws=None, wsb=0, st=None)
SAMPLE = dict(z=P, ldz=100, dt=1, R=2, V=100, u=P, f64=0, t=1.0, k=0, p=1.0, m=0.0, tr=None, kr=None, pr=None, mr=None,
              tok=P, lp=P, ws=P, wsb=1 << 30, st=None)
ACT8_BWD = dict(q=P, scale=P, W=P, dt=0, idx=P, logit=P, mask=None, T=64, d=64, V=1000, K=10, tau=1.0, chunk=32, rl=P,
                gl=None, gH=P, ghdt=1, gW=P, acc=0, gWb=None, ws=P, wsb=1 << 40, status=None, st=None)


@pytest.mark.parametrize("name,base,kw,code", [
    ("kd_act8_quantize", QUANT, k, c) for k, c in
    [(dict(x=None), 1), (dict(q=None), 1), (dict(scale=None), 1), (dict(dt=2), 5), (dict(T=0), 2), (dict(d=0), 2),
     (dict(ldx=63), 2), (dict(T=(1 << 24) + 1), 2), (dict(d=(1 << 24) + 1, ldx=1 << 25), 2), (dict(x=P + 1), 2),
     (dict(scale=P + 2), 2)]
] + [
    ("kd_act8_dequantize", DEQUANT, k, c) for k, c in
    [(dict(q=None), 1), (dict(scale=None), 1), (dict(out=None), 1), (dict(dt=-1), 5), (dict(T=0), 2), (dict(d=-3), 2),
     (dict(dt=1, out=P + 2), 2)]
] + [
    ("kd_layer_norm_fwd", FWD, k, c) for k, c in
    [(dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
     (dict(q=P), 1), (dict(scale=P), 1), (dict(dt=3), 5), (dict(dt=1, wdt=0), 5), (dict(wdt=7), 5), (dict(T=0), 2),
     (dict(d=0), 2), (dict(d=32769, ldx=32769), 2), (dict(ldx=10), 2), (dict(eps=-1e-9), 10), (dict(eps=NAN), 10),
     (dict(eps=INF), 10), (dict(x=P + 1), 2), (dict(mean=P + 2), 2), (dict(wdt=1, w=P + 2), 2)]
] + [
    ("kd_layer_norm_bwd", BWD, k, c) for k, c in
    [(dict(dy=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
     (dict(q=P, scale=P), 1), (dict(x=None, q=P), 1), (dict(dx=None, dw=None, db=None), 1), (dict(dt=9), 5),
     (dict(T=0), 2), (dict(d=40000, ldx=40000), 2), (dict(ldx=3), 2), (dict(ws=None), 6), (dict(wsb=100), 6),
     (dict(ws=P + 64), 6), (dict(dy=P + 1), 2), (dict(dw=P + 2), 2)]
] + [
    ("kd_head_logits", LOGITS, k, c) for k, c in
    [(dict(h=None), 1), (dict(W=None), 1), (dict(z=None), 1), (dict(dt=4), 5), (dict(T=0), 2), (dict(d=0), 2),
     (dict(V=0), 2), (dict(V=(1 << 24) + 1), 2), (dict(ldh=8), 2), (dict(h=P + 1), 2), (dict(z=P + 2), 2),
     (dict(T=65, d=63), 6), (dict(T=65, d=63, ws=P + 16, wsb=1 << 30), 6), (dict(T=65, h=P + 2), 6), (dict(T=65, W=P + 4), 2)]
] + [
    ("kd_sample", SAMPLE, k, c) for k, c in
    [(dict(z=None), 1), (dict(u=None), 1), (dict(tok=None), 1), (dict(dt=2), 5), (dict(R=0), 2), (dict(V=0), 2),
     (dict(V=(1 << 24) + 1, ldz=1 << 25), 2), (dict(R=(1 << 21) + 1), 2), (dict(R=1 << 17, V=1 << 20, ldz=1 << 20), 2),
     (dict(ldz=99), 2), (dict(t=-1.0), 10), (dict(t=NAN), 10), (dict(t=INF), 10), (dict(k=-1), 10), (dict(p=0.0), 10),
     (dict(p=1.5), 10), (dict(p=NAN), 10), (dict(m=-0.1), 10), (dict(m=1.01), 10), (dict(m=NAN), 10), (dict(ws=None), 6),
     (dict(wsb=10), 6), (dict(ws=P + 8), 6), (dict(z=P + 2), 2), (dict(f64=1, u=P + 4), 2), (dict(tr=P + 4), 2)]
] + [
    ("kd_topk_kl_bwd_act8", ACT8_BWD, k, c) for k, c in
    [(dict(q=None), 1), (dict(scale=None), 1), (dict(W=None), 1), (dict(rl=None), 1), (dict(gH=None, gW=None), 1),
     (dict(T=0), 2), (dict(tau=0.0), 3), (dict(chunk=0), 4), (dict(dt=3), 5), (dict(wsb=1000), 6)]
])
def test_host_argument_errors(name, base, kw, code):
    assert _run(name, base, kw) == code


def test_workspace_sizes():
    L = kd.lib()
    assert L.kd_layer_norm_bwd_workspace_bytes(0, 8) == 0 and L.kd_layer_norm_bwd_workspace_bytes(8, 32769) == 0
    # partial rows: bounded however many rows there are, one at least
    assert L.kd_layer_norm_bwd_workspace_bytes(1, 2880) == 2880 * 8
    a, b = L.kd_layer_norm_bwd_workspace_bytes(1 << 20, 2880), L.kd_layer_norm_bwd_workspace_bytes(1 << 24, 2880)
    assert a == b and a % 256 == 0
    assert kd.sample_workspace_bytes(0, 5) == 0 and kd.sample_workspace_bytes(5, 0) == 0
    assert kd.sample_workspace_bytes(1, 1) == 4 * 256
    assert kd.sample_workspace_bytes(256, 201088) < 256 * 201088 * 4 // 3          # a third of fp32 logits
    assert kd.head_logits_workspace_bytes(64, 63, 1000, 0) == 0            # few rows: none
    assert kd.head_logits_workspace_bytes(512, 63, 1000, 0) == 1000 * 64 * 2 + 512 * 64 * 2
    assert kd.head_logits_workspace_bytes(512, 64, 0, 0) == 0
    shape = (512, 64, 1000, 10, 128, 0)
    # the chunk's rows brought back, where the width alone needs no padded copy
    assert L.kd_topk_kl_bwd_act8_workspace_bytes(*shape) == kd.bwd_workspace_bytes(*shape) + 256 * 64 * 2
    assert L.kd_topk_kl_bwd_act8_workspace_bytes(0, 8, 8, 1, 1, 0) == 0


def test_binding_refuses_host_tensors_and_bad_kinds():
    x, w = torch.zeros(4, 8), torch.ones(8)
    for call in (lambda: kd.act8_quantize(x), lambda: kd.layer_norm_fwd(x, w), lambda: kd.layer_norm(x, w),
                 lambda: kd.layer_norm_bwd(x, x, w, w, w), lambda: kd.head_logits(x, x),
                 lambda: kd.sample(x, torch.zeros(4)),
                 lambda: kd.act8_dequantize(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="checkpoint"):
        kd.kd_topk_kl_loss(x, x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), checkpoint="int4")


def test_names_are_public():
    for n in ("layer_norm", "layer_norm_fwd", "layer_norm_bwd", "act8_quantize", "act8_dequantize", "head_logits", "sample",
              "KdLayerNormFunction"):
        assert n in kd.__all__ and getattr(kd, n)
