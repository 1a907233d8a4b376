"""What is measured of the operators around the output head: layer norm
(forward and backward), 8-bit activation checkpoints, head logits and token
sampling; their plain forms in elementary torch operations, the framework's
calls, and their definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BLOCK = 128                    # elements of a row that share one scale of an 8-bit checkpoint
EPS = 1e-5


def listed():
    return [
        # the final norm of a toy student, fp32 end to end: launch latency
        dict(name="norm_tiny_f32", kind="norm", T=512, d=256, dtype="f32", ckpt=False),
        # one 8K sequence in bf16, the exact input kept for the backward pass
        dict(name="norm_8k_bf16", kind="norm", T=8192, d=2880, dtype="bf16", ckpt=False),
        # a packed batch whose length and width are odd, the input kept in 8 bits
        dict(name="norm_odd_bf16_int8", kind="norm", T=5003, d=1999, dtype="bf16", ckpt=True),
        # one 128K sequence: where the 8-bit checkpoint's memory counts
        dict(name="norm_128k_bf16_int8", kind="norm", T=131072, d=2880, dtype="bf16", ckpt=True),
        # a chunk of hidden states kept for the backward pass and brought back
        dict(name="act8_chunk_bf16", kind="act8", T=2048, d=2880, dtype="bf16"),
        # a 32K sequence of fp32 activations
        dict(name="act8_32k_f32", kind="act8", T=32768, d=2880, dtype="f32"),
        # one sequence answering: a single token's logits
        dict(name="logits_1", kind="logits", T=1, d=2880, V=201088, dtype="bf16"),
        # a small batch answering
        dict(name="logits_24", kind="logits", T=24, d=2880, V=128256, dtype="bf16"),
        # scoring a prompt: every position's logits
        dict(name="logits_512", kind="logits", T=512, d=2880, V=201088, dtype="bf16"),
        # one sequence answering, the usual filters
        dict(name="sample_1_topk_topp", kind="sample", R=1, V=201088, dtype="f32", temperature=0.8, top_k=50,
             top_p=0.95, min_p=0.0),
        # a batch in bf16 with min-p
        dict(name="sample_64_minp_bf16", kind="sample", R=64, V=128256, dtype="bf16", temperature=1.2, top_k=0,
             top_p=1.0, min_p=0.05),
        # a large rollout batch, nucleus alone: nuclei from a few ids to most of the vocabulary
        dict(name="sample_256_topp", kind="sample", R=256, V=201088, dtype="f32", temperature=1.0, top_k=0,
             top_p=0.95, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cap(x, most):
    return max(1, min(int(x), int(most)))


def draw(rng):
    kind = rng.choice(["norm", "norm", "act8", "logits", "sample", "sample"])
    if kind == "norm":
        dtype, d, ckpt = rng.choice(["bf16", "bf16", "f32"]), _log(rng, 64, 8192), rng.random() < 0.5
        T = _cap(_log(rng, 1, 131072), 131072 * 2880 * 2 // (SIZE[dtype] * d))
        return dict(kind=kind, T=T, d=d, dtype=dtype, ckpt=ckpt)
    if kind == "act8":
        dtype, d = rng.choice(["bf16", "f32"]), _log(rng, 64, 8192)
        return dict(kind=kind, T=_cap(_log(rng, 1, 131072), 32768 * 2880 * 4 // (SIZE[dtype] * d)), d=d, dtype=dtype)
    if kind == "logits":
        # widths of heads are multiples of 64; the tiny fp32 head among them
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = 64 * _log(rng, 4, 64)
        V = _cap(_log(rng, 4096, 201088), 201088 * 2880 // d)
        T = _cap(_log(rng, 1, 512), (512 if dtype == "bf16" else 64) * 2880 * 201088 // (d * V))
        return dict(kind=kind, T=min(T, 512), d=d, V=V, dtype=dtype)
    V, mode = _log(rng, 4096, 201088), rng.choice(["none", "k", "p", "kp", "m", "kpm"])
    return dict(kind=kind, R=_cap(_log(rng, 1, 256), 256 * 201088 // V), V=V, dtype=rng.choice(["bf16", "f32"]),
                temperature=rng.choice([1.0, round(rng.uniform(0.5, 1.5), 2)]),
                top_k=_log(rng, 1, 200) if "k" in mode else 0, top_p=round(rng.uniform(0.5, 0.99), 3) if "p" in mode else 1.0,
                min_p=round(rng.uniform(0.01, 0.2), 3) if "m" in mode else 0.0)


def work(case):
    k, e = case["kind"], SIZE[case["dtype"]]
    if k == "sample":
        n = case["R"] * case["V"]
        return {"bytes": n * e + 12 * case["R"], "flops": 4 * n}
    n = case["T"] * case["d"]
    if k == "logits":
        z = case["T"] * case["V"]
        return {"bytes": (n + case["V"] * case["d"]) * e + 4 * z, "flops": 2 * z * case["d"]}
    kept = case["T"] * (case["d"] + 4 * -(-case["d"] // BLOCK))     # an 8-bit checkpoint of the input
    if k == "act8":
        return {"bytes": 2 * n * e + 2 * kept, "flops": 6 * n}
    # forward: x in, y out; backward: dy and x (or its checkpoint) in, dx out
    saved = 2 * kept if case["ckpt"] else n * e
    return {"bytes": 4 * n * e + saved + 16 * case["d"], "flops": 24 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * (seed + 1))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, T, d, dt):
    """Residual-stream values: a width-wise scale that varies, a small mean and a few channels that stand out."""
    col = torch.exp(0.5 * _randn(g, d))
    col[torch.randint(0, d, (max(1, d // 500),), generator=g, device=DEV)] *= 20.0
    x = _randn(g, T, d)
    x.mul_(col).add_(0.1)
    return x.to(dt)


def prepare(case, seed):
    g, k, dt = _gen(seed), case["kind"], DT[case["dtype"]]
    s = dict(case)
    if k == "sample":
        # logits of rows from flat to peaked, with the ids past the tokenizer's last one masked out
        R, V = case["R"], case["V"]
        width = torch.exp(torch.rand(R, 1, generator=g, device=DEV) * math.log(4.0))
        z = _randn(g, R, V).mul_(width)
        z[:, V - V // 200:] = -math.inf
        s["logits"] = z.to(dt)
        s["u"] = torch.rand(R, generator=g, device=DEV)
        return s
    T, d = case["T"], case["d"]
    if k == "logits":
        h = _randn(g, T, d)
        s["hidden"] = (h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)).to(dt)
        s["W"] = _randn(g, case["V"], d).mul_(0.02).to(dt)
        return s
    s["x"] = _activations(g, T, d, dt)
    if k == "norm":
        s["dy"] = _randn(g, T, d).mul_(1e-3).to(dt)
        s["weight"] = (1.0 + 0.1 * _randn(g, d)).to(dt)
        s["bias"] = (0.1 * _randn(g, d)).to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantised(x):
    """(values that an 8-bit checkpoint of x [T, d] stands for, scales [T, blocks]), in 32 bits."""
    T, d = x.shape
    nb = -(-d // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - d)).view(T, nb, BLOCK)
    scale = (v.abs().amax(2) * torch.tensor(1.0 / 127.0, device=x.device, dtype=torch.float32)).clamp_min(2.0 ** -126)
    q = torch.round(v * (torch.ones_like(scale) / scale)[:, :, None]).clamp(-127.0, 127.0)
    return (q * scale[:, :, None]).view(T, nb * BLOCK)[:, :d], scale


def _plain_norm(x, dy, weight, bias, ckpt):
    v, w, b = x.float(), weight.float(), bias.float()
    mean = v.mean(1, keepdim=True)
    c = v - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    y = (c * rstd * w + b).to(x.dtype)
    xh = ((_quantised(x)[0] if ckpt else v) - mean) * rstd
    gy = dy.float()
    g = gy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return y, dx.to(x.dtype), (gy * xh).sum(0), gy.sum(0)


def _plain_sample(z, u, temperature, top_k, top_p, min_p):
    V = z.shape[1]
    v, ids = torch.sort(z.float(), dim=1, descending=True, stable=True)     # equal logits: the lower id first
    w = torch.exp((v.double() - v[:, :1].double()) / temperature)
    if 0 < top_k < V:
        w[:, top_k:] = 0.0
    if top_p < 1.0:
        c = torch.cumsum(w, 1)
        w = torch.where(c - w < top_p * c[:, -1:], w, torch.zeros_like(w))
    w = torch.where(w >= min_p, w, torch.zeros_like(w))
    by_id = torch.zeros_like(w).scatter_(1, ids, w)
    c = torch.cumsum(by_id, 1)
    token = ((c > u.double()[:, None] * c[:, -1:]) & (by_id > 0)).int().argmax(1)
    p = torch.gather(by_id, 1, token[:, None])[:, 0] / c[:, -1]
    return token.int(), torch.log(p).float()


def _plain(s):
    k = s["kind"]
    if k == "norm":
        return _plain_norm(s["x"], s["dy"], s["weight"], s["bias"], s["ckpt"])
    if k == "act8":
        x, scale = _quantised(s["x"])
        return x.to(s["x"].dtype), scale
    if k == "logits":
        return s["hidden"].float() @ s["W"].float().T
    return _plain_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _kernels(s):
    import chunked_top_kl_lm_amd as kd
    k = s["kind"]
    if k == "norm":
        if s["ckpt"]:
            y, mean, rstd, q, scale = kd.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS, checkpoint="int8")
            dx, dw, db = kd.layer_norm_bwd(s["dy"], (q, scale), s["weight"], mean, rstd)
        else:
            y, mean, rstd = kd.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS)
            dx, dw, db = kd.layer_norm_bwd(s["dy"], s["x"], s["weight"], mean, rstd)
        return y, dx, dw, db
    if k == "act8":
        q, scale = kd.act8_quantize(s["x"])
        return kd.act8_dequantize(q, scale, s["x"].dtype), scale
    if k == "logits":
        return kd.head_logits(s["hidden"], s["W"])
    return kd.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_checkpoint(x):
    """The checkpoint's scale and integers are defined by single-precision steps: taken on the host by numpy, the values they stand for in 64 bits."""
    a = x.float().cpu().numpy()
    T, d = a.shape
    out, scales = np.empty((T, d), np.float64), np.empty((T, -(-d // BLOCK)), np.float32)
    for j in range(scales.shape[1]):
        part = a[:, j * BLOCK:(j + 1) * BLOCK]
        scale = np.maximum(np.abs(part).max(1) * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126))
        whole = np.clip(np.rint(part * (np.float32(1) / scale)[:, None]), -127, 127)
        out[:, j * BLOCK:(j + 1) * BLOCK] = whole.astype(np.float64) * scale.astype(np.float64)[:, None]
        scales[:, j] = scale
    return torch.from_numpy(out).to(x.device), torch.from_numpy(scales).to(x.device)


def _exact_norm(s):
    x, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
    d = x.shape[1]
    mu = x.sum(1) / d
    rs = (torch.sum(torch.square(x - mu[:, None]), 1) / d + EPS).pow(-0.5)
    y = torch.addcmul(s["bias"].double()[None, :], (x - mu[:, None]) * rs[:, None], w[None, :])
    if s["ckpt"]:
        x = _exact_checkpoint(s["x"])[0]
    xh = (x - mu[:, None]) * rs[:, None]
    a, b = (dy @ w) / d, ((dy * xh) @ w) / d
    dx = (dy * w[None, :] - a[:, None] - xh * b[:, None]) * rs[:, None]
    one = torch.ones(1, x.shape[0], dtype=torch.float64, device=x.device)
    return y, dx, (one @ (dy * xh))[0], (one @ dy)[0]


def _exact_row(z, u, temperature, top_k, top_p, min_p):
    order = np.lexsort((np.arange(z.size), -z))
    if top_k > 0:
        order = order[:top_k]
    w = np.exp((z[order] - z[order[0]]) / temperature)
    before = np.concatenate(([0.0], np.cumsum(w)))
    n = order.size if top_p >= 1.0 else int(np.searchsorted(before[:-1], top_p * before[-1], side="left"))
    n = max(1, min(n, int(np.count_nonzero(w >= min_p)) if min_p > 0 else n))
    kept = np.argsort(order[:n], kind="stable")
    mass = np.cumsum(w[:n][kept])
    at = int(np.searchsorted(mass, u * mass[-1], side="right"))
    pick = kept[min(at, n - 1)]
    return int(order[pick]), float(np.log(w[pick] / mass[-1]))


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k == "norm":
        return _exact_norm(s)
    if k == "act8":
        return _exact_checkpoint(s["x"])
    if k == "logits":
        return s["hidden"].double() @ s["W"].double().T
    z, u = s["logits"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        rows = [_exact_row(z[r], u[r], case["temperature"], case["top_k"], case["top_p"], case["min_p"]) for r in range(case["R"])]
    return (torch.tensor([r[0] for r in rows], dtype=torch.int32, device=DEV),
            torch.tensor([r[1] for r in rows], dtype=torch.float64, device=DEV))
