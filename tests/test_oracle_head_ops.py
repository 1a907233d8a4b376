"""The oracle of the operators around the head, pinned by other means: finite
differences and float64 autograd for layer norm, bounds and special blocks for
8-bit checkpoints, brute force in plain Python for sampling."""
import math
import random

import numpy as np
import pytest

from oracle import head_ops as o


@pytest.mark.parametrize("d", [1, 2, 7, 64])
def test_layer_norm_against_autograd_and_differences(d):
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(d)
    x, w, b, dy = r.normal(size=(5, d)), r.normal(size=d), r.normal(size=d), r.normal(size=(5, d))
    y, mean, rstd = o.layer_norm(x, w, b, 1e-3)
    tx, tw, tb = (torch.tensor(a, requires_grad=True) for a in (x, w, b))
    ty = torch.nn.functional.layer_norm(tx, (d,), tw, tb, 1e-3)
    ty.backward(torch.tensor(dy))
    assert np.allclose(y, ty.detach().numpy(), atol=1e-12)
    dx, dw, db = o.layer_norm_grads(dy, x, w, mean, rstd)
    for a, t in ((dx, tx), (dw, tw), (db, tb)):
        assert np.allclose(a, t.grad.numpy(), atol=1e-10)
    h = 1e-5
    for i in range(d):
        e = np.zeros_like(x)
        e[2, i] = h
        num = ((o.layer_norm(x + e, w, b, 1e-3)[0] - o.layer_norm(x - e, w, b, 1e-3)[0]) * dy).sum() / (2 * h)
        assert abs(num - dx[2, i]) <= 1e-6 * max(1.0, abs(num))


@pytest.mark.parametrize("d", [1, 127, 128, 129, 300])
def test_act8_is_within_half_a_step(d):
    r = np.random.default_rng(d)
    x = (r.normal(size=(6, d)) * np.exp(r.normal(size=(6, 1)) * 5)).astype(np.float32)
    x[1] = 0
    x[2] = np.float32(1e-44)                       # subnormal: kept within the scale's floor
    q, s = o.act8(x)
    v = o.act8_values(q, s)
    amax = np.repeat([[np.abs(x[t, j:j + 128]).max() for j in range(0, d, 128)] for t in range(6)], 128, axis=1)[:, :d]
    # half a step of amax / 127, a few single-precision roundings of it, and half the floor
    assert (np.abs(v - x) <= amax / 254 * (1 + 2.0 ** -15) + 2.0 ** -127).all()
    assert (v[1] == 0).all() and np.isfinite(v).all()
    x[3, 0], x[4, d - 1] = np.inf, np.nan
    v = o.act8_values(*o.act8(x))
    assert np.isnan(v[3, :128]).all() and np.isnan(v[4, (d - 1) // 128 * 128:]).all()
    assert np.isfinite(v[3, 128:]).all()


def _brute(z, u, t, k, p, mp):
    z = [-math.inf if math.isnan(a) else a for a in z]
    m = max(z)
    ids = sorted(range(len(z)), key=lambda i: (-z[i], i))
    if k:
        ids = ids[:k]
    w = {i: math.exp((z[i] - m) / t) if z[i] > -math.inf else 0.0 for i in ids}
    total = math.fsum(w.values())
    kept, run = [], []
    for i in ids:
        if kept and math.fsum(run) >= p * total:
            break
        kept.append(i)
        run.append(w[i])
    kept = sorted(i for i in kept if w[i] >= mp and w[i] > 0)
    mass = math.fsum(w[i] for i in kept)
    for n, i in enumerate(kept):
        if math.fsum(w[j] for j in kept[:n + 1]) > u * mass:
            return i, math.log(w[i] / mass)
    return kept[-1], math.log(w[kept[-1]] / mass)


def test_sample_against_brute_force():
    rng = random.Random(5)
    for n in range(400):
        V = rng.choice([1, 2, 5, 17])
        z = [rng.choice([rng.gauss(0, 2), round(rng.gauss(0, 1)), -math.inf, math.nan]) for _ in range(V)]
        if all(math.isnan(a) or a == -math.inf for a in z):
            assert o.sample(z, 0.5) == (-1, -math.inf)
            continue
        a = (rng.random(), rng.choice([0.5, 1.0, 2.0]), rng.choice([0, 0, 1, 3, 40]), rng.choice([1.0, 0.3, 0.9]),
             rng.choice([0.0, 0.2, 1.0]))
        got, want = o.sample(z, *a), _brute(z, *a)
        assert got[0] == want[0] and abs(got[1] - want[1]) < 1e-12, (z, a)


def test_sample_planted():
    z = [0.0, 3.0, 3.0, 1.0]
    assert o.sample(z, 0.99, temperature=0.0)[0] == 1            # lowest id of the largest
    assert o.sample(z, 0.0, top_k=2)[0] == 1 and o.sample(z, 0.5, top_k=2)[0] == 2
    assert o.sample(z, 0.9999, top_p=0.01)[0] == 1
    assert o.sample([math.inf, 0.0, math.inf], 0.5)[0] == 2
    low = float(np.finfo(np.float32).min)
    assert o.sample([low] * 4, 0.75)[0] == 3 and o.sample([low, 0.0], 0.9)[0] == 1
