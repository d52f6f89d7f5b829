"""Distillation (include/lora_distill.h) where exponents are large: logits, or their quotient by the temperature, far
beyond what a softmax meets in ordinary use, on every row and on rows between ordinary ones.

Tolerances are those of test_gpu_distill.py: a logarithm of a probability is off by 2e-5 + 2^-21 of its distance from
the row's largest (differences of bf16 numbers in fp32, one product), whatever the logits' level.  A probability, or a
gradient, below fp32's smallest normal number, 2^-126, may come out as 0 (the exponential flushes it): 1.2e-38, where
that file allows 1e-38 absolute.  So may a loss, of which fp32 holds nothing below 2^-149 and less than its 24 bits
below 2^-126: T^2 log V at a temperature of 1e-25 is 7e-50."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import api
from lora_fine_tuning_mlp_b200 import build as libbuild
from oracle import distill as ods
from test_gpu_distill import f64, make, padded, tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def check(z, values, ids, dloss, T, s, cap, loss, dz):
    z64 = f64(z)
    rl, rd, q, P = ods.run(z64, f64(values), ids.numpy().astype(np.int64), dloss, None, T, s, cap)
    tl, td = tolerances(z64, T, s, cap, dloss, q, P, rl, rd)
    td = td + 2.0 ** -126 * (1.0 + np.abs(dloss) * T * abs(s))[:, None]
    for got, ref, tol in ((loss, rl, tl + 2.0 ** -126), (dz, rd, td)):
        if got is not None:
            bad = ~(np.abs(got - ref) <= tol)
            assert not np.any(bad), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


def run_and_check(z, values, ids, dloss, T=1.0, s=1.0, cap=0.0):
    """Loss, gradient, the gradient beside the loss and the one in place, against the oracle."""
    dev, full = padded(z)
    V = z.shape[1]
    args = (dev, values.cuda(), ids.cuda())
    up = torch.from_numpy(dloss).cuda()
    kw = dict(temperature=T, logit_scale=s, softcap=cap)
    T, s, cap = (float(np.float32(x)) for x in (T, s, cap))
    loss, dz = api.distill_forward(*args, **kw), api.distill_backward(*args, up, **kw)
    check(z, values, ids, dloss, T, s, cap, f64(loss), f64(dz))
    _, dr = api.distill_loss(*args, reduction="sum", **kw)
    check(z, values, ids, np.ones(len(dloss)), T, s, cap, None, f64(dr))
    api.distill_backward(*args, up, inplace=True, **kw)
    assert torch.equal(dev, dz) and torch.all(full[:, V:] == 7.0)
    assert api.step_device_status() == 0


def levels(rng, z, ids, level, s):
    """Rows of five kinds in turn: all logits at `level`; some of them at it, the others twice that far below; ordinary
    ones; one logit of `level` among ordinary ones, no teacher's entry; ordinary ones."""
    N, V = z.shape
    at = level / s
    kind = torch.arange(N) % 5
    z[kind == 0] = at
    part = torch.from_numpy(rng.random((N, V)) < 0.01)
    part[torch.arange(N), ids[:, 0]] = True
    z[(kind == 1)[:, None] & part] = at
    z[(kind == 1)[:, None] & ~part] = (level - 2 * abs(level)) / s
    free = torch.tensor([next(j for j in range(V) if j not in set(r.tolist())) for r in ids])
    rows = torch.nonzero(kind == 3)[:, 0]
    z[rows, free[rows]] = at
    return z


SIZES = [(40, 1003), (700, 9000), (60, 40003), (1500, 777)]


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("s", [1.0, -0.5])
@pytest.mark.parametrize("level", [1e3, -1e3, 1e5, -1e5, 1e6, -1e6, 1e9, -1e9, 1e11, -1e11, 1e20, -1e20])
def test_levels(N, V, s, level):
    rng = np.random.default_rng(V)
    z, values, ids = make(rng, N, V, 6)
    z = levels(rng, z, ids, level, s)
    run_and_check(z, values, ids, rng.uniform(0.5, 1.5, N).astype(np.float32), s=s)


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("level", [1e5, 1e6])
def test_spread_around_a_level(N, V, level):
    """bf16 numbers near a level lie 512 (4096) apart: a few different ones, many times each."""
    rng = np.random.default_rng(V + 1)
    z, values, ids = make(rng, N, V, 6)
    z[::2] = torch.from_numpy(level * (1.0 + rng.integers(0, 4, z[::2].shape) * 2.0 ** -7)).to(z.dtype)
    run_and_check(z, values, ids, rng.uniform(-1.5, 1.5, N).astype(np.float32))


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("T", [0.02, 1e-4, 1e-6, 1e-12, 1e-25])
def test_small_temperatures(N, V, T):
    rng = np.random.default_rng(V + 2)
    z, values, ids = make(rng, N, V, 6)
    z[::3] += 8.0
    z[1::3] = 8.0
    run_and_check(z, values, ids, rng.uniform(0.5, 1.5, N).astype(np.float32), T=T)


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("level", [1e5, -1e5])
@pytest.mark.parametrize("cap,T", [(1e5, 1.0), (30.0, 3e-4)])
def test_softcap_far_above_the_temperature(N, V, level, cap, T):
    rng = np.random.default_rng(V + 3)
    z, values, ids = make(rng, N, V, 6, 10.0)
    z = levels(rng, z, ids, level, 1.0)
    run_and_check(z, values, ids, rng.uniform(0.5, 1.5, N).astype(np.float32), T=T, cap=cap)


def test_all_of_a_cluster_at_a_masks_value():
    """Every row wholly at a usual mask value: a uniform softmax, row after row."""
    rng = np.random.default_rng(9)
    N, V = 900, 1000
    z, values, ids = make(rng, N, V, 4)
    z[:] = -1e9
    run_and_check(z, values, ids, np.full(N, 0.5, dtype=np.float32))
    dz = api.distill_backward(padded(z)[0], values.cuda(), ids.cuda(), torch.full((N,), 0.5, device="cuda"))
    assert float(dz.float().max()) <= 0.5 / V * (1 + 2.0 ** -7)


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("s,T", [(1.0, 1.0), (-0.5, 2.0)])
def test_softcap_slope_far_from_zero(N, V, s, T):
    """dt/dz where tanh is near -1 or 1, down to 10^-8, at the teacher's entries and others.

    Tolerance, relative to the slope itself: 2^-8 of the result for its rounding, 2^-17 for the slope's (an exponent of
    at most 30 off by 2^-23 of it, 2.5e-6, twice), and the probabilities' d of test_gpu_distill.py."""
    rng = np.random.default_rng(V + 4)
    cap = 30.0
    z, values, ids = make(rng, N, V, 6, 10.0, abs(s))
    z[::2] = torch.from_numpy(rng.uniform(-300.0, 300.0, z[::2].shape)).to(z.dtype) / abs(s)
    dev, _ = padded(z)
    dloss = rng.uniform(0.5, 1.5, N).astype(np.float32)
    kw = dict(temperature=T, logit_scale=s, softcap=cap)
    dz = f64(api.distill_backward(dev, values.cuda(), ids.cuda(), torch.from_numpy(dloss).cuda(), **kw))
    z64 = f64(z)
    rl, rd, q, P = ods.run(z64, f64(values), ids.numpy().astype(np.int64), dloss, None, T, s, cap)
    x = cap * np.tanh(s * z64 / cap) / T
    d = 2e-5 + 2.0 ** -21 * (x.max(axis=1, keepdims=True) - x) + 2.0 ** -19 * cap / T
    slope = abs(s) / np.cosh(s * z64 / cap) ** 2
    tol = (2.0 ** -8 + 2.0 ** -17) * np.abs(rd) + (T * dloss)[:, None] * slope * (q + P) * d + 2.0 ** -126
    bad = ~(np.abs(dz - rd) <= tol)
    assert not np.any(bad), (np.argwhere(bad)[:4], dz[bad][:4], rd[bad][:4], tol[bad][:4])


WIDE = [(1e3, 1.0), (1e5, 1.0), (1e7, 1.0), (1e30, 1.0), (30.0, 0.01), (130.0, 1.0), (50.0, 0.3)]


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("s", [1.0, -0.25])
@pytest.mark.parametrize("cap,T", WIDE)
def test_caps_far_above_the_temperature_cost_no_precision(N, V, s, cap, T):
    """Ordinary logits, and some near the cap, under caps of more than 128 temperatures.

    t = cap tanh(s z / cap) is off by 2^-21 of itself (the quotient 2^-23, tanh 2^-22 by its two units in the last place,
    the product 2^-24), so a logarithm of a probability by 2^-20 of the row's largest |t| / T beside the d of
    test_gpu_distill.py without softcapping; nothing grows with the cap.  dt/dz as in the test before."""
    rng = np.random.default_rng(V + 5)
    z, values, ids = make(rng, N, V, 6, 2.0, abs(s))
    z[::4] *= 5.0
    if cap < 1e20:
        z[1::4] = torch.from_numpy(rng.uniform(-3.0 * cap, 3.0 * cap, z[1::4].shape)).to(z.dtype) / abs(s)
    dev, _ = padded(z)
    dloss = rng.uniform(0.5, 1.5, N).astype(np.float32)
    kw = dict(temperature=T, logit_scale=s, softcap=cap)
    args = (dev, values.cuda(), ids.cuda())
    loss = f64(api.distill_forward(*args, **kw))
    dz = f64(api.distill_backward(*args, torch.from_numpy(dloss).cuda(), **kw))
    z64 = f64(z)
    cap, T = float(np.float32(cap)), float(np.float32(T))
    rl, rd, q, P = ods.run(z64, f64(values), ids.numpy().astype(np.int64), dloss, None, T, s, cap)
    x = cap * np.tanh(s * z64 / cap) / T
    span = x.max(axis=1, keepdims=True) - x
    d = 2e-5 + 2.0 ** -21 * span + 2.0 ** -20 * np.abs(x).max(axis=1, keepdims=True)
    row = T * T * (np.max(d * (P > 0), axis=1) + 2.0 ** -20 * (np.max(span * (P > 0), axis=1) + 20.0))
    slope = abs(s) / np.cosh(s * z64 / cap) ** 2
    el = (2.0 ** -8 + 2.0 ** -17) * np.abs(rd) + (T * dloss)[:, None] * slope * (q + P) * d + 2.0 ** -126
    for got, ref, tol in ((loss, rl, row), (dz, rd, el)):
        bad = ~(np.abs(got - ref) <= tol)
        assert not np.any(bad), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])
    _, dr = api.distill_loss(*args, reduction="sum", **kw)
    unit = ods.run(z64, f64(values), ids.numpy().astype(np.int64), np.ones(N), None, T, s, cap)[1]
    assert np.all(np.abs(f64(dr) - unit) <= el / dloss[:, None] + 2.0 ** -126)
    assert api.step_device_status() == 0
