"""GPU parity of distillation from a teacher's top logits
(include/lora_distill.h) against the fp64 oracle.

Tolerances, from the arithmetic: a log-probability x - lse is off by
d = 2e-5 + 2^-21 |x - max| (fp32 sums of up to 2^18 exponentials with a
relative error of 2^-21 each; the difference rounded and scaled) and, with
softcapping, by 2^-19 cap / T (t = cap - 2 cap r with r within 2^-21).  A row's
loss is within T^2 d plus 2^-20 of its terms' magnitudes.  A gradient element
is rounded to bf16 (2^-8 |ref|) after an error of d (q + p), and with
softcapping 2^-18 (q + p) from 1 - (t / cap)^2, times dloss T |s|."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild
from oracle import distill as ods

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
IGN = -100
LOWEST = float(torch.finfo(torch.bfloat16).min)


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def f64(t):
    return t.detach().double().cpu().numpy()


def padded(z, ld=None):
    """Logits on the device in rows of ld elements (V rounded up to 8), canaries behind V."""
    N, V = z.shape
    full = torch.full((N, (V + 7) // 8 * 8 if ld is None else ld), 7.0, dtype=BF16, device="cuda")
    full[:, :V] = z.cuda()
    return full[:, :V], full


def make(rng, N, V, K, std=2.0, scale=1.0):
    z = torch.from_numpy((rng.standard_normal((N, V)) * std / scale).astype(np.float32)).to(BF16)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)])
    values = np.sort(rng.standard_normal((N, K)) * 2.0 + 6.0, axis=1)[:, ::-1].copy()
    return z, torch.from_numpy(values).float(), torch.from_numpy(ids)


def tolerances(z, T, s, cap, dloss, q, P, loss, dz):
    x = s * z
    if cap > 0:
        x = cap * np.tanh(x / cap)
    x = np.where(np.isfinite(x), x, 0.0) / T
    span = np.abs(x - x.max(axis=1, keepdims=True))
    d = 2e-5 + 2.0 ** -21 * span + (2.0 ** -19 * cap / T if cap > 0 else 0.0)
    row = T * T * np.max(d * (P > 0), axis=1) + 2.0 ** -20 * T * T * (np.max(span * (P > 0), axis=1) + 20.0)
    el = 2.0 ** -8 * np.abs(dz) + (np.abs(dloss) * T * abs(s))[:, None] * (q + P) * (d + (2.0 ** -18 if cap else 0.0))
    return row, el + 1e-38


def check(z, values, ids, labels, dloss, T, s, cap, loss, dz):
    z64, v64, i64 = f64(z), f64(values), ids.cpu().numpy().astype(np.int64)
    lab = None if labels is None else labels.cpu().numpy()
    rl, rd, q, P = ods.run(z64, v64, i64, dloss, lab, T, s, cap, IGN)
    tl, td = tolerances(z64, T, s, cap, np.asarray(dloss), q, P, rl, rd)
    if loss is not None:
        bad = ~(np.abs(loss - rl) <= tl)
        assert not np.any(bad), (np.argwhere(bad)[:4], loss[bad][:4], rl[bad][:4], tl[bad][:4])
    if dz is not None:
        bad = ~(np.abs(dz - rd) <= td)
        assert not np.any(bad), (np.argwhere(bad)[:4], dz[bad][:4], rd[bad][:4], td[bad][:4])
    return rl, rd


CASES = [
    # N, V, K, T, s, cap, values, ids
    (1, 1, 1, 1.0, 1.0, 0.0, F32, torch.int64),            # one logit, one entry
    (3, 7, 7, 1.0, 1.0, 0.0, F32, torch.int32),            # the whole vocabulary, less than a vector
    (5, 8, 1, 2.0, 1.0, 0.0, BF16, torch.int64),
    (37, 1003, 8, 1.0, 1.0, 0.0, F32, torch.int64),
    (20, 2051, 33, 0.5, -0.25, 0.0, BF16, torch.int32),    # a negative logit scale
    (11, 4097, 100, 3.0, 1.0, 30.0, F32, torch.int64),
    (400, 1500, 20, 1.0, 1.0, 0.0, F32, torch.int64),      # rows enough for one block each
    (3, 32776, 64, 1.0, 0.0625, 0.0, BF16, torch.int64),   # a cluster of two
    (2, 50257, 512, 2.0, -1.0, 50.0, F32, torch.int32),
    (2, 128256, 64, 2.0, 1.0, 0.0, BF16, torch.int32),
    (1, 262147, 1024, 1.0, 1.0, 30.0, F32, torch.int64),   # eight blocks, more than 64 KB each
]


@pytest.mark.parametrize("N,V,K,T,s,cap,vt,it", CASES)
def test_loss_and_gradient(N, V, K, T, s, cap, vt, it):
    rng = np.random.default_rng(N * 31 + V)
    z, values, ids = make(rng, N, V, K, 10.0 if cap else 2.0, abs(s))
    values, ids = values.to(vt).cuda(), ids.to(it).cuda()
    dloss = rng.uniform(0.5, 1.5, N).astype(np.float32)
    labels = torch.from_numpy(np.where(rng.random(N) < 0.1, IGN, 5)) if N > 1 else None
    labels = None if labels is None else labels.cuda()
    dev, full = padded(z, (V + 7) // 8 * 8 + 16)
    kw = dict(labels=labels, temperature=T, logit_scale=s, softcap=cap)
    loss = api.distill_forward(dev, values, ids, **kw)
    dz = api.distill_backward(dev, values, ids, torch.from_numpy(dloss).cuda(), **kw)
    rl, rd = check(z, values, ids, labels, dloss, T, s, cap, f64(loss), f64(dz))
    # reduced, with the gradient in the same pass
    taking = N if labels is None else int((labels != IGN).sum())
    for reduction, factor in (("sum", 1.0), ("mean", 1.0 / max(1, taking))):
        out, dr = api.distill_loss(dev, values, ids, reduction=reduction, **kw)
        assert abs(float(out[1]) - factor) <= 2.0 ** -24 * factor
        assert abs(float(out[0]) - factor * f64(loss).sum()) <= 2.0 ** -22 * factor * np.abs(f64(loss)).sum()
        check(z, values, ids, labels, np.full(N, float(out[1])), T, s, cap, None, f64(dr))
        # without the gradient the row is summed in another order: twice the rows' tolerance
        only, none = api.distill_loss(dev, values, ids, reduction=reduction, with_grad=False, **kw)
        tol = 2 * factor * tolerances(f64(z), T, s, cap, dloss, *(ods.run(
            f64(z), f64(values), f64(ids).astype(np.int64), dloss, None if labels is None else labels.cpu().numpy(),
            T, s, cap, IGN)[j] for j in (2, 3, 0, 1)))[0].sum()
        assert none is None and only[1] == out[1] and abs(float(only[0]) - float(out[0])) <= tol
    # in place: the same bits, and nothing behind the vocabulary
    api.distill_backward(dev, values, ids, torch.from_numpy(dloss).cuda(), inplace=True, **kw)
    assert torch.equal(dev, dz) and torch.all(full[:, V:] == 7.0)


def test_absent_repeated_and_empty_entries():
    rng = np.random.default_rng(3)
    N, V, K = 8, 900, 12
    z, values, ids = make(rng, N, V, K)
    ids[0, 5:] = -1                      # fewer entries
    ids[1, :] = -1                       # none
    ids[2, 1], ids[2, 7] = ids[2, 0], ids[2, 0]   # one id three times
    values[3, :] = -np.inf               # nothing left by the teacher's mask
    values[4, 2:] = -np.inf              # two left
    values[5, :] = torch.finfo(torch.float32).min
    ids[6, ::2] = -1                     # gaps
    ids[7, 3:] = ids[7, 2]
    dloss = np.ones(N, dtype=np.float32)
    dev, _ = padded(z)
    args = (dev, values.cuda(), ids.cuda())
    loss, dz = api.distill_forward(*args), api.distill_backward(*args, torch.ones(N, device="cuda"))
    check(z, values, ids, None, dloss, 1.0, 1.0, 0.0, f64(loss), f64(dz))
    assert loss[1] == 0 and loss[3] == 0 and torch.all(dz[[1, 3]] == 0)
    assert api.step_device_status() == 0


def test_masked_and_extreme_students():
    rng = np.random.default_rng(4)
    N, V, K = 7, 3001, 5
    z, values, ids = make(rng, N, V, K)
    z[0, :2000] = -float("inf")          # a masked vocabulary,
    ids[0] = torch.tensor([2000, 2500, 3000, 2001, 2999])
    z[1, :2900] = LOWEST                 # ... masked with the type's lowest value
    ids[1] = torch.tensor([2900, 2950, 3000, 2999, 2901])
    z[2, :] = LOWEST                     # nothing else left: uniform
    z[3, :] = 0.0
    z[4, 17] = 3.0e4                     # one logit takes all
    ids[4, 0], values[4, 0] = 17, 1e4
    z[5, :] = 1.0e4
    z[6, :] = -1.0e4
    dev, _ = padded(z)
    args = (dev, values.cuda(), ids.cuda())
    loss, dz = api.distill_forward(*args), api.distill_backward(*args, torch.ones(N, device="cuda"))
    z64 = f64(z)
    z64[1][z64[1] == LOWEST] = z64[2][:] = -1e30   # the same softmax, without fp64 overflow in the checks
    z64[0][np.isinf(z64[0])] = -1e30
    z64[2][:] = 0.0
    zt = torch.from_numpy(z64)
    check(zt, values, ids, None, np.ones(N), 1.0, 1.0, 0.0, f64(loss), f64(dz))
    # a teacher on a masked entry: an infinite loss in that row alone, as the formula says
    ids[0, 4] = 0
    loss = api.distill_forward(dev, values.cuda(), ids.cuda())
    assert torch.isinf(loss[0]) and torch.all(torch.isfinite(loss[1:]))
    # NaN stays in its row
    dev[3, 9] = float("nan")
    loss, dz = api.distill_forward(dev, values.cuda(), ids.cuda()), api.distill_backward(
        dev, values.cuda(), ids.cuda(), torch.ones(N, device="cuda"))
    assert torch.isnan(loss[3]) and torch.all(torch.isfinite(loss[4:])) and torch.all(torch.isfinite(dz[4:]))


@pytest.mark.parametrize("N,V,cap,s", [(700, 9000, 0.0, 1.0), (700, 9000, 0.0, -0.5), (300, 40003, 0.0, 1.0),
                                       (300, 40003, 20.0, 1.0), (2000, 777, 0.0, 1.0)])
def test_rows_of_very_different_levels_follow_one_another(N, V, cap, s):
    """A row far above or below the last, masked rows, ignored ones and rows
    without a teacher between them, many to a cluster, also in place."""
    rng = np.random.default_rng(11)
    z, values, ids = make(rng, N, V, 6)
    kind = torch.from_numpy(rng.integers(0, 8, N))
    z[kind == 1] += 1000.0
    z[kind == 2] -= 1000.0
    keep = torch.zeros(V, dtype=torch.bool)
    keep[rng.choice(V, 50, replace=False)] = True
    for k, mask in ((3, -float("inf")), (4, LOWEST)):
        # the lowest value is the lowest exponent for a positive scale
        z[torch.outer(kind == k, ~keep)] = mask if s > 0 else -mask
    kept = torch.from_numpy(np.flatnonzero(keep.numpy())[:6])
    ids[(kind == 3) | (kind == 4)] = kept
    ids[kind == 5] = -1
    labels = torch.where(kind == 6, IGN, 1).cuda()
    dloss = rng.uniform(-1.0, 1.0, N).astype(np.float32)
    dev, full = padded(z)
    kw = dict(labels=labels, softcap=cap, logit_scale=s)
    args = (dev, values.cuda(), ids.cuda())
    loss = api.distill_forward(*args, **kw)
    dz = api.distill_backward(*args, torch.from_numpy(dloss).cuda(), **kw)
    z64 = z.double()
    masked = torch.outer((kind == 3) | (kind == 4), ~keep)
    z64[masked] = -2000.0 * np.sign(s)         # the same softmax, and tanh, without fp64's infinities in the checks
    check(z64, values, ids, labels, dloss, 1.0, s, cap, f64(loss), f64(dz))
    out, dr = api.distill_loss(*args, reduction="sum", **kw)
    check(z64, values, ids, labels, np.ones(N), 1.0, s, cap, None, f64(dr))
    assert abs(float(out[0]) - f64(loss).sum()) <= 2.0 ** -18 * np.abs(f64(loss)).sum()
    api.distill_backward(*args, torch.from_numpy(dloss).cuda(), inplace=True, **kw)
    assert torch.equal(dev, dz) and torch.all(full[:, V:] == 7.0)
    assert api.step_device_status() == 0


def test_bad_ids_are_reported():
    rng = np.random.default_rng(5)
    N, V, K = 4, 500, 6
    z, values, ids = make(rng, N, V, K)
    ids[1, 2], ids[2, 0] = V, -2
    dev, _ = padded(z)
    loss = api.distill_forward(dev, values.cuda(), ids.cuda())
    assert api.step_device_status() == _lib.ERR_INVALID_ARG and api.step_device_status() == 0
    assert torch.equal(torch.isnan(loss).cpu(), torch.tensor([False, True, True, False]))
    dz = api.distill_backward(dev, values.cuda(), ids.cuda(), torch.ones(N, device="cuda"))
    assert api.step_device_status() == _lib.ERR_INVALID_ARG
    ids[1, 2], ids[2, 0] = -1, -1        # they count as absent
    check(z, values, ids, None, np.ones(N), 1.0, 1.0, 0.0, None, f64(dz))


def test_all_rows_ignored():
    rng = np.random.default_rng(6)
    z, values, ids = make(rng, 3, 100, 4)
    dev, _ = padded(z)
    labels = torch.full((3,), IGN, device="cuda")
    out, dz = api.distill_loss(dev, values.cuda(), ids.cuda(), labels=labels)
    assert float(out[0]) == 0.0 and float(out[1]) == 1.0 and torch.all(dz == 0)


def test_autograd_function_and_differences():
    rng = np.random.default_rng(7)
    N, V, K, T, s, cap = 3, 40, 6, 2.0, 0.5, 20.0
    z, values, ids = make(rng, N, V, K, 5.0)
    labels = torch.tensor([1, IGN, 2]).cuda()
    dev = z.cuda().requires_grad_(True)
    loss = api.DistillFunction.apply(dev, values.cuda(), ids.cuda(), labels, T, s, cap, IGN)
    (3.0 * loss).backward()
    z64, v64, i64, lab = f64(z), f64(values), ids.numpy(), labels.cpu().numpy()

    def value(x):
        return 1.5 * ods.run(x, v64, i64, np.ones(N), lab, T, s, cap, IGN)[0].sum()

    h = 1e-4
    for r, j in ((0, int(ids[0, 0])), (0, 3), (2, 39), (1, 5)):
        up, down = z64.copy(), z64.copy()
        up[r, j] += h
        down[r, j] -= h
        ref = (value(up) - value(down)) / (2 * h)
        assert abs(f64(dev.grad)[r, j] - ref) <= 2.0 ** -8 * abs(ref) + 1e-5   # 1e-5: the kernel's d, and h^2
    # backward twice over a kept graph gives the same again; in place bumps the version
    dev.grad = None
    loss = api.DistillFunction.apply(dev, values.cuda(), ids.cuda(), labels, T, s, cap, IGN)
    loss.backward(retain_graph=True)
    once = dev.grad.clone()
    loss.backward()
    assert torch.equal(dev.grad, once + once)
    leaf = z.cuda().requires_grad_(True)
    mine = leaf * 1.0
    version = mine._version
    api.DistillFunction.apply(mine, values.cuda(), ids.cuda(), labels, T, s, cap, IGN, True).backward()
    assert torch.equal(leaf.grad, once) and mine._version > version


def test_determinism_graph_replay_and_two_streams():
    rng = np.random.default_rng(8)
    N, V, K = 64, 50000, 16
    z, values, ids = make(rng, N, V, K)
    dev, values, ids, ws = padded(z)[0], values.cuda(), ids.cuda(), api.Workspace()
    api.distill_loss(dev, values, ids, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, dz = api.distill_loss(dev, values, ids, workspace=ws)
    dev.copy_(make(rng, N, V, K)[0])
    g.replay()
    ref = api.distill_loss(dev, values, ids)
    assert torch.equal(out, ref[0]) and torch.equal(dz, ref[1])
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(api.distill_loss(dev, values, ids))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[0]) and torch.equal(d, ref[1]) for o, d in outs)


def test_refusals():
    z = torch.zeros(2, 64, dtype=BF16, device="cuda")
    v, i = torch.zeros(2, 4, device="cuda"), torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    fwd = api.distill_forward
    with pytest.raises(TypeError):
        fwd(z.float(), v, i)
    with pytest.raises(TypeError):
        fwd(z, v.double(), i)
    with pytest.raises(TypeError):
        fwd(z, v, i.short())
    with pytest.raises(ValueError):
        fwd(z, v, i[:, :3])
    with pytest.raises(ValueError):
        fwd(z, v.t().contiguous().t(), i)
    with pytest.raises(ValueError):
        fwd(z.t().contiguous().t(), v, i)
    with pytest.raises(ValueError):
        api.distill_loss(z, v, i, reduction="none")
    with pytest.raises(ValueError):
        api.distill_loss(z, v, i, grad_out=torch.zeros(2, 72, dtype=BF16, device="cuda")[:, :64])
    for kw in ({"temperature": 0.0}, {"temperature": float("nan")}, {"logit_scale": 0.0}, {"softcap": -1.0}):
        with pytest.raises(_lib.LoraMLPError):
            fwd(z, v, i, **kw)
    with pytest.raises(_lib.LoraMLPError):
        fwd(torch.zeros(2, 68, dtype=BF16, device="cuda")[:, :64], v, i)         # a row stride of 68
    with pytest.raises(_lib.LoraMLPError):
        fwd(z, torch.zeros(2, 1025, device="cuda"), torch.zeros(2, 1025, dtype=torch.int64, device="cuda"))
