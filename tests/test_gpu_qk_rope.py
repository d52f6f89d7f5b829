"""GPU parity of the queries' and keys' norm and rotation
(include/lora_qk_rope.h) against the fp64 oracle.

Tolerances, from the arithmetic, u = 2^-24: a normed element is off by
(D + 8) u relative (the sum of D squares, the root, three products), a turned
one by that and 3 u of its pair's magnitudes, then rounded to bf16 (2^-8 of
the result).  Backward, the mean of D products adds (D + 8) u of the mean of
their magnitudes.  A gain's gradient adds up n = tokens x heads terms, each off
by (D + 12) u of its magnitudes: (n + D + 12) u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild
from oracle import qk_rope as oqk

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def f64(t):
    return t.detach().double().cpu().numpy()


def heads(rng, layout, B, S, H, D):
    """A bf16 [B, S, H, D] view on the device, of the given memory layout."""
    x = torch.from_numpy(rng.standard_normal((B, S, H, D)).astype(np.float32)).to(BF16).cuda()
    if layout == "bhsd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "packed":  # columns of a wider projection
        wide = torch.full((B, S, (H + 3) * D), float("nan"), dtype=BF16, device="cuda")
        wide[..., D:(H + 1) * D] = x.reshape(B, S, H * D)
        return wide[..., D:(H + 1) * D].view(B, S, H, D)
    return x


def pair_mag(x, rot, interleaved):
    """|a| + |b| of each element's pair (|x| for elements that do not turn)."""
    m = np.abs(x)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    both = m[..., a] + m[..., b]
    m[..., a], m[..., b] = both, both
    return m


def check(got, ref, tol):
    bad = ~(np.abs(got - ref) <= tol)
    assert not np.any(bad), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


def check_all(x, gain, eps, cos, sin, interleaved, y, dy=None, dx=None, dgain=None):
    """All arrays [T, H, D] in fp64; cos and sin of each token."""
    D, rot = x.shape[-1], 2 * cos.shape[-1]
    n = oqk.forward(x, gain, eps, cos[:, :0], sin[:, :0], interleaved)
    ref = oqk.forward(x, gain, eps, cos, sin, interleaved)
    check(y, ref, 2.0 ** -8 * np.abs(ref) + (D + 12) * U * pair_mag(n, rot, interleaved))
    if dy is None:
        return
    rdx, rdg = oqk.backward(x, gain, eps, cos, sin, dy, interleaved)
    mag = pair_mag(dy, rot, interleaved)
    if gain is None:
        check(dx, rdx, 2.0 ** -8 * np.abs(rdx) + 4 * U * mag)
        return
    rstd = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xh, gm = np.abs(x) * rstd, mag * np.abs(gain)
    check(dx, rdx, 2.0 ** -8 * np.abs(rdx) + 3 * (D + 12) * U * rstd * (gm + xh * np.mean(gm * xh, -1, keepdims=True)))
    if dgain is not None:
        terms = x.shape[0] * x.shape[1]
        check(dgain, rdg, (terms + D + 12) * U * np.sum(mag * xh, axis=(0, 1)))


CASES = [
    # B, S, Hq, Hk, D, rot, interleaved, layout
    (1, 1, 1, 1, 16, 16, False, "bshd"),      # one head of one token, one thread
    (1, 1, 32, 8, 128, 128, False, "bshd"),   # a decoding step
    (2, 37, 5, 3, 64, 64, False, "packed"),
    (3, 50, 14, 2, 96, 48, True, "bhsd"),     # six threads of eight, half the head turned
    (1, 129, 4, 4, 80, 32, False, "bhsd"),
    (2, 9, 9, 1, 256, 256, True, "bshd"),
    (1, 33, 3, 2, 512, 512, False, "packed"), # a head a warp
    (1, 5, 70, 1, 32, 16, True, "bshd"),      # more heads than a unit
    (4, 300, 6, 2, 48, 32, False, "bshd"),
    (5, 211, 1, 1, 128, 128, False, "packed"),  # units of several tokens, across sequences
    (2, 61, 40, 9, 64, 64, True, "bshd"),     # units of one token, the last of them partly empty
]


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "rotation"])
@pytest.mark.parametrize("B,S,Hq,Hk,D,rot,interleaved,layout", CASES)
def test_forward_and_backward(B, S, Hq, Hk, D, rot, interleaved, layout, norm):
    rng = np.random.default_rng(B * 1000 + S * 10 + D)
    P, eps = 5000, 1e-5
    cos, sin = api.rope_table(P, rot, base=500000.0, device="cuda")
    pos = torch.from_numpy(rng.integers(0, P, (B, S))).cuda()
    q, k = heads(rng, layout, B, S, Hq, D), heads(rng, layout, B, S, Hk, D)
    dq, dk = heads(rng, "bshd", B, S, Hq, D), heads(rng, "bhsd", B, S, Hk, D)
    gains = [torch.from_numpy(rng.uniform(-1.5, 1.5, D).astype(np.float32)).to(BF16).cuda() if norm else None
             for _ in range(2)]
    kw = {"positions": pos, "q_gain": gains[0], "k_gain": gains[1], "eps": eps, "interleaved": interleaved}
    out = api.qk_norm_rope_forward(q, k, cos, sin, **kw)
    grads = api.qk_norm_rope_backward(q, k, cos, sin, dq, dk, **kw)
    again = api.qk_norm_rope_backward(q, k, cos, sin, dq, dk, gain_grads=False, **kw)
    assert again[2] is None and torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])
    assert api.step_device_status() == 0
    c, s = f64(cos[pos.flatten()]), f64(sin[pos.flatten()])
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        flat = lambda t: f64(t).reshape(B * S, -1, D)  # noqa: E731
        check_all(flat(x), None if not norm else f64(gains[i]), float(np.float32(eps)), c, s, interleaved,
                  flat(out[i]), flat(d), flat(grads[i]), None if not norm else f64(grads[2 + i]))
        assert (grads[2 + i] is None) == (not norm)


def test_outputs_into_views_and_default_positions():
    """Results into a heads-first cache slot; no positions means 0 .. S-1; one [S] row serves every sequence."""
    rng = np.random.default_rng(3)
    B, S, D = 2, 21, 64
    q, k = heads(rng, "bshd", B, S, 4, D), heads(rng, "packed", B, S, 2, D)
    cos, sin = api.rope_table(64, D, device="cuda")
    ref = api.qk_norm_rope_forward(q, k, cos, sin)
    cache = torch.full((B, 2, 40, D), 7.0, dtype=BF16, device="cuda")
    slot = cache[:, :, 5:5 + S].transpose(1, 2)
    pos = torch.arange(S, device="cuda")
    q_out, k_out = api.qk_norm_rope_forward(q, k, cos, sin, positions=pos, k_out=slot)
    assert k_out is slot and torch.equal(q_out, ref[0]) and torch.equal(slot, ref[1])
    assert torch.all(cache[:, :, :5] == 7.0) and torch.all(cache[:, :, 5 + S:] == 7.0)
    # three axes: one sequence
    one = api.qk_norm_rope_forward(q[1], k[1], cos, sin)
    assert one[0].shape == (S, 4, D) and torch.equal(one[0], ref[0][1]) and torch.equal(one[1], ref[1][1])


def test_broadcast_gradient_and_gains_shared_by_heads():
    """A gradient that is one head expanded over all, read in place; the gain's gradient adds up over heads."""
    rng = np.random.default_rng(4)
    S, H, D = 30, 6, 32
    q, k = heads(rng, "bshd", 1, S, H, D), heads(rng, "bshd", 1, S, 2, D)
    gain = torch.full((D,), 0.75, dtype=BF16, device="cuda")
    cos, sin = api.rope_table(S, D, device="cuda")
    d1 = heads(rng, "bshd", 1, S, 1, D)
    args = dict(q_gain=gain, k_gain=gain)
    wide = api.qk_norm_rope_backward(q, k, cos, sin, d1.expand(1, S, H, D), k, **args)
    full = api.qk_norm_rope_backward(q, k, cos, sin, d1.expand(1, S, H, D).contiguous(), k, **args)
    assert all(torch.equal(a, b) for a, b in zip(wide, full))


def test_autograd_function_and_differences():
    rng = np.random.default_rng(5)
    B, S, D, eps = 1, 4, 16, 1e-3
    q, k = (heads(rng, "bshd", B, S, h, D).requires_grad_(True) for h in (2, 1))
    gq, gk = (torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32)).to(BF16).cuda().requires_grad_(True)
              for _ in range(2))
    cos, sin = api.rope_table(100, D, device="cuda")
    pos = torch.tensor([[3, 99, 0, 17]], device="cuda")
    wq, wk = heads(rng, "bshd", B, S, 2, D), heads(rng, "bhsd", B, S, 1, D)
    qo, ko = api.QKNormRopeFunction.apply(q, k, cos, sin, pos, gq, gk, eps, False)
    ((qo.float() * wq.float()).sum() + (ko.float() * wk.float()).sum()).backward()
    c, s = f64(cos[pos[0]]), f64(sin[pos[0]])
    x, g, w = f64(q)[0], f64(gq), f64(wq)[0]

    def value(x, g):
        return float(np.sum(oqk.forward(x, g, eps, c, s) * w))

    h = 1e-4
    for at in ((0, 0, 0), (1, 1, 9), (3, 0, 15)):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        ref = (value(up, g) - value(down, g)) / (2 * h)
        assert abs(f64(q.grad)[0][at] - ref) <= 2.0 ** -8 * abs(ref) + 1e-5   # 1e-5: h^2 and the differences' rounding
    for e in (0, 7, 15):
        up, down = g.copy(), g.copy()
        up[e] += h
        down[e] -= h
        ref = (value(x, up) - value(x, down)) / (2 * h)
        assert abs(f64(gq.grad)[e] - ref) <= 2.0 ** -8 * abs(ref) + 1e-5
    assert k.grad is not None and gk.grad is not None and gk.grad.dtype == BF16
    # the rotation alone, frozen: gradients of q and k only
    q2 = q.detach().clone().requires_grad_(True)
    qo, _ = api.QKNormRopeFunction.apply(q2, k.detach(), cos, sin, pos, None, None, eps, True)
    qo.sum().backward()
    assert q2.grad.shape == q2.shape


def test_bad_positions_are_reported_and_stay_in_their_tokens():
    rng = np.random.default_rng(6)
    S, D = 9, 64
    q, k = heads(rng, "bshd", 1, S, 3, D), heads(rng, "bshd", 1, S, 2, D)
    gain = torch.ones(D, dtype=BF16, device="cuda")
    cos, sin = api.rope_table(S, D, device="cuda")
    good = torch.arange(S, device="cuda")
    bad = good.clone()
    bad[2], bad[7] = -1, S
    kw = dict(q_gain=gain, k_gain=gain)
    ref = api.qk_norm_rope_forward(q, k, cos, sin, positions=good, **kw)
    got = api.qk_norm_rope_forward(q, k, cos, sin, positions=bad, **kw)
    assert api.step_device_status() == _lib.ERR_INVALID_ARG and api.step_device_status() == 0
    keep = torch.ones(S, dtype=torch.bool, device="cuda")
    keep[[2, 7]] = False
    dq, dk, dgq, dgk = api.qk_norm_rope_backward(q, k, cos, sin, q, k, positions=bad, **kw)
    assert api.step_device_status() == _lib.ERR_INVALID_ARG
    for a, b in zip(got, ref):
        assert torch.equal(a[:, keep], b[:, keep]) and torch.all(torch.isnan(a[:, ~keep]))
    assert torch.all(torch.isnan(dq[:, ~keep])) and torch.all(torch.isfinite(dq[:, keep]))
    assert torch.all(torch.isfinite(dgq)) and torch.all(torch.isfinite(dgk))


def test_bad_positions_among_many_heads():
    rng = np.random.default_rng(16)
    S, D = 5, 64
    q, k = heads(rng, "bshd", 1, S, 48, D), heads(rng, "bshd", 1, S, 32, D)
    cos, sin = api.rope_table(S, D, device="cuda")
    pos = torch.arange(S, device="cuda")
    ref = api.qk_norm_rope_forward(q, k, cos, sin, positions=pos)
    pos[3] = 2 ** 40
    got = api.qk_norm_rope_forward(q, k, cos, sin, positions=pos)
    assert api.step_device_status() == _lib.ERR_INVALID_ARG and api.step_device_status() == 0
    for a, b in zip(got, ref):
        assert torch.equal(a[:, :3], b[:, :3]) and torch.equal(a[:, 4], b[:, 4]) and torch.all(torch.isnan(a[:, 3]))


def test_zero_heads_and_infinities_stay_apart():
    rng = np.random.default_rng(7)
    q, k = heads(rng, "bshd", 1, 6, 4, 32), heads(rng, "bshd", 1, 6, 4, 32)
    q[0, 1, 2] = 0.0
    q[0, 3, 1, 5] = float("inf")       # an element of a pair that turns
    k[0, 2, 0, 31] = float("nan")      # an element behind rot
    cos, sin = api.rope_table(6, 16, device="cuda")
    gain = torch.ones(32, dtype=BF16, device="cuda")
    qo, ko = api.qk_norm_rope_forward(q, k, cos, sin)
    assert int((~torch.isfinite(qo)).sum()) == 2 and int((~torch.isfinite(ko)).sum()) == 1
    qo, ko = api.qk_norm_rope_forward(q, k, cos, sin, q_gain=gain, k_gain=gain)
    assert torch.all(qo[0, 1, 2] == 0.0)
    finite = torch.isfinite(qo).all(-1)
    assert int((~finite).sum()) == 1 and int((~torch.isfinite(ko).all(-1)).sum()) == 1


def test_graph_replay_and_two_streams():
    rng = np.random.default_rng(8)
    B, S, D = 2, 64, 128
    q, k = heads(rng, "bshd", B, S, 8, D), heads(rng, "bshd", B, S, 2, D)
    cos, sin = api.rope_table(S, D, device="cuda")
    gain = torch.ones(D, dtype=BF16, device="cuda")
    kw, ws = dict(q_gain=gain, k_gain=gain), api.Workspace()

    def step():
        return [*api.qk_norm_rope_forward(q, k, cos, sin, **kw),
                *api.qk_norm_rope_backward(q, k, cos, sin, q, k, workspace=ws, **kw)]

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    q.copy_(heads(rng, "bshd", B, S, 8, D))
    g.replay()
    ref = step()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(api.qk_norm_rope_backward(q, k, cos, sin, q, k, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, ref[2:]))


def test_refusals():
    q = torch.zeros(1, 4, 2, 64, dtype=BF16, device="cuda")
    cos, sin = api.rope_table(8, 64, device="cuda")
    fwd = api.qk_norm_rope_forward
    with pytest.raises(TypeError):
        fwd(q.float(), q, cos, sin)
    with pytest.raises(ValueError):
        fwd(q, q[:, :3], cos, sin)
    with pytest.raises(ValueError):
        fwd(q, q, cos, sin[:, :16])
    with pytest.raises(ValueError):
        fwd(q, q, cos, sin, q_gain=torch.ones(64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        fwd(q, q, cos, sin, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        fwd(q.transpose(2, 3), q, cos, sin)
    with pytest.raises(ValueError):
        fwd(q, q, cos, sin, q_out=q[:, :1].expand(1, 4, 2, 64))
    with pytest.raises(ValueError):
        fwd(torch.zeros(1, 4, 2, 68, dtype=BF16, device="cuda")[..., :64], q, cos, sin)   # strides of 68
    with pytest.raises(_lib.LoraMLPError):
        fwd(q, q, cos[:2], sin[:2])                       # four positions, a table of two
    with pytest.raises(_lib.LoraMLPError):
        fwd(q, q, cos[:, :20].contiguous(), sin[:, :20].contiguous())   # rot 40
    with pytest.raises(_lib.LoraMLPError):
        fwd(q[..., :32], q[..., :32], cos, sin)           # rot 64 of 32
    with pytest.raises(_lib.LoraMLPError):
        fwd(q[..., 4:52], q[..., :48], *api.rope_table(8, 48, device="cuda"))   # an address off 16 bytes
    with pytest.raises(_lib.LoraMLPError):
        fwd(q, q, cos, sin, q_gain=torch.ones(64, dtype=BF16, device="cuda"),
            k_gain=torch.ones(64, dtype=BF16, device="cuda"), eps=float("nan"))
