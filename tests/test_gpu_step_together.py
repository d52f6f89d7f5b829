"""The operators around the dense layers in one training step: scaled embedding, norm and rotation of queries and
keys between the LoRA projections, and distillation of the logits, with the gradient of every parameter.

Tolerance of a gradient, relative in the 2-norm, against the same step in fp64: about 16 tensors are rounded to bf16
on the way from a parameter to the loss and back, each off by at most 2^-8 of its elements, and a map of the step
passes a relative error on at most twice: 2 x 16 x 2^-8 = 0.125.  A lost or wrong term is an error of order 1."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import api
from lora_fine_tuning_mlp_b200 import build as libbuild

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
IGN = -100
B, S, V, D, HQ, HK, HD, R, K = 2, 45, 1003, 256, 4, 2, 64, 8, 12
SCALE, ALPHA, EPS, TAU, CAP = 16.0, 16.0, 1e-5, 2.0, 30.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def parameters(g):
    def rand(*shape, std):
        return (torch.randn(*shape, generator=g, dtype=torch.float32) * std).to(BF16).cuda()
    p = {"E": rand(V, D, std=1.0 / SCALE), "gq": 1.0 + rand(HD, std=0.1), "gk": 1.0 + rand(HD, std=0.1)}
    for name, d_out, d_in in (("q", HQ * HD, D), ("k", HK * HD, D), ("v", HK * HD, D), ("o", D, HQ * HD)):
        p["W" + name] = rand(d_out, d_in, std=d_in ** -0.5)
        p["A" + name] = rand(R, d_in, std=d_in ** -0.5)
        p["B" + name] = rand(d_out, R, std=0.05)
    return p


TRAINED = ["E", "gq", "gk"] + [x + n for n in "qkvo" for x in "AB"]


def batch(g):
    ids = torch.randint(1, V, (B, S), generator=g)
    ids[1, 30:] = 0                                    # a padded sequence
    labels = torch.where(ids == 0, IGN, ids)
    positions = torch.arange(S).expand(B, S).contiguous() + torch.tensor([[0], [100]])
    tids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(B * S)])
    tvals = torch.randn(B * S, K, generator=g) * 2.0
    return ids.cuda(), labels.reshape(-1).cuda(), positions.cuda(), tids.cuda(), tvals.cuda()


def attention(q, k, v):
    k, v = (x.repeat_interleave(HQ // HK, dim=2) for x in (k, v))
    a = torch.einsum("bqhd,bkhd->bhqk", q, k) * HD ** -0.5
    a = a.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), -float("inf")).softmax(-1)
    return torch.einsum("bhqk,bkhd->bqhd", a, v)


def ours(p, data, table):
    ids, labels, pos, tids, tvals = data
    ones = torch.ones(D, dtype=BF16, device="cuda")

    def linear(x, n):
        w = api.LinearWeights(W=p["W" + n], A=p["A" + n], B=p["B" + n], alpha=ALPHA)
        return api.LoRALinearFunction.apply(x, w, p["A" + n], p["B" + n])

    x = api.EmbeddingFunction.apply(ids.reshape(-1), p["E"], SCALE, 0)
    h = api.RMSNormFunction.apply(x, ones, EPS)
    q, k, v = (linear(h, n).view(B, S, -1, HD) for n in "qkv")
    q, k = api.QKNormRopeFunction.apply(q, k, *table, pos, p["gq"], p["gk"], EPS, False)
    o = attention(q.float(), k.float(), v.float()).to(BF16)
    x = x + linear(o.reshape(B * S, -1), "o")
    f = api.RMSNormFunction.apply(x, ones, EPS)
    head = torch.cat([p["E"], p["E"].new_zeros(-V % 8, D)])   # rows of logits a multiple of 8 apart
    logits = (f @ head.t())[:, :V]
    return api.DistillFunction.apply(logits, tvals, tids, labels, TAU, 1.0, CAP, IGN)


def plain(p, data, table):
    """The same step in fp64."""
    ids, labels, pos, tids, tvals = data

    def norm(x, gain=1.0):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain

    def linear(x, n):
        return x @ (p["W" + n] + ALPHA / R * p["B" + n] @ p["A" + n]).t()

    def turn(x):
        c, s = (t.to(F64)[pos][:, :, None] for t in table)
        a, b = x[..., :HD // 2], x[..., HD // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    E = p["E"]
    table_rows = torch.cat([E[:1].detach(), E[1:]])           # no gradient to the padding's row through the lookup
    x = SCALE * table_rows[ids.reshape(-1)]
    h = norm(x)
    q, k, v = (linear(h, n).view(B, S, -1, HD) for n in "qkv")
    o = attention(turn(norm(q, p["gq"])), turn(norm(k, p["gk"])), v)
    x = x + linear(o.reshape(B * S, -1), "o")
    z = norm(x) @ E.t()
    logq = (CAP * torch.tanh(z / CAP) / TAU).log_softmax(-1).gather(1, tids)
    logp = (tvals.to(F64) / TAU).log_softmax(-1)
    rows = TAU * TAU * (logp.exp() * (logp - logq)).sum(-1)
    return rows[labels != IGN].mean()


@pytest.mark.parametrize("seed", [1, 2])
def test_training_step(seed):
    g = torch.Generator().manual_seed(seed)
    p, data, table = parameters(g), batch(g), api.rope_table(256, HD, device="cuda")
    p64 = {n: t.detach().to(F64) for n, t in p.items()}
    for n in TRAINED:
        p[n].requires_grad_(True)
        p64[n].requires_grad_(True)
    loss, ref = ours(p, data, table), plain(p64, data, table)
    loss.backward()
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) <= 0.125 * abs(float(ref.detach()))
    for n in TRAINED:
        got, want = p[n].grad.to(F64), p64[n].grad
        assert got.shape == want.shape and float((got - want).norm() / want.norm()) <= 0.125, n
    assert api.step_device_status() == 0


def test_captured_step_replays_on_new_batches():
    """Lookup, projection, rotation, projection and the distillation, forward and back, in one graph: the bits of the
    same calls without it."""
    g = torch.Generator().manual_seed(3)
    p, table = parameters(g), api.rope_table(256, HD, device="cuda")
    N = B * S
    wq = api.LinearWeights(W=p["Wq"], A=p["Aq"], B=p["Bq"], alpha=ALPHA)
    head = api.LinearWeights(W=torch.randn(1008, HQ * HD, generator=g).mul(0.05).to(BF16).cuda(),
                             A=torch.randn(R, HQ * HD, generator=g).mul(0.05).to(BF16).cuda(),
                             B=torch.randn(1008, R, generator=g).mul(0.05).to(BF16).cuda(), alpha=ALPHA)

    def step(ids, labels, pos, tids, tvals):
        x = api.embedding_forward(ids.reshape(-1), p["E"], scale=SCALE)
        q, saved = api.linear_forward(x, wq)
        q = q.view(B, S, HQ, HD)
        k = q[:, :, :HK]
        qr, kr = api.qk_norm_rope_forward(q, k, *table, positions=pos, q_gain=p["gq"], k_gain=p["gk"])
        y = qr.reshape(N, -1)
        logits, saved_h = api.linear_forward(y, head)
        out, dz = api.distill_loss(logits[:, :V], tvals, tids, labels=labels, temperature=TAU)
        full = logits.new_zeros(logits.shape)
        full[:, :V] = dz
        dy, dA, dB = api.linear_backward(y, head, saved_h, full)
        dq, dk, dgq, dgk = api.qk_norm_rope_backward(q, k, *table, dy.view(B, S, HQ, HD), kr, positions=pos,
                                                     q_gain=p["gq"], k_gain=p["gk"])
        dx, dAq, dBq = api.linear_backward(x, wq, saved, dq.reshape(N, -1))
        dE = api.embedding_backward(dx, ids.reshape(-1), V, scale=SCALE, padding_idx=0)
        return [out, dA, dB, dk, dgq, dgk, dAq, dBq, dE]

    data = batch(g)
    step(*data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*data)
    for seed in (4, 5):
        new = batch(torch.Generator().manual_seed(seed))
        for t, n in zip(data, new):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        captured = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(captured, step(*new)))
    assert np.isfinite(float(got[0][0])) and api.step_device_status() == 0
