"""The norm and rotation of queries and keys written over their inputs: the bits of the same call into new memory, and
refusals of results that begin where another view does."""
import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def heads(g, layout, B, S, H, D):
    x = torch.randn(B, S, H, D, generator=g).to(BF16).cuda()
    if layout == "bhsd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "packed":
        wide = torch.zeros(B, S, (H + 3) * D, dtype=BF16, device="cuda")
        wide[..., D:(H + 1) * D] = x.reshape(B, S, H * D)
        return wide[..., D:(H + 1) * D].view(B, S, H, D)
    return x


@pytest.mark.parametrize("norm", [True, False], ids=["norm", "rotation"])
@pytest.mark.parametrize("B,S,Hq,Hk,D,rot,inter,layout", [
    (1, 1, 1, 1, 16, 16, False, "bshd"), (2, 37, 5, 3, 64, 64, False, "packed"), (3, 50, 14, 2, 96, 48, True, "bhsd"),
    (1, 33, 3, 2, 512, 512, False, "packed"), (5, 611, 1, 1, 128, 128, False, "bshd"),
    (2, 2001, 32, 8, 128, 128, False, "packed"), (2, 61, 40, 9, 64, 64, True, "bhsd")])
def test_same_bits_in_place(B, S, Hq, Hk, D, rot, inter, layout, norm):
    g = torch.Generator().manual_seed(S)
    cos, sin = api.rope_table(S, rot, device="cuda")
    gains = {n: torch.randn(D, generator=g).to(BF16).cuda() if norm else None for n in ("q_gain", "k_gain")}
    kw = dict(interleaved=inter, **gains)

    def fresh():
        gen = torch.Generator().manual_seed(S + 1)
        return [heads(gen, layout, B, S, h, D) for h in (Hq, Hk)] + [heads(gen, "bshd", B, S, h, D) for h in (Hq, Hk)]

    q, k, dq, dk = fresh()
    ref = api.qk_norm_rope_forward(q, k, cos, sin, **kw)
    back = api.qk_norm_rope_backward(q, k, cos, sin, dq, dk, **kw)
    a, b, _, _ = fresh()
    got = api.qk_norm_rope_forward(a, b, cos, sin, q_out=a, k_out=b, **kw)
    assert got[0] is a and torch.equal(a, ref[0]) and torch.equal(b, ref[1])
    q, k, dq, dk = fresh()
    got = api.qk_norm_rope_backward(q, k, cos, sin, dq, dk, dq=dq, dk=dk, **kw)   # over the gradients that come in
    assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(got, back))
    if norm:                                                                      # over the forward's inputs
        q, k, dq, dk = fresh()
        got = api.qk_norm_rope_backward(q, k, cos, sin, dq, dk, dq=q, dk=k, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, back))


def test_other_overlaps_are_refused():
    q, k, o = (torch.zeros(2, 4, 2, 64, dtype=BF16, device="cuda") for _ in range(3))
    cos, sin = api.rope_table(4, 64, device="cuda")
    gain = torch.ones(64, dtype=BF16, device="cuda")
    fwd, bwd = api.qk_norm_rope_forward, api.qk_norm_rope_backward
    turned = q.view(4, 2, 2, 64).transpose(0, 1)           # q's memory in another order
    with_gains = dict(q_gain=gain, k_gain=gain)
    for call in (lambda: fwd(q, k, cos, sin, q_out=k), lambda: fwd(q, k, cos, sin, k_out=q),
                 lambda: fwd(q, k, cos, sin, q_out=o, k_out=o), lambda: fwd(q, q, cos, sin, q_out=q),
                 lambda: fwd(q, k, cos, sin, q_out=turned),
                 lambda: bwd(q, k, cos, sin, o, k, dq=k), lambda: bwd(q, k, cos, sin, o, q, dk=o),
                 lambda: bwd(q, k, cos, sin, q, k, dq=o, dk=o),
                 lambda: bwd(q, k, cos, sin, o, o.clone(), dq=k, **with_gains),
                 lambda: bwd(q, k, cos, sin, o, o.clone(), dq=turned, **with_gains)):
        with pytest.raises(_lib.LoraMLPError) as e:
            call()
        assert e.value.code == _lib.ERR_INVALID_ARG
    with pytest.raises(_lib.LoraMLPError) as e:
        fwd(q, k, cos, sin, q_out=torch.zeros(10000, dtype=BF16, device="cuda").as_strided(q.shape, (1024, 128, 8, 1)))
    assert e.value.code == _lib.ERR_UNSUPPORTED_SHAPE
    fwd(q, k, cos, sin, q_out=q, k_out=k)
    bwd(q, k, cos, sin, o, o.clone(), dq=k)                # without gains q and k are not read
    assert api.step_device_status() == 0
