"""A second derivative through the autograd functions is an error, not a term that is silently lost."""
import pytest
import torch

from lora_fine_tuning_mlp_b200 import api
from lora_fine_tuning_mlp_b200 import build as libbuild

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def leaf(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(1)).to(BF16).cuda().requires_grad_(True)


def embedding():
    E = leaf(9, 16)
    return E, api.EmbeddingFunction.apply(torch.arange(5, device="cuda"), E, 2.0)


def rotation():
    q, gain = leaf(1, 4, 2, 32), torch.ones(32, dtype=BF16, device="cuda")
    return q, api.QKNormRopeFunction.apply(q, q.detach(), *api.rope_table(4, 32, device="cuda"), None, gain, gain)[0]


def distillation():
    z = leaf(3, 40)
    ids = torch.arange(6, device="cuda").view(3, 2)
    return z, api.DistillFunction.apply(z, torch.ones(3, 2, device="cuda"), ids)


def mlp():
    x, r, d, f = leaf(128, 64), 8, 64, 128
    w = api.MLPWeights(*(leaf(*shape).detach() * 0.1 for shape in
                         ((f, d), (f, d), (d, f), (r, d), (f, r), (r, d), (f, r), (r, f), (d, r))), alpha=16.0)
    return x, w, (w.Ag, w.Bg, w.Au, w.Bu, w.Ad, w.Bd)


def dense():
    x, w, adapters = mlp()
    return x, api.LoRAMLPFunction.apply(x, w, *adapters)


def block():
    x, w, adapters = mlp()
    return x, api.LoRAMLPBlockFunction.apply(x, w, torch.ones(64, dtype=BF16, device="cuda"), 1e-5, *adapters)


def projection():
    x = leaf(128, 64)
    w = api.LinearWeights(W=leaf(128, 64).detach(), A=leaf(8, 64).detach(), B=leaf(128, 8).detach(), alpha=16.0)
    return x, api.LoRALinearFunction.apply(x, w, w.A, w.B)


def norm():
    x = leaf(128, 64)
    return x, api.RMSNormFunction.apply(x, torch.ones(64, dtype=BF16, device="cuda"), 1e-5)


def cross_entropy():
    z = leaf(3, 40)
    return z, api.CrossEntropyFunction.apply(z, torch.tensor([1, 2, 39], device="cuda"))


@pytest.mark.parametrize("make", [embedding, rotation, distillation, dense, block, projection, norm, cross_entropy])
def test_second_derivative(make):
    x, y = make()
    (y.float() ** 2).sum().backward(retain_graph=True)
    first = x.grad.clone()
    (g,) = torch.autograd.grad((y.float() ** 2).sum(), x, create_graph=True)
    assert torch.equal(g.detach(), first)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g.float() ** 2).sum() + x.float().sum()).backward()
