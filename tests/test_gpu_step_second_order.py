"""A second derivative through the operators around the dense layers is an error, not a term that is silently lost."""
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


@pytest.mark.parametrize("make", [embedding, rotation, distillation])
def test_second_derivative(make):
    x, y = make()
    (y.float() ** 2).sum().backward(retain_graph=True)
    first = x.grad.clone()
    (g,) = torch.autograd.grad((y.float() ** 2).sum(), x, create_graph=True)
    assert torch.equal(g.detach(), first)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        ((g.float() ** 2).sum() + x.float().sum()).backward()
