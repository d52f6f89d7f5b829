"""The distillation's bounded waits, without a GPU fault: the test hook lets no wait of its kernels be over, with a
limit of about a millisecond.  Every warp gives up, the kernels return, the status word says so (before any id that is
out of its range), and the next ordinary call is right."""
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


@pytest.fixture
def forced():
    """Switches the hook on, and off again however the test ends."""
    yield lambda on: _lib.step_debug_force_timeout(on, 2_000_000)
    _lib.step_debug_force_timeout(False)


def inputs(N, V, K=5):
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, (V + 7) // 8 * 8, generator=g).to(BF16).cuda()[:, :V]
    return z, torch.randn(N, K, generator=g).cuda(), torch.randint(0, V, (N, K), generator=g).cuda()


@pytest.mark.parametrize("cap", [0.0, 30.0, 1e4])
@pytest.mark.parametrize("N,V", [(1, 1), (2000, 777), (300, 9000), (3, 262_147), (40, 128_256)])
def test_waits_that_run_out(forced, N, V, cap):
    args, kw = inputs(N, V), {"softcap": cap}
    ones = torch.ones(N, device="cuda")
    calls = [lambda: [api.distill_forward(*args, **kw)], lambda: [api.distill_backward(*args, ones, **kw)],
             lambda: list(api.distill_loss(*args, **kw))]
    ref = [c() for c in calls]
    assert api.step_device_status() == 0
    for call, want in zip(calls, ref):
        forced(True)
        call()
        torch.cuda.synchronize()                 # it ended by itself, without a CUDA error
        forced(False)
        assert api.step_device_status() == _lib.ERR_DEVICE_TIMEOUT
        assert api.step_device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert api.step_device_status() == 0


@pytest.mark.parametrize("first", [True, False])
def test_a_timeout_outranks_an_id_out_of_range(forced, first):
    z, values, ids = inputs(50, 5000)
    bad = ids.clone()
    bad[7, 1] = 5000
    E, q = torch.zeros(9, 64, dtype=BF16, device="cuda"), torch.zeros(1, 2, 1, 64, dtype=BF16, device="cuda")
    cos, sin = api.rope_table(4, 64, device="cuda")

    def out_of_range():
        api.distill_forward(z, values, bad)
        api.embedding_forward(torch.tensor([9], device="cuda"), E)
        api.embedding_backward(torch.zeros(1, 64, dtype=BF16, device="cuda"), torch.tensor([-1], device="cuda"), 9)
        gain = torch.ones(64, dtype=BF16, device="cuda")
        pos = torch.tensor([4, 0], device="cuda")
        api.qk_norm_rope_forward(q, q, cos, sin, positions=pos)
        api.qk_norm_rope_backward(q, q, cos, sin, q, q, positions=pos, q_gain=gain, k_gain=gain)

    if first:
        out_of_range()
    forced(True)
    api.distill_forward(z, values, ids)
    torch.cuda.synchronize()
    forced(False)
    if not first:
        out_of_range()
    assert api.step_device_status() == _lib.ERR_DEVICE_TIMEOUT and api.step_device_status() == 0
    out_of_range()
    assert api.step_device_status() == _lib.ERR_INVALID_ARG


def test_the_hook_refuses_a_limit_of_nothing():
    with pytest.raises(_lib.LoraMLPError):
        _lib.step_debug_force_timeout(True, 0)
