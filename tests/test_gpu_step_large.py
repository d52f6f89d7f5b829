"""Offsets past 32 bits in the operators around the dense layers: tensors of more than 2^31 elements, whose last rows
are compared with the same rows in small tensors; and calls on a stream that is not the current one, from two host
threads.

Embedding and rotation: the same bits.  Distillation: two sums of a row in different orders, each within 2^-20 of its
terms, and two roundings to bf16 (2^-8 of the value); its loss within 2^-18 T^2 of the sum of magnitudes, at most 40."""
import threading

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
    api.step_device_status()
    yield
    torch.cuda.empty_cache()


def test_embedding_of_a_large_table():
    V, d, n = 300_001, 8192, 64                              # 2.5e9 elements
    E = torch.empty(V, d, dtype=BF16, device="cuda")
    E[-100:].normal_()
    ids = torch.arange(V - n, V, device="cuda").flip(0).contiguous()
    assert torch.equal(api.embedding_forward(ids, E), E[ids])
    dOut = torch.randn(n, d, device="cuda").to(BF16)
    api.embedding_backward(dOut, ids, V, dE=E)               # every row is written, most with zeros
    assert torch.equal(E[ids], dOut)
    E[ids] = 0
    assert not torch.any(E.view(torch.int16))


def test_lookup_of_many_tokens():
    N, d = 300_001, 8192                                     # the output passes 2^31 elements
    E = torch.randn(11, d, device="cuda").to(BF16)
    ids = torch.arange(N, device="cuda") % 11
    out = api.embedding_forward(ids, E)
    assert torch.equal(out[-1000:], E[ids[-1000:]])
    dE = api.embedding_backward(out, ids, 11, dtype=torch.float32)
    n = torch.bincount(ids, minlength=11)[:, None].float()
    # n equal terms: sums of at most 30000 of them in fp32 in any order, n 2^-24 of their magnitude
    assert torch.all((dE - n * E.float()).abs() <= n * 2.0 ** -24 * n * E.float().abs())


@pytest.mark.parametrize("Hq,Hk,norm", [(100, 28, True), (5, 2, False)])
def test_rotation_past_32_bits(Hq, Hk, norm):
    D, S = 128, 2 ** 31 // 128 // Hq + 1000
    x = torch.empty(1, S, Hq + Hk, D, dtype=BF16, device="cuda")
    x.normal_()
    q, k = x[:, :, :Hq], x[:, :, Hq:]
    cos, sin = api.rope_table(512, D, device="cuda")
    pos = torch.arange(S, device="cuda") % 512
    gain = torch.ones(D, dtype=BF16, device="cuda") if norm else None
    kw = dict(q_gain=gain, k_gain=gain)
    qo, ko = api.qk_norm_rope_forward(q, k, cos, sin, positions=pos, **kw)
    cut = slice(S - 300, S)
    few = api.qk_norm_rope_forward(q[:, cut], k[:, cut], cos, sin, positions=pos[cut].contiguous(), **kw)
    assert torch.equal(qo[:, cut], few[0]) and torch.equal(ko[:, cut], few[1])
    dq, dk, _, _ = api.qk_norm_rope_backward(q, k, cos, sin, qo, ko, positions=pos, gain_grads=False, **kw)
    few = api.qk_norm_rope_backward(q[:, cut], k[:, cut], cos, sin, qo[:, cut], ko[:, cut],
                                    positions=pos[cut].contiguous(), gain_grads=False, **kw)
    assert torch.equal(dq[:, cut], few[0]) and torch.equal(dk[:, cut], few[1])
    assert api.step_device_status() == 0


def test_distillation_past_32_bits_in_place():
    N, V, K = 8400, 256_008, 4                               # 2.15e9 logits
    z = torch.empty(N, V, dtype=BF16, device="cuda")
    z.normal_()
    ids = torch.randint(0, V, (N, K), device="cuda")
    values = torch.randn(N, K, device="cuda")
    last = z[-3:].clone()
    loss = api.distill_forward(z, values, ids)
    few = api.distill_forward(last, values[-3:].contiguous(), ids[-3:].contiguous())
    assert torch.all((loss[-3:] - few).abs() <= 2.0 ** -18 * 40)
    ref = api.distill_backward(last, values[-3:].contiguous(), ids[-3:].contiguous(), torch.ones(3, device="cuda"))
    api.distill_backward(z, values, ids, torch.ones(N, device="cuda"), inplace=True)
    got = z[-3:].float()
    # a gradient at a teacher's entry is a difference q - p: its terms are at most 1
    assert torch.all((got - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 2.0 ** -20)
    assert api.step_device_status() == 0


def test_another_stream_and_two_host_threads():
    g = torch.Generator().manual_seed(1)
    E = torch.randn(500, 256, generator=g).to(BF16).cuda()
    ids = torch.randint(0, 500, (3000,), generator=g).cuda()
    dOut = torch.randn(3000, 256, generator=g).to(BF16).cuda()
    q = torch.randn(1, 300, 6, 64, generator=g).to(BF16).cuda()
    gain = torch.ones(64, dtype=BF16, device="cuda")
    table = api.rope_table(300, 64, device="cuda")
    z = torch.randn(70, 5000, generator=g).to(BF16).cuda()
    tids = torch.randint(0, 5000, (70, 9), generator=g).cuda()
    tvals = torch.randn(70, 9, generator=g).cuda()

    def calls(stream):
        out, dz = api.distill_loss(z, tvals, tids, stream=stream)
        return [api.embedding_backward(dOut, ids, 500, stream=stream), out, dz,
                *api.qk_norm_rope_backward(q, q, *table, q, q, q_gain=gain, k_gain=gain, stream=stream)]

    ref = calls(None)
    torch.cuda.synchronize()
    results = [[], []]

    def work(mine):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        for _ in range(20):
            got = calls(s)
            s.synchronize()
            mine.append(all(torch.equal(a, b) for a, b in zip(got, ref)))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(r,)) for r in results]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(len(r) == 20 and all(r) for r in results)
