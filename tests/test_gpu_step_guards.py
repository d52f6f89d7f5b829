"""Guard zones around every output and workspace of the operators around the dense layers, on ragged sizes: no byte
beside them changes, every element of an output is written, and a workspace of the size that is asked for, with other
contents, gives the same bits."""
import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


class Guards:
    def __init__(self):
        self.all = []

    def bytes(self, n, fill):
        buf = torch.full((GUARD + (n + 255) // 256 * 256 + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        buf[GUARD:GUARD + n] = fill
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n]

    def tensor(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype)
        return self.bytes(t.numel() * t.element_size(), 0xFF).view(dtype).view(shape)  # 0xFF..: NaN

    def workspace(self, n, fill):
        ws = api.Workspace()
        ws.buf = self.bytes(n, fill)
        return ws

    def intact(self):
        return all(bool(torch.all(b[:GUARD] == 0x5A)) and bool(torch.all(b[GUARD + n:] == 0x5A)) for b, n in self.all)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,V,d", [(1, 3, 8), (777, 131, 200), (5000, 70, 1048), (9001, 4003, 24), (33, 9, 4104)])
def test_embedding(N, V, d, dtype):
    g = torch.Generator().manual_seed(N)
    ids = torch.randint(0, V, (N,), generator=g)
    ids[N // 2:] = V - 1
    ids, dOut = ids.cuda(), torch.randn(N, d, generator=g).to(BF16).cuda()
    z, need, outs = Guards(), _lib.embedding_sizes(N, V, d), []
    for fill in (0x00, 0xA5):
        dE = z.tensor((V, d), dtype)
        api.embedding_backward(dOut, ids, V, dtype=dtype, dE=dE, workspace=z.workspace(need, fill))
        outs.append(dE)
    out = z.tensor((N, d), BF16)
    api.embedding_forward(ids, outs[0].to(BF16), out=out)
    torch.cuda.synchronize()
    assert z.intact() and torch.equal(*outs) and not torch.any(torch.isnan(outs[0])) and not torch.any(torch.isnan(out))


@pytest.mark.parametrize("B,S,Hq,Hk,D,rot,inter", [(1, 1, 1, 1, 16, 16, False), (3, 41, 5, 2, 96, 48, True),
                                                   (2, 17, 33, 9, 128, 128, False), (1, 7, 3, 1, 512, 512, False)])
def test_norm_and_rotation(B, S, Hq, Hk, D, rot, inter):
    g = torch.Generator().manual_seed(S)
    q, k = (torch.randn(B, S, h, D, generator=g).to(BF16).cuda() for h in (Hq, Hk))
    gain = torch.randn(D, generator=g).to(BF16).cuda()
    cos, sin = api.rope_table(S, rot, device="cuda")
    shape = _lib.QKShape(B, S, Hq, Hk, D, rot, S, 0, 1e-6, 0)
    z, need, outs = Guards(), _lib.qk_rope_sizes(shape), []
    for fill in (0x00, 0xA5):
        o = [z.tensor(t.shape, BF16) for t in (q, k, q, k)]
        kw = dict(q_gain=gain, k_gain=gain, interleaved=inter)
        api.qk_norm_rope_forward(q, k, cos, sin, q_out=o[0], k_out=o[1], **kw)
        grads = api.qk_norm_rope_backward(q, k, cos, sin, o[0], o[1], dq=o[2], dk=o[3],
                                          workspace=z.workspace(need, fill), **kw)
        outs.append(o + list(grads[2:]))
    torch.cuda.synchronize()
    assert z.intact()
    assert all(torch.equal(a, b) and not torch.any(torch.isnan(a)) for a, b in zip(*outs))


@pytest.mark.parametrize("N,V,K,cap", [(1, 1, 1, 0.0), (19, 1003, 9, 0.0), (5, 4099, 130, 30.0), (301, 9001, 3, 0.0),
                                       (2, 130_007, 64, 20.0)])
def test_distillation(N, V, K, cap):
    g = torch.Generator().manual_seed(V)
    ld = (V + 7) // 8 * 8
    logits = torch.randn(N, ld, generator=g).to(BF16).cuda()
    ids, values = torch.randint(0, V, (N, K), generator=g).cuda(), torch.randn(N, K, generator=g).cuda()
    shape = _lib.DistillShape(N, V, ld, K, 1.0, 1.0, cap, _lib.DISTILL_VALUES_FP32, _lib.DISTILL_IDS_INT64, -100)
    z, need, outs = Guards(), _lib.distill_sizes(shape), []
    for fill in (0x00, 0xA5):
        dz = z.tensor((N, ld), BF16)
        out, _ = api.distill_loss(logits[:, :V], values, ids, softcap=cap, grad_out=dz[:, :V],
                                  workspace=z.workspace(need, fill))
        outs.append((out, dz[:, :V].clone()))
        assert torch.all(torch.isnan(dz[:, V:]))
    torch.cuda.synchronize()
    assert z.intact()
    assert all(torch.equal(a, b) and not torch.any(torch.isnan(a)) for a, b in zip(*outs))
    assert api.step_device_status() == 0
