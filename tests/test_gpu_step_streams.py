"""Calls on a stream of their own beside calls on the current one, with nothing between them that waits: each
gives the bits of a call by itself."""
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


class Inputs:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.ids = torch.randint(0, 2001, (20000,), generator=g).cuda()
        self.dOut = torch.randn(20000, 512, generator=g).to(BF16).cuda()
        self.q = torch.randn(1, 3000, 8, 128, generator=g).to(BF16).cuda()
        self.gain = torch.randn(128, generator=g).to(BF16).cuda()
        self.z = torch.randn(600, 20008, generator=g).to(BF16).cuda()
        self.values = torch.randn(600, 9, generator=g).cuda()
        self.tids = torch.randint(0, 20008, (600, 9), generator=g).cuda()
        self.table = api.rope_table(3000, 128, device="cuda")
        self.E = self.dOut[:2001].contiguous()

    def calls(self, stream):
        kw = {"stream": stream}
        rope = dict(q_gain=self.gain, k_gain=self.gain)
        return [api.embedding_forward(self.ids, self.E, **kw), api.embedding_backward(self.dOut, self.ids, 2001, **kw),
                *api.qk_norm_rope_forward(self.q, self.q, *self.table, **rope, **kw),
                *api.qk_norm_rope_backward(self.q, self.q, *self.table, self.q, self.q, **rope, **kw),
                api.distill_forward(self.z, self.values, self.tids, **kw),
                *api.distill_loss(self.z, self.values, self.tids, **kw)]


def test_interleaved_with_the_current_stream():
    torch.cuda.empty_cache()
    a, b = Inputs(1), Inputs(2)
    ref = {x: [t.clone() for t in x.calls(None)] for x in (a, b)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for i in range(12):
        kept.append((a, a.calls(None)))
        kept.append((b, b.calls(side)))
        if i % 3 == 2:                       # results go while their kernels are queued, their memory comes back
            kept = kept[-2:]
    torch.cuda.synchronize()
    assert all(torch.equal(t, r) for x, got in kept for t, r in zip(got, ref[x]))
    assert api.step_device_status() == 0


def test_a_result_that_goes_while_the_current_stream_reads_it():
    x = Inputs(3)
    ref = x.calls(None)[1].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sums = []
    for _ in range(10):
        dE = api.embedding_backward(x.dOut, x.ids, 2001, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2_000_000)
        sums.append(dE.clone())
        del dE
    torch.cuda.synchronize()
    assert all(torch.equal(s, ref) for s in sums)


def test_a_workspace_from_one_stream_to_the_other():
    x, ws = Inputs(4), api.Workspace()
    side = torch.cuda.Stream()
    ref = x.calls(None)[1].clone()
    for stream in (None, side, None, side):
        small = api.embedding_backward(x.dOut[:100], x.ids[:100], 2001, workspace=ws, stream=stream)
        dE = api.embedding_backward(x.dOut, x.ids, 2001, workspace=ws, stream=stream)
        torch.cuda.synchronize()             # a workspace belongs to one call at a time
        assert torch.equal(dE, ref) and small.shape == dE.shape
        ws.buf = ws.buf[:0]                  # grown again at the next call


def test_a_call_on_a_side_stream_of_a_capture():
    x = Inputs(5)
    ref = [t.clone() for t in x.calls(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = x.calls(side)
        torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, r) for t, r in zip(got, ref))


def test_dense_layers_norms_and_losses_beside_the_current_stream():
    def make(seed):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).to(BF16).cuda()

        n, d, f, r = 1024, 512, 1024, 8
        w = api.MLPWeights(rand(f, d), rand(f, d), rand(d, f), rand(r, d), rand(f, r), rand(r, d), rand(f, r),
                           rand(r, f), rand(d, r), alpha=16.0)
        lw = api.LinearWeights(W=rand(f, d), A=rand(r, d), B=rand(f, r), alpha=16.0)
        x, dy, dz, gamma = rand(n, d), rand(n, d), rand(n, f), rand(d)
        labels, ones = torch.randint(0, f, (n,), generator=g).cuda(), torch.ones(n, device="cuda")

        def calls(stream):
            kw = {"stream": stream}
            out, saved = api.forward(x, w, **kw)
            dx, grads = api.backward(x, w, saved, dy, **kw)
            bo, bsaved = api.block_forward(x, w, gamma, 1e-5, **kw)
            bx, bgrads = api.block_backward(x, w, gamma, bsaved, dy, **kw)
            y, lsaved = api.linear_forward(x, lw, **kw)
            h, rstd = api.rmsnorm_forward(x, gamma, 1e-5, **kw)
            loss, lse = api.ce_loss(dz, labels, **kw)
            return [out, dx, *grads.values(), bo, bx, *bgrads.values(), y,
                    *api.linear_backward(x, lw, lsaved, dz, **kw), h,
                    api.rmsnorm_backward(x, gamma, rstd, dy, **kw), loss,
                    api.ce_backward(dz, labels, lse, ones, **kw)]
        return calls

    a, b = make(1), make(2)
    ref = {x: [t.clone() for t in x(None)] for x in (a, b)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for i in range(6):
        kept.append((a, a(None)))
        kept.append((b, b(side)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, r) for x, got in kept for t, r in zip(got, ref[x]))
