"""GPU parity of the scaled embedding lookup and its gradient by sorted tokens
(include/lora_embedding.h) against the fp64 oracle.

Tolerances, from the arithmetic: the lookup rounds one fp32 product to bf16,
2^-8 |ref| + 2^-23 |ref|.  A row of the gradient adds n tokens in fp32, an
error of at most n 2^-24 times the sum of magnitudes (any order), is scaled
(2^-24) and, for bf16, rounded (2^-8 |ref|)."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild
from oracle import embedding as oemb

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    assert api.step_device_status() in (0, _lib.ERR_INVALID_ARG)  # start from a clear word


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(BF16)


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("N,V,d,scale", [
    (1, 1, 8, 1.0),          # one token, one row, one vector
    (1, 5, 4096, 1.0),
    (3, 7, 16, 2.5),
    (257, 100, 72, 0.3),     # a row that is no power of two of vectors
    (1000, 777, 2056, 45.25),
    (33, 50, 8200, 1.0),     # a row longer than one trip of the block
])
def test_forward(N, V, d, scale):
    rng = np.random.default_rng(N * 131 + d)
    E, ids = bf16(rng, V, d), torch.from_numpy(rng.integers(0, V, N))
    got = f64(api.embedding_forward(ids.cuda(), E.cuda(), scale=scale))
    ref = oemb.forward(ids.numpy(), f64(E), np.float32(scale).astype(np.float64))
    assert np.all(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))
    if scale == 1.0:
        assert np.array_equal(got, ref)


def make_ids(rng, kind, N, V):
    if kind == "uniform":
        return rng.integers(0, V, N)
    if kind == "same":
        return np.full(N, V - 1)
    if kind == "heavy":  # one id takes most tokens, in the middle of the rest
        ids = rng.integers(0, V, N)
        ids[rng.random(N) < 0.7] = V // 2
        return ids
    if kind == "runs":   # ids with exactly, just under and just over whole chunks of tokens
        ids = np.concatenate([np.full(n, i % V) for i, n in enumerate((64, 63, 65, 128, 1, 127, 129, 200, 2))])
        ids = np.concatenate([ids, rng.integers(0, V, max(0, N - len(ids)))])[:N]
        return rng.permutation(ids)
    return np.minimum(np.exp(rng.random(N) * np.log(V + 1.0)).astype(np.int64) - 1, V - 1)  # zipf


def check_grad(dOut, ids, V, scale, dtype, padding_idx, got):
    s32 = float(np.float32(scale))
    ref, mag, n = oemb.backward(f64(dOut), ids, V, s32, padding_idx)
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if dtype == BF16 else 0.0)
    bad = np.abs(got - ref) > tol
    assert not np.any(bad), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
    assert np.all(got[n == 0] == 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind,N,V,d", [
    ("uniform", 1, 1, 8),
    ("uniform", 1, 300, 64),
    ("uniform", 63, 40, 24),
    ("same", 64, 9, 40),         # exactly one whole chunk
    ("same", 65, 1, 2056),       # a vocabulary of one row, two slices of columns
    ("same", 8192, 3, 264),      # the largest that one block sorts
    ("runs", 900, 20, 4104),
    ("runs", 900, 1000, 136),
    ("heavy", 5000, 333, 520),
    ("zipf", 4097, 5003, 1032),
    ("uniform", 8193, 700, 72),  # the smallest that many blocks sort
    ("zipf", 20000, 30011, 264),
    ("heavy", 30000, 2, 64),
    ("zipf", 9000, 300007, 32),  # ids of 19 bits: three passes
    ("uniform", 700, 270001, 8),
    ("zipf", 1500, 900, 16),     # two and four tokens a thread of the one block's sort
    ("heavy", 3000, 70, 24),
    ("zipf", 140001, 3001, 8),   # wider tiles of the many-block sort
    ("heavy", 40000, 300, 1032), # more chunks than blocks are worth: wider slices
])
def test_gradient(kind, N, V, d, dtype):
    rng = np.random.default_rng(N * 7 + V)
    ids, dOut = make_ids(rng, kind, N, V), bf16(rng, N, d)
    scale = 1.0 if N % 2 else 3.7
    pad = None if N % 3 else int(ids[0])
    dE = torch.full((V, d), float("nan"), dtype=dtype, device="cuda")
    args = (dOut.cuda(), torch.from_numpy(ids).cuda(), V)
    got = api.embedding_backward(*args, scale=scale, padding_idx=pad, dtype=dtype, dE=dE)
    assert got is dE
    check_grad(dOut, ids, V, scale, dtype, pad, f64(got))
    # the same bits again, over a workspace of other contents
    ws = api.Workspace()
    ws.get(_lib.embedding_sizes(N, V, d), torch.device("cuda", 0)).fill_(0xA5)
    again = api.embedding_backward(*args, scale=scale, padding_idx=pad, dtype=dtype, workspace=ws)
    assert torch.equal(again.view(torch.uint8), got.view(torch.uint8))


def test_bad_ids_are_reported_and_leave_the_rest_alone():
    rng = np.random.default_rng(5)
    N, V, d = 300, 50, 128
    ids = rng.integers(0, V, N)
    ids[[3, 77, 299]] = [-1, V, 2 ** 40]
    E, dOut, dev = bf16(rng, V, d), bf16(rng, N, d), torch.from_numpy(ids).cuda()
    out = f64(api.embedding_forward(dev, E.cuda()))
    assert api.step_device_status() == _lib.ERR_INVALID_ARG and api.step_device_status() == 0
    assert np.array_equal(out, oemb.forward(ids, f64(E)), equal_nan=True)
    dE = f64(api.embedding_backward(dOut.cuda(), dev, V))
    assert api.step_device_status() == _lib.ERR_INVALID_ARG and api.step_device_status() == 0
    check_grad(dOut, ids, V, 1.0, BF16, None, dE)


def test_infinities_stay_in_their_rows():
    rng = np.random.default_rng(6)
    N, V, d = 200, 30, 64
    ids, dOut = rng.integers(1, V, N), bf16(rng, N, d)
    ids[10], ids[11] = 0, 5
    dOut[10, 3], dOut[11, 4] = float("inf"), float("nan")
    dE = f64(api.embedding_backward(dOut.cuda(), torch.from_numpy(ids).cuda(), V))
    assert dE[0, 3] == np.inf and np.isnan(dE[5, 4])
    dE[0, 3] = dE[5, 4] = 0.0
    assert np.all(np.isfinite(dE))
    skipped = f64(api.embedding_backward(dOut.cuda(), torch.from_numpy(ids).cuda(), V, padding_idx=0))
    assert np.all(skipped[0] == 0.0)


def test_autograd_function_against_differences():
    """d/dE of a weighted sum of the lookup, by central differences of the (linear) oracle, and through autograd."""
    rng = np.random.default_rng(8)
    N, V, d, scale = 40, 12, 16, 1.5
    ids, E, w = torch.from_numpy(rng.integers(0, V, N)), bf16(rng, V, d), bf16(rng, N, d)
    leaf = E.cuda().requires_grad_(True)
    out = api.EmbeddingFunction.apply(ids.cuda(), leaf, scale, 3)
    (out * w.cuda()).sum().backward()
    got = f64(leaf.grad)
    E64, w64 = f64(E), f64(w)
    for v, j in ((0, 0), (5, 7), (11, 15)):
        up, down = E64.copy(), E64.copy()
        up[v, j] += 0.5
        down[v, j] -= 0.5
        ref = ((oemb.forward(ids.numpy(), up, scale) - oemb.forward(ids.numpy(), down, scale)) * w64).sum()
        assert abs(got[v, j] - ref) <= 2.0 ** -8 * abs(ref) + 42 * 2.0 ** -24 * scale * np.abs(w64[:, j]).sum()
    assert np.all(got[3] == 0.0)


def test_graph_replay_and_another_stream():
    """A captured backward replays on new values of its inputs; two streams at once do not meet."""
    rng = np.random.default_rng(9)
    N, V, d = 9000, 4001, 256
    dOut, ids = bf16(rng, N, d).cuda(), torch.from_numpy(make_ids(rng, "zipf", N, V)).cuda()
    dE, ws = torch.empty((V, d), dtype=BF16, device="cuda"), api.Workspace()
    api.embedding_backward(dOut, ids, V, dE=dE, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.embedding_backward(dOut, ids, V, dE=dE, workspace=ws)
    new_ids = torch.from_numpy(make_ids(rng, "heavy", N, V))
    ids.copy_(new_ids)
    g.replay()
    torch.cuda.synchronize()
    check_grad(dOut.cpu(), new_ids.numpy(), V, 1.0, BF16, None, f64(dE))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            outs.append(api.embedding_backward(dOut, ids, V))
    torch.cuda.synchronize()
    assert all(torch.equal(o, dE) for o in outs)


def test_refusals():
    E, ids = torch.zeros(10, 16, dtype=BF16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dOut = torch.zeros(4, 16, dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        api.embedding_forward(ids.int(), E)
    with pytest.raises(TypeError):
        api.embedding_forward(ids, E.float())
    with pytest.raises(ValueError):
        api.embedding_forward(ids, E.t())
    with pytest.raises(_lib.LoraMLPError):
        api.embedding_forward(ids, E[:, :12].contiguous())    # 12 columns
    with pytest.raises(_lib.LoraMLPError):
        api.embedding_forward(ids[:0], E)                     # no tokens
    with pytest.raises(ValueError):
        api.embedding_backward(dOut, ids[:3], 10)
    with pytest.raises(ValueError):
        api.embedding_backward(dOut, ids, 10, padding_idx=10)
    with pytest.raises(TypeError):
        api.embedding_backward(dOut, ids, 10, dtype=torch.float16)
    with pytest.raises(_lib.LoraMLPError):
        api.embedding_backward(dOut, ids, 10, scale=float("nan"))
