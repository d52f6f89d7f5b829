"""The embedding's gradient where runs of equal ids meet the chunks that the sorted tokens are cut into (32 tokens):
lengths around one and two chunks, at every offset to the chunks' borders, and borders between a run and the tokens
that take no part.

Tolerance as in test_gpu_embedding.py: n terms in fp32, (n + 2) 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from lora_fine_tuning_mlp_b200 import api
from lora_fine_tuning_mlp_b200 import build as libbuild
from oracle import embedding as oemb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    api.step_device_status()


def run(lengths, d, padding_idx=None, seed=0):
    """Ids 0, 1, ... with `lengths` tokens each, in any order."""
    rng = np.random.default_rng(seed)
    ids = rng.permutation(np.repeat(np.arange(len(lengths)), lengths))
    V = len(lengths) + 1
    dOut = torch.from_numpy(rng.standard_normal((len(ids), d)).astype(np.float32)).to(torch.bfloat16)
    got = api.embedding_backward(dOut.cuda(), torch.from_numpy(ids).cuda(), V, dtype=torch.float32,
                                 padding_idx=padding_idx).double().cpu().numpy()
    ref, mag, n = oemb.backward(dOut.double().numpy(), ids, V, 1.0, padding_idx)
    assert np.all(np.abs(got - ref) <= (n[:, None] + 2) * 2.0 ** -24 * mag)
    assert np.all(got[n == 0] == 0.0)


@pytest.mark.parametrize("d", [8, 264, 1032, 4104])
@pytest.mark.parametrize("first", [0, 1, 15, 31, 32, 33])
def test_runs_around_whole_chunks(first, d):
    """The tokens before a run shift it against the chunks."""
    for n in (1, 31, 32, 33, 63, 64, 65, 95, 96, 97):
        run(([first] if first else []) + [n, 3], d, seed=n)


@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65])
def test_runs_at_the_end_of_the_tokens(n):
    run([5, n], 72)
    run([n], 72)


@pytest.mark.parametrize("N", [8192, 8193])
def test_many_runs_of_each_length(N):
    """The largest number of tokens that one block sorts, and one more."""
    lengths = [n for n in (31, 32, 33, 63, 64, 65, 1, 2) for _ in range(28)]
    lengths += [N - sum(lengths)]
    run(lengths, 40)


@pytest.mark.parametrize("n", [31, 32, 33, 64, 65])
def test_padding_behind_a_run(n):
    """Tokens that take no part are sorted behind all others."""
    run([n, 40, n], 264, padding_idx=1)
    run([n, 40], 264, padding_idx=1)
    run([n], 264, padding_idx=0)
