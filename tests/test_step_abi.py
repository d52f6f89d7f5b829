"""Host-side checks of the operators around the dense layers (lora_step.h and
the headers that include it): the binding covers the headers, sizes are what
the kernels need, bad arguments are refused with the documented codes, and the
Python entry points take no host tensors.  No GPU."""
import os
import re

import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = ("lora_step.h", "lora_embedding.h")
FAKE = 0x10000  # aligned, never dereferenced: no device owns it, so the last check refuses it
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def L():
    libbuild.build()
    return _lib.lib()


def test_binding_covers_the_headers(L):
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in HEADERS)
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(lora_(?:step|embedding|qk|distill)_\w+)\s*\(", text)))
    assert names == sorted(_lib.STEP_SYMBOLS)
    for name in names:
        assert hasattr(L, name), name


def test_timing_and_counts_without_gpu(L):
    _lib.timing_enable(True)
    _lib.timing_enable(False)
    assert _lib.timing_collect() == [] and _lib.launch_count() == 0
    assert L.lora_step_device_status(None, None) == _lib.ERR_INVALID_ARG


# ----------------------------------------------------------------------------- embedding


def code_of(fn, *args):
    with pytest.raises(_lib.LoraMLPError) as e:
        fn(*args)
    return e.value.code


def test_embedding_sizes():
    # sorted ids and tokens, twice, and fp32 sums of whole 64-token chunks
    assert _lib.embedding_sizes(4096, 128256, 4096) >= 4 * 4096 * 4 + 64 * 4096 * 4
    assert _lib.embedding_sizes(1, 1, 8) > 0
    assert _lib.embedding_sizes(65536, 32000, 2048) > _lib.embedding_sizes(8192, 32000, 2048)
    assert code_of(_lib.embedding_sizes, 0, 10, 8) == _lib.ERR_INVALID_ARG
    assert code_of(_lib.embedding_sizes, 4, 0, 8) == _lib.ERR_INVALID_ARG
    assert code_of(_lib.embedding_sizes, 4, 10, 12) == _lib.ERR_UNSUPPORTED_SHAPE
    assert code_of(_lib.embedding_sizes, 2 ** 30 + 1, 10, 8) == _lib.ERR_UNSUPPORTED_SHAPE
    assert code_of(_lib.embedding_sizes, 4, 2 ** 31 - 1, 8) == _lib.ERR_UNSUPPORTED_SHAPE


def test_embedding_argument_errors():
    fwd = _lib.embedding_forward
    assert fwd(4, 10, 12, 1.0, FAKE, FAKE, FAKE, None) == _lib.ERR_UNSUPPORTED_SHAPE
    assert fwd(4, 10, 16, float("inf"), FAKE, FAKE, FAKE, None) == _lib.ERR_INVALID_ARG
    assert fwd(4, 10, 16, 1.0, None, FAKE, FAKE, None) == _lib.ERR_INVALID_ARG
    assert fwd(4, 10, 16, 1.0, FAKE + 4, FAKE, FAKE, None) == _lib.ERR_MISALIGNED
    assert fwd(4, 10, 16, 1.0, FAKE, FAKE + 8, FAKE, None) == _lib.ERR_MISALIGNED
    assert fwd(4, 10, 16, 1.0, FAKE, FAKE, FAKE, None) == _lib.ERR_INVALID_ARG   # no device's memory
    bwd = _lib.embedding_backward
    ws = _lib.embedding_sizes(4, 10, 16)
    assert bwd(4, 10, 16, 1.0, -1, 2, FAKE, FAKE, FAKE, FAKE, ws, None) == _lib.ERR_INVALID_ARG
    assert bwd(4, 10, 16, 1.0, -1, 0, FAKE, FAKE, FAKE, FAKE, ws - 1, None) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert bwd(4, 10, 16, 1.0, -1, 0, FAKE, FAKE, None, FAKE, ws, None) == _lib.ERR_INVALID_ARG
    assert bwd(4, 10, 16, 1.0, -1, 1, FAKE, FAKE + 2, FAKE, FAKE, ws, None) == _lib.ERR_MISALIGNED


def test_embedding_refuses_host_tensors():
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises((ValueError, TypeError), match="CUDA"):
        api.embedding_forward(ids, torch.zeros(10, 16, dtype=BF16))
    with pytest.raises((ValueError, TypeError), match="CUDA"):
        api.embedding_backward(torch.zeros(4, 16, dtype=BF16), ids, 10)
