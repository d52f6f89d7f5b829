"""Host-side checks of the operators around the dense layers (lora_step.h and
the headers that include it): the binding covers the headers, sizes are what
the kernels need, bad arguments are refused with the documented codes, and the
Python entry points take no host tensors.  No GPU."""
import ctypes
import os
import re

import pytest
import torch

from lora_fine_tuning_mlp_b200 import _lib, api
from lora_fine_tuning_mlp_b200 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = ("lora_step.h", "lora_embedding.h", "lora_qk_rope.h", "lora_distill.h")
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


# ----------------------------------------------------------------------------- queries' and keys' norm and rotation


def qk_shape(B=2, S=5, Hq=4, Hk=2, D=64, rot=64, P=100, stride=5, eps=1e-6, interleaved=0):
    return _lib.QKShape(B, S, Hq, Hk, D, rot, P, stride, eps, interleaved)


def view(data=FAKE, sb=1280, ss=256, sh=64):
    return _lib.QKView(data, sb, ss, sh)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), _lib.ERR_INVALID_ARG),
    (dict(S=-1), _lib.ERR_INVALID_ARG),
    (dict(Hk=0), _lib.ERR_INVALID_ARG),
    (dict(P=0), _lib.ERR_INVALID_ARG),
    (dict(rot=80), _lib.ERR_INVALID_ARG),             # more than the head
    (dict(eps=-1.0), _lib.ERR_INVALID_ARG),
    (dict(eps=float("inf")), _lib.ERR_INVALID_ARG),
    (dict(stride=-1), _lib.ERR_INVALID_ARG),
    (dict(D=72), _lib.ERR_UNSUPPORTED_SHAPE),
    (dict(rot=40), _lib.ERR_UNSUPPORTED_SHAPE),
    (dict(D=528), _lib.ERR_UNSUPPORTED_SHAPE),
    (dict(B=2 ** 20, S=2 ** 20), _lib.ERR_UNSUPPORTED_SHAPE),
])
def test_qk_shape_validation(L, kw, code):
    ws = ctypes.c_size_t()
    assert L.lora_qk_rope_sizes(ctypes.byref(qk_shape(**kw)), ctypes.byref(ws)) == code


def test_qk_argument_errors():
    def fwd(sh=None, q=None, out=None, gains=(None, None), cos=FAKE, pos=None):
        return _lib.qk_rope_forward(sh or qk_shape(), q or view(), view(), *gains, cos, FAKE, pos, out or view(),
                                    view(), None)

    assert fwd(gains=(FAKE, None)) == _lib.ERR_INVALID_ARG
    assert fwd(q=view(None)) == _lib.ERR_INVALID_ARG
    assert fwd(q=view(FAKE + 8)) == _lib.ERR_MISALIGNED
    assert fwd(q=view(ss=260)) == _lib.ERR_UNSUPPORTED_SHAPE
    assert fwd(out=view(sh=4)) == _lib.ERR_UNSUPPORTED_SHAPE
    assert fwd(cos=None) == _lib.ERR_INVALID_ARG
    assert fwd(cos=FAKE + 4) == _lib.ERR_MISALIGNED
    assert fwd(pos=FAKE + 4) == _lib.ERR_MISALIGNED
    assert fwd(sh=qk_shape(S=101)) == _lib.ERR_INVALID_ARG      # no positions, and a table of 100
    assert fwd() == _lib.ERR_INVALID_ARG                        # no device's memory

    ws = _lib.qk_rope_sizes(qk_shape())

    def bwd(gains=(FAKE, FAKE), dgains=(FAKE, FAKE), q=None, work=FAKE, nbytes=ws):
        return _lib.qk_rope_backward(qk_shape(), q or view(), view(), *gains, FAKE, FAKE, None, view(), view(), view(),
                                     view(), *dgains, work, nbytes, None)

    assert bwd(gains=(None, None)) == _lib.ERR_INVALID_ARG      # gradients of gains that are not there
    assert bwd(dgains=(FAKE, None)) == _lib.ERR_INVALID_ARG
    assert bwd(dgains=(FAKE + 2, FAKE)) == _lib.ERR_MISALIGNED
    assert bwd(nbytes=ws - 1) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert bwd(work=None) == _lib.ERR_INVALID_ARG
    assert bwd(q=view(None)) == _lib.ERR_INVALID_ARG


# ----------------------------------------------------------------------------- distillation


def ds_shape(N=4, V=100, ld=104, K=8, T=1.0, s=1.0, cap=0.0, vt=1, it=1):
    return _lib.DistillShape(N, V, ld, K, T, s, cap, vt, it, -100)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), _lib.ERR_INVALID_ARG),
    (dict(V=0), _lib.ERR_INVALID_ARG),
    (dict(K=0), _lib.ERR_INVALID_ARG),
    (dict(ld=96), _lib.ERR_INVALID_ARG),
    (dict(T=0.0), _lib.ERR_INVALID_ARG),
    (dict(T=-1.0), _lib.ERR_INVALID_ARG),
    (dict(T=1e-39), _lib.ERR_INVALID_ARG),           # 1 / T is out of fp32's range
    (dict(cap=1e-39), _lib.ERR_INVALID_ARG),
    (dict(s=1e20, T=1e-20), _lib.ERR_INVALID_ARG),
    (dict(T=float("inf")), _lib.ERR_INVALID_ARG),
    (dict(s=0.0), _lib.ERR_INVALID_ARG),
    (dict(cap=-2.0), _lib.ERR_INVALID_ARG),
    (dict(vt=2), _lib.ERR_INVALID_ARG),
    (dict(it=-1), _lib.ERR_INVALID_ARG),
    (dict(ld=100), _lib.ERR_UNSUPPORTED_SHAPE),
    (dict(K=1025), _lib.ERR_UNSUPPORTED_SHAPE),
    (dict(V=327681, ld=327688), _lib.ERR_UNSUPPORTED_SHAPE),
])
def test_distill_shape_validation(L, kw, code):
    ws = ctypes.c_size_t()
    assert L.lora_distill_sizes(ctypes.byref(ds_shape(**kw)), ctypes.byref(ws)) == code


def test_distill_argument_errors():
    sh = ds_shape()
    ws = _lib.distill_sizes(sh)
    assert ws >= 4 * 4
    fwd = _lib.distill_forward
    assert fwd(sh, None, FAKE, FAKE, None, FAKE, None) == _lib.ERR_INVALID_ARG
    assert fwd(sh, FAKE + 8, FAKE, FAKE, None, FAKE, None) == _lib.ERR_MISALIGNED
    assert fwd(sh, FAKE, FAKE + 2, FAKE, None, FAKE, None) == _lib.ERR_MISALIGNED      # fp32 values
    assert fwd(sh, FAKE, FAKE, FAKE + 4, None, FAKE, None) == _lib.ERR_MISALIGNED      # int64 ids
    assert fwd(sh, FAKE, FAKE, FAKE, FAKE + 4, FAKE, None) == _lib.ERR_MISALIGNED      # labels
    assert fwd(sh, FAKE, FAKE, FAKE, None, FAKE, None) == _lib.ERR_INVALID_ARG         # no device's memory
    bwd = _lib.distill_backward
    assert bwd(sh, FAKE, FAKE, FAKE, None, None, FAKE, None) == _lib.ERR_INVALID_ARG
    assert bwd(sh, FAKE, FAKE, FAKE, None, FAKE, FAKE + 2, None) == _lib.ERR_MISALIGNED
    red = _lib.distill_backward_reduced
    assert red(sh, FAKE, FAKE, FAKE, None, FAKE, FAKE + 4, FAKE, None) == _lib.ERR_MISALIGNED
    loss = _lib.distill_loss
    assert loss(sh, FAKE, FAKE, FAKE, None, 0, FAKE, None, FAKE, ws, None) == _lib.ERR_INVALID_ARG
    assert loss(sh, FAKE, FAKE, FAKE, None, 2, FAKE + 4, None, FAKE, ws, None) == _lib.ERR_MISALIGNED
    assert loss(sh, FAKE, FAKE, FAKE, None, 2, FAKE, None, FAKE, ws - 1, None) == _lib.ERR_WORKSPACE_TOO_SMALL
    assert loss(sh, FAKE, FAKE, FAKE, None, 2, FAKE, FAKE + 8, FAKE, ws, None) == _lib.ERR_MISALIGNED


def test_qk_and_distill_refuse_host_tensors():
    q = torch.zeros(1, 2, 2, 64, dtype=BF16)
    cos = torch.zeros(4, 32)
    with pytest.raises((ValueError, TypeError), match="CUDA"):
        api.qk_norm_rope_forward(q, q, cos, cos)
    with pytest.raises((ValueError, TypeError), match="CUDA"):
        api.distill_forward(torch.zeros(2, 64, dtype=BF16), torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int64))


def test_rope_table_keeps_far_angles():
    """The table's angles are formed in fp64: at position 10^6 the first pair's sine is right to fp32."""
    cos, sin = api.rope_table(1_000_001, 16, base=10000.0)
    import math
    for p in (1, 999_999, 1_000_000):
        for i in range(8):
            a = p * 10000.0 ** (-2 * i / 16)
            assert abs(float(sin[p, i]) - math.sin(a)) <= 2.0 ** -24 + 1e-9
            assert abs(float(cos[p, i]) - math.cos(a)) <= 2.0 ** -24 + 1e-9
    with pytest.raises(ValueError):
        api.rope_table(4, 15)
