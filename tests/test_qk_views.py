"""Which written views the norm and rotation of queries and keys refuses on the host: those that overlap themselves.
No GPU: FAKE is an address that no device owns, which the last check refuses with another code."""
import pytest

from lora_fine_tuning_mlp_b200 import _lib
from lora_fine_tuning_mlp_b200 import build as libbuild

FAKE = 0x10000
B, S, H, D = 2, 5, 4, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()


def view(sb, ss, sh, data=FAKE):
    return _lib.QKView(data, sb, ss, sh)


def codes(written, B=B, S=S, H=H):
    """Of the forward and the backward with `written` as each of their results."""
    shape = _lib.QKShape(B, S, H, H, D, D, 100, 0, 1e-6, 0)
    ok = [view(S * H * D, H * D, D, FAKE * (i + 2)) for i in range(4)]
    return {_lib.qk_rope_forward(shape, *ok[:2], None, None, FAKE, FAKE, None, written, ok[2], None),
            _lib.qk_rope_forward(shape, *ok[:2], None, None, FAKE, FAKE, None, ok[2], written, None),
            _lib.qk_rope_backward(shape, None, None, None, None, FAKE, FAKE, None, *ok[:2], written, ok[2], None, None,
                                  None, 0, None),
            _lib.qk_rope_backward(shape, None, None, None, None, FAKE, FAKE, None, *ok[:2], ok[2], written, None, None,
                                  None, 0, None)}


@pytest.mark.parametrize("strides", [
    (S * H * D, H * D, 8),           # heads eight elements apart
    (S * H * D, H * D, 0),
    (S * H * D, H * D, 56),
    (S * H * D, H * D - 8, D),       # a position's last head in the next one's first
    (S * H * D - 8, H * D, D),       # sequences
    (8, H * D, D),
    (S * H * D, H * D, -8),          # strides below zero
    (H * S * D, D, S * D - 8),       # heads first
    (2 ** 61, 2 ** 60, 2 ** 59),     # spans past 64 bits do not wrap
])
def test_overlapping_results_are_refused(strides):
    assert codes(view(*strides)) == {_lib.ERR_UNSUPPORTED_SHAPE}


@pytest.mark.parametrize("strides", [
    (S * H * D, H * D, D),
    (H * S * D, D, S * D),           # heads first
    (H * 40 * D, D, 40 * D),         # a part of a longer cache
    (D, B * H * D, B * D),           # sequences innermost
    (S * H * D, H * D, -D),
    (2 ** 62, 2 ** 59, 2 ** 57),
])
def test_others_are_not(strides):
    assert codes(view(*strides)) == {_lib.ERR_INVALID_ARG}


def test_strides_of_single_entries_do_not_matter():
    assert codes(view(0, 0, 0), B=1, S=1, H=1) == {_lib.ERR_INVALID_ARG}
    assert codes(view(8, 0, D), B=1, S=1) == {_lib.ERR_INVALID_ARG}
