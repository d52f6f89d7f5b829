"""The current stream's address without torch's private names, which another version may lack."""
import torch

from lora_fine_tuning_mlp_b200 import api


class Stream:
    cuda_stream = 0x1230


def test_the_public_way_stands_in(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    for missing in ("_raw_stream", "_current_device"):
        with monkeypatch.context() as m:
            m.setattr(api, missing, None)
            assert api._stream(None) == 0x1230
    monkeypatch.setattr(api, "_raw_stream", lambda d: 0x4560 + d)
    monkeypatch.setattr(api, "_current_device", lambda: 3)
    assert api._stream(None) == 0x4563 and api._stream(Stream) == 0x1230
