"""How the calls around the attention layers are enqueued, without a GPU: the tensors' GPU is made the
current one for the call, and a stream of another GPU is refused."""
import contextlib

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


def test_the_tensors_gpu_is_current(monkeypatch):
    now, seen = [0], []

    @contextlib.contextmanager
    def device(index):
        old, now[0] = now[0], index
        yield
        now[0] = old

    monkeypatch.setattr(gdn, "_this_gpu", lambda: now[0])
    monkeypatch.setattr(gdn, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    gdn._launch("x", lambda queue: seen.append((queue, now[0])), 0, None)
    gdn._launch("x", lambda queue: seen.append((queue, now[0])), 2, None)
    gdn._launch("x", lambda queue: seen.append((queue, now[0])), 2, Stream(2))
    assert seen == [(1000, 0), (1002, 2), (77, 2)] and now == [0]
    with pytest.raises(ValueError, match="stream"):
        gdn._launch("x", lambda queue: seen.append(queue), 0, Stream(1))
    with pytest.raises(gdn.GdnError, match="x: "):
        gdn._launch("x", lambda queue: 2, 2, None)
    assert len(seen) == 3 and now == [0]
