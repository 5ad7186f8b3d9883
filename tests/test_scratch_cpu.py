"""Where the binding's own scratch comes from (streams faked: no GPU)."""
import contextlib

import pytest
import torch

import rank_joint_qkv_b200 as q


class Stream:
    def __init__(self, name):
        self.cuda_stream = self.name = name


@pytest.fixture
def streams(monkeypatch):
    """current, side; every allocation notes the stream that is current then and the streams it is kept for."""
    current, side = Stream("current"), Stream("side")
    now, made = [current], []

    class Block:
        def __init__(self):
            self.pool, self.kept_for = now[-1], []
            made.append(self)

        def record_stream(self, s):
            self.kept_for.append(s)

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Block())
    return current, side, made


def test_scratch_comes_from_the_calls_stream(streams):
    """A block of the current stream's pool may still be in use there when a call on another stream writes it."""
    current, side, made = streams
    assert q._scratch(10, "cuda", side).pool is side and made[0].kept_for == [current]
    assert q._scratch(10, "cuda", current).pool is current and made[1].kept_for == []
    assert q._scratch(10, "cuda", None).pool is current and made[2].kept_for == []


def test_any_holder_of_a_stream_will_do(streams, monkeypatch):
    current, side, made = streams
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(("external", handle)))

    class Holder:
        cuda_stream = 77

    q._scratch(10, "cuda", Holder())
    assert made[0].pool.name == ("external", 77)
