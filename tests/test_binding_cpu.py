"""What the Python binding does around the library's calls (devices faked: no GPU)."""
import contextlib
import types

import pytest
import torch

import rank_joint_qkv_b200 as q


def tensor(index):
    return types.SimpleNamespace(is_cuda=index is not None, device=types.SimpleNamespace(index=index))


@pytest.fixture
def device(monkeypatch):
    now = [0]

    @contextlib.contextmanager
    def on(d):
        now.append(d.index)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(q, "_several_devices", lambda: True)
    return now


def test_a_call_runs_on_its_tensors_device(device):
    """The library launches on the current device: its kernels would be given another GPU's memory."""
    ran = q._on_the_tensors_device(lambda *a, **k: device[-1])
    assert ran("dims", tensor(None), tensor(1), tensor(0)) == 1
    assert ran("dims", None, cache=tensor(1)) == 1
    assert ran("dims", tensor(0)) == 0 and ran("dims") == 0
    assert ran("dims", tensor(0), stream=tensor(1)) == 1    # the stream says where
    assert ran("dims", tensor(1), stream=None) == 1
    assert device == [0]


def test_every_call_is_made_that_way():
    calls = [n for n in q._sigs if n != "qsvd_testing_set_score_wait_ns"]
    assert all(getattr(q, n).on_the_tensors_device for n in calls)


def test_one_gpu_needs_no_choice(monkeypatch):
    monkeypatch.setattr(q, "_several_devices", lambda: False)
    call = lambda: None  # noqa: E731
    assert q._on_the_tensors_device(call) is call


def test_an_error_leaves_the_current_device(device):
    def fails(*a, **k):
        raise q.QsvdError(q.QSVD_ERR_INVALID_ARG, "here")
    with pytest.raises(q.QsvdError):
        q._on_the_tensors_device(fails)(tensor(1))


def test_eviction_in_place_takes_no_destinations_sizes():
    d = q.make_dims(64, 1, 64, 64, 1, 100, cache="f16")
    t = torch.zeros(1)
    for extra in (dict(dst_max_len=50), dict(dst_scales=t)):
        with pytest.raises(ValueError, match="need dst_cache"):
            q.qsvd_evict_rows(d, t, t, 10, t, **extra)
