"""Which buffer a call without a workspace gets: one per stream outside graph capture, and one per capture
within.  The captures are made up; buffers lie on the host."""
import torch

from speculative_decoding_verification_verify_gb300 import binding


def kept(monkeypatch, make=torch.zeros):
    now = dict(capture=0)
    monkeypatch.setattr(binding, "_capture_id", lambda device, stream, raw: now["capture"])
    return binding._Workspaces(make), now


def test_a_capture_has_its_own(monkeypatch):
    w, now = kept(monkeypatch)
    a = w.get(100, "cpu", None, 5)
    assert a.numel() >= 100 and not a.any()
    now["capture"] = 7
    b = w.get(100, "cpu", None, 5)
    assert b is not a and w.get(50, "cpu", None, 5) is b
    b.fill_(1)  # what a graph's calls left there is not another graph's beginning
    now["capture"] = 8
    c = w.get(100, "cpu", None, 5)
    assert c is not a and c is not b and not c.any()
    assert w.get(100, "cpu", None, 6) is not c  # a second stream of the same capture
    now["capture"] = 0
    assert w.get(100, "cpu", None, 5) is a  # no graph's buffer outside, no other stream's


def test_a_larger_need_outside_leaves_captures_alone(monkeypatch):
    w, now = kept(monkeypatch)
    a = w.get(100, "cpu", None, 5)
    now["capture"] = 7
    b = w.get(100, "cpu", None, 5)
    now["capture"] = 0
    big = w.get(a.numel() + 1, "cpu", None, 5)
    assert big is not a and big.numel() > a.numel() and w.get(1, "cpu", None, 5) is big
    now["capture"] = 7
    assert w.get(100, "cpu", None, 5) is b
    assert w.get(b.numel() + 1, "cpu", None, 5).numel() > b.numel()


def test_streams_and_devices_do_not_share(monkeypatch):
    w, _ = kept(monkeypatch)
    a = w.get(1, "cpu", None, 5)
    assert w.get(1, "cpu", None, 6) is not a
    assert w.get(1, torch.device("cpu"), None, 5) is not a


def test_the_planner_keeps_apart():
    assert binding._plan_workspaces is not binding._workspaces


def test_capture_id_on_the_host(monkeypatch):
    from speculative_decoding_verification_verify_gb300 import _build

    _build.build()
    assert binding.load_library().spec_verify_capture_id(None, None) == binding.EINVAL
    assert binding._capture_id(0, None, 0) == 0


def test_forgetting_gives_new_zeros(monkeypatch):
    w, _ = kept(monkeypatch)
    monkeypatch.setattr(binding, "_workspaces", w)
    a = w.get(100, "cpu", None, 5)
    a.fill_(1)  # what a wait that ran out leaves behind
    assert w.get(100, "cpu", None, 5) is a
    binding.spec_verify_reset_workspaces()
    b = w.get(100, "cpu", None, 5)
    assert b is not a and not b.any()
