"""spec_verify_reset_workspaces forgets the buffers of every entry point that keeps some.  Buffers lie on the host."""
import inspect

import pytest
import torch

import speculative_decoding_verification_verify_gb300 as sv
from speculative_decoding_verification_verify_gb300 import binding, binding_cache

KEPT = ["_workspaces", "_plan_workspaces", "_chunk_workspaces"]


@pytest.mark.parametrize("name", KEPT)
def test_all_are_forgotten(monkeypatch, name):
    monkeypatch.setattr(binding, "_capture_id", lambda device, stream, raw: 0)
    for other in KEPT:
        monkeypatch.setattr(binding, other, binding._Workspaces(torch.zeros))
    a = getattr(binding, name).get(100, "cpu", None, 5)
    assert getattr(binding, name).get(100, "cpu", None, 5) is a
    sv.spec_verify_reset_workspaces()
    assert getattr(binding, name).get(100, "cpu", None, 5) is not a


def test_no_other_is_kept():
    for module in (binding, binding_cache):
        assert {n for n, x in vars(module).items() if isinstance(x, binding._Workspaces)} <= set(KEPT)
    assert "_chunk_workspaces.get(" in inspect.getsource(binding_cache.spec_verify_attention_chunk)
