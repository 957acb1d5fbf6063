"""The entry points of binding_cache reach the library with their tensors' device current, as test_current_device_cpu.py
has it for binding's."""
import inspect

import pytest
import torch

import test_current_device_cpu as base
from speculative_decoding_verification_verify_gb300 import binding_cache
from test_current_device_cpu import BF, CACHE, K, KW, Q, WS, now, t  # noqa: F401

F32 = torch.float32
ROWS = t(20, 80, dtype=torch.uint8)
OUT = dict(out=t(2, 3, 2, 64, dtype=BF))
CALLS = {
    "spec_verify_kv_append_ex": lambda f, c, kw: f(Q, K, K, c, c, t(2, 9), t(2), None, q_out=t(2, 3, 2, 64, dtype=BF),
                                                   q_norm=t(64, dtype=BF), **KW),
    "spec_verify_kv_read": lambda f, c, kw: f(c, c, t(2, 9), t(2), 3, head_dim=64, dtype=BF, k_out=t(2, 3, 1, 64, dtype=BF),
                                              v_out=t(2, 3, 1, 64, dtype=BF), **kw, **KW),
    "spec_verify_attention_chunk": lambda f, c, kw: f(Q, c, c, t(2, 9), t(2), lse=t(2, 3, 2, dtype=F32), **OUT, **WS, **kw,
                                                      **KW),
    "spec_verify_attention_e4m3": lambda f, c, kw: f(Q, ROWS, ROWS, t(2, 9), t(2), kv_heads=1, **OUT, **WS, **KW),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("rows", [False, True])
def test_the_tensors_device_is_current(now, monkeypatch, name, current, rows):  # noqa: F811
    monkeypatch.setattr(binding_cache, "spec_verify_kv_e4m3_row_bytes", lambda heads, dim: 80)
    now["device"] = current
    CALLS[name](getattr(binding_cache, name), ROWS if rows else CACHE, dict(kv_heads=1) if rows else {})
    assert now["seen"] == [(name, 1)]
    assert now["device"] == current


def test_no_entry_point_is_left_out():
    launching = {n for n, f in vars(binding_cache).items()
                 if n.startswith("spec_verify_") and "stream" in inspect.signature(f).parameters}
    assert launching == set(CALLS) and base.binding is binding_cache.b
