"""Every entry point reaches the library with its tensors' device current.  The second device, the streams and
the library are made up: nothing is launched."""
import contextlib
import types

import pytest
import torch

from speculative_decoding_verification_verify_gb300 import binding


class OnOne(torch.Tensor):
    """A host tensor that says that it lies on cuda:1."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda:1"))

    def get_device(self):
        return 1


def t(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnOne)


@pytest.fixture()
def now(monkeypatch):
    state = dict(device=0, seen=[])

    @contextlib.contextmanager
    def enter(device):
        before, state["device"] = state["device"], device
        try:
            yield
        finally:
            state["device"] = before

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                if name.endswith("_bytes"):
                    return 1024
                state["seen"].append((name, state["device"]))
                return 0
            return entry

    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_current_device", lambda: state["device"])
    monkeypatch.setattr(binding.torch.cuda, "device", enter)
    monkeypatch.setattr(binding, "_plan_workspaces", types.SimpleNamespace(get=lambda *a: t(8)))
    return state


BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
STREAM = types.SimpleNamespace(cuda_stream=5)
KW = dict(stream=STREAM)
WS = dict(workspace=t(8, dtype=torch.uint8), dev_status=t(1))
OUT = dict(out_tokens=t(2, 3), accept_len=t(2))
RNG = dict(temperature=1.0, seed=0, offset=0)
X, D = t(2, 3, 9, dtype=BF), t(2, 2)
CACHE = t(20, 1, 64, dtype=BF)
Q = t(2, 3, 2, 64, dtype=BF)
K = t(2, 3, 1, 64, dtype=BF)
TREE = dict(out_tokens=t(2, 3), accept_index=t(2, 3), accept_len=t(2))
CALLS = {
    "spec_verify_greedy": lambda f: f(X, D, **OUT, **WS, **KW),
    "spec_verify_rejection": lambda f: f(X, D, **RNG, **OUT, **WS, **KW),
    "spec_verify_block": lambda f: f(X, D, **RNG, **OUT, **WS, **KW),
    "spec_verify_rejection_ex": lambda f: f(X, D, **OUT, **WS, **KW),
    "spec_verify_rejection_noalloc": lambda f: f(X, D, **RNG, **OUT, **KW),
    "spec_verify_tree": lambda f: f(X, t(2, 3), t(2, 3), mode=0, **TREE, **WS, **KW),
    "spec_verify_tree_ex": lambda f: f(X, t(2, 3), t(2, 3), **TREE, **WS, **KW),
    "spec_verify_kv_compact": lambda f: f(CACHE, t(2, 9), t(2), t(2, 3), t(2), committed_out=t(2), dev_status=t(1), **KW),
    "spec_verify_plan_budget": lambda f: f(t(2, 2, dtype=F32), t(5, dtype=F64), admitted=t(2), budget=t(1),
                                           best_rate=t(1, dtype=F64), **KW),
    "spec_verify_philox": lambda f: f(1, 2, 3, 4, out=t(3, 4, 4), device="cuda:1", **KW),
    "spec_verify_kv_append": lambda f: f(Q, K, K, CACHE, CACHE, t(2, 9), t(2), None, q_out=t(2, 3, 2, 64, dtype=BF), **KW),
    "spec_verify_attention": lambda f: f(Q, CACHE, CACHE, t(2, 9), t(2), out=t(2, 3, 2, 64, dtype=BF), **WS, **KW),
    "spec_verify_logprobs": lambda f: f(X, t(2, 3), logprobs=t(2, 3, dtype=F32), entropy=t(2, 3, dtype=F32), ranks=t(2, 3),
                                        **WS, **KW),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current(now, name, current):
    now["device"] = current
    CALLS[name](getattr(binding, name))
    assert now["seen"] == [(name, 1)]
    assert now["device"] == current


def test_captures_are_looked_up_on_the_streams_device(now, monkeypatch):
    monkeypatch.setattr(binding.torch.cuda, "is_current_stream_capturing", lambda: False)
    binding._capture_id(1, None, 5)  # the current stream of a device that is not current
    binding._capture_id(0, None, 5)  # of the current one: torch has said no
    assert now["seen"] == [("spec_verify_capture_id", 1)]


def test_no_entry_point_is_left_out():
    import inspect

    launching = {n for n, f in vars(binding).items()
                 if n.startswith("spec_verify_") and "stream" in inspect.signature(f).parameters}
    assert launching == set(CALLS)
