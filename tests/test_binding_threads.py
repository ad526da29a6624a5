"""Host threads that share a stream: a call's kernels are enqueued as a whole, since they hand data
to one another through the stream's workspace (runs without a GPU, the library faked)."""
import threading
import time
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_verification_32_gb300 as sv
from speculative_decoding_verification_32_gb300 import _binding


class Launches:
    """Stands in for an entry point that takes a while to enqueue its kernels."""

    def __init__(self):
        self.inside, self.most, self.count, self.lock = 0, 0, 0, threading.Lock()

    def __call__(self, *args):
        with self.lock:
            self.inside += 1
            self.count += 1
            self.most = max(self.most, self.inside)
        time.sleep(0.002)  # other threads run, as they do during a foreign call
        with self.lock:
            self.inside -= 1
        return 0


@pytest.fixture
def launches(monkeypatch):
    calls = Launches()
    fake = SimpleNamespace(spec_verify_chain=calls, spec_verify_chain_truncated=calls, spec_verify_tree=calls,
                           spec_drift_residuals=calls, spec_verify_chain_workspace_size=lambda *a: 64,
                           spec_verify_chain_truncated_workspace_size=lambda *a: 64,
                           spec_verify_tree_workspace_size=lambda *a: 64)
    monkeypatch.setattr(_binding, "lib", lambda: fake)
    monkeypatch.setattr(_binding, "_fn", lambda name, nargs: calls)
    monkeypatch.setattr(_binding, "_kv_cache", lambda *a: (2, 8, 64, 1, 9, 1024, 1024, 16, 16))
    monkeypatch.setattr(_binding, "_capturing", lambda: False)
    monkeypatch.setattr(_binding, "_attention_bytes", lambda a: 64)
    monkeypatch.setattr(_binding, "_raw_stream", lambda index: 7)
    monkeypatch.setattr(_binding, "_stream", lambda device, stream: (SimpleNamespace(cuda_stream=7), 7))
    monkeypatch.setattr(_binding, "_ws", {})
    for name in ("_on", "_device"):
        monkeypatch.setattr(_binding, name, lambda *a: _binding._here)
    return calls


def attention():
    sv.spec_prefix_attention(torch.zeros(2, 3, 8, 64).bfloat16(), torch.zeros(2, 2, 9, 8, 64).bfloat16(),
                             torch.zeros(2, dtype=torch.int32))


def tree():
    sv.spec_verify_tree(torch.zeros(2, 3, 50), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32))


def chain():
    sv.spec_verify_chain(torch.zeros(2, 4, 50), torch.zeros(2, 3, 50), torch.zeros(2, 3, dtype=torch.int32),
                         u_accept=torch.zeros(2, 3), u_sample=torch.zeros(2, 4))


def truncated():
    sv.spec_verify_chain(torch.zeros(2, 4, 50), torch.zeros(2, 3, 50), torch.zeros(2, 3, dtype=torch.int32),
                         u_accept=torch.zeros(2, 3), u_sample=torch.zeros(2, 4), top_k=torch.ones(2, dtype=torch.int32))


def drift():
    sv.spec_drift_residuals(torch.zeros(2, 4, 50), torch.zeros(2, 3, 50), m=4)


@pytest.mark.parametrize("calls", [(attention,) * 4, (tree,) * 4, (chain, truncated, drift, chain)])
def test_calls_on_one_stream_are_enqueued_one_by_one(launches, calls):
    threads = [threading.Thread(target=lambda c=c: [c() for _ in range(10)]) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert launches.count == 40 and launches.most == 1


def test_a_call_within_a_call_does_not_wait_for_itself(launches, monkeypatch):
    """An allocation may run a finaliser, and that may make a call."""
    plain = _binding.workspace

    def workspace(*a):
        monkeypatch.setattr(_binding, "workspace", plain)
        tree()
        return plain(*a)
    monkeypatch.setattr(_binding, "workspace", workspace)
    t = threading.Thread(target=tree, daemon=True)
    t.start()
    t.join(20)
    assert not t.is_alive() and launches.count == 2
