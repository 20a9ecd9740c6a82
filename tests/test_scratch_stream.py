"""A workspace that a call allocates for itself belongs to the stream the call is
given: the allocator may otherwise hand out memory on which kernels of the current
stream are still pending."""
import contextlib

import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B


class FakeLib:
    """Stands for the library: sizes, and calls that only note their name."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        return lambda *a: self.called.append(name) or 0


class FakeStream:
    cuda_stream = 7


@pytest.fixture
def watched(monkeypatch):
    """The stream that is current at each allocation of 4096 bytes."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty

    def noting(*a, **kw):
        if a[0] == 4096:
            seen.append(current[-1])
        return empty(*a, **kw)

    fake = FakeLib()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_lib", fake)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", noting)
    monkeypatch.setattr(B, "_attn_call", lambda fn, q, s: fn(0, s))
    return seen


def paged(stream):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    B.gdn_attn_paged(q, kc, kc, torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32),
                     None, torch.zeros_like(q), stream=stream)


def kda(stream):
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    B.gdn_kda_varlen(x, x, x, torch.zeros(2, 2, 128), torch.zeros(2, 2), torch.zeros(1, 2, 128, 128),
                     torch.tensor([0, 2], dtype=torch.int32), torch.zeros_like(x), stream=stream)


@pytest.mark.parametrize("call", [paged, kda])
def test_allocated_on_the_calls_stream(call, watched):
    s = FakeStream()
    call(s)
    assert watched == [s]


@pytest.mark.gpu
def test_paged_leaves_pending_memory_alone(cuda_device):
    """A block freed while a kernel of the current stream still has to read it is not
    the scratch of a call on another stream."""
    dev, N, D = cuda_device, 16, 128
    g = torch.Generator().manual_seed(9)
    q = torch.randn(N, 8, D, generator=g).to(torch.bfloat16).to(dev)
    kc = torch.randn(N * 32, 2, 16, D, generator=g).to(torch.bfloat16).to(dev)
    table = torch.arange(N * 32, dtype=torch.int32, device=dev).view(N, 32)
    kv = torch.full((N,), 500, dtype=torch.int32, device=dev)
    eager, out = torch.empty_like(q), torch.empty_like(q)
    nbytes = B.gdn_attn_paged_workspace_bytes(N, N, 8, 2, D, 0)
    assert nbytes > 0
    B.gdn_attn_paged(q, kc, kc, table, kv, None, eager)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    block = torch.full((nbytes,), 5, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)       # about 0.1 s on the current stream
    kept.copy_(block)
    del block
    B.gdn_attn_paged(q, kc, kc, table, kv, None, out, stream=side)
    torch.cuda.synchronize()
    B.gdn_read_device_status()
    assert (kept == 5).all()
    assert torch.equal(out, eager)
