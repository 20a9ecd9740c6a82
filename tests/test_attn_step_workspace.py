"""The step helper's workspace on a cache in 8 bits: it grows with the table's width, and a smaller
one is kept only for a graph that was captured with it."""
import gc
import weakref

import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from gated_delta_rule_44_gb300 import layer

BF = torch.bfloat16


class Calls:
    """Stands for the library: workspaces in proportion to the table's width."""

    def __getattr__(self, name):
        if name == "gdn_attn8_paged_workspace_bytes":
            return lambda T, N, Hq, Hkv, D, mq, dt, width, page: 1000 * width
        if name.endswith("workspace_bytes"):
            return lambda *a: 64
        return lambda *a: 0


@pytest.fixture
def step(monkeypatch):
    fake, capturing = Calls(), [False]
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_lib", fake)
    monkeypatch.setattr(B, "_attn_call", lambda fn, q, s: None)
    monkeypatch.setattr(layer, "_capturing", lambda stream: capturing[0], raising=False)
    s = layer.AttnStep(4, 2, 0, 4, 2, 64, BF, torch.device("cpu"), max_q_len=4)

    def run(width, captured=False, eight=True):
        capturing[0] = captured
        q, k = torch.zeros(4, 4, 64, dtype=BF), torch.zeros(4, 2, 64, dtype=BF)
        kind = torch.float8_e4m3fn if eight else BF
        cache = torch.zeros(8, 2, 16, 64, dtype=torch.uint8 if eight else BF)
        cache = cache.view(kind) if eight else cache
        scales = dict(k_scale=torch.ones(8, 2, 1), v_scale=torch.ones(8, 2, 1)) if eight else {}
        cu = torch.tensor([0, 2, 4], dtype=torch.int32)
        s.run(q, k, k, cu, torch.tensor([9, 9], dtype=torch.int32), torch.zeros(2, width, dtype=torch.int32), cache, cache,
              cu_seqlens_prefill=cu, **scales)
        return weakref.ref(s.workspace), s.workspace.numel()
    return run


def alive(refs):
    gc.collect()
    return [r() is not None for r in refs]


def test_outgrown_workspaces_are_dropped(step):
    """A table that widens step by step: one workspace at a time."""
    seen = [step(w) for w in range(1, 40)]
    assert [n for _, n in seen] == [1000 * w for w in range(1, 40)]
    assert sum(alive([r for r, _ in seen])) == 1


@pytest.mark.parametrize("eight", [True, False])
def test_captured_workspaces_stay(step, eight):
    """Those that a graph was captured with are kept, and the next is at least twice as large."""
    first, n = step(3)
    if not eight:
        step(3, captured=True, eight=False)
    else:
        step(3, captured=True)
    second, m = step(4)
    assert m >= 2 * n
    third, o = step(100)
    assert o == 100000
    assert alive([first, second, third]) == [True, False, True]
    again, p = step(5, captured=True)      # fits
    assert again() is third() and p == o


def test_captures_at_growing_widths_are_bounded(step):
    """A graph for every width: what is kept beside the last workspace is no more than that."""
    sizes = {}
    for w in range(1, 200):
        r, n = step(w, captured=True)
        sizes[r] = n
    kept = [n for r, n in sizes.items() if alive([r])[0]]
    assert sum(kept) <= 2 * max(kept)


@pytest.mark.gpu
def test_memory_of_a_table_that_widens(cuda_device):
    """A prompt in chunks over a table as wide as its context so far: the memory in use is that of
    the last workspace, and steps on another stream leave nothing of an old one to overwrite."""
    dev, T, Hq, Hkv, D, page = cuda_device, 300, 8, 2, 128, 64
    g = torch.Generator(device=dev).manual_seed(1)
    pages = 600
    codes = [torch.randn(pages, Hkv, page, D, generator=g, device=dev).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = dict(k_scale=torch.ones(pages, Hkv, 2, device=dev), v_scale=torch.ones(pages, Hkv, 2, device=dev))
    q, k = (torch.randn(T, h, D, generator=g, device=dev).to(BF) for h in (Hq, Hkv))
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    table = torch.arange(pages, dtype=torch.int32, device=dev)[None]
    step = layer.AttnStep(T, 1, 0, Hq, Hkv, D, BF, dev, max_q_len=T)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def run(width, stream):
        kv = torch.tensor([width * page - 7], dtype=torch.int32, device=dev)
        torch.cuda.current_stream().synchronize()
        out = step.run(q, k, k, cu, kv, table[:, :width].contiguous(), *codes, cu_seqlens_prefill=cu, stream=stream, **scales)
        side.synchronize()
        return out.clone()

    before = torch.cuda.memory_allocated()
    for width in range(20, pages, 20):
        run(width, side if width % 40 else None)
        grown = torch.cuda.memory_allocated() - before
        assert grown <= step.workspace.numel() + (64 << 20), (width, grown)
    assert not step.outgrown
    B.gdn_read_device_status()
