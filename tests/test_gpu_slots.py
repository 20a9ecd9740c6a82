"""GPU: gdn_copy_slots, byte for byte against indexing."""
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B

pytestmark = pytest.mark.gpu


def make_pools(g, slots, dev):
    """Pools of several types, sizes and strides (some not in 16-byte units)."""
    def r(*shape):
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
    wide = r(slots, 5 * 4096).to(dev)
    joint = r(slots, 2, 96 * 16).to(dev)
    return [
        r(slots, 3 * 65536).to(dev).view(torch.float32).view(slots, 3, 128, 128),   # pieces of a slot
        r(slots, 48).to(dev).view(torch.int32),
        r(slots, 20).to(dev).view(torch.float32),                                   # words
        r(slots, 4).to(dev),
        wide[:, 4096:4096 * 2 + 16],                                                # strided slots
        wide[:, :4092],                                                             # strided words
        joint[:, 0].view(torch.bfloat16), joint[:, 1],
        r(slots + 9, 40976).to(dev).view(torch.float8_e4m3fn),                      # more slots, a ragged piece
    ]


def want_of(pools, dst, src):
    out = []
    for p in pools:
        b = p.clone().view(torch.uint8) if p.is_contiguous() else p.clone().contiguous().view(torch.uint8)
        new = b.clone()
        for d, s in zip(dst, src):
            new[d] = b[s]
        out.append(new)
    return out


def same(pools, want):
    for i, (p, w) in enumerate(zip(pools, want)):
        assert torch.equal(p.contiguous().view(torch.uint8), w), i


@pytest.mark.parametrize("groups,W", [(1, 1), (1, 2), (5, 3), (7, 4), (2, 16), (1, 64), (3, 33), (1, 128)])
def test_groups(groups, W, cuda_device):
    """Cycles, fans and places that stay, in place; outside the groups nothing changes."""
    dev = cuda_device
    g = torch.Generator().manual_seed(groups * 100 + W)
    slots = groups * W + 4
    pools = make_pools(g, slots, dev)
    dst = torch.randperm(slots, generator=g)[:groups * W].view(groups, W).to(torch.int32)
    src = torch.randint(0, W, (groups, W), generator=g).to(torch.int32)
    src[0] = torch.roll(torch.arange(W), 1)     # one cycle
    flat_src = torch.gather(dst, 1, src.long())
    want = want_of(pools, dst.view(-1).tolist(), flat_src.view(-1).tolist())
    B.gdn_copy_slots(pools, dst.to(dev), src.to(dev), groups=True, dst_host=dst, src_host=src)
    B.gdn_read_device_status()
    same(pools, want)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 300, 1500])
def test_lists(n, cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(n)
    slots = 2 * n + 5
    order = torch.randperm(slots, generator=g).to(torch.int32)
    dst, src = order[:n], order[n:][torch.randint(0, n + 5, (n,), generator=g)]
    pools = make_pools(g, slots, dev)[1 if n > 300 else 0:]
    want = want_of(pools, dst.tolist(), src.tolist())
    B.gdn_copy_slots(pools, dst.to(dev), src.to(dev), dst_host=dst, src_host=src)
    B.gdn_read_device_status()
    same(pools, want)


def test_nothing_moves(cuda_device):
    """Negative entries, parents of -1, places without a slot, slots onto themselves."""
    dev = cuda_device
    g = torch.Generator().manual_seed(1)
    pools = make_pools(g, 12, dev)
    want = want_of(pools, [3, 5], [4, 0])
    dst = torch.tensor([-1, 3, 2, 5, 7], dtype=torch.int32, device=dev)
    src = torch.tensor([1, 4, -1, 0, 7], dtype=torch.int32, device=dev)
    B.gdn_copy_slots(pools, dst, src)
    same(pools, want)
    want = want_of(pools, [0, 8], [1, 9])
    dst = torch.tensor([[0, 1, -1], [8, 9, 10]], dtype=torch.int32, device=dev)
    src = torch.tensor([[1, 2, 0], [1, -1, 2]], dtype=torch.int32, device=dev)   # 1 <- a place without a slot
    B.gdn_copy_slots(pools, dst, src, groups=True)
    B.gdn_read_device_status()
    same(pools, want)


@pytest.mark.parametrize("dst,src,groups", [
    ([3, 40, 2], [1, 0, 5], False), ([3, 2], [1, 99], False), ([2 ** 31 - 1, 4], [0, 1], False),
    ([[3, 4], [5, 6]], [[0, 2], [1, 0]], True), ([[3, 77]], [[1, 0]], True),
])
def test_out_of_range(dst, src, groups, cuda_device):
    """Entries out of range are raised and move nothing; the others move."""
    dev = cuda_device
    g = torch.Generator().manual_seed(1)
    pools = make_pools(g, 12, dev)[:8]
    d, s = (torch.tensor(x, dtype=torch.int32) for x in (dst, src))
    moved = []
    for r in range(d.shape[0] if groups else 1):
        dd, ss = (d[r], s[r]) if groups else (d, s)
        for j in range(len(dd)):
            f = int(ss[j])
            if groups:
                if not 0 <= f < len(dd):
                    continue
                f = int(dd[f])
            if 0 <= int(dd[j]) < 12 and 0 <= f < 12:
                moved.append((int(dd[j]), f))
    want = want_of(pools, [m[0] for m in moved], [m[1] for m in moved])
    B.gdn_copy_slots(pools, d.to(dev), s.to(dev), groups=groups)
    with pytest.raises(B.GdnError) as e:
        B.gdn_read_device_status()
    assert e.value.code == B.GDN_ERR_DEVICE_CHECK
    same(pools, want)


@pytest.mark.parametrize("dst,src,groups", [
    ([3, 3], [1, 2], False), ([3, 4], [4, 1], False), ([[3, 4], [4, 5]], [[0, 0], [1, 1]], True),
])
def test_named_twice(dst, src, groups, cuda_device):
    """A destination named twice, or a source that is one: raised, and other slots are as they
    were."""
    dev = cuda_device
    g = torch.Generator().manual_seed(1)
    pools = [torch.randint(0, 256, (400000, size), generator=g, dtype=torch.uint8).to(dev) for size in (48, 20, 4)]
    before = [p.clone() for p in pools]
    d, s = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (dst, src))
    B.gdn_copy_slots(pools, d, s, groups=groups)
    with pytest.raises(B.GdnError):
        B.gdn_read_device_status()
    rest = [i for i in range(12) if i not in set(d.view(-1).tolist())]
    for p, b in zip(pools, before):
        assert torch.equal(p[rest], b[rest])
    far = torch.tensor([399999, 7], dtype=torch.int32, device=dev)
    if not groups:     # beyond the first window of the check
        B.gdn_copy_slots(pools, far, torch.tensor([1, 399999], dtype=torch.int32, device=dev))
        with pytest.raises(B.GdnError):
            B.gdn_read_device_status()


def test_many_pools_stream_and_graph(cuda_device):
    """More pools than one launch takes; another stream; a graph replayed: two swaps are none."""
    dev = cuda_device
    g = torch.Generator().manual_seed(1)
    pools = [torch.randn(6, 40 + 4 * i, generator=g).to(dev) for i in range(101)]
    before = [p.clone() for p in pools]
    dst = torch.tensor([[1, 2, 5]], dtype=torch.int32, device=dev)
    src = torch.tensor([[1, 0, 2]], dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.gdn_copy_slots(pools, dst, src, groups=True, stream=side)
    torch.cuda.synchronize()
    for p, b in zip(pools, before):
        assert torch.equal(p[[1, 2, 5, 0]], b[[2, 1, 5, 0]])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdn_copy_slots(pools, dst, src, groups=True)
    graph.replay()
    torch.cuda.synchronize()
    for p, b in zip(pools, before):
        assert torch.equal(p, b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    B.gdn_read_device_status()
    for p, b in zip(pools, before):
        assert torch.equal(p, b)


@pytest.mark.parametrize("groups", [False, True])
def test_many_pairs_and_offsets_past_32_bits(groups, cuda_device):
    """A pool of more than 2^32 bytes next to one of many small slots; lists of 60000, right, and
    wrong in their last pair."""
    dev, n, slots = cuda_device, 60000, 1_100_000
    g = torch.Generator().manual_seed(7)
    big = torch.empty(slots, 1024, dtype=torch.int32, device=dev)
    small = torch.arange(slots, dtype=torch.int32, device=dev).view(-1, 1).clone()
    order = torch.randperm(slots, generator=g)
    last = int((order == slots - 1).nonzero()[0, 0])
    order[last] = order[0]
    order[0] = slots - 1
    dst = order[:n].to(torch.int32)
    if groups:
        dst = dst.view(-1, 5)
        src = torch.randint(0, 5, dst.shape, generator=g).to(torch.int32)
        want = torch.gather(dst, 1, src.long())
    else:
        src = want = order[n:2 * n].to(torch.int32)
    big[:, 0] = small[:, 0]
    big[:, 1023] = small[:, 0]
    B.gdn_copy_slots([big, small], dst.to(dev), src.to(dev), groups=groups)
    B.gdn_read_device_status()
    d = dst.view(-1).long().to(dev)
    w = want.reshape(-1).to(dev)
    assert torch.equal(small[d, 0], w) and torch.equal(big[d, 0], w) and torch.equal(big[d, 1023], w)
    wrong = dst.clone()
    wrong.view(-1)[-1] = wrong.view(-1)[3]
    B.gdn_copy_slots([small], wrong.to(dev), src.to(dev), groups=groups)
    with pytest.raises(B.GdnError):
        B.gdn_read_device_status()
    del big
    torch.cuda.empty_cache()
