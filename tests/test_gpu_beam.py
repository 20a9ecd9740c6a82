"""GPU: gdn_beam_select against its definition in 64 bits.

The library's log-sums carry f32 exponentials: |d lse| <= 2^-20 (2 ulp of ex2 and the
rounding of its argument, up to 16, relative to the sum; each part of the sum counts once).
Beams and tokens have to be those of the definition wherever no two candidates of different
beams lie nearer than twice that; the tests' inputs are looked at for it."""
import numpy as np
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LSE = 2.0 ** -20


def definition(logits, scores, K, finished=None, pad=0):
    """parents, tokens, scores (f64), and the smallest gap between neighbours of different
    beams among the first K + 1."""
    x = logits.double().cpu().numpy()
    n, W, V = x.shape
    par, tok = np.full((n, K), -1), np.full((n, K), -1)
    best = np.full((n, K), -np.inf)
    gap = np.inf
    for b in range(n):
        s = np.full((W, V), -np.inf)
        for w in range(W):
            sc = float(scores[b, w])
            if not np.isfinite(sc):
                continue
            if finished is not None and finished[b, w]:
                s[w, pad] = sc
                continue
            row = x[b, w]
            top = row.max()
            if not np.isfinite(top) or np.isnan(row).any():
                continue
            with np.errstate(divide="ignore"):
                s[w] = sc + (row - top) - np.log(np.exp(row - top).sum())
        flat = s.reshape(-1)
        order = np.argsort(-flat, kind="stable")[:K + 1]
        order = order[np.isfinite(flat[order])]
        for i, j in zip(order[:-1], order[1:]):
            if i // V != j // V:
                gap = min(gap, flat[i] - flat[j])
        order = order[:K]
        par[b, :len(order)], tok[b, :len(order)] = order // V, order % V
        best[b, :len(order)] = flat[order]
    return par, tok, best, gap


def select(logits, scores, K, dev, finished=None, pad=0, **over):
    n = logits.shape[0]
    par = torch.full((n, K), 77, dtype=torch.int32, device=dev)
    tok, best = torch.full_like(par, 77), torch.full((n, K), 77.0, device=dev)
    B.gdn_beam_select(logits, scores, par, tok, best, finished=finished, pad_token=pad, **over)
    B.gdn_read_device_status()
    return par, tok, best


def check(got, want):
    par, tok, best, gap = want
    assert gap > 2 * LSE, f"the inputs' nearest beams differ by {gap}"
    assert np.array_equal(got[0].cpu().numpy(), par)
    assert np.array_equal(got[1].cpu().numpy(), tok)
    g = got[2].cpu().numpy().astype(np.float64)
    fin = np.isfinite(best)
    assert np.array_equal(g[~fin], best[~fin])
    err = np.abs(g[fin] - best[fin])
    assert (err <= LSE + 2.0 ** -24 * np.abs(best[fin])).all(), err.max()


@pytest.mark.parametrize("n,W,V,K,dtype", [
    (1, 1, 1, 1, F32), (1, 1, 5, 8, BF), (2, 3, 7, 4, F32), (3, 4, 211, 8, BF), (1, 4, 32003, 4, F32),
    (2, 8, 32003, 16, BF), (5, 2, 4097, 128, F32), (1, 64, 1000, 64, BF), (2, 1, 131072, 2, BF),
    (70, 5, 8191, 10, BF), (1, 3, 200001, 128, F32), (2, 2, 100, 128, F32),
])
def test_select(n, W, V, K, dtype, cuda_device):
    g = torch.Generator().manual_seed(V + K)
    x = (torch.randn(n, W, V, generator=g) * 3).to(dtype)
    s = -torch.rand(n, W, generator=g) * 6
    check(select(x.to(cuda_device), s.to(cuda_device), K, cuda_device), definition(x, s, K))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ended_dead_and_masked(dtype, cuda_device):
    """Beams that ended or never lived, tokens that may not come, rows with NaN, infinities or
    nothing; more places than candidates."""
    g = torch.Generator().manual_seed(2)
    n, W, V = 4, 6, 3001
    x = torch.randn(n, W, V, generator=g) * 2
    s = -torch.rand(n, W, generator=g) * 3
    fin = torch.zeros(n, W, dtype=torch.bool)
    fin[0, 2] = fin[0, 5] = True
    x[0, 2] = float("nan")                     # not read
    x[0, 1, ::2] = float("-inf")
    x[1, 0, 17], x[1, 1, 5], x[1, 2] = float("nan"), float("inf"), float("-inf")
    s[1, 3], s[1, 4] = float("-inf"), float("nan")
    s[2, 1:] = float("-inf")                   # a search's first step
    s[2, 1] = float("inf")
    x[3] = float("-inf")
    x[3, 4, 1234], x[3, 4, 2999], x[3, 2, 0] = 1.0, 2.0, -5.0
    x = x.to(dtype)
    for K in (6, 12):
        got = select(x.to(cuda_device), s.to(cuda_device), K, cuda_device, finished=fin.to(cuda_device), pad=11)
        check(got, definition(x, s, K, fin.numpy(), 11))
    assert (got[0].cpu()[3, 3:] == -1).all()


@pytest.mark.parametrize("n,W,V,K,dtype", [(200, 4, 9001, 8, F32), (9, 3, 70001, 5, BF), (1, 7, 130001, 7, F32),
                                           (150, 8, 301, 16, F32)])
def test_many_rows_with_some_that_take_no_part(n, W, V, K, dtype, cuda_device):
    """Rows that end inside a block's share, next to ended and dead ones."""
    g = torch.Generator().manual_seed(n + V)
    x = (torch.randn(n, W, V, generator=g) * 3).to(dtype)
    s = -torch.rand(n, W, generator=g) * 6
    fin = torch.rand(n, W, generator=g) < 0.3
    dead = torch.rand(n, W, generator=g) < 0.2
    s[dead & ~fin] = float("-inf")
    x[fin] = float("nan")
    got = select(x.to(cuda_device), s.to(cuda_device), K, cuda_device, finished=fin.to(cuda_device), pad=3)
    check(got, definition(x, s, K, fin.numpy(), 3))


@pytest.mark.parametrize("dtype,V", [(BF, 50001), (F32, 9000), (BF, 1500)])
def test_equal_logits(dtype, V, cuda_device):
    """Rows of one value, of two, of zeros of either sign: the lowest indices, though more
    logits tie than a list has room for."""
    dev = cuda_device
    x = torch.zeros(3, 2, V)
    x[0] = 1.5
    x[0, 0, V // 2:] = 1.75
    x[1, :, 1::2] = -0.0
    x[2, 0] = (torch.arange(V) % 7).float()
    x[2, 1] = -4.0
    x = x.to(dtype)
    s = torch.tensor([[-1.0, -1.5], [-0.25, -3.0], [-1.0, -30.0]])
    K = 24
    check(select(x.to(dev), s.to(dev), K, dev), definition(x, s, K))


def test_equal_beams(cuda_device):
    """Beams with the same row and score tie bit for bit: the lower beam first."""
    dev = cuda_device
    g = torch.Generator().manual_seed(8)
    row = torch.randn(1, 1, 40000, generator=g)
    x = row.expand(1, 4, -1).contiguous().to(dev)
    got = select(x, torch.full((1, 4), -2.0, device=dev), 8, dev)
    top = row[0, 0].topk(2).indices.tolist()
    assert got[0].tolist() == [[0, 1, 2, 3] * 2]
    assert got[1].tolist() == [[top[0]] * 4 + [top[1]] * 4]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_alignment(dtype, cuda_device):
    """Rows at any element: views of wider, shifted and transposed logits."""
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    n, W, V, K = 3, 4, 5003, 9
    s = -torch.rand(n, W, generator=g)
    wide = (torch.randn(n, W, V + 13, generator=g) * 2).to(dtype)
    for off in (0, 1, 3, 8, 13):
        x = wide.to(dev)[..., off:off + V]
        check(select(x, s.to(dev), K, dev), definition(wide[..., off:off + V], s, K))
    t = wide.transpose(0, 1).contiguous().to(dev).transpose(0, 1)[..., 5:5 + V]
    check(select(t, s.to(dev), K, dev), definition(wide[..., 5:5 + V], s, K))


def test_in_place_streams_and_graphs(cuda_device):
    """out_scores over scores, another stream, and a graph replayed over changed inputs."""
    dev = cuda_device
    g = torch.Generator().manual_seed(4)
    n, W, V = 6, 4, 20000
    x = torch.randn(n, W, V, generator=g).to(BF).to(dev)
    x2 = torch.randn(n, W, V, generator=g).to(BF).to(dev)
    s = (-torch.rand(n, W, generator=g)).to(dev)
    want, want2 = select(x, s, W, dev), select(x2, s, W, dev)
    own = s.clone()
    par, tok = torch.empty(n, W, dtype=torch.int32, device=dev), torch.empty(n, W, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.gdn_beam_select(x, own, par, tok, own, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(own, want[2]) and torch.equal(par, want[0]) and torch.equal(tok, want[1])
    ws = torch.empty(B.gdn_beam_select_workspace_bytes(n, W, V, W), dtype=torch.uint8, device=dev)
    buf, best = x.clone(), torch.empty_like(s)
    B.gdn_beam_select(buf, s, par, tok, best, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdn_beam_select(buf, s, par, tok, best, workspace=ws)
    for src, w in ((x2, want2), (x, want)):
        buf.copy_(src)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(par, w[0]) and torch.equal(tok, w[1]) and torch.equal(best, w[2])


def test_offsets_past_32_bits(cuda_device):
    """Rows more than 2^32 elements apart."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    n, W, V, K = 3, 2, 2001, 4
    x = (torch.randn(n, W, V, generator=g) * 2).to(BF)
    far = torch.empty(2 ** 32 + 100 + 3 * V, dtype=BF, device=dev)
    step = 2 ** 31 + 7
    rows = far.as_strided((n, W, V), (step, V + 5, 1))
    rows.copy_(x)
    s = -torch.rand(n, W, generator=g)
    check(select(rows, s.to(dev), K, dev), definition(x, s, K))
    del far, rows
    torch.cuda.empty_cache()
