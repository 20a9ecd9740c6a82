"""GPU: gdn_beam_select over logits of any finite size: masks of large finite values, rows that hold
nothing else, logits far from zero; and sums of many equal terms.  Against the definition in 64
bits, as in test_gpu_beam.py."""
import numpy as np
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from test_gpu_beam import BF, F32, LSE, check, definition, select

pytestmark = pytest.mark.gpu

LOWEST = {BF: torch.finfo(BF).min, F32: torch.finfo(F32).min}


def value(mask, dtype):
    return LOWEST[dtype] if mask == "lowest" else float(mask)


def masked_but(n, W, V, keep, mask, dtype, g):
    """Normal logits at `keep` tokens of each row, the rest masked."""
    x = torch.full((n, W, V), value(mask, dtype))
    for b in range(n):
        for w in range(W):
            at = torch.randperm(V, generator=g)[:keep]
            x[b, w, at] = torch.randn(keep, generator=g) * 2
    return x.to(dtype)


MASKS = [-1e4, -1e9, -1e10, -1e12, -1e18, -1e20, -1e30, -1e32, "lowest"]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", MASKS)
def test_masks_of_large_finite_values(mask, dtype, cuda_device):
    """A few tokens of each row are allowed; whole chunks and most threads see the mask only."""
    g = torch.Generator().manual_seed(1)
    n, W, V, K = 2, 3, 40011, 5
    x = masked_but(n, W, V, 20, mask, dtype, g)
    x[0, 0] = (torch.randn(V, generator=g) * 2).to(dtype)       # an ordinary row, its first chunks masked
    x[0, 0, :17000] = value(mask, dtype)
    s = -torch.rand(n, W, generator=g) * 4
    check(select(x.to(cuda_device), s.to(cuda_device), K, cuda_device), definition(x, s, K))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", [-1e9, -1e20, "lowest"])
def test_fewer_allowed_tokens_than_places(mask, dtype, cuda_device):
    """Masked tokens are finite candidates: they take the places that are left, lowest first."""
    g = torch.Generator().manual_seed(2)
    n, W, V, K = 2, 1, 9001, 12
    x = masked_but(n, W, V, 4, mask, dtype, g)
    s = -torch.rand(n, W, generator=g)
    check(select(x.to(cuda_device), s.to(cuda_device), K, cuda_device), definition(x, s, K))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("level", [-1e7, -1e10, -1e20, -1e30, -1.6e38, "lowest", 2.8e6, 1e10, 1.5 * 2.0 ** 32, 1e20, 1.2e38,
                                   3e38])
@pytest.mark.parametrize("V", [5, 1000, 33001])
def test_rows_far_from_zero(V, level, dtype, cuda_device):
    """Rows of one value: each token's score is score - ln V, whatever the value.  Beside them a row
    of several values near it, and an ordinary one."""
    g = torch.Generator().manual_seed(3)
    K = 4
    x = torch.full((3, 2, V), value(level, dtype)).to(dtype)
    step = float(x[0, 0, 0].abs()) * float(torch.finfo(dtype).eps)
    x[1, 0] = (x[1, 0].double() + step * torch.randint(-3 if level != "lowest" else 0, 4, (V,), generator=g).double()).to(dtype)
    x[2, 1] = (torch.randn(V, generator=g) * 2).to(dtype)
    s = torch.tensor([[-1.0, -2.5], [-0.5, -40.0], [-30.0, -0.25]])
    want = definition(x, s, K)
    got = select(x.to(cuda_device), s.to(cuda_device), K, cuda_device)
    check(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_low_and_high_parts_of_a_row(dtype, cuda_device):
    """Rows whose parts lie far apart: only the highest has weight; NaN and infinities still take a
    row out wherever they are."""
    V, K = 70000, 24
    x = torch.zeros(8, 1, V)
    x[0, 0, :40000] = -1e12
    x[1, 0, 40000:] = 1e12
    x[2, 0, :40000], x[2, 0, 40000:] = -1e30, -1e31
    x[3, 0, :40000], x[3, 0, 40000:] = 1e30, 1e31
    x[4] = -1e20
    x[4, 0, 69999] = float("nan")
    x[5] = -1e20
    x[5, 0, 7] = float("inf")
    x[6] = 1e20
    x[6, 0, 5] = float("nan")
    x[7] = float("-inf")
    x[7, 0, 69000:] = -1e25
    x = x.to(dtype)
    s = -torch.arange(1.0, 9.0)[:, None]
    check(select(x.to(cuda_device), s.to(cuda_device), K, cuda_device), definition(x, s, K))


@pytest.mark.parametrize("n,W,V,dtype", [(152, 2, 131072, F32), (152, 2, 262144, F32), (160, 2, 131071, BF), (320, 1, 262147, BF),
                                         (2, 2, 1 << 20, F32)])
def test_sums_of_many_equal_terms(n, W, V, dtype, cuda_device):
    """Flat rows: every term of a thread's sum is the same, and what an addition loses is lost at
    each.  The score is score - ln V."""
    dev = cuda_device
    x = torch.empty(n, W, V, dtype=dtype, device=dev)
    s = torch.zeros(n, W, device=dev)
    for flat in (0.3, -1.1, 5.6, -17.3):
        x.fill_(flat)
        got = select(x, s, 1, dev)
        err = (got[2].double() + np.log(V)).abs().max().item()
        print(f"{flat}: log-sum off by {err:.2e}")
        assert err <= LSE + 2.0 ** -24 * np.log(V)
    g = torch.Generator(device=dev).manual_seed(V)
    x.copy_(torch.randn(1, 1, V, generator=g, device=dev).to(dtype).expand(n, W, V))
    got = select(x, s, 1, dev)
    y = x[0, 0].double()
    want = (y.max() - torch.logsumexp(y, 0)).item()
    assert (got[2].double() - want).abs().max().item() <= LSE + 2.0 ** -24 * abs(want)


@pytest.mark.parametrize("n,W,V,dtype", [(1, 4, 40001, F32), (100, 4, 40003, BF), (3, 5, 131071, BF), (1, 64, 5001, F32)])
def test_equal_beams_at_different_places(n, W, V, dtype, cuda_device):
    """Equal rows that begin at different elements and are divided differently: each token comes
    from every beam before the next best one, the beams' scores within the log-sums' 2^-19."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(V)
    row = torch.randn(V, generator=g, device=dev).to(dtype)
    row[torch.tensor([7, V // 2], device=dev)] = torch.tensor([9.0, 8.0], device=dev).to(dtype)
    x = row.expand(n, W, V).contiguous()
    par, tok, best = select(x, torch.full((n, W), -2.0, device=dev), 2 * W, dev)
    assert (par.view(n, 2, W).sort(-1).values == torch.arange(W, device=dev)).all()
    assert torch.equal(tok, torch.tensor([7] * W + [V // 2] * W, dtype=torch.int32, device=dev).expand(n, -1))
    want = -2.0 - torch.logsumexp(row.double(), 0) + torch.tensor([9.0, 8.0], dtype=torch.float64, device=dev)
    assert ((best.view(n, 2, W).double() - want[:, None]).abs() <= 2 * LSE + 2.0 ** -24 * 20).all()
