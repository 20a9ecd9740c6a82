"""GPU: one long context over an 8-bit cache, cut between many blocks of threads, whose parts have
value scales far apart: the sums of the parts refer to different scales when they are joined."""
import math

import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("D,G", [(64, 8), (128, 16), (256, 4)])
@pytest.mark.parametrize("low,high", [(-64, 0), (-64, 55), (-64, 84), (-20, 84), (-64, 100)])
def test_parts_with_value_scales_far_apart(D, G, low, high, cuda_device):
    dev, L, page, block = cuda_device, 200000, 64, 64
    g = torch.Generator(device=dev).manual_seed(D + high)
    P = L // page
    k, v = (torch.randn(L, D, generator=g, device=dev) for _ in range(2))
    ks = torch.full((P, 1, 1), 2.0 ** -6, device=dev)
    vs = torch.full((P, 1, 1), 2.0 ** low, device=dev)
    vs[P // 2:] = 2.0 ** high
    kc = (k * 2.0 ** 6).clamp(-448, 448).to(E4M3)
    vc = (v * 2.0 ** 6).clamp(-448, 448).to(E4M3)
    k = kc.double() * 2.0 ** -6
    v = vc.double() * vs.double().view(-1).repeat_interleave(page)[:, None]
    q = (torch.randn(1, G, D, generator=g, device=dev) * 1.5).to(BF)
    table = torch.arange(P, dtype=torch.int32, device=dev)[None]
    out, lse = torch.empty_like(q), torch.empty(1, G, device=dev)
    B.gdn_attn8_paged(q, kc.view(P, 1, page, D), vc.view(P, 1, page, D), ks, vs, table,
                      torch.tensor([L], dtype=torch.int32, device=dev), None, out, lse=lse)
    B.gdn_read_device_status()
    x = q[0].double()
    sc = (x @ k.T) * D ** -0.5
    top = sc.amax(1, keepdim=True)
    w = torch.exp(sc - top)
    z = w.sum(1, keepdim=True)
    # tests/attn_reference.py's bound; ranges of 1300 keys and less are summed apart and then joined,
    # so that 4096 terms stand for what the sums lose.
    ds = D ** -0.5 * (D + 4) * 2 * R.U * (x.abs() @ k.abs().T).amax(1)
    S = (top - sc).amax(1).clamp(max=104.0)
    rel = 2 * ds + (2 * 4096 + S + 64) * R.U
    want = (top + z.log())[:, 0]
    assert ((lse[0].double() - want).abs() <= rel + 4 * R.U * want.abs()).all(), (lse[0].double() - want).abs().max()
    ref, A = (w @ v) / z, (w @ v.abs()) / z
    tol = A * (rel[:, None] + 2.0 ** -8) + R.half_step(BF) * ref.abs()
    err = ((out[0].double() - ref).abs() / tol).max().item()
    print(f"worst error {err:.3f} of its bound")
    assert math.isfinite(err) and err <= 1.0
