"""GPU: attention over an 8-bit cache where one key takes most of a row: the others' weights are
small beside the largest and still make up the output (the heavy key's value is 0, as that of
a first token often is).  All sequences share one context, and there are as many that a block has
whole contexts of its own, whose weights are then all relative to the heavy key's."""
import math

import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, F32, cu_of

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
N = 304          # two contexts, or one, for each block of a grid of 152 or 304
SHOWN = range(0, N, 19)

# D, query heads of the kv head, tokens of a sequence: 8 to 128 rows
SHAPES = [(64, 8, 1), (128, 8, 1), (256, 8, 1), (128, 4, 4), (256, 16, 1), (128, 8, 4), (256, 8, 4), (64, 16, 4),
          (128, 16, 4), (256, 16, 4), (128, 16, 8)]


def context(L, D, score, flat, gen, dev):
    """Codes and scales of one kv head's context of L tokens; key 0 scores `score` with a q whose
    first value is 8, the others normally distributed scores (flat: 0)."""
    page, block = 64, 16
    P = L // page
    k = torch.zeros(L, D, device=dev) if flat else torch.randn(L, D, generator=gen, device=dev)
    v = torch.randn(L, D, generator=gen, device=dev).abs_()
    k[:, 0] = 0.0
    k[0] = 0.0
    k[0, 0] = score * math.sqrt(D) / 8.0
    v[0] = 0.0
    ks = torch.full((P, 1, page // block), 2.0 ** -5, device=dev)
    vs = torch.full((P, 1, page // block), 2.0 ** -6, device=dev)
    ks[0, 0, 0] = 2.0 ** -3
    out = []
    for x, s in ((k, ks), (v, vs)):
        rows = s.repeat_interleave(block, 2).view(L, 1)
        codes = (x / rows).clamp(-448, 448).to(E4M3)
        out.append((codes.view(P, 1, page, D), s, codes.double() * rows.double()))
    return out


def run(D, G, n, L, score, flat, dev, std=1.5):
    g = torch.Generator(device=dev).manual_seed(L + D + G)
    (kc, ks, k), (vc, vs, v) = context(L, D, score, flat, g, dev)
    T = N * n
    q = (torch.randn(T, G, D, generator=g, device=dev) * std).to(BF)
    q[..., 0] = 8.0
    table = torch.arange(L // 64, dtype=torch.int32, device=dev).expand(N, -1).contiguous()
    out, lse = torch.empty_like(q), torch.empty(T, G, device=dev)
    kv = torch.full((N,), L, dtype=torch.int32, device=dev)
    B.gdn_attn8_paged(q, kc, vc, ks, vs, table, kv, cu_of([n] * N, dev), out, max_q_len=n, lse=lse)
    B.gdn_read_device_status()
    worst = 0.0
    for s in SHOWN:
        x = q[s * n:(s + 1) * n].double().view(n * G, D)
        sc = (x @ k.T) * D ** -0.5
        last = L - n + torch.arange(n, device=dev).repeat_interleave(G)
        sees = torch.arange(L, device=dev)[None, :] <= last[:, None]
        sc = torch.where(sees, sc, torch.full_like(sc, -math.inf))
        top = sc.amax(1, keepdim=True)
        w = torch.exp(sc - top)
        z = w.sum(1, keepdim=True)
        ref, A = (w @ v) / z, (w @ v.abs()) / z
        # tests/attn_reference.py's bound, all rows at once
        ds = D ** -0.5 * (D + 4) * 2 * R.U * (x.abs() @ k.abs().T).amax(1)
        S = (top - torch.where(sees, sc, top)).amax(1).clamp(max=104.0)
        rel = 2 * ds + (2 * L + S + 64) * R.U + 2.0 ** -8
        tol = (A * rel[:, None] + R.half_step(BF) * ref.abs() + 1e-37).view(n, G, D)
        got = out[s * n:(s + 1) * n].double()
        err = ((got - ref.view(n, G, D)).abs() / tol).max().item()
        worst = max(worst, err if math.isfinite(err) else math.inf)
        want = (top + z.log()).view(n, G)
        slack = (ds + (2 * L + S + 64) * R.U).view(n, G) + 4 * R.U * want.abs()
        assert ((lse[s * n:(s + 1) * n].double() - want).abs() <= slack).all()
    print(f"worst error {worst:.3f} of its bound")
    assert worst <= 1.0, f"error {worst:.2f} times its bound"


@pytest.mark.parametrize("L,share", [(4096, 0.9), (65536, 0.5), (65536, 0.97)])
@pytest.mark.parametrize("D,G,n", SHAPES)
def test_a_first_key_with_most_of_the_weight(D, G, n, L, share, cuda_device):
    """The others' scores are spread by 1.5 nats."""
    score = math.log(L) + 1.5 ** 2 / 2 + math.log(share / (1.0 - share))
    run(D, G, n, L, score, False, cuda_device)


@pytest.mark.parametrize("L,nats", [(4096, 8.0), (16384, 11.0), (65536, 12.13), (65536, 14.0)])
@pytest.mark.parametrize("D,G,n", [(64, 8, 1), (128, 4, 4), (256, 8, 1), (256, 16, 4)])
def test_a_heavy_key_over_a_flat_tail(D, G, n, L, nats, cuda_device):
    """Every other key has the same small weight, e^-nats of the largest: what each loses adds up."""
    run(D, G, n, L, nats, True, cuda_device)
