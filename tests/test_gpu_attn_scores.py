"""GPU: rows of attention whose scores are infinite or far from zero, against the
64-bit forms of tests/attn_reference.py.

The keys are made so that a row's scores are known: q is 1 in its first dims and 0 in
the others, scale is ln 2, so that a score in units of log2 is the sum of the key's
first dims."""
import math

import numpy as np
import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, F32, cu_of

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(math.log(2.0)))
TILE = 128


def unit_q(T, Hq, D, dtype, dims):
    q = torch.zeros(T, Hq, D)
    q[..., :dims] = 1.0
    return q.to(dtype)


def keys_with(score, Hkv, D, dtype):
    """Keys [L, Hkv, D] whose first dims are the rows of score [L, Hkv, n]."""
    k = torch.zeros(score.shape[0], Hkv, D)
    k[..., :score.shape[2]] = score
    out = k.to(dtype)
    assert torch.equal(out.float(), k)    # every score is exact
    return out


def as_pages(k, v, lens, page, dev, gen):
    """Packed keys and values of contexts `lens` in a shuffled paged cache."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    kc, vc = (torch.zeros(sum(need), x.shape[1], page, x.shape[2], dtype=x.dtype) for x in (k, v))
    a = at = 0
    for s, n in enumerate(lens):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        for i in range(n):
            kc[table[s, i // page], :, i % page] = k[a + i]
            vc[table[s, i // page], :, i % page] = v[a + i]
        a += n
    return kc.to(dev), vc.to(dev), table.to(dev)


def reference(q, k, v, q_lens, kv_lens):
    """Row by row over the visible keys whose score is finite: the others have weight
    0 and take no part."""
    q, k, v = R.f64(q), R.f64(k), R.f64(v)
    Hq, G = q.shape[1], q.shape[1] // k.shape[1]
    outs, lses, pieces = [], [], []
    a = c = 0
    for n, L in zip(q_lens, kv_lens):
        for i in range(n):
            vis = L - n + i + 1
            head = []
            for h in range(Hq):
                kk, vv = k[c:c + vis, h // G:h // G + 1], v[c:c + vis, h // G:h // G + 1]
                keep = np.isfinite(kk).all(axis=(1, 2))
                head.append(R.attention_rows(q[a + i:a + i + 1, h:h + 1], kk[keep], vv[keep],
                                             int(keep.sum()) - 1, SCALE))
            outs.append(np.concatenate([x[0] for x in head], 1))
            lses.append(np.concatenate([x[1] for x in head], 1))
            pieces.append([np.concatenate([x[2][j] for x in head], 1) for j in range(4)])
        a += n
        c += L
    return (np.concatenate(outs), np.concatenate(lses),
            tuple(np.concatenate([p[j] for p in pieces]) for j in range(4)))


def run(q, k, v, q_lens, kv_lens, page, dev, gen):
    """page None: packed prompts (kv_lens are q_lens)."""
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    cu = cu_of(q_lens, dev)
    if page is None:
        B.gdn_attn_varlen(q.to(dev), k.to(dev), v.to(dev), cu, out, scale=SCALE, lse=lse)
    else:
        kc, vc, table = as_pages(k, v, kv_lens, page, dev, gen)
        B.gdn_attn_paged(q.to(dev), kc, vc, table, torch.tensor(kv_lens, dtype=torch.int32, device=dev),
                         cu, out, max_q_len=max(q_lens), scale=SCALE, lse=lse)
    B.gdn_read_device_status()
    return out, lse


# q_lens, kv_lens, page (None: packed), Hq, Hkv
FORMS = [
    ([300], [300], None, 4, 2),
    ([1, 1], [300, 900], 16, 4, 2),        # few rows
    ([3], [6000], 64, 4, 1),               # few rows, many key ranges
    ([200], [500], 64, 4, 2),
    ([150], [6000], 128, 2, 1),            # a chunk whose keys are cut into ranges
]


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (128, F32), (32, BF)])
@pytest.mark.parametrize("q_lens,kv_lens,page,Hq,Hkv", FORMS)
def test_low_scores_beside_infinite_ones(q_lens, kv_lens, page, Hq, Hkv, D, dtype, cuda_device):
    """Every other block of 128 keys scores -inf, the first one among them; the other
    scores lie around -126, where a weight relative to 0 would leave the range of f32."""
    g = torch.Generator().manual_seed(D + sum(kv_lens))
    L = sum(kv_lens)
    score = -torch.randint(110, 141, (L, Hkv, 1), generator=g).float()
    a = 0
    for n in kv_lens:
        score[a:a + n][(torch.arange(n) // TILE) % 2 == 0] = -math.inf
        a += n
    q = unit_q(sum(q_lens), Hq, D, dtype, 1)
    k, v = keys_with(score, Hkv, D, dtype), torch.randn(L, Hkv, D, generator=g).to(dtype)
    out, lse = run(q, k, v, q_lens, kv_lens, page, cuda_device, g)
    ro, rl, pieces = reference(q, k, v, q_lens, kv_lens)
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, dtype == BF), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,page,Hq,Hkv", [
    ([1500], [1500], None, 2, 1),
    ([1] * 64, [2048] * 64, 16, 1, 1),     # few rows: several key tiles per SM
    ([1100], [2300], 64, 2, 1),
])
def test_scores_far_below_zero(q_lens, kv_lens, page, Hq, Hkv, D, cuda_device):
    """Scores around -19966, blocks of 128 keys at -20028 between them: the running
    reference moves up by 62 and has to stay within f32's range of the scores."""
    g = torch.Generator().manual_seed(D + len(kv_lens))
    L = sum(kv_lens)
    score = torch.empty(L, Hkv, 2)
    score[..., 0] = -19968.0
    score[..., 1] = torch.randint(0, 129, (L, Hkv), generator=g).float() / 32
    a = 0
    for n in kv_lens:
        score[a:a + n, :, 1][(torch.arange(n) // TILE) % 2 == 0] -= 64.0
        a += n
    score[..., 1] = score[..., 1].to(BF).float()
    q = unit_q(sum(q_lens), Hq, D, BF, 2)
    k, v = keys_with(score, Hkv, D, BF), torch.randn(L, Hkv, D, generator=g).to(BF)
    out, lse = run(q, k, v, q_lens, kv_lens, page, cuda_device, g)
    ro, rl, (A, ds, S, keys) = reference(q, k, v, q_lens, kv_lens)
    # The scores are exact in f32.  What is left of their error in a weight is that of
    # the factor to log2 units (two roundings) on a difference of at most 68 of them,
    # and one rounding of the difference.
    ds = np.full_like(ds, 68 * math.log(2.0) * 4 * R.U)
    R.check(R.f64(out), ro, R.bound(ro, (A, ds, S, keys), BF, True), "out")
    # lse: that factor, the one back and a sum, on a value of 13840.
    R.check(R.f64(lse), rl, R.lse_bound(rl, (A, ds, S, keys)) + 8 * R.U * np.abs(rl), "lse")


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (128, F32), (32, BF)])
@pytest.mark.parametrize("q_lens,kv_lens,page,Hq,Hkv", FORMS)
def test_infinite_values_at_keys_without_weight(q_lens, kv_lens, page, Hq, Hkv, D, dtype, cuda_device):
    """Keys that score -inf take no part, whatever their value is and wherever among
    the others they stand."""
    g = torch.Generator().manual_seed(D + 1 + sum(kv_lens))
    L = sum(kv_lens)
    score = torch.randint(-8, 9, (L, Hkv, 1), generator=g).float() / 4
    out_of = torch.rand(L, generator=g) < 0.01
    out_of[[0, L // 2, L - 1]] = True
    score[out_of] = -math.inf
    q = unit_q(sum(q_lens), Hq, D, dtype, 1)
    k, v = keys_with(score, Hkv, D, dtype), torch.randn(L, Hkv, D, generator=g).to(dtype)
    bad = v.clone()
    bad[out_of] = math.inf
    out, lse = run(q, k, bad, q_lens, kv_lens, page, cuda_device, g)
    ro, rl, pieces = reference(q, k, v, q_lens, kv_lens)
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, dtype == BF), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")
