"""The step helper of the full-attention layer, and the small hybrid stack that
runs it beside the gated-delta-rule layers."""
import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from gated_delta_rule_44_gb300 import hybrid_example as E
from gated_delta_rule_44_gb300.layer import AttnStep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new_prompts", [True, False])
def test_mixed_step(new_prompts, cuda_device):
    """Three decode rows and two prompts (or chunks over an earlier context) in one
    batch, against the 64-bit forms on the rows the step stored."""
    dev, bf = cuda_device, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    Hq, Hkv, D, page = 8, 2, 128, 16
    ql = [1, 1, 1, 40, 150]
    kl = [5, 300, 1, 40, 150] if new_prompts else [5, 300, 1, 90, 170]
    T, N, nd = sum(ql), 5, 3
    width = 20
    kc = torch.randn(N * width, Hkv, page, D, generator=g).to(bf).to(dev)
    vc = torch.randn(N * width, Hkv, page, D, generator=g).to(bf).to(dev)
    table = torch.randperm(N * width, generator=g).to(torch.int32).view(N, width).to(dev)
    row = torch.randn(T, (2 * Hq + 2 * Hkv) * D, generator=g).to(bf).to(dev)
    qg = row[:, :2 * Hq * D].view(T, Hq, 2 * D)
    kv = row[:, 2 * Hq * D:].view(T, 2 * Hkv, D)
    cs = torch.randn(320, 64, generator=g).to(dev)
    cu = torch.tensor([0] + ql).cumsum(0).to(torch.int32).to(dev)
    step = AttnStep(T, N, nd, Hq, Hkv, D, bf, dev, max_q_len=150, new_prompts=new_prompts)
    out = step.run(qg[..., :D], kv[:, :Hkv], kv[:, Hkv:], cu,
                   torch.tensor(kl, dtype=torch.int32, device=dev), table, kc, vc,
                   cu_seqlens_prefill=(cu[nd:] - nd).contiguous(), gate=qg[..., D:], cos_sin=cs)
    B.gdn_read_device_status()
    ro, _, pieces = R.paged(step.q, kc, vc, table, kl, ql, D ** -0.5, qg[..., D:])
    R.check(R.f64(out), ro, R.bound(ro, pieces, bf, True), "out")


def test_hybrid_stack_serves_what_it_computes_whole(cuda_device):
    """Prompts and then single tokens, against the same sequences in one batch.  The
    two round in other places (every layer's rows are stored in bf16, the decode
    recurrence is not the chunked one), by a few 2^-8 of a row after eight stored
    projections."""
    prompts, more = [37, 130, 1], 5
    total = [n + more for n in prompts]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(sum(total), E.HybridStack.HID, generator=g).to(torch.bfloat16).to(cuda_device)
    served = E.generate(E.HybridStack(3, max(total), cuda_device), x, prompts, total).float()
    whole = E.generate(E.HybridStack(3, max(total), cuda_device), x, total, total).float()
    B.gdn_read_device_status()
    assert torch.isfinite(served).all()
    rms = whole.square().mean().sqrt().item()
    err = (served - whole).square().mean().sqrt().item()
    assert err <= 16 * 2.0 ** -8 * rms, (err, rms)
