"""GPU: single rows whose evaluation key by key outlasts any wait of the kernel."""
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 256])
def test_one_row_over_two_million_keys(D, cuda_device):
    """A prompt of 2^21 + 2 tokens, an infinite value at the last but one: the two rows
    that see it are alone in their tile and take some 2 s each, twice the limit of a
    wait."""
    dev, T = cuda_device, 2 ** 21 + 2
    g = torch.Generator(device=dev).manual_seed(D)
    q, k, v = (torch.randn(T, 1, D, generator=g, device=dev).to(BF) for _ in range(3))
    v += 1.0
    cu = cu_of([T], dev)
    clean = torch.full_like(q, float("nan"))
    B.gdn_attn_varlen(q, k, v, cu, clean)
    v[T - 2, 0, 5] = float("inf")
    out = torch.full_like(q, float("nan"))
    B.gdn_attn_varlen(q, k, v, cu, out)
    B.gdn_read_device_status()
    assert torch.equal(out[:T - 2], clean[:T - 2])
    assert (out[T - 2:, :, 5] == float("inf")).all()
    rest = [d for d in range(D) if d != 5]
    # Values around 1: the tiled form's weights rounded to bf16 and two stores.
    torch.testing.assert_close(out[T - 2:, :, rest], clean[T - 2:, :, rest], rtol=2.0 ** -7, atol=2.0 ** -7)
