"""gdn_attn8_prepare reads k and v while it writes q_out and k_out: outputs over those rows are
refused (CPU: fake device addresses, never dereferenced; GPU: the binding's call)."""
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from test_attn8_refusals import cache8, call
from test_attn_refusals import FAKE, prepare_args, rows

BF = torch.bfloat16
T, Hq, Hkv, D = 4, 4, 2, 64
FAR = FAKE + (1 << 30)


def at(address, H, **over):
    r = rows(T, H, D)
    r.data = address
    for k, v in over.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("which", ["q_out", "k_out"])
@pytest.mark.parametrize("over", ["k", "v"])
@pytest.mark.parametrize("shift", [0, 16, -16, 2 * T * Hkv * D - 16])
def test_outputs_over_k_or_v(which, over, shift):
    place = dict(q=at(FAR * 2, Hq), k=at(FAR * 3, Hkv), v=at(FAR * 4, Hkv), q_out=FAR * 5, k_out=FAR * 6, k_out_len=T * Hkv * D)
    place[which] = place[over].data + shift
    rc, msg = call(prepare_args, cache8(), T=T, Hq=Hq, Hkv=Hkv, D=D, **place)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT
    assert msg == f"gdn_attn8_prepare q_out and k_out must not overlap the {'key' if over == 'k' else 'value'} rows"


def test_outputs_between_rows_of_a_projection():
    """k's last head of the last token is the end of what may not be written; its first one of the
    first the beginning."""
    wide = 1024
    k = at(FAR * 3, Hkv, token_stride=wide, len=3 * wide + Hkv * D)
    end = k.data + 2 * (3 * wide + Hkv * D)
    for q_out in (end - 16, k.data - 2 * T * Hq * D + 16, k.data + 2 * wide):
        rc, msg = call(prepare_args, cache8(), T=T, Hq=Hq, Hkv=Hkv, D=D, q=at(FAR * 2, Hq), k=k, v=at(FAR * 4, Hkv), q_out=q_out)
        assert rc == B.GDN_ERR_INVALID_ARGUMENT and "key rows" in msg


@pytest.mark.gpu
def test_neighbours_are_taken_and_overlaps_refused(cuda_device):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(1)
    n = T * Hkv * D
    one = torch.randn(6 * n, generator=g, device=dev).to(BF)
    q = torch.randn(T, Hq, D, generator=g, device=dev).to(BF)
    k, v = one[n:2 * n].view(T, Hkv, D), one[4 * n:5 * n].view(T, Hkv, D)
    kc, vc = (torch.zeros(1, Hkv, 16, D, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
    c = dict(k_cache=kc, v_cache=vc, k_scale=torch.zeros(1, Hkv, 1, device=dev), v_scale=torch.zeros(1, Hkv, 1, device=dev),
             block_table=torch.zeros(1, 1, dtype=torch.int32, device=dev))
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    keys = k.clone()
    B.gdn_attn8_prepare(q, k, v, cu, one[2 * n:4 * n].view(T, Hq, D), k_out=one[:n].view(T, Hkv, D), **c)
    B.gdn_read_device_status()
    assert torch.equal(one[2 * n:4 * n].view(T, Hq, D), q) and torch.equal(one[:n].view(T, Hkv, D), keys)
    before = one.clone()
    for over in (dict(k_out=k), dict(k_out=v), dict(k_out=one[n - 8:2 * n - 8].view(T, Hkv, D))):
        with pytest.raises(B.GdnError) as e:
            B.gdn_attn8_prepare(q, k, v, cu, torch.empty_like(q), **over, **c)
        assert e.value.code == B.GDN_ERR_INVALID_ARGUMENT
    with pytest.raises(B.GdnError):
        B.gdn_attn8_prepare(q, k, v, cu, one[n:3 * n].view(T, Hq, D), **c)
    torch.cuda.synchronize()
    assert torch.equal(one, before)
