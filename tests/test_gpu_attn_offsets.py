"""GPU: offsets that fall somewhere among thousands of tokens raise the device status
in every form of the full-attention calls, wherever the searches over them land."""
import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, F32, cu_of, randn

pytestmark = pytest.mark.gpu

STEPS = [2 * i for i in range(65)]
BAD = [
    [0, 2000, 500, 2000],
    [0, 3000, 1000, 1500, 4000],
    [0, 2500, 100, 2600, 3000],
    STEPS[:33] + [STEPS[32] - 1] + STEPS[34:],   # one of many, by one token
]


def flagged():
    with pytest.raises(B.GdnError) as e:
        B.gdn_read_device_status()
    return e.value.code == B.GDN_ERR_DEVICE_CHECK


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (32, BF), (128, F32)])
def test_varlen(cu, D, dtype, cuda_device):
    T = cu[-1]
    g = torch.Generator(device=cuda_device).manual_seed(T)
    q = torch.randn(T, 4, D, generator=g, device=cuda_device).to(dtype)
    k = torch.randn(T, 2, D, generator=g, device=cuda_device).to(dtype)
    out = torch.empty_like(q)
    B.gdn_attn_varlen(q, k, k, torch.tensor(cu, dtype=torch.int32, device=cuda_device), out)
    assert flagged()
    B.gdn_attn_varlen(q, k, k, cu_of([T - 70, 0, 70], cuda_device), out)
    B.gdn_read_device_status()


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("D,dtype,page,max_q", [
    (128, BF, 16, 0), (256, BF, 64, 0), (64, BF, 16, 30),     # tiles, tiles, few rows
    (128, F32, 16, 0), (64, F32, 16, 8), (128, BF, 5, 0),     # CUDA cores: tiles, rows, tiles
])
def test_paged(cu, D, dtype, page, max_q, cuda_device):
    dev, T, N = cuda_device, cu[-1], len(cu) - 1
    g = torch.Generator(device=dev).manual_seed(T)
    q = torch.randn(T, 4, D, generator=g, device=dev).to(dtype)
    width = -(-200 // page)
    kc = torch.randn(N * width, 2, page, D, generator=g, device=dev).to(dtype)
    table = torch.arange(N * width, dtype=torch.int32, device=dev).view(N, width)
    kv = torch.full((N,), 200, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    B.gdn_attn_paged(q, kc, kc, table, kv, torch.tensor(cu, dtype=torch.int32, device=dev), out,
                     max_q_len=max_q)
    assert flagged()


@pytest.mark.parametrize("dtype,page,max_q", [(BF, 16, 0), (BF, 16, 8), (F32, 16, 0), (F32, 16, 4)])
def test_length_of_an_empty_sequence(dtype, page, max_q, cuda_device):
    """A context length outside the table is flagged for a sequence without new
    tokens, too."""
    dev, D = cuda_device, 64
    lens = [8, 0, 8, 0, 4] if max_q == 8 else [4, 0, 4, 0, 4] if max_q else [300, 0, 300, 0, 300]
    g = torch.Generator().manual_seed(1)
    T, N = sum(lens), len(lens)
    q = randn(g, T, 2, D, dtype=dtype).to(dev)
    kc = randn(g, N * 20, 2, page, D, dtype=dtype).to(dev)
    table = torch.arange(N * 20, dtype=torch.int32, device=dev).view(N, 20)
    out, cu = torch.empty_like(q), cu_of(lens, dev)
    for bad in (-1, 20 * page + 1):
        kv = torch.tensor([310, 5, 310, bad, 310], dtype=torch.int32, device=dev)
        B.gdn_attn_paged(q, kc, kc, table, kv, cu, out, max_q_len=max_q)
        assert flagged()
        B.gdn_attn_prepare(q, q, q, cu, out, kv_lens=kv, block_table=table, k_cache=kc.clone(), v_cache=kc.clone())
        assert flagged()
    kv = torch.tensor([310, 5, 310, 0, 310], dtype=torch.int32, device=dev)
    B.gdn_attn_paged(q, kc, kc, table, kv, cu, out, max_q_len=max_q)
    B.gdn_attn_prepare(q, q, q, cu, out, kv_lens=kv, block_table=table, k_cache=kc.clone(), v_cache=kc.clone())
    B.gdn_read_device_status()


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("D,dtype", [(64, BF), (256, F32)])
def test_prepare(cu, D, dtype, cuda_device):
    dev, T = cuda_device, cu[-1]
    g = torch.Generator().manual_seed(T)
    x = randn(g, T, 2, D, dtype=dtype).to(dev)
    q_out, k_out = torch.empty_like(x), torch.empty_like(x)
    B.gdn_attn_prepare(x, x, None, torch.tensor(cu, dtype=torch.int32, device=dev), q_out, k_out=k_out)
    assert flagged()
    B.gdn_attn_prepare(x, x, None, cu_of([T - 7, 0, 7], dev), q_out, k_out=k_out)
    B.gdn_read_device_status()


def test_prepare_many_sequences(cuda_device):
    """More sequences than one CTA looks at, the fallen offset among the last."""
    dev, N = cuda_device, 5000
    x = torch.randn(2 * N, 1, 32, device=dev).to(BF)
    out, k_out = torch.empty_like(x), torch.empty_like(x)
    cu = 2 * torch.arange(N + 1, dtype=torch.int32, device=dev)
    B.gdn_attn_prepare(x, x, None, cu, out, k_out=k_out)
    B.gdn_read_device_status()
    cu[4901] = cu[4900] - 1
    B.gdn_attn_prepare(x, x, None, cu, out, k_out=k_out)
    assert flagged()
