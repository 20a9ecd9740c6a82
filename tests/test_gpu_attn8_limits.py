"""GPU: the calls on an 8-bit cache where their indices could go wrong: offsets that fall,
lengths that cannot be, more tokens than announced, caches past 32 bits, many sequences, contexts
widened a group at a time, and what lies around every buffer."""
import numpy as np
import pytest
import torch

import attn8_reference as Q
import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, F32, Guarded, cu_of, randn
from test_gpu_attn8 import E4M3, bounds, make_cache8
from test_gpu_attn_offsets import BAD, flagged

pytestmark = pytest.mark.gpu

# Hq, Hkv, D, dtype, max_q: on the codes (few rows, several tiles of them), widened, rows
FORMS = [(4, 2, 128, BF, 4), (8, 2, 64, BF, 60), (4, 2, 256, BF, 0), (4, 2, 32, BF, 2), (4, 2, 64, F32, 0),
         (2, 2, 128, F32, 4)]


def cache8(gen, pages, Hkv, page, D, block, dev):
    codes = [torch.randn(pages, Hkv, page, D, generator=gen, device=dev).to(E4M3) for _ in range(2)]
    scales = [torch.ones(pages, Hkv, page // block, device=dev) for _ in range(2)]
    return dict(k_cache=codes[0], v_cache=codes[1], k_scale=scales[0], v_scale=scales[1])


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("Hq,Hkv,D,dtype,max_q", FORMS)
def test_offsets_that_fall(cu, Hq, Hkv, D, dtype, max_q, cuda_device):
    dev, T, N, page = cuda_device, cu[-1], len(cu) - 1, 32
    g = torch.Generator(device=dev).manual_seed(T)
    c = cache8(g, N * 7, Hkv, page, D, 16, dev)
    table = torch.arange(N * 7, dtype=torch.int32, device=dev).view(N, 7)
    q, k = (torch.randn(T, h, D, generator=g, device=dev).to(dtype) for h in (Hq, Hkv))
    kv = torch.full((N,), 200, dtype=torch.int32, device=dev)
    off = torch.tensor(cu, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    B.gdn_attn8_paged(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], table, kv, off, out, max_q_len=max_q)
    assert flagged()
    B.gdn_attn8_prepare(q, k, k, off, out, kv_lens=kv, block_table=table, **c)
    assert flagged()


@pytest.mark.parametrize("Hq,Hkv,D,dtype,max_q", FORMS)
def test_lengths_that_cannot_be(Hq, Hkv, D, dtype, max_q, cuda_device):
    """Contexts outside the table, of sequences with and without tokens; a sequence with more
    tokens than max_q_len; then the same call as it should be."""
    dev, page = cuda_device, 16
    n = max_q or 130
    lens = [n, 0, n, 0, n]
    g = torch.Generator(device=dev).manual_seed(1)
    c = cache8(g, 100, Hkv, page, D, 16, dev)
    table = torch.arange(100, dtype=torch.int32, device=dev).view(5, 20)
    q = torch.randn(sum(lens), Hq, D, generator=g, device=dev).to(dtype)
    out = torch.empty_like(q)

    def call(kv, cu):
        B.gdn_attn8_paged(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], table,
                          torch.tensor(kv, dtype=torch.int32, device=dev), cu_of(cu, dev), out, max_q_len=n)

    for kv in ([310, 5, 310, -1, 310], [310, 5, 310, 321, 310], [310, 5, -2 ** 31, 0, 310],
               [2 ** 31 - 1, 0, 310, 5, 310]):
        call(kv, lens)
        assert flagged()
    call([310, 5, 310, 0, 310], [n + 1, 0, n - 1, 0, n])
    assert flagged()
    call([310, 5, 310, 0, 310], lens)
    B.gdn_read_device_status()


@pytest.mark.parametrize("Hq,Hkv,D,dtype,max_q", [f for f in FORMS if f[2] >= 64])
def test_offsets_past_32_bits(Hq, Hkv, D, dtype, max_q, cuda_device):
    """Codes past 2^32 bytes: the pages used are the last ones."""
    dev, page, block = cuda_device, 64, 32
    pages = 2 ** 32 // (Hkv * page * D) + 40
    g = torch.Generator().manual_seed(4)
    lens = [1000, 333]
    small, (_, _, _, _, t) = make_cache8(g, lens, Hkv, D, page, block, dev, poison=False)
    n, n_q = small["k_cache"].shape[0], max_q or 70
    big = {}
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        big[name] = torch.empty((pages, *small[name].shape[1:]), dtype=small[name].dtype, device=dev)
        big[name][pages - n:] = small[name]
    table = torch.where(t >= 0, t + (pages - n), t).to(dev)
    q, k = (randn(g, 2 * n_q, h, D, dtype=dtype).to(dev) for h in (Hq, Hkv))
    kv = torch.tensor(lens, dtype=torch.int32, device=dev)
    outs, q_out = [], torch.empty_like(q)
    for c, tb in ((small, t.to(dev)), (big, table)):
        caches = {m: c[m] for m in ("k_cache", "v_cache", "k_scale", "v_scale")}
        out = torch.empty_like(q)
        B.gdn_attn8_prepare(q, k, k, cu_of([n_q, n_q], dev), q_out, kv_lens=kv, block_table=tb, **caches)
        B.gdn_attn8_paged(q, *caches.values(), tb, kv, cu_of([n_q, n_q], dev), out, max_q_len=n_q)
        outs.append(out)
    B.gdn_read_device_status()
    assert torch.equal(*outs)
    for name in ("k_cache", "k_scale", "v_cache", "v_scale"):
        assert torch.equal(big[name][pages - n:].view(torch.uint8), small[name].view(torch.uint8)), name
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,Hq,n_q", [(BF, 2, 1), (BF, 64, 5), (F32, 2, 1)])
def test_many_sequences(dtype, Hq, n_q, cuda_device):
    """More sequences than threads in a block, most of them empty."""
    dev, D, page = cuda_device, 64, 16
    kv_lens = [(i * 37) % 50 if i % 3 == 0 else 0 for i in range(1100)]
    q_lens = [n_q if i % 2 == 0 else 0 for i in range(1100)]
    g = torch.Generator().manual_seed(2)
    c, (kc, ks, vc, vs, table) = make_cache8(g, kv_lens, 1, D, page, 16, dev)
    q = randn(g, sum(q_lens), Hq, D, dtype=dtype)
    out = torch.empty_like(q, device=dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    B.gdn_attn8_paged(q.to(dev), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["block_table"], kv,
                      cu_of(q_lens, dev), out, max_q_len=n_q)
    B.gdn_read_device_status()
    ro, _, pieces = Q.paged(q, kc, ks, vc, vs, table, kv_lens, q_lens, D ** -0.5, None)
    R.check(R.f64(out), ro, bounds(pieces, ro, dtype), "out")


@pytest.mark.parametrize("dtype,Hq,n_q", [(BF, 32, 70), (F32, 128, 1), (F32, 32, 9)])
def test_widened_in_groups(dtype, Hq, n_q, cuda_device):
    """A table so wide that the contexts of four sequences (two in f32) fill the workspace's
    share: nine are taken in groups."""
    dev, Hkv, D, page = cuda_device, 8, 128, 64
    kv_lens = [300, 70, 0, 129, 90, 1000, 64, 200, 75]
    g = torch.Generator().manual_seed(5)
    c, (kc, ks, vc, vs, table) = make_cache8(g, kv_lens, Hkv, D, page, 32, dev)
    wide = torch.full((9, 1024), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q_lens = [n_q] * 9
    q = randn(g, 9 * n_q, Hq, D, dtype=dtype)
    out, lse = torch.empty_like(q, device=dev), torch.empty(9 * n_q, Hq, device=dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    B.gdn_attn8_paged(q.to(dev), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], wide.to(dev), kv,
                      None if n_q == 1 else cu_of(q_lens, dev), out, max_q_len=n_q, lse=lse)
    B.gdn_read_device_status()
    ro, rl, pieces = Q.paged(q, kc, ks, vc, vs, table, kv_lens, q_lens, D ** -0.5, None)
    R.check(R.f64(out), ro, bounds(pieces, ro, dtype), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


@pytest.mark.parametrize("Hq,Hkv,D,dtype,max_q", FORMS)
def test_nothing_is_written_outside(Hq, Hkv, D, dtype, max_q, cuda_device):
    dev, page, block = cuda_device, 32, 16
    gd = Guarded(dev)
    g = torch.Generator().manual_seed(D)
    n = max_q or 130
    for ql, kl in (([1, 1, 1], [3, 700, 0]), ([n, 1, n], [40, 1, 500])):
        T, N, width = sum(ql), 3, -(-max(kl) // page)
        codes = [gd.new((N * width, Hkv, page, D), torch.uint8, 0) for _ in range(2)]
        scales = [gd.new((N * width, Hkv, page // block), F32, 0) for _ in range(2)]
        c = dict(k_cache=codes[0].view(E4M3), v_cache=codes[1].view(E4M3), k_scale=scales[0], v_scale=scales[1])
        table = torch.randperm(N * width, generator=g).to(torch.int32).view(N, width).to(dev)
        kv = torch.tensor(kl, dtype=torch.int32, device=dev)
        q, k, v = (randn(g, T, h, D, dtype=dtype).to(dev) for h in (Hq, Hkv, Hkv))
        q_out, k_out = gd.new((T, Hq, D), dtype), gd.new((T, Hkv, D), dtype)
        out, lse = gd.new((T, Hq, D), dtype), gd.new((T, Hq), F32)
        need = B.gdn_attn8_paged_workspace_bytes(T, N, Hq, Hkv, D, max(ql), B._dt(q), width, page)
        ws = gd.new((max(need, 256),), torch.uint8, 0)
        cs = torch.randn(max(kl) + 1, 32, generator=g).to(dev)
        B.gdn_attn8_prepare(q, k, v, cu_of(ql, dev), q_out, kv_lens=kv, block_table=table, k_out=k_out, cos_sin=cs, **c)
        B.gdn_attn8_paged(q_out, c["k_cache"], c["v_cache"], scales[0], scales[1], table, kv, cu_of(ql, dev), out,
                          max_q_len=max(ql), lse=lse, workspace=ws)
        gd.check()
    B.gdn_read_device_status()
