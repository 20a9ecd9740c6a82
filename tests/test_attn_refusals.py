"""Refusals of the full-attention calls, on the CPU: nothing is launched.  The
binding checks what it sees of the tensors; the C entries check sizes, strides,
alignment, host metadata and the workspace (fake device addresses, never
dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B

FAKE = 0x100000


def rows(T, H, D, **over):
    a = dict(data=FAKE, len=T * H * D, token_stride=0, head_stride=0)
    a.update(over)
    return B.gdn_attn_rows(**a)


def cache(Hkv, D, pages=8, page=16, max_pages=4, N=2, **over):
    n = pages * Hkv * page * D
    a = dict(k=FAKE, k_len=n, v=FAKE, v_len=n, num_pages=pages, page_size=page, block_table=FAKE,
             max_pages=max_pages)
    a.update(over)
    return B.gdn_attn_cache(**a)


def paged_args(T=4, N=2, Hq=4, Hkv=2, D=64, c=None, **over):
    c = cache(Hkv, D) if c is None else c
    a = dict(T=T, N=N, Hq=Hq, Hkv=Hkv, D=D, max_q_len=0, act_dtype=B.GDN_DTYPE_BF16, scale=-1.0,
             q=rows(T, Hq, D), cu_seqlens=FAKE, kv_lens=FAKE, cache=ctypes.pointer(c), out=FAKE,
             out_len=T * Hq * D, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(over)
    return B.gdn_attn_paged_args(**a)


def varlen_args(T=4, N=2, Hq=4, Hkv=2, D=64, **over):
    a = dict(T=T, N=N, Hq=Hq, Hkv=Hkv, D=D, act_dtype=B.GDN_DTYPE_BF16, scale=-1.0,
             q=rows(T, Hq, D), k=rows(T, Hkv, D), v=rows(T, Hkv, D), cu_seqlens=FAKE, out=FAKE,
             out_len=T * Hq * D)
    a.update(over)
    return B.gdn_attn_varlen_args(**a)


def prepare_args(T=4, N=2, Hq=4, Hkv=2, D=64, c=None, **over):
    c = cache(Hkv, D) if c is None else c
    a = dict(T=T, N=N, Hq=Hq, Hkv=Hkv, D=D, rot_dim=32, act_dtype=B.GDN_DTYPE_BF16, norm_eps=1e-6,
             q=rows(T, Hq, D), k=rows(T, Hkv, D), v=rows(T, Hkv, D), q_norm_weight=FAKE,
             q_norm_weight_len=D, k_norm_weight=FAKE, k_norm_weight_len=D, cos_sin=FAKE,
             cos_sin_len=32 * 100, cu_seqlens=FAKE, kv_lens=FAKE, cache=ctypes.pointer(c),
             q_out=FAKE, q_out_len=T * Hq * D)
    a.update(over)
    return B.gdn_attn_prepare_args(**a)


def call(a):
    L = B.lib()
    fn = {B.gdn_attn_paged_args: L.gdn_attn_paged, B.gdn_attn_varlen_args: L.gdn_attn_varlen,
          B.gdn_attn_prepare_args: L.gdn_attn_prepare}[type(a)]
    rc = fn(ctypes.byref(a), None)
    return rc, L.gdn_last_error_message().decode()


MAKERS = [paged_args, varlen_args, prepare_args]


@pytest.mark.parametrize("make", MAKERS)
def test_shapes(make):
    assert call(make(T=0))[0] == B.GDN_ERR_SHAPE
    assert call(make(N=0))[0] == B.GDN_ERR_SHAPE
    rc, msg = call(make(Hq=3))
    assert rc == B.GDN_ERR_SHAPE and msg == "attention query_heads 3 must be divisible by kv_heads 2"
    assert call(make(D=48))[0] == B.GDN_ERR_UNSUPPORTED
    assert call(make(Hq=130, Hkv=2))[0] == B.GDN_ERR_UNSUPPORTED
    assert call(make(T=1 << 40))[0] == B.GDN_ERR_UNSUPPORTED
    assert call(make(act_dtype=5))[0] == B.GDN_ERR_DTYPE
    rc, msg = call(make(q=rows(4, 4, 64, len=4 * 4 * 64 - 1)))
    assert rc == B.GDN_ERR_SHAPE and msg == "attention query length 1023 < expected 1024"
    assert call(make(q=rows(4, 4, 64, len=1 << 30, token_stride=1 << 61)))[0] == B.GDN_ERR_SHAPE
    assert call(make(q=rows(4, 4, 64, len=1 << 30, token_stride=-256)))[0] == B.GDN_ERR_SHAPE
    assert call(make(q=rows(4, 4, 64, len=1 << 30, token_stride=257)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(q=rows(4, 4, 64, len=1 << 30, head_stride=65)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(q=rows(4, 4, 64, data=FAKE + 8)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(q=rows(4, 4, 64, data=None)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    fn = {paged_args: "gdn_attn_paged", varlen_args: "gdn_attn_varlen",
          prepare_args: "gdn_attn_prepare"}[make]
    assert getattr(B.lib(), fn)(None, None) == B.GDN_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("make", MAKERS)
def test_cu_seqlens_mirror(make):
    def cu(*v):
        a = (ctypes.c_int32 * len(v))(*v)
        return call(make(cu_seqlens_host=ctypes.addressof(a)))
    assert cu(0, 2, 3)[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert cu(1, 2, 4)[0] == B.GDN_ERR_INVALID_ARGUMENT
    rc, msg = cu(0, 5, 4)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and "sequence 0 has range 0..5" in msg


@pytest.mark.parametrize("make", [paged_args, prepare_args])
def test_cache(make):
    assert call(make(c=cache(2, 64, k_len=8 * 2 * 16 * 64 - 1)))[0] == B.GDN_ERR_SHAPE
    assert call(make(c=cache(2, 64, v=None)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(c=cache(2, 64, k=FAKE + 2)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(c=cache(2, 64, block_table=None)))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(c=cache(2, 64, page=0)))[0] == B.GDN_ERR_SHAPE
    assert call(make(c=cache(2, 64, table_stride=3)))[0] == B.GDN_ERR_SHAPE
    assert call(make(c=cache(2, 64, table_stride=1 << 62)))[0] == B.GDN_ERR_SHAPE
    assert call(make(c=cache(2, 64, k_page_stride=1 << 61)))[0] == B.GDN_ERR_SHAPE
    assert call(make(c=cache(2, 64, k_len=1 << 30, k_token_stride=68)))[0] == \
        B.GDN_ERR_INVALID_ARGUMENT
    assert call(make(c=cache(2, 64, max_pages=1 << 30)))[0] == B.GDN_ERR_UNSUPPORTED
    kv = (ctypes.c_int32 * 2)(5, 65)
    rc, msg = call(make(kv_lens_host=ctypes.addressof(kv)))
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and "sequence 1 has kv_len 65, not 0..64" in msg
    kv = (ctypes.c_int32 * 2)(5, 17)
    table = (ctypes.c_int32 * 8)(0, -9, -9, -9, 1, 8, -9, -9)
    rc, msg = call(make(c=cache(2, 64, block_table_host=ctypes.addressof(table)),
                        kv_lens_host=ctypes.addressof(kv)))
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and "sequence 1 names page 8 of 8" in msg


def test_paged_only():
    assert call(paged_args(cache=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args(kv_lens=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args(cu_seqlens=None))[0] == B.GDN_ERR_INVALID_ARGUMENT  # 4 tokens, 2 sequences
    assert call(paged_args(max_q_len=-1))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args(out_len=4 * 4 * 64 - 1))[0] == B.GDN_ERR_SHAPE
    assert call(paged_args(lse=FAKE, lse_len=15))[0] == B.GDN_ERR_SHAPE
    cu = (ctypes.c_int32 * 3)(0, 3, 4)
    rc, msg = call(paged_args(max_q_len=2, cu_seqlens_host=ctypes.addressof(cu)))
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and "not 0..2 tokens" in msg
    need = B.gdn_attn_paged_workspace_bytes(4, 2, 4, 2, 64)
    assert need > 0
    rc, msg = call(paged_args(workspace_bytes=need - 1))
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and f"needs {need} bytes" in msg
    assert call(paged_args(workspace=FAKE + 128))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args(workspace=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert B.gdn_attn_paged_workspace_bytes(0, 2, 4, 2, 64) == 0
    assert B.gdn_attn_paged_workspace_bytes(4, 2, 4, 2, 64, -1) == 0


def test_prepare_only():
    for rot in (8, 80, -16):
        assert call(prepare_args(rot_dim=rot))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(prepare_args(cos_sin=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(prepare_args(cos_sin_len=31))[0] == B.GDN_ERR_SHAPE
    assert call(prepare_args(norm_eps=float("nan")))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(prepare_args(norm_eps=-1.0))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(prepare_args(cache=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(prepare_args(q_norm_weight_len=63))[0] == B.GDN_ERR_SHAPE
    assert call(prepare_args(k_out=FAKE, k_out_len=511))[0] == B.GDN_ERR_SHAPE
    assert call(prepare_args(v=rows(4, 2, 64, data=None)))[0] == B.GDN_ERR_INVALID_ARGUMENT


def test_binding_refuses_wrong_tensors():
    """Shapes, types, broadcast views and devices, before the library is asked."""
    T, Hq, Hkv, D = 4, 4, 2, 64
    def mk():
        bf = torch.bfloat16
        return dict(q=torch.zeros(T, Hq, D, dtype=bf), k=torch.zeros(T, Hkv, D, dtype=bf),
                    v=torch.zeros(T, Hkv, D, dtype=bf),
                    cu_seqlens=torch.tensor([0, 1, 4], dtype=torch.int32),
                    out=torch.zeros(T, Hq, D, dtype=bf))

    def refused(code, **over):
        a = mk()
        a.update(over)
        with pytest.raises(B.GdnError) as e:
            B.gdn_attn_varlen(a["q"], a["k"], a["v"], a["cu_seqlens"], a["out"],
                              gate=a.get("gate"), lse=a.get("lse"))
        assert e.value.code == code, e.value

    bf = torch.bfloat16
    refused(B.GDN_ERR_INVALID_ARGUMENT)  # nothing wrong but the device
    refused(B.GDN_ERR_SHAPE, v=torch.zeros(T, 1, D, dtype=bf))
    refused(B.GDN_ERR_DTYPE, k=torch.zeros(T, Hkv, D))
    refused(B.GDN_ERR_DTYPE, **{n: torch.zeros(T, h, D, dtype=torch.float16)
                               for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv), ("out", Hq))})
    refused(B.GDN_ERR_DTYPE, cu_seqlens=torch.tensor([0, 1, 4]))
    refused(B.GDN_ERR_INVALID_ARGUMENT, k=torch.zeros(T, 1, D, dtype=bf).expand(T, Hkv, D))
    refused(B.GDN_ERR_INVALID_ARGUMENT, q=torch.zeros(T, D, Hq, dtype=bf).transpose(1, 2))
    refused(B.GDN_ERR_INVALID_ARGUMENT, out=torch.zeros(T, 2 * Hq, D, dtype=bf)[:, ::2])
    refused(B.GDN_ERR_SHAPE, gate=torch.zeros(T, Hkv, D, dtype=bf))
    refused(B.GDN_ERR_DTYPE, lse=torch.zeros(T, Hq, dtype=bf))
    kc = torch.zeros(8, Hkv, 16, D, dtype=bf)
    a = mk()
    for table, code in ((torch.zeros(3, 4, dtype=torch.int32), B.GDN_ERR_SHAPE),
                        (torch.zeros(2, 4), B.GDN_ERR_DTYPE),
                        (torch.zeros(4, 2, dtype=torch.int32).t(), B.GDN_ERR_INVALID_ARGUMENT),
                        (torch.zeros(4, dtype=torch.int32), B.GDN_ERR_SHAPE)):
        with pytest.raises(B.GdnError) as e:
            B.gdn_attn_paged(a["q"], kc, kc, table, torch.ones(2, dtype=torch.int32),
                             a["cu_seqlens"], a["out"])
        assert e.value.code == code, e.value


def test_reference_sees_a_mask_off_by_one():
    """A causal mask shifted by one key breaks the bound the kernels are held to."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(9, 2, 64, generator=g) for _ in range(3))
    out, lse, pieces = R.varlen(q, k, v, [9], 0.125)
    wrong, wlse, _ = R.attention_rows(R.f64(q), R.f64(k), R.f64(v), 1, 0.125)
    tol = R.bound(out, pieces, torch.bfloat16, True)
    assert (np.abs(wrong[:8] - out[:8]) > tol[:8]).mean() > 0.5
    assert (np.abs(wlse[:8] - lse[:8]) > R.lse_bound(lse, pieces)[:8]).all()
