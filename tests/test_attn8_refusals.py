"""Refusals of the calls on an 8-bit cache, on the CPU: nothing is launched (fake device
addresses, never dereferenced)."""
import ctypes

import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B
from test_attn_refusals import FAKE, cache, paged_args, prepare_args


def cache8(Hkv=2, D=64, page=16, block=16, pages=8, **over):
    codes = {k: over.pop(k) for k in list(over) if k not in ("k_scale", "v_scale", "k_scale_len", "v_scale_len")}
    n = pages * Hkv * (page // block if block else 0)
    a = dict(codes=cache(Hkv, D, pages=pages, page=page, **codes), k_scale=FAKE, k_scale_len=n, v_scale=FAKE,
             v_scale_len=n, block=block)
    a.update(over)
    return B.gdn_attn_cache8(**a)


def call(make, c, base_cache=None, **over):
    base = make(**over)
    base.cache = base_cache
    cls, fn = ((B.gdn_attn8_paged_args, "gdn_attn8_paged") if make is paged_args
               else (B.gdn_attn8_prepare_args, "gdn_attn8_prepare"))
    a = cls(base=base, cache=None if c is None else ctypes.pointer(c))
    L = B.lib()
    return getattr(L, fn)(ctypes.byref(a), None), L.gdn_last_error_message().decode()


@pytest.mark.parametrize("make", [paged_args, prepare_args])
def test_cache8(make):
    L = B.lib()
    assert L.gdn_attn8_paged(None, None) == B.GDN_ERR_INVALID_ARGUMENT
    assert L.gdn_attn8_prepare(None, None) == B.GDN_ERR_INVALID_ARGUMENT
    rc, msg = call(make, None)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and msg == "cache is NULL"
    rc, msg = call(make, cache8(), base_cache=ctypes.pointer(cache(2, 64)))
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and "not in base.cache" in msg
    for block in (0, 8, 24, 256, -16):
        rc, msg = call(make, cache8(block=block))
        assert rc == B.GDN_ERR_UNSUPPORTED and "16, 32, 64 or 128" in msg
    rc, msg = call(make, cache8(page=48, block=32))
    assert rc == B.GDN_ERR_SHAPE and "multiple of the scale block" in msg
    rc, msg = call(make, cache8(k_scale_len=15))
    assert rc == B.GDN_ERR_SHAPE and msg == "attention k_scale length 15 < expected 16"
    assert call(make, cache8(v_scale_len=15))[0] == B.GDN_ERR_SHAPE
    assert call(make, cache8(v_scale=None))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make, cache8(k_scale=FAKE + 4))[0] == B.GDN_ERR_INVALID_ARGUMENT
    # lengths and strides count codes
    assert call(make, cache8(k_len=8 * 2 * 16 * 64 - 1))[0] == B.GDN_ERR_SHAPE
    assert call(make, cache8(v_len=1 << 30, v_token_stride=72))[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(make, cache8(k=FAKE + 8))[0] == B.GDN_ERR_INVALID_ARGUMENT


def test_paged8_sizes():
    assert call(paged_args, cache8(pages=2, v_len=1 << 50, v_page_stride=1 << 41))[0] == B.GDN_ERR_UNSUPPORTED
    rc, msg = call(paged_args, cache8(), T=40, N=2, workspace_bytes=16)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and msg.startswith("gdn_attn8_paged workspace needs")
    assert call(paged_args, cache8(), max_q_len=-1)[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args, cache8(), kv_lens=None)[0] == B.GDN_ERR_INVALID_ARGUMENT
    assert call(paged_args, cache8(), D=48)[0] == B.GDN_ERR_UNSUPPORTED
    f = B.gdn_attn8_paged_workspace_bytes
    assert f(4, 2, 4, 2, 48) == 0 and f(4, 2, 3, 2, 64) == 0 and f(4, 2, 4, 2, 64, -1) == 0
    assert f(4, 2, 4, 2, 64, 0, B.GDN_DTYPE_BF16, 0, 16) == 0
    assert f(4, 2, 4, 2, 64, 0, B.GDN_DTYPE_BF16, 1 << 30, 1 << 10) == 0


def test_wide_workspace_grows_with_the_table_up_to_a_group():
    """A chunk's workspace holds widened contexts: per sequence up to 1 GiB, then one
    sequence at a time."""
    f = B.gdn_attn8_paged_workspace_bytes
    one = f(2048, 1, 32, 4, 128, 2048, B.GDN_DTYPE_BF16, 256, 128)
    assert one >= 256 * 128 * 4 * 128 * 2 * 2
    many = f(2048 * 100, 100, 32, 4, 128, 2048, B.GDN_DTYPE_BF16, 256, 128)
    assert many < 3 << 30
    long = f(2048, 2, 32, 4, 128, 2048, B.GDN_DTYPE_BF16, 1 << 14, 128)
    assert long >= (1 << 14) * 128 * 4 * 128 * 2 * 2


def test_binding():
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(8, 2, 32, 64, dtype=torch.float8_e4m3fn)
    sc = torch.zeros(8, 2, 2)
    table, kv = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    good = dict(k_cache=kc, v_cache=kc, k_scale=sc, v_scale=sc, block_table=table)

    def paged(**over):
        a = dict(good, **over)
        with pytest.raises(B.GdnError) as e:
            B.gdn_attn8_paged(q, a["k_cache"], a["v_cache"], a["k_scale"], a["v_scale"], a["block_table"], kv,
                              None, torch.empty_like(q))
        return e.value

    def prep(**over):
        with pytest.raises(B.GdnError) as e:
            B.gdn_attn8_prepare(q, q[:, :2], q[:, :2], None, torch.empty_like(q), kv_lens=kv, **dict(good, **over))
        return e.value

    for f in (paged, prep):
        assert f(k_cache=kc.view(torch.uint8)).code == B.GDN_ERR_DTYPE
        assert f(v_cache=torch.zeros(8, 2, 32, 64, dtype=torch.bfloat16)).code == B.GDN_ERR_DTYPE
        assert f(k_scale=torch.zeros(8, 2, 3)).code == B.GDN_ERR_SHAPE
        assert f(k_scale=torch.zeros(8, 2)).code == B.GDN_ERR_SHAPE
        assert f(k_scale=torch.zeros(8, 2, 0)).code == B.GDN_ERR_SHAPE
        assert f(v_scale=torch.zeros(8, 2, 1)).code == B.GDN_ERR_SHAPE
        assert f(v_scale=torch.zeros(8, 2, 2, dtype=torch.float64)).code == B.GDN_ERR_DTYPE
        assert f(k_scale=torch.zeros(8, 2, 4)[..., ::2]).code == B.GDN_ERR_INVALID_ARGUMENT
        assert f(k_cache=kc[:, :1].expand(8, 2, 32, 64)).code == B.GDN_ERR_INVALID_ARGUMENT
        assert "CUDA device" in f().msg
    for name in good:
        assert prep(**{name: None}).code == B.GDN_ERR_INVALID_ARGUMENT
