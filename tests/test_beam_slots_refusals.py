"""Refusals of gdn_beam_select and gdn_copy_slots, on the CPU: nothing is launched (fake
device addresses, never dereferenced)."""
import ctypes

import pytest
import torch

from gated_delta_rule_44_gb300 import binding as B

FAKE = 0x100000


def beam(n=2, W=4, V=100, K=4, **over):
    a = dict(B=n, W=W, V=V, K=K, dtype=B.GDN_DTYPE_BF16, logits=FAKE, logits_len=n * W * V, scores=FAKE,
             scores_len=n * W, parents=FAKE, parents_len=n * K, tokens=FAKE, tokens_len=n * K, out_scores=FAKE,
             out_scores_len=n * K, workspace=FAKE, workspace_bytes=1 << 40)
    a.update(over)
    args = B.gdn_beam_select_args(**a)
    return B.lib().gdn_beam_select(ctypes.byref(args), None), B.lib().gdn_last_error_message().decode()


def test_beam():
    SHAPE, ARG, UNS = B.GDN_ERR_SHAPE, B.GDN_ERR_INVALID_ARGUMENT, B.GDN_ERR_UNSUPPORTED
    assert B.lib().gdn_beam_select(None, None) == ARG
    for name in ("n", "W", "V", "K"):
        assert beam(**{name: 0})[0] == SHAPE
        assert beam(**{name: -1})[0] == SHAPE
    assert beam(dtype=9)[0] == B.GDN_ERR_DTYPE
    assert beam(W=65)[0] == UNS and beam(K=129)[0] == UNS
    assert beam(W=64, V=1 << 26)[0] == UNS
    rc, msg = beam(logits_len=799)
    assert rc == SHAPE and msg == "beam_select logits length 799 < expected 800"
    assert beam(beam_stride=101)[0] == SHAPE and beam(batch_stride=500)[0] == SHAPE
    assert beam(beam_stride=-100)[0] == SHAPE and beam(batch_stride=1 << 62)[0] == SHAPE
    for name, least in (("scores", 8), ("parents", 8), ("tokens", 8), ("out_scores", 8)):
        assert beam(**{name + "_len": least - 1})[0] == SHAPE
        assert beam(**{name: None})[0] == ARG
    assert beam(finished=FAKE, finished_len=7)[0] == SHAPE
    assert beam(finished=FAKE, finished_len=8, pad_token=100)[0] == ARG
    assert beam(finished=FAKE, finished_len=8, pad_token=-1)[0] == ARG
    assert beam(logits=FAKE + 1)[0] == ARG and beam(logits=None)[0] == ARG
    rc, msg = beam(workspace_bytes=8)
    assert rc == ARG and msg.startswith("gdn_beam_select workspace needs")
    assert beam(workspace=FAKE + 64)[0] == ARG
    f = B.gdn_beam_select_workspace_bytes
    assert f(2, 4, 100, 4) > 0 and f(0, 4, 100, 4) == 0 and f(2, 65, 100, 4) == 0


def test_beam_workspace_does_for_smaller_calls():
    f = B.gdn_beam_select_workspace_bytes
    for W, V, K in ((1, 131072, 1), (4, 32003, 8), (8, 131072, 16), (3, 200, 3), (64, 5000, 128)):
        needs = [f(n, W, V, K) for n in range(1, 700)]
        assert needs == sorted(needs)
        assert f(50, W, V - 100, K) <= f(50, W, V, K) and f(50, W, V, K) <= f(50, W, V, K + 1 if K < 128 else K)
        # a list for every chunk of 4096, or a row's two ends and what 304 blocks cut
        assert needs[-1] <= (304 + 2 * 699 * W) * (16 + 8 * K)


def pool(**over):
    a = dict(data=FAKE, len=10 * 64, slots=10, slot_bytes=64, slot_stride=0)
    a.update(over)
    return B.gdn_slot_pool(**a)


def slots(*pools, n=4, group=0, dst_host=None, src_host=None, **over):
    arr = (B.gdn_slot_pool * max(1, len(pools)))(*pools)
    keep = [None if h is None else (ctypes.c_int32 * len(h))(*h) for h in (dst_host, src_host)]
    a = dict(pools=arr, num_pools=len(pools), n=n, group=group, dst=FAKE, src=FAKE)
    for name, k in zip(("dst_host", "src_host"), keep):
        a[name] = None if k is None else ctypes.addressof(k)
    a.update(over)
    args = B.gdn_copy_slots_args(**a)
    return B.lib().gdn_copy_slots(ctypes.byref(args), None), B.lib().gdn_last_error_message().decode()


def test_slots():
    SHAPE, ARG, UNS = B.GDN_ERR_SHAPE, B.GDN_ERR_INVALID_ARGUMENT, B.GDN_ERR_UNSUPPORTED
    assert B.lib().gdn_copy_slots(None, None) == ARG
    assert slots()[0] == SHAPE and slots(pool(), n=-1)[0] == SHAPE and slots(pool(), group=-2)[0] == SHAPE
    assert slots(pool(), n=0) == (B.GDN_OK, "")
    assert slots(pool(), group=129, n=129)[0] == UNS
    assert slots(pool(), group=3)[0] == SHAPE
    assert slots(pool(), dst=None)[0] == ARG and slots(pool(), src=None)[0] == ARG
    assert slots(pool(), n=1 << 33)[0] == UNS
    assert slots(pool(slots=0))[0] == SHAPE and slots(pool(slot_bytes=0))[0] == SHAPE
    assert slots(pool(len=639))[0] == SHAPE and slots(pool(slot_stride=60))[0] == SHAPE
    assert slots(pool(len=1 << 50, slot_stride=1 << 62))[0] == SHAPE
    assert slots(pool(slot_bytes=62))[0] == ARG and slots(pool(data=FAKE + 2))[0] == ARG
    assert slots(pool(len=1 << 20, slot_stride=66))[0] == ARG and slots(pool(data=None))[0] == ARG
    rc, msg = slots(pool(), pool())
    assert rc == ARG and msg == "copy_slots pool 1 is given twice"


@pytest.mark.parametrize("dst,src,group,text", [
    ([1, 2, 3, 10], [4, 5, 6, 7], 0, "names 10 from 7"),
    ([1, 2, 3, 8], [4, 5, 6, 10], 0, "names 8 from 10"),
    ([1, 2, 1, 8], [4, 5, 6, 7], 0, "slot 1 is a destination twice"),
    ([1, 2, 3, 8], [4, 5, 6, 2], 0, "slot 2 is both a source and a destination"),
    ([1, 2, 3, 8], [0, 1, 2, 0], 2, "groups of 2"),
    ([1, 2, 3, 1], [0, 1, 1, 0], 2, "slot 1 is a destination twice"),
])
def test_slots_mirrors(dst, src, group, text):
    rc, msg = slots(pool(), group=group, dst_host=dst, src_host=src)
    assert rc == B.GDN_ERR_INVALID_ARGUMENT and text in msg


def test_slots_mirrors_that_are_right():
    """Negative entries, slots onto themselves and cycles pass the checks, and fail at the
    device lookup of a machine without one."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for dst, src, group in (([1, -1, 3, 8], [4, 1, 3, -1], 0), ([1, 2, 3, -1], [1, 0, -1, 0], 2)):
        rc, msg = slots(pool(), group=group, dst_host=dst, src_host=src, dst=FAKE)
        assert rc == B.GDN_ERR_CUDA, msg


def test_binding():
    x, s = torch.zeros(2, 3, 50), torch.zeros(2, 3)
    i32, f = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)

    def sel(logits=x, scores=s, parents=i32, tokens=i32, best=f, **over):
        with pytest.raises(B.GdnError) as e:
            B.gdn_beam_select(logits, scores, parents, tokens, best, **over)
        return e.value

    assert sel(x[0]).code == B.GDN_ERR_SHAPE
    assert sel(scores=s[:, :2]).code == B.GDN_ERR_SHAPE
    assert sel(scores=s.double()).code == B.GDN_ERR_DTYPE
    assert sel(tokens=i32.long()).code == B.GDN_ERR_DTYPE
    assert sel(tokens=i32[:, :3]).code == B.GDN_ERR_SHAPE
    assert sel(best=torch.zeros(4, 2).t()).code == B.GDN_ERR_INVALID_ARGUMENT
    assert sel(logits=x.half()).code == B.GDN_ERR_DTYPE
    assert sel(logits=torch.zeros(2, 50, 3).transpose(1, 2)).code == B.GDN_ERR_INVALID_ARGUMENT
    assert sel(logits=x[:, :1].expand(2, 3, 50)).code == B.GDN_ERR_INVALID_ARGUMENT
    assert sel(finished=torch.zeros(2, 3)).code == B.GDN_ERR_DTYPE
    assert "CUDA device" in sel().msg

    d = torch.zeros(4, dtype=torch.int32)

    def copy(pools=None, dst=d, src=d, **over):
        with pytest.raises(B.GdnError) as e:
            B.gdn_copy_slots([torch.zeros(5, 8)] if pools is None else pools, dst, src, **over)
        return e.value

    assert copy(pools=[]).code == B.GDN_ERR_SHAPE
    assert copy(dst=d.long()).code == B.GDN_ERR_DTYPE
    assert copy(src=d[:3]).code == B.GDN_ERR_SHAPE
    assert copy(groups=True).code == B.GDN_ERR_SHAPE
    assert copy(dst=d.view(2, 2), src=d.view(2, 2)).code == B.GDN_ERR_SHAPE
    assert copy(pools=[torch.zeros(5, 0)]).code == B.GDN_ERR_SHAPE
    assert copy(pools=[torch.zeros(8, 5).t()]).code == B.GDN_ERR_INVALID_ARGUMENT
    assert copy(pools=[torch.zeros(1, 8).expand(5, 8)]).code == B.GDN_ERR_INVALID_ARGUMENT
    assert "CUDA device" in copy().msg
