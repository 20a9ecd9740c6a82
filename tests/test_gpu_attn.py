"""GPU parity of the full-attention calls against the plain 64-bit forms of
tests/attn_reference.py, within bounds computed from the reference's values."""
import numpy as np
import pytest
import torch

import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def cu_of(lens, dev):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)


def randn(gen, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def strided(t, pad):
    """The same values in rows `pad` elements wider per token (a view)."""
    if not pad:
        return t
    T, H, D = t.shape
    wide = torch.full((T, H * D + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, :H * D].view(T, H, D)
    view.copy_(t)
    return view


def make_paged(gen, kv_lens, Hkv, D, page, dtype, dev, layout="head", poison=True):
    """A shuffled cache; places no sequence owns hold NaN."""
    need = [-(-n // page) for n in kv_lens]
    pages, width = sum(need) + 2, max(max(need), 1) + 1
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    k = torch.full((pages, Hkv, page, D), float("nan") if poison else 0.0)
    v = k.clone()
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
        for i in range(n):
            rows = min(page, kv_lens[s] - i * page)
            k[table[s, i], :, :rows] = torch.randn(Hkv, rows, D, generator=gen)
            v[table[s, i], :, :rows] = torch.randn(Hkv, rows, D, generator=gen)
    k, v = k.to(dtype).to(dev), v.to(dtype).to(dev)
    if layout == "token":     # [pages, page, Hkv, D] memory
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
        v = v.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "joint":   # one tensor [pages, 2, Hkv, page, D]
        kv = torch.stack([k, v], 1)
        k, v = kv[:, 0], kv[:, 1]
    return k, v, table.to(dev)


def ref_cache(t):
    return torch.nan_to_num(t.float(), nan=0.0)


# ---- packed prompts -------------------------------------------------------------

VARLEN = [
    # lens, Hq, Hkv, D, dtype, gate, pad
    ([1], 1, 1, 64, BF, False, 0),
    ([1, 2, 3], 8, 1, 128, BF, True, 64),
    ([64], 4, 4, 128, BF, False, 0),
    ([127, 1, 130], 4, 2, 64, BF, False, 16),
    ([300], 6, 2, 128, BF, True, 0),          # group of 3: tiles of 42 tokens
    ([129, 0, 255], 5, 1, 128, BF, False, 8),  # an empty sequence, a group of 5
    ([257, 33], 16, 2, 256, BF, True, 0),
    ([40, 300], 4, 1, 256, BF, False, 0),
    ([200], 64, 1, 64, BF, False, 0),         # the widest group
    ([90, 41], 7, 1, 64, BF, False, 0),
    ([77, 130], 4, 2, 32, BF, False, 0),
    ([1, 65, 130], 4, 2, 128, F32, True, 4),
    ([70], 6, 2, 256, F32, False, 0),
    ([33, 1], 3, 1, 64, F32, False, 0),
    ([50], 2, 2, 32, F32, False, 0),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,gated,pad", VARLEN)
def test_varlen(lens, Hq, Hkv, D, dtype, gated, pad, cuda_device):
    g = torch.Generator().manual_seed(sum(lens) + D)
    T = sum(lens)
    q, k, v = (randn(g, T, h, D, dtype=dtype, std=s) for h, s in ((Hq, 1.5), (Hkv, 1), (Hkv, 1)))
    gate = randn(g, T, Hq, D, dtype=dtype) if gated else None
    dev = cuda_device
    out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    lse = torch.full((T, Hq), float("nan"), device=dev)
    cu = cu_of(lens, dev)
    B.gdn_attn_varlen(strided(q.to(dev), pad), strided(k.to(dev), pad), strided(v.to(dev), pad), cu,
                      out, gate=None if gate is None else strided(gate.to(dev), pad), lse=lse,
                      cu_seqlens_host=cu)
    B.gdn_read_device_status()
    ro, rl, pieces = R.varlen(q, k, v, lens, D ** -0.5, gate)
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, dtype == BF), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


def test_varlen_scale_and_large_scores(cuda_device):
    """Scores of several hundred: the running maximum has to move often."""
    g = torch.Generator().manual_seed(3)
    lens, Hq, Hkv, D = [700], 4, 1, 128
    q = randn(g, 700, Hq, D)
    # keys grow along the sequence, so later tiles raise the maximum
    k = (torch.randn(700, Hkv, D, generator=g) * torch.linspace(0.1, 6, 700)[:, None, None]).to(BF)
    v = randn(g, 700, Hkv, D)
    out = torch.empty(700, Hq, D, dtype=BF, device=cuda_device)
    B.gdn_attn_varlen(q.to(cuda_device), k.to(cuda_device), v.to(cuda_device),
                      cu_of(lens, cuda_device), out, scale=1.0)
    ro, rl, pieces = R.varlen(q, k, v, lens, 1.0)
    R.check(R.f64(out), ro, R.bound(ro, pieces, BF, True), "out")


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (128, F32)])
def test_varlen_sequences_do_not_mix(D, dtype, cuda_device):
    """NaN and infinities in one sequence, or in later tokens of the same one,
    leave every row that does not attend to them bit for bit as it was."""
    g = torch.Generator().manual_seed(D)
    lens, Hq, Hkv = [70, 90, 140], 4, 2
    T = sum(lens)
    q, k, v = (randn(g, T, h, D, dtype=dtype).to(cuda_device) for h in (Hq, Hkv, Hkv))
    cu = cu_of(lens, cuda_device)
    clean = torch.empty(T, Hq, D, dtype=dtype, device=cuda_device)
    B.gdn_attn_varlen(q, k, v, cu, clean)
    kb, vb = k.clone(), v.clone()
    kb[75:160] = float("nan")
    vb[75:160] = float("inf")
    vb[260, 1] = float("inf")      # a late token of the last sequence, kv head 1
    kb[261, 0] = float("-inf")
    out = torch.empty_like(clean)
    B.gdn_attn_varlen(q, kb, vb, cu, out)
    tol = dict(rtol=2.0 ** -7, atol=1e-2) if dtype == BF else dict(rtol=1e-4, atol=1e-4)
    for a, b in ((0, 75), (160, 260)):
        torch.testing.assert_close(out[a:b], clean[a:b], **tol)
    torch.testing.assert_close(out[260:261, :2], clean[260:261, :2], **tol)
    assert not torch.isfinite(out[75:160].float()).any()
    assert not torch.isfinite(out[260:, 2:].float()).any()


def test_varlen_malformed_offsets_are_flagged(cuda_device):
    dev = cuda_device
    q = torch.randn(8, 2, 64, device=dev, dtype=BF)
    out = torch.empty_like(q)
    for bad in ([0, 5, 3, 8], [0, 4, 9, 8], [0, 4, 6, 7], [1, 4, 6, 8], [-4, 4, 6, 8]):
        B.gdn_attn_varlen(q, q, q, torch.tensor(bad, dtype=torch.int32, device=dev), out)
        with pytest.raises(B.GdnError) as e:
            B.gdn_read_device_status()
        assert e.value.code == B.GDN_ERR_DEVICE_CHECK, bad
    B.gdn_attn_varlen(q, q, q, cu_of([8], dev), out)
    B.gdn_read_device_status()


# ---- paged ----------------------------------------------------------------------

PAGED = [
    # q_lens (None: one token each), kv_lens, Hq, Hkv, D, page, dtype, gate, layout
    (None, [1], 1, 1, 64, 16, BF, False, "head"),
    (None, [1, 16, 17, 128, 129, 0, 300], 8, 2, 128, 16, BF, True, "head"),
    (None, [1000, 3], 16, 2, 256, 64, BF, True, "token"),
    (None, [2100], 4, 1, 128, 128, BF, False, "joint"),     # split over the keys
    (None, [500, 700], 6, 2, 64, 32, BF, False, "token"),
    (None, [260, 31], 64, 1, 64, 256, BF, False, "head"),
    (None, [100, 40], 4, 2, 32, 16, BF, False, "head"),
    (None, [100, 41, 0], 4, 2, 128, 5, BF, False, "head"),   # pages of 5 rows
    ([4, 1, 3, 0, 2], [300, 64, 3, 9, 1], 8, 2, 128, 16, BF, False, "head"),  # L < q_len last
    ([5, 2], [700, 129], 16, 2, 256, 64, BF, False, "joint"),
    ([8, 8], [130, 1030], 8, 1, 64, 16, BF, True, "head"),
    ([70, 1, 200], [70, 500, 801], 4, 2, 128, 64, BF, False, "token"),  # chunks
    ([300], [1200], 8, 2, 128, 16, BF, True, "head"),
    ([260, 9], [263, 700], 8, 1, 256, 128, BF, False, "head"),
    ([40, 130], [41, 390], 10, 2, 64, 48, BF, False, "head"),  # pages of 48
    ([5, 300], [3, 290], 4, 1, 128, 32, BF, False, "head"),   # rows before any key
    (None, [1, 70, 0, 515], 4, 2, 128, 16, F32, True, "head"),
    ([3, 70], [200, 75], 6, 2, 64, 16, F32, False, "token"),
    ([2, 1], [1500, 2], 4, 1, 256, 64, F32, False, "joint"),
]


def run_paged(case, dev, seed=0, **kw):
    q_lens, kv_lens, Hq, Hkv, D, page, dtype, gated, layout = case
    g = torch.Generator().manual_seed(sum(kv_lens) + D + seed)
    ql = q_lens or [1] * len(kv_lens)
    T = sum(ql)
    q = randn(g, T, Hq, D, dtype=dtype, std=1.5)
    gate = randn(g, T, Hq, D, dtype=dtype) if gated else None
    kc, vc, table = make_paged(g, kv_lens, Hkv, D, page, dtype, dev, layout)
    out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    lse = torch.full((T, Hq), float("nan"), device=dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    cu = cu_of(ql, dev) if q_lens else None
    B.gdn_attn_paged(q.to(dev), kc, vc, table, kv, cu, out, lse=lse,
                     gate=None if gate is None else gate.to(dev), max_q_len=max(ql), **kw)
    ro, rl, pieces = R.paged(q, ref_cache(kc), ref_cache(vc), table, kv_lens, ql, D ** -0.5, gate)
    return out, lse, ro, rl, pieces, dtype


@pytest.mark.parametrize("case", PAGED)
def test_paged(case, cuda_device):
    out, lse, ro, rl, pieces, dtype = run_paged(case, cuda_device)
    B.gdn_read_device_status()
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, dtype == BF), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


def test_paged_host_mirrors_and_workspace(cuda_device):
    """Mirrors are accepted, a workspace full of NaN changes nothing."""
    dev = cuda_device
    g = torch.Generator().manual_seed(1)
    kv_lens, Hq, Hkv, D = [900, 31], 8, 2, 128
    kc, vc, table = make_paged(g, kv_lens, Hkv, D, 16, BF, dev)
    q = randn(g, 2, Hq, D).to(dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    outs = []
    for fill in (0, 255):
        ws = torch.full((B.gdn_attn_paged_workspace_bytes(2, 2, Hq, Hkv, D, 1),), fill,
                        dtype=torch.uint8, device=dev)
        out = torch.empty_like(q)
        B.gdn_attn_paged(q, kc, vc, table, kv, None, out, workspace=ws, kv_lens_host=kv,
                         block_table_host=table)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    B.gdn_read_device_status()
    with pytest.raises(B.GdnError):
        B.gdn_attn_paged(q, kc, vc, table, kv, None, out, kv_lens_host=kv + 10 ** 6)


def test_paged_bad_metadata_is_flagged(cuda_device):
    """Pages outside the cache and lengths outside the table: flagged, nothing
    read out of bounds (the kernels clamp lengths and read such pages as 0)."""
    dev = cuda_device
    g = torch.Generator().manual_seed(2)
    for D, page, dtype in ((128, 16, BF), (64, 5, BF), (64, 16, F32)):
        kc, vc, table = make_paged(g, [100, 60], 2, D, page, dtype, dev, poison=False)
        q = randn(g, 2, 4, D, dtype=dtype).to(dev)
        out = torch.empty_like(q)

        def call(tb, kv, cu=None, qq=q, o=out, mq=0):
            B.gdn_attn_paged(qq, kc, vc, tb, torch.tensor(kv, dtype=torch.int32, device=dev), cu, o,
                             max_q_len=mq)

        for pg in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
            tb = table.clone()
            tb[1, 2] = pg
            call(tb, [100, 60])
            with pytest.raises(B.GdnError) as e:
                B.gdn_read_device_status()
            assert e.value.code == B.GDN_ERR_DEVICE_CHECK
        for kv in ([-1, 60], [100, 10 ** 6], [2 ** 31 - 1, 60]):
            tb = table.clamp(min=0)
            call(tb, kv)
            with pytest.raises(B.GdnError):
                B.gdn_read_device_status()
        q3 = randn(g, 6, 4, D, dtype=dtype).to(dev)
        call(table, [100, 60], cu_of([4, 2], dev), q3, torch.empty_like(q3), mq=2)
        with pytest.raises(B.GdnError):
            B.gdn_read_device_status()
        call(table, [100, 60])
        B.gdn_read_device_status()


def test_paged_many_sequences(cuda_device):
    """More sequences than threads in a block, most of them empty."""
    case = (None, [(i * 37) % 50 if i % 3 == 0 else 0 for i in range(1100)], 2, 1, 64, 16, BF, False,
            "head")
    out, lse, ro, rl, pieces, dtype = run_paged(case, cuda_device)
    B.gdn_read_device_status()
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, True), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


def test_paged_offsets_past_32_bits(cuda_device):
    """A cache of more than 2^32 elements: the pages used are its last ones."""
    dev, Hkv, page, D = cuda_device, 8, 64, 128
    pages = 2 ** 32 // (Hkv * page * D) + 40
    kc = torch.empty(pages, Hkv, page, D, dtype=BF, device=dev)
    g = torch.Generator().manual_seed(4)
    kv_lens = [1000, 333]
    small_k, small_v, small_t = make_paged(g, kv_lens, Hkv, D, page, BF, dev, poison=False)
    n = small_k.shape[0]
    kc[pages - n:] = small_k
    vc = torch.empty_like(kc)
    vc[pages - n:] = small_v
    q = randn(g, 2, 16, D).to(dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    small, big = torch.empty_like(q), torch.empty_like(q)
    B.gdn_attn_paged(q, small_k, small_v, small_t, kv, None, small)
    table = torch.where(small_t >= 0, small_t + (pages - n), small_t)
    B.gdn_attn_paged(q, kc, vc, table, kv, None, big)
    assert torch.equal(small, big)
    q2 = randn(g, 300, 16, D).to(dev)
    cu = cu_of([200, 100], dev)
    a, b = torch.empty_like(q2), torch.empty_like(q2)
    B.gdn_attn_paged(q2, small_k, small_v, small_t, kv, cu, a)
    B.gdn_attn_paged(q2, kc, vc, table, kv, cu, b)
    assert torch.equal(a, b)
    # and the prepare that writes there
    k_new = randn(g, 2, Hkv, D).to(dev)
    q_out = torch.empty_like(q)
    B.gdn_attn_prepare(q, k_new, k_new, None, q_out, kv_lens=kv, block_table=table, k_cache=kc,
                       v_cache=vc)
    torch.cuda.synchronize()
    for s, L in enumerate(kv_lens):
        pg = int(table[s, (L - 1) // page])
        assert torch.equal(kc[pg, :, (L - 1) % page], k_new[s])
        assert torch.equal(vc[pg, :, (L - 1) % page], k_new[s])
    del kc, vc
    torch.cuda.empty_cache()


def test_paged_equals_varlen(cuda_device):
    """A prompt computed whole equals the same prompt in two chunks over a cache
    that gdn_attn_prepare filled (same keys; sums in another order)."""
    dev = cuda_device
    g = torch.Generator().manual_seed(8)
    L, Hq, Hkv, D, page = 333, 8, 2, 128, 16
    q, k, v = (randn(g, L, h, D).to(dev) for h in (Hq, Hkv, Hkv))
    whole = torch.empty_like(q)
    B.gdn_attn_varlen(q, k, v, cu_of([L], dev), whole)
    pages = -(-L // page)
    kc = torch.zeros(pages, Hkv, page, D, dtype=BF, device=dev)
    vc = torch.zeros_like(kc)
    table = torch.randperm(pages, generator=g).to(torch.int32).view(1, -1).to(dev)
    parts = []
    for a, b in ((0, 200), (200, L)):
        kv = torch.tensor([b], dtype=torch.int32, device=dev)
        qo = torch.empty(b - a, Hq, D, dtype=BF, device=dev)
        cu = cu_of([b - a], dev)
        B.gdn_attn_prepare(q[a:b], k[a:b], v[a:b], cu, qo, kv_lens=kv, block_table=table,
                           k_cache=kc, v_cache=vc)
        assert torch.equal(qo, q[a:b])
        o = torch.empty_like(qo)
        B.gdn_attn_paged(qo, kc, vc, table, kv, cu, o, max_q_len=b - a)
        parts.append(o)
    torch.testing.assert_close(torch.cat(parts), whole, rtol=2.0 ** -6, atol=2e-3)
    B.gdn_read_device_status()


# ---- prepare --------------------------------------------------------------------

PREPARE = [
    # q_lens (None: one each), kv_lens, Hq, Hkv, D, rot, page, dtype, norm, gated rows, layout
    (None, [1, 17, 64, 0], 8, 2, 128, 128, 16, BF, True, False, "head"),
    ([70, 1, 0, 33], [70, 300, 5, 40], 4, 1, 256, 64, 64, BF, True, True, "token"),
    ([5, 130], [3, 131], 6, 3, 64, 16, 7, BF, False, False, "joint"),   # tokens before the context
    ([40], [40], 3, 1, 32, 32, 16, BF, True, False, "head"),
    ([1, 64], [77, 64], 4, 2, 128, 0, 16, F32, True, False, "head"),
    ([33, 2], [33, 500], 4, 2, 256, 256, 32, F32, True, True, "token"),
    ([3, 90], [9, 95], 2, 1, 64, 48, 16, F32, False, False, "head"),    # a pair 3 lanes apart
    ([500], [500], 1, 1, 32, 16, 64, F32, True, False, "head"),
    ([2000, 48], [2000, 3000], 16, 4, 128, 64, 64, BF, True, True, "head"),
]


@pytest.mark.parametrize("case", PREPARE)
@pytest.mark.parametrize("own_positions", [False, True])
def test_prepare(case, own_positions, cuda_device):
    q_lens, kv_lens, Hq, Hkv, D, rot, page, dtype, norm, gated, layout = case
    dev = cuda_device
    g = torch.Generator().manual_seed(D + rot)
    ql = q_lens or [1] * len(kv_lens)
    T = sum(ql)
    per = 2 * D if gated else D
    row = randn(g, T, Hq * per + 2 * Hkv * D, dtype=dtype).to(dev)
    q = row[:, :Hq * per].view(T, Hq, per)[:, :, :D]
    k = row[:, Hq * per:Hq * per + Hkv * D].view(T, Hkv, D)
    v = row[:, Hq * per + Hkv * D:].view(T, Hkv, D)
    qw = (torch.rand(D, generator=g) + 0.5).to(dtype).to(dev) if norm else None
    kw = (torch.rand(D, generator=g) + 0.5).to(dtype).to(dev) if norm else None
    cs = torch.randn(max(max(kv_lens), 1) + 3, rot, generator=g).to(dev) if rot else None
    kc, vc, table = make_paged(g, kv_lens, Hkv, D, page, dtype, dev, layout, poison=False)
    before_k, before_v = kc.clone(), vc.clone()
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(ql, kv_lens)] or [[]]).astype(int)
    seq = np.repeat(np.arange(len(ql)), ql)
    rpos = (pos * 7 + 3) % max(1, cs.shape[0] if rot else 1) if own_positions else pos
    q_out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    k_out = torch.full((T, Hkv, D), float("nan"), dtype=dtype, device=dev)
    B.gdn_attn_prepare(q, k, v, cu_of(ql, dev) if q_lens else None, q_out, kv_lens=kv,
                       block_table=table, k_cache=kc, v_cache=vc, k_out=k_out, q_norm_weight=qw,
                       k_norm_weight=kw, norm_eps=1e-5, cos_sin=cs,
                       positions=torch.tensor(rpos, dtype=torch.int32, device=dev)
                       if own_positions else None)
    B.gdn_read_device_status()
    shown = pos >= 0
    cos = sin = None
    if rot:
        tab = R.f64(cs)[np.where(shown, rpos, 0)]
        cos, sin = tab[:, :rot // 2], tab[:, rot // 2:]
    for x, w, got, what in ((q, qw, q_out, "q"), (k, kw, k_out, "k")):
        y, mag = R.norm_rotate(R.f64(x), None if w is None else R.f64(w), 1e-5, cos, sin)
        y, mag = y * shown[:, None, None], mag * shown[:, None, None]
        R.check(R.f64(got), y, R.prepare_bound(y, mag, D, dtype), what)
    # the cache holds k_out's rows and v's, and is otherwise untouched
    want_k, want_v = before_k, before_v
    for t in np.flatnonzero(shown):
        pg = int(table[seq[t], pos[t] // page])
        want_k[pg, :, pos[t] % page] = k_out[t]
        want_v[pg, :, pos[t] % page] = v[t]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_prepare_without_cache(cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(0)
    x = randn(g, 37, 3, 64).to(dev)
    q_out, k_out = torch.empty(37, 2, 64, dtype=BF, device=dev), torch.empty(37, 1, 64, dtype=BF,
                                                                             device=dev)
    B.gdn_attn_prepare(x[:, :2], x[:, 2:], x[:, 2:], cu_of([30, 7], dev), q_out, k_out=k_out)
    assert torch.equal(q_out, x[:, :2]) and torch.equal(k_out, x[:, 2:])
    B.gdn_read_device_status()


def test_prepare_bad_metadata_is_flagged(cuda_device):
    """Nothing is written for the bad token: its q row is zero."""
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    kc, vc, table = make_paged(g, [20, 20], 1, 64, 16, BF, dev, poison=False)
    x = randn(g, 2, 1, 64).to(dev)
    cs = torch.ones(64, 64, device=dev)

    def call(tb=table, kv=(20, 20), cu=None, positions=None):
        k0, v0 = kc.clone(), vc.clone()
        q_out = torch.full_like(x, float("nan"))
        B.gdn_attn_prepare(x, x, x, cu, q_out, kv_lens=torch.tensor(kv, dtype=torch.int32, device=dev),
                           block_table=tb, k_cache=k0, v_cache=v0, cos_sin=cs, positions=positions)
        with pytest.raises(B.GdnError) as e:
            B.gdn_read_device_status()
        assert e.value.code == B.GDN_ERR_DEVICE_CHECK
        return q_out, (k0 != kc).any() or (v0 != vc).any()

    for pg in (-1, kc.shape[0], 2 ** 31 - 1):
        tb = table.clone()
        tb[:, 1] = pg
        assert not call(tb=tb)[1]
    for kv in ((-1, -5), (10 ** 6, 49), (2 ** 31 - 1, 49)):
        assert not call(kv=kv)[1]
    for p in (-1, 64, 2 ** 31 - 1):
        q_out, wrote = call(positions=torch.tensor([p, p], dtype=torch.int32, device=dev))
        assert not wrote and not q_out.any()
    assert not call(cu=torch.tensor([0, 5, 2], dtype=torch.int32, device=dev))[1]
    q_out = torch.empty_like(x)
    B.gdn_attn_prepare(x, x, x, None, q_out, kv_lens=torch.tensor([20, 20], dtype=torch.int32, device=dev),
                       block_table=table, k_cache=kc, v_cache=vc, cos_sin=cs)
    B.gdn_read_device_status()


# ---- streams and graphs ---------------------------------------------------------

def test_side_stream_and_graph_replay(cuda_device):
    """Prepare and paged attention captured once, replayed with other lengths
    and rows (a padded sequence among them): equal to the eager calls."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    N, Hq, Hkv, D, page = 5, 8, 2, 128, 16
    kv_sets = [[40, 1, 300, 17, 0], [41, 2, 301, 0, 500], [700, 3, 1, 18, 64]]
    most = [max(s[i] for s in kv_sets) for i in range(N)]
    kc, vc, table = make_paged(g, most, Hkv, D, page, BF, dev, poison=False)
    rows = [randn(g, N, (Hq + 2 * Hkv) * D).to(dev) for _ in kv_sets]
    row = torch.empty_like(rows[0])
    kv = torch.zeros(N, dtype=torch.int32, device=dev)
    cs = torch.randn(1024, D, generator=g).to(dev)
    ws = torch.empty(B.gdn_attn_paged_workspace_bytes(N, N, Hq, Hkv, D, 1), dtype=torch.uint8,
                     device=dev)

    def step(row, kv, k0, v0, q_out, out, stream=None):
        q = row[:, :Hq * D].view(N, Hq, D)
        k = row[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
        v = row[:, (Hq + Hkv) * D:].view(N, Hkv, D)
        B.gdn_attn_prepare(q, k, v, None, q_out, kv_lens=kv, block_table=table, k_cache=k0,
                           v_cache=v0, cos_sin=cs, stream=stream)
        B.gdn_attn_paged(q_out, k0, v0, table, kv, None, out, workspace=ws, stream=stream)

    def bufs():
        return kc.clone(), vc.clone(), torch.empty(N, Hq, D, dtype=BF, device=dev), \
            torch.empty(N, Hq, D, dtype=BF, device=dev)

    eager, e = [], bufs()
    for r, s in zip(rows, kv_sets):
        step(r, torch.tensor(s, dtype=torch.int32, device=dev), *e)
        eager.append(e[3].clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = bufs()
    torch.cuda.synchronize()
    got = []
    for r, s in zip(rows, kv_sets):     # the explicit stream argument
        kv_s = torch.tensor(s, dtype=torch.int32, device=dev)
        torch.cuda.synchronize()
        step(r, kv_s, *b, stream=side)
        side.synchronize()
        got.append(b[3].clone())
    c = bufs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(row, kv, *c)
    replay = []
    for r, s in zip(rows, kv_sets):
        row.copy_(r)
        kv.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        replay.append(c[3].clone())
    for x, y, z in zip(eager, got, replay):
        assert torch.equal(x, y) and torch.equal(x, z)
    assert torch.equal(e[0], c[0]) and torch.equal(e[1], c[1])
    B.gdn_read_device_status()


# ---- f32 and other sizes: few rows, clusters of key shares -------------------------

@pytest.mark.parametrize("case", [
    (None, [700, 5, 0, 64], 16, 1, 64, 16, F32, True, "head"),     # 16 rows at D = 64
    (None, [300, 129], 8, 1, 128, 64, F32, False, "token"),        # 8 rows
    ([2, 1, 2], [900, 1, 2], 4, 2, 128, 7, F32, True, "joint"),    # 2 tokens x 2 heads
    ([1, 4], [33, 600], 1, 1, 256, 16, F32, False, "head"),        # 4 rows at D = 256
    ([3, 2], [40, 500], 6, 2, 32, 3, BF, False, "head"),           # 9 rows at D = 32
    ([9, 30], [9, 1500], 8, 2, 256, 16, F32, True, "head"),        # tiles in clusters
    ([200], [900], 12, 4, 64, 9, BF, False, "head"),               # bf16, pages of 9
])
def test_paged_cuda_cores(case, cuda_device):
    out, lse, ro, rl, pieces, dtype = run_paged(case, cuda_device)
    B.gdn_read_device_status()
    R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, dtype == BF), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


def test_paged_poisoned_rows_cuda_cores(cuda_device):
    """A later token's infinite value, in f32: earlier rows of the same call keep
    their results (few rows, and tiles in clusters)."""
    dev = cuda_device
    g = torch.Generator().manual_seed(12)
    for q_len, D in ((2, 128), (40, 64)):
        kc, vc, table = make_paged(g, [400], 1, D, 16, F32, dev, poison=False)
        q = torch.randn(q_len, 2, D, generator=g).to(dev)
        kv = torch.tensor([400], dtype=torch.int32, device=dev)
        cu = cu_of([q_len], dev)
        clean, out = torch.empty_like(q), torch.empty_like(q)
        B.gdn_attn_paged(q, kc, vc, table, kv, cu, clean, max_q_len=q_len)
        vc[table[0, 24], 0, 15] = float("inf")  # position 399, the last token's own
        B.gdn_attn_paged(q, kc, vc, table, kv, cu, out, max_q_len=q_len)
        torch.testing.assert_close(out[:-1], clean[:-1], rtol=1e-5, atol=1e-6)
        assert not torch.isfinite(out[-1]).any()


# ---- what is written ------------------------------------------------------------------

class Guarded:
    """Buffers with 4 KB of a NaN bit pattern on either side."""

    def __init__(self, dev):
        self.dev, self.all = dev, []

    def new(self, shape, dtype, fill=0.0):
        n = int(np.prod(shape))
        pad = 4096 // torch.empty(0, dtype=dtype).element_size()
        raw = torch.empty(n + 2 * pad, dtype=dtype, device=self.dev)
        raw.view(torch.uint8).fill_(0x7F)
        raw.view(torch.uint8).add_(0x80)  # 0xff bytes
        body = raw[pad:pad + n]
        body.fill_(fill)
        self.all.append((raw, pad, n))
        return body.view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, pad, n in self.all:
            for side in (raw[:pad], raw[pad + n:]):
                assert (side.view(torch.uint8) == 0xFF).all()


@pytest.mark.parametrize("dtype,D,page", [(BF, 128, 16), (BF, 256, 64), (BF, 64, 5), (F32, 128, 16),
                                          (F32, 32, 16)])
def test_nothing_is_written_outside(dtype, D, page, cuda_device):
    dev = cuda_device
    gd = Guarded(dev)
    g = torch.Generator().manual_seed(D)
    Hq, Hkv = 6, 2
    for ql, kl in (([1, 1, 1], [3, 700, 0]), ([3, 1, 2], [40, 1, 500]), ([130, 5], [130, 900])):
        T, N = sum(ql), len(ql)
        width = -(-max(kl) // page)
        kc = gd.new((N * width, Hkv, page, D), dtype)
        vc = gd.new((N * width, Hkv, page, D), dtype)
        table = torch.randperm(N * width, generator=g).to(torch.int32).view(N, width).to(dev)
        kv = torch.tensor(kl, dtype=torch.int32, device=dev)
        q, k, v = (randn(g, T, h, D, dtype=dtype).to(dev) for h in (Hq, Hkv, Hkv))
        q_out, k_out = gd.new((T, Hq, D), dtype), gd.new((T, Hkv, D), dtype)
        out, lse = gd.new((T, Hq, D), dtype), gd.new((T, Hq), F32)
        need = B.gdn_attn_paged_workspace_bytes(T, N, Hq, Hkv, D, max(ql), B._dt(q))
        ws = gd.new((need,), torch.uint8, 0)
        cs = torch.randn(max(kl) + 1, 32, generator=g).to(dev)
        cu = cu_of(ql, dev)
        B.gdn_attn_prepare(q, k, v, cu, q_out, kv_lens=kv, block_table=table, k_cache=kc, v_cache=vc,
                           k_out=k_out, cos_sin=cs)
        B.gdn_attn_paged(q_out, kc, vc, table, kv, cu, out, max_q_len=max(ql), lse=lse, workspace=ws)
        B.gdn_attn_varlen(q_out, k_out, v, cu, out, lse=lse)
        gd.check()
    B.gdn_read_device_status()


def test_results_repeat_bit_for_bit(cuda_device):
    """No sum's order depends on timing: key ranges over SMs and clusters included."""
    dev = cuda_device
    g = torch.Generator().manual_seed(2)
    for dtype, D, ql, kl in ((BF, 128, [1] * 5, [900, 31, 4000, 0, 77]), (BF, 256, [2, 3], [3000, 50]),
                             (F32, 64, [1, 1], [2000, 300]), (F32, 128, [70], [300]),
                             (BF, 128, [300, 200], [300, 2000])):
        kc, vc, table = make_paged(g, kl, 2, D, 16, dtype, dev, poison=False)
        q = randn(g, sum(ql), 8, D, dtype=dtype).to(dev)
        kv = torch.tensor(kl, dtype=torch.int32, device=dev)
        outs = []
        for _ in range(20):
            out = torch.empty_like(q)
            B.gdn_attn_paged(q, kc, vc, table, kv, cu_of(ql, dev), out, max_q_len=max(ql))
            outs.append(out)
        assert all(torch.equal(outs[0], o) for o in outs[1:])
    q, k = randn(g, 3000, 8, 128).to(dev), randn(g, 3000, 2, 128).to(dev)
    cu = cu_of([1700, 300, 1000], dev)
    outs = []
    for _ in range(20):
        out = torch.empty_like(q)
        B.gdn_attn_varlen(q, k, k, cu, out)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_varlen_long_against_key_blocks(D, cuda_device):
    """A prompt of many key tiles and items per SM, against the f64 form of some of
    its rows (the whole would take too long)."""
    dev = cuda_device
    g = torch.Generator().manual_seed(D)
    lens, Hq, Hkv = [2999, 1500, 700], 16, 2
    T = sum(lens)
    q, k, v = (randn(g, T, h, D, std=s) for h, s in ((Hq, 1.5), (Hkv, 1), (Hkv, 1)))
    out = torch.empty(T, Hq, D, dtype=BF, device=dev)
    for _ in range(3):  # back to back: the later calls find the SMs' memory used
        B.gdn_attn_varlen(q.to(dev), k.to(dev), v.to(dev), cu_of(lens, dev), out)
    B.gdn_read_device_status()
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    for a, n in zip(starts, lens):
        for i in sorted({0, 1, 127, 128, n // 2, n - 129, n - 2, n - 1}):
            ro, rl, pieces = R.attention_rows(R.f64(q[a + i:a + i + 1]), R.f64(k[a:a + n]),
                                              R.f64(v[a:a + n]), i, D ** -0.5)
            R.check(R.f64(out[a + i:a + i + 1]), ro, R.bound(ro, pieces, BF, True), f"row {i} of {n}")


# ---- heads of 256: two row tiles share their keys --------------------------------

def test_varlen_256_short_items(cuda_device):
    """Hundreds of items of one or two key tiles, each with a last key inside the
    tile: tiles whose second half has no row, full ones, empty sequences."""
    dev = cuda_device
    g = torch.Generator().manual_seed(21)
    lens = [(i * 29) % 67 if i % 7 else 0 for i in range(150)] + [130, 1, 257]
    T, Hq, Hkv, D = sum(lens), 8, 2, 256
    q, k, v = (randn(g, T, h, D, std=s) for h, s in ((Hq, 1.5), (Hkv, 1), (Hkv, 1)))
    cu = cu_of(lens, dev)
    outs = []
    for _ in range(10):
        out = torch.full((T, Hq, D), float("nan"), dtype=BF, device=dev)
        lse = torch.full((T, Hq), float("nan"), device=dev)
        B.gdn_attn_varlen(q.to(dev), k.to(dev), v.to(dev), cu, out, lse=lse)
        outs.append(out)
    B.gdn_read_device_status()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    ro, rl, pieces = R.varlen(q, k, v, lens, D ** -0.5, None)
    R.check(R.f64(outs[0]), ro, R.bound(ro, pieces, BF, True), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


@pytest.mark.parametrize("case", [
    ([300, 20], [4000, 1021], 8, 1, 256, 16, BF, True, "head"),     # few items: key ranges
    ([130, 33, 0, 64], [130, 2000, 7, 900], 16, 2, 256, 48, BF, False, "token"),
    ([90] * 30, [90 + 31 * i for i in range(30)], 16, 4, 256, 128, BF, False, "joint"),  # many
])
def test_paged_256(case, cuda_device):
    first = None
    for _ in range(2):
        out, lse, ro, rl, pieces, dtype = run_paged(case, cuda_device)
        B.gdn_read_device_status()
        R.check(R.f64(out), ro, R.bound(ro, pieces, dtype, True), "out")
        R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")
        assert first is None or torch.equal(first, out)
        first = out


@pytest.mark.parametrize("D,dtype,q_len,kv", [(128, BF, 200, 9000), (256, BF, 100, 9001), (64, BF, 300, 3003),
                                              (256, BF, 3, 20001), (128, F32, 70, 2000),
                                              (32, F32, 2, 3001)])
def test_paged_infinite_value_in_sight(D, dtype, q_len, kv, cuda_device):
    """An infinite value that every row sees: its dim is infinite, the others are
    what they are without it, and no wait runs out over the rows' evaluation."""
    dev = cuda_device
    g = torch.Generator().manual_seed(D + q_len)
    Hq, Hkv, page = 8, 2, 16
    kc, vc, table = make_paged(g, [kv], Hkv, D, page, dtype, dev, poison=False)
    q = randn(g, q_len, Hq, D, dtype=dtype).to(dev)
    lens = torch.tensor([kv], dtype=torch.int32, device=dev)
    cu = cu_of([q_len], dev)
    j = 1003
    vc[table[0, j // page], 1, j % page, 5] = 0.0
    clean, out = torch.empty_like(q), torch.empty_like(q)
    lse, lse0 = (torch.empty(q_len, Hq, device=dev) for _ in range(2))
    B.gdn_attn_paged(q, kc, vc, table, lens, cu, clean, max_q_len=q_len, lse=lse0)
    vc[table[0, j // page], 1, j % page, 5] = float("inf")
    B.gdn_attn_paged(q, kc, vc, table, lens, cu, out, max_q_len=q_len, lse=lse)
    B.gdn_read_device_status()
    assert (out[:, 4:, 5] == float("inf")).all()
    out[:, 4:, 5] = clean[:, 4:, 5]
    # Both sides carry the tiled form's error: P rounded to bf16 (2^-8 of each weight,
    # of values of size 1), and a store's rounding; in f32 sums in two orders.
    tol = dict(rtol=2.0 ** -7, atol=2.0 ** -7) if dtype == BF else dict(rtol=1e-4, atol=1e-5)
    torch.testing.assert_close(out, clean, **tol)
    torch.testing.assert_close(lse, lse0, rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("D,Hq,Hkv,q_len", [(128, 32, 4, 1216), (256, 16, 2, 1216)])
def test_paged_long_evaluation_is_not_a_timeout(D, Hq, Hkv, q_len, cuda_device):
    """Rows evaluated key by key for longer than any wait of the kernel may last (about
    a second): the waits of the other roles, and of a pair's other CTA, go on."""
    dev = cuda_device
    kv, page = 70000, 64
    g = torch.Generator(device=dev).manual_seed(D)
    pages = -(-kv // page)
    kc, vc = (torch.randn(pages, Hkv, page, D, generator=g, device=dev).to(BF) for _ in range(2))
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(1, -1)
    q = torch.randn(q_len, Hq, D, generator=g, device=dev).to(BF)
    lens = torch.tensor([kv], dtype=torch.int32, device=dev)
    cu = cu_of([q_len], dev)
    vc[table[0, 0], :, 3, 5] = 0.0
    clean, out = torch.empty_like(q), torch.empty_like(q)
    B.gdn_attn_paged(q, kc, vc, table, lens, cu, clean, max_q_len=q_len)
    for i in range(0, pages, 8):  # in every key range, should there be several
        vc[table[0, i], :, 3, 5] = float("inf")
    B.gdn_attn_paged(q, kc, vc, table, lens, cu, out, max_q_len=q_len)
    B.gdn_read_device_status()
    assert (out[:, :, 5] == float("inf")).all()
    rest = [d for d in range(D) if d != 5]
    torch.testing.assert_close(out[..., rest], clean[..., rest], rtol=2.0 ** -7, atol=2.0 ** -7)
