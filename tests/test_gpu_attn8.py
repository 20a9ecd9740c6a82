"""GPU parity of the calls on an 8-bit cache against the plain forms of
tests/attn8_reference.py.  What is written without a norm and rotary positions is
compared bit for bit; the rest within bounds computed from the reference's values."""
import numpy as np
import pytest
import torch

import attn8_reference as Q
import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from test_gpu_attn import BF, F32, cu_of, randn, strided

pytestmark = pytest.mark.gpu
E4M3 = Q.E4M3


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


def make_cache8(gen, kv_lens, Hkv, D, page, block, dev, layout="head", poison=True, spread=1.0):
    """A shuffled 8-bit cache; places no sequence owns hold NaN codes, and blocks without an
    owned row NaN scales.  Returns device tensors and CPU copies (codes, scales, table)."""
    need = [-(-n // page) for n in kv_lens]
    pages, width = sum(need) + 2, max(max(need), 1) + 1
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    bad = float("nan") if poison else 0.0
    cpu = []
    for _ in range(2):
        x = torch.full((pages, Hkv, page, D), bad)
        sc = torch.full((pages, Hkv, page // block), bad)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
            for i in range(n):
                rows = min(page, kv_lens[s] - i * page)
                pg = int(table[s, i])
                x[pg, :, :rows] = torch.randn(Hkv, rows, D, generator=gen)
                nb = -(-rows // block)
                sc[pg, :, :nb] = 2.0 ** torch.randint(-8, -5, (Hkv, nb), generator=gen).float() * spread
        step = sc.repeat_interleave(block, 2)[..., None]
        cpu.append(((x / step).clamp(-448, 448).to(E4M3), sc))
    (kc, ks), (vc, vs) = cpu

    def place(t):
        if layout == "token":     # [pages, page, Hkv, D] memory
            return t.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
        return t.to(dev)
    dk, dv = place(kc.view(torch.uint8)), place(vc.view(torch.uint8))
    if layout == "joint":         # one tensor [pages, 2, Hkv, page, D]
        kv = torch.stack([dk, dv], 1)
        dk, dv = kv[:, 0], kv[:, 1]
    return (dict(k_cache=dk.view(E4M3), v_cache=dv.view(E4M3), k_scale=ks.to(dev), v_scale=vs.to(dev),
                 block_table=table.to(dev)), (kc, ks, vc, vs, table))


# ---- the cache's rows --------------------------------------------------------------

WRITE = [
    # q_lens, kv_lens, Hkv, D, page, block, dtype, layout
    ([1], [1], 1, 64, 16, 16, BF, "head"),
    ([1, 1, 1, 1], [17, 16, 40, 1], 2, 128, 32, 16, BF, "head"),
    ([5, 0, 40, 33], [21, 9, 40, 100], 3, 64, 32, 32, BF, "token"),
    ([300, 1], [300, 64], 2, 256, 64, 64, BF, "joint"),
    ([130, 7], [391, 130], 1, 128, 128, 128, BF, "head"),
    ([6, 3], [2, 0], 2, 32, 16, 16, BF, "head"),          # tokens without a position
    ([70, 1, 2], [133, 48, 50], 2, 32, 48, 16, F32, "token"),
    ([200], [500], 4, 256, 128, 128, F32, "head"),
    ([65, 20], [65, 35], 5, 64, 64, 32, F32, "joint"),
]


@pytest.mark.parametrize("q_lens,kv_lens,Hkv,D,page,block,dtype,layout", WRITE)
def test_write_bits(q_lens, kv_lens, Hkv, D, page, block, dtype, layout, cuda_device):
    """Codes, scales and every byte around them; k without norm and rotary positions is
    written as v is."""
    dev = cuda_device
    g = torch.Generator().manual_seed(sum(q_lens) * 7 + D)
    T, Hq = sum(q_lens), Hkv * 2
    c, (kc, ks, vc, vs, table) = make_cache8(g, kv_lens, Hkv, D, page, block, dev, layout)
    q = randn(g, T, Hq, D, dtype=dtype)
    # Magnitudes that grow along the tokens make blocks that held rows round them again.
    grow = torch.exp2(torch.randint(-6, 7, (T, Hkv, 1), generator=g).float())
    k, v = ((torch.randn(T, Hkv, D, generator=g) * grow).to(dtype) for _ in range(2))
    q_out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    k_out = torch.full((T, Hkv, D), float("nan"), dtype=dtype, device=dev)
    cu, kv = cu_of(q_lens, dev), torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    B.gdn_attn8_prepare(strided(q.to(dev), 16), strided(k.to(dev), 16), strided(v.to(dev), 16), cu,
                        q_out, kv_lens=kv, k_out=k_out, cu_seqlens_host=cu, kv_lens_host=kv, **c)
    B.gdn_read_device_status()
    a = 0
    for s, n in enumerate(q_lens):
        first = kv_lens[s] - n
        Q.write_rows(kc, ks, table[s], first, k[a:a + n].float(), block)
        Q.write_rows(vc, vs, table[s], first, v[a:a + n].float(), block)
        seen = torch.arange(first, first + n) >= 0
        assert torch.equal(q_out.cpu()[a:a + n], q[a:a + n] * seen[:, None, None])
        assert torch.equal(k_out.cpu()[a:a + n], k[a:a + n] * seen[:, None, None])
        a += n
    for name, want in (("k_scale", ks), ("v_scale", vs)):
        assert torch.equal(c[name].cpu().nan_to_num(-1), want.nan_to_num(-1)), name
    for name, want in (("k_cache", kc), ("v_cache", vc)):
        got = c[name].cpu().float()
        same = (got == want.float()) | (got.isnan() & want.float().isnan())
        assert same.all(), name


def test_write_step_by_step(cuda_device):
    """The same rows a token, some tokens and a rollback at a time, each step against the
    plain form; without offsets for the single tokens."""
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    Hkv, D, page, block, N = 2, 64, 32, 16, 3
    c, (kc, ks, vc, vs, table) = make_cache8(g, [64] * N, Hkv, D, page, block, dev)
    lens = [0, 3, 15]
    for step, n in enumerate([1, 1, 7, 1, -4, 1, 1, 2, 1, 16, 1]):
        if n < 0:      # drafts refused: their rows are written again
            lens = [max(0, x + n) for x in lens]
            continue
        T = N * n
        grow = torch.exp2(torch.randint(-4, 9, (T, Hkv, 1), generator=g).float())
        k, v = ((torch.randn(T, Hkv, D, generator=g) * grow).to(BF) for _ in range(2))
        lens = [x + n for x in lens]
        cu = None if n == 1 else cu_of([n] * N, dev)
        out = torch.empty(T, Hkv, D, dtype=BF, device=dev)
        B.gdn_attn8_prepare(k.to(dev), k.to(dev), v.to(dev), cu, out,
                            kv_lens=torch.tensor(lens, dtype=torch.int32, device=dev), **c)
        B.gdn_read_device_status()
        for s in range(N):
            Q.write_rows(kc, ks, table[s], lens[s] - n, k[s * n:(s + 1) * n].float(), block)
            Q.write_rows(vc, vs, table[s], lens[s] - n, v[s * n:(s + 1) * n].float(), block)
        for name, want in (("k_scale", ks), ("v_scale", vs), ("k_cache", kc), ("v_cache", vc)):
            assert torch.equal(c[name].cpu().float().nan_to_num(-1), want.float().nan_to_num(-1)), (step, name)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_write_extremes(dtype, cuda_device):
    """Zeros, infinities, NaN, the largest and the smallest values: each block by itself."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    Hkv, D, page, block = 1, 64, 32, 16
    c, (kc, ks, vc, vs, table) = make_cache8(g, [192], Hkv, D, page, block, dev, poison=False)
    x = torch.randn(192, Hkv, D, generator=g)
    x[:16] = 0.0
    x[17, 0, 3], x[18, 0, 4] = float("inf"), float("nan")
    x[32:48] = float("-inf")
    x[48:64] *= 2.0 ** 125
    x[64:80] *= 2.0 ** -120
    x[80] = torch.finfo(dtype).max
    x[96:112] = 448.0 * 2.0 ** -3              # exactly the border
    x[112:128] = 448.0
    x[128, 0, 0] = 450.0
    x[130, 0, 1] = 2.0 ** -9 * 1.5             # ties of the smallest codes
    x[131, 0, 1] = 2.0 ** -10
    x = x.to(dtype)
    out = torch.empty(192, Hkv, D, dtype=dtype, device=dev)
    B.gdn_attn8_prepare(x.to(dev), x.to(dev), x.to(dev), cu_of([192], dev), out,
                        kv_lens=torch.tensor([192], dtype=torch.int32, device=dev), **c)
    B.gdn_read_device_status()
    Q.write_rows(vc, vs, table[0], 0, x.float(), block)
    for name, want in (("v_scale", vs), ("k_scale", vs), ("v_cache", vc), ("k_cache", vc)):
        assert torch.equal(c[name].cpu().float().nan_to_num(-1), want.float().nan_to_num(-1)), name


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,rot,page,block,dtype", [
    ([1, 1, 1], [1, 30, 77], 4, 2, 128, 128, 32, 32, BF),
    ([100, 3], [150, 3], 6, 2, 256, 64, 64, 64, BF),
    ([40, 1], [61, 20], 4, 4, 64, 32, 16, 16, F32),
    ([33], [33], 2, 1, 32, 32, 32, 16, F32),
])
def test_write_norm_and_rotary(q_lens, kv_lens, Hq, Hkv, D, rot, page, block, dtype, cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(D + rot)
    T = sum(q_lens)
    c, (kc, ks, vc, vs, table) = make_cache8(g, kv_lens, Hkv, D, page, block, dev)
    q, k, v = (randn(g, T, h, D, dtype=dtype) for h in (Hq, Hkv, Hkv))
    qw, kw = ((torch.rand(D, generator=g) + 0.5).to(dtype) for _ in range(2))
    ang = torch.rand(max(kv_lens), rot // 2, generator=g, dtype=torch.float64) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    q_out = torch.empty(T, Hq, D, dtype=dtype, device=dev)
    B.gdn_attn8_prepare(q.to(dev), k.to(dev), v.to(dev), cu_of(q_lens, dev), q_out,
                        kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=dev),
                        q_norm_weight=qw.to(dev), k_norm_weight=kw.to(dev), cos_sin=cs.to(dev), **c)
    B.gdn_read_device_status()
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(q_lens, kv_lens)])
    cos, sin = R.f64(cs)[pos, :rot // 2], R.f64(cs)[pos, rot // 2:]
    y, mag = R.norm_rotate(R.f64(q), R.f64(qw), 1e-6, cos, sin)
    R.check(R.f64(q_out), y, R.prepare_bound(y, mag, D, dtype), "q")
    y, mag = R.norm_rotate(R.f64(k), R.f64(kw), 1e-6, cos, sin)
    ybound = mag * (D / 2 + 16) * 2 * R.U
    old = R.f64(ks)
    got, sc = R.f64(c["k_cache"].cpu().float()), R.f64(c["k_scale"])
    a = 0
    for s, n in enumerate(q_lens):
        for b0 in range((kv_lens[s] - n) // block * block, kv_lens[s], block):
            lo = max(b0, kv_lens[s] - n)
            hi = min(b0 + block, kv_lens[s])
            rows = np.arange(a + lo - (kv_lens[s] - n), a + hi - (kv_lens[s] - n))
            pg, r0, bl = int(table[s, lo // page]), lo % page, lo % page // block
            for h in range(Hkv):
                yy, eb = y[rows, h], ybound[rows, h]
                top, slack = np.abs(yy).max(), eb.max()
                choices = {Q.need(top - slack), Q.need(top + slack)}
                if lo > b0:
                    choices = {max(x, old[pg, h, bl]) for x in choices}
                S = sc[pg, h, bl]
                assert S in choices
                err = np.abs(got[pg, h, r0:r0 + len(rows)] - yy / S)
                assert (err <= Q.half_code(yy / S) * (1 + 2.0 ** -10) + eb / S).all()
        a += n


@pytest.mark.parametrize("T,Hkv,D,rot,dtype", [(2000, 2, 128, 128, BF), (700, 1, 256, 64, BF), (900, 3, 64, 64, F32),
                                               (1500, 2, 32, 32, BF), (400, 2, 128, 64, F32)])
@pytest.mark.parametrize("single", [False, True])
def test_write_codes_of_the_exact_values(T, Hkv, D, rot, dtype, single, cuda_device):
    """A key's codes are those of its exact value, in one prompt and token by token: equal to
    the 64-bit value's, which itself is off by 2^-44 of the row's magnitude at most."""
    dev = cuda_device
    g = torch.Generator().manual_seed(T + D)
    page = block = 16
    n = -(-T // page)
    N = T if single else 1
    if single:      # one token per sequence, a page each
        n = T
    table = torch.arange(n, dtype=torch.int32).view(N, -1).to(dev)
    kc = torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device=dev).view(E4M3)
    vc = torch.zeros_like(kc.view(torch.uint8)).view(E4M3)
    ks, vs = torch.zeros(n, Hkv, 1, device=dev), torch.zeros(n, Hkv, 1, device=dev)
    k = randn(g, T, Hkv, D, dtype=dtype)
    kw = (torch.rand(D, generator=g) + 0.5).to(dtype)
    ang = torch.rand(T, rot // 2, generator=g, dtype=torch.float64) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    B.gdn_attn8_prepare(k.to(dev), k.to(dev), k.to(dev), None if single else cu_of([T], dev),
                        torch.empty(T, Hkv, D, dtype=dtype, device=dev),
                        kv_lens=torch.full((N,), 1 if single else T, dtype=torch.int32, device=dev),
                        k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=table, positions=pos,
                        k_norm_weight=kw.to(dev), cos_sin=cs.to(dev))
    B.gdn_read_device_status()
    y, mag = R.norm_rotate(R.f64(k), R.f64(kw), float(np.float32(1e-6)), R.f64(cs)[:, :rot // 2], R.f64(cs)[:, rot // 2:])
    S = R.f64(ks)[:, :, 0] if single else np.repeat(R.f64(ks)[:, :, 0], page, 0)[:T]
    got = R.f64(kc.cpu().float())
    got = got[:, :, 0] if single else got.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T]
    for t in range(0, T, page if not single else 1):       # the scales, from the exact maxima
        rows = slice(t, min(t + (1 if single else page), T))
        for h in range(Hkv):
            top = np.abs(y[rows, h]).max()
            if Q.need(top * (1 - 1e-6)) == Q.need(top * (1 + 1e-6)):
                assert S[t, h] == Q.need(top)
    z = y / S[..., None]
    half = Q.half_code(z)
    slack = 2.0 ** -44 * mag / S[..., None]
    assert (np.abs(got - z) <= half + slack).all()


def test_write_bad_metadata(cuda_device):
    """Pages, lengths and positions that cannot be right: raised, nothing written for them."""
    dev = cuda_device
    g = torch.Generator().manual_seed(9)
    c, (kc, ks, vc, vs, table) = make_cache8(g, [32, 32], 2, 64, 16, 16, dev)
    x = randn(g, 4, 2, 64).to(dev)
    out = torch.empty_like(x)

    def call(kv, **over):
        cc = dict(c, **over)
        B.gdn_attn8_prepare(x, x, x, cu_of([2, 2], dev), out,
                            kv_lens=torch.tensor(kv, dtype=torch.int32, device=dev), **cc)
        with pytest.raises(B.GdnError) as e:
            B.gdn_read_device_status()
        assert e.value.code == B.GDN_ERR_DEVICE_CHECK

    before = {n: bits(c[n]) for n in ("k_cache", "v_cache")}
    wrong = table.clone()
    wrong[:, :2] = torch.tensor([[10 ** 6, -5], [2 ** 31 - 1, 99]], dtype=torch.int32)
    call([32, 32], block_table=wrong.to(dev))
    call([-3, 10 ** 6])
    for n, b in before.items():
        assert torch.equal(bits(c[n]), b), n
    good = torch.tensor([32, 32], dtype=torch.int32, device=dev)
    cos_sin = torch.ones(31, 64, device=dev)
    B.gdn_attn8_prepare(x, x, x, cu_of([2, 2], dev), out, kv_lens=good, cos_sin=cos_sin, **c)
    with pytest.raises(B.GdnError):
        B.gdn_read_device_status()
    # position 31 has no table row: its cache row is as it was
    for s in range(2):
        pg = int(table[s, 1])
        assert torch.equal(bits(c["k_cache"])[pg, :, 15], before["k_cache"][pg, :, 15])


# ---- attention over the cache --------------------------------------------------------

PAGED = [
    # q_lens, kv_lens, Hq, Hkv, D, page, block, dtype, gate, layout
    ([1], [1], 1, 1, 64, 16, 16, BF, False, "head"),
    ([1], [300], 8, 1, 128, 64, 32, BF, True, "head"),
    ([1, 1, 1], [129, 0, 700], 16, 2, 256, 64, 64, BF, True, "token"),
    ([1] * 5, [5, 128, 127, 1000, 31], 4, 4, 64, 32, 16, BF, False, "joint"),
    ([2, 4, 1, 3], [200, 90, 33, 400], 8, 2, 128, 16, 16, BF, False, "head"),
    ([5, 8], [300, 8], 12, 2, 128, 48, 16, BF, False, "token"),
    ([16, 1], [150, 77], 4, 1, 64, 32, 32, BF, True, "head"),
    ([3, 2], [260, 140], 16, 1, 256, 128, 128, BF, False, "head"),
    ([1, 2], [70, 300], 64, 1, 128, 32, 32, BF, False, "head"),       # the widest group
    ([4, 6], [2, 40], 5, 1, 64, 16, 16, BF, False, "head"),            # tokens without a key
    ([40, 7], [300, 7], 8, 2, 128, 64, 32, BF, True, "head"),          # several tiles of rows
    ([20, 1, 0, 40], [500, 300, 9, 41], 12, 2, 128, 32, 16, BF, False, "token"),
    ([4, 3], [700, 2], 64, 1, 64, 64, 32, BF, True, "head"),
    ([9, 16, 5], [129, 1100, 260], 15, 1, 256, 48, 16, BF, False, "head"),
    ([90, 7], [300, 7], 8, 2, 128, 64, 32, BF, True, "head"),          # many rows: widened
    ([130], [200], 4, 1, 256, 16, 16, BF, False, "token"),
    ([17, 100], [400, 100], 6, 2, 64, 112, 16, BF, False, "head"),
    ([1, 3, 0], [90, 40, 9], 4, 2, 32, 32, 16, BF, False, "head"),
    ([60], [130], 2, 1, 32, 16, 16, BF, True, "head"),
    ([1, 1], [333, 40], 4, 2, 128, 32, 16, F32, True, "token"),
    ([2, 1], [90, 300], 2, 1, 256, 64, 64, F32, False, "head"),
    ([1, 4], [200, 64], 12, 3, 64, 16, 16, F32, False, "joint"),
    ([50, 3], [80, 200], 6, 1, 128, 32, 32, F32, False, "head"),
    ([1, 1, 1], [50, 0, 200], 16, 1, 64, 32, 32, F32, False, "head"),  # no offsets, widened
]


def bounds(pieces, ref, dtype):
    """attn_reference's, with the rounding of a weight that the tensor-core forms keep (2^-8
    of it: hi + lo e4m3 parts, or bf16), and two more products per score and value."""
    return R.bound(ref, pieces, dtype, dtype == BF) + 4 * R.U * np.abs(pieces[0])


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page,block,dtype,gated,layout", PAGED)
def test_paged8(q_lens, kv_lens, Hq, Hkv, D, page, block, dtype, gated, layout, cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(sum(kv_lens) + D)
    T = sum(q_lens)
    c, (kc, ks, vc, vs, table) = make_cache8(g, kv_lens, Hkv, D, page, block, dev, layout)
    q = randn(g, T, Hq, D, dtype=dtype, std=1.5)
    gate = randn(g, T, Hq, D, dtype=dtype) if gated else None
    out = torch.full((T, Hq, D), float("nan"), dtype=dtype, device=dev)
    lse = torch.full((T, Hq), float("nan"), device=dev)
    kv = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    cu = None if all(n == 1 for n in q_lens) else cu_of(q_lens, dev)
    B.gdn_attn8_paged(strided(q.to(dev), 16), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                      c["block_table"], kv, cu, out, max_q_len=max(q_lens), lse=lse, kv_lens_host=kv,
                      gate=None if gate is None else strided(gate.to(dev), 32))
    B.gdn_read_device_status()
    ro, rl, pieces = Q.paged(q, kc, ks, vc, vs, table, kv_lens, q_lens, D ** -0.5, gate)
    R.check(R.f64(out), ro, bounds(pieces, ro, dtype), "out")
    R.check(R.f64(lse), rl, R.lse_bound(rl, pieces), "lse")


@pytest.mark.parametrize("q_lens,Hq,D,dtype", [([1], 8, 128, BF), ([3], 4, 64, BF), ([2], 8, 256, BF),
                                               ([30], 8, 128, BF), ([1], 4, 128, F32), ([40], 2, 64, F32)])
def test_paged8_not_finite(q_lens, Hq, D, dtype, cuda_device):
    """NaN codes where no row looks change nothing; a NaN key that is seen makes the rows that
    see it NaN, and only those of its kv head; so does a NaN scale."""
    dev = cuda_device
    g = torch.Generator().manual_seed(D)
    n, L, Hkv, page, block = q_lens[0], 200, 2, 32, 16
    c, (kc, ks, vc, vs, table) = make_cache8(g, [L], Hkv, D, page, block, dev)
    q = randn(g, n, Hq, D, dtype=dtype).to(dev)
    kv = torch.tensor([L], dtype=torch.int32, device=dev)

    def run(codes_k, codes_v, sk, sv):
        out = torch.empty(n, Hq, D, dtype=dtype, device=dev)
        B.gdn_attn8_paged(q, codes_k.to(dev), codes_v.to(dev), sk.to(dev), sv.to(dev), c["block_table"], kv,
                          cu_of(q_lens, dev), out, max_q_len=n)
        B.gdn_read_device_status()
        return out.float().cpu()

    clean = run(kc, vc, ks, vs)
    assert torch.isfinite(clean).all()
    pg, row = int(table[0, (L - 1) // page]), (L - 1) % page
    for which in range(2):
        codes = [kc.clone(), vc.clone()]
        codes[which].view(torch.uint8)[pg, 0, row] = 0x7F     # the last position: only the last token sees it
        got = run(codes[0], codes[1], ks, vs)
        tol = dict(rtol=2.0 ** -7, atol=1e-2) if dtype == BF else dict(rtol=1e-4, atol=1e-4)
        torch.testing.assert_close(got[:n - 1], clean[:n - 1], **tol)
        torch.testing.assert_close(got[:, Hq // 2:], clean[:, Hq // 2:], **tol)
        assert got[n - 1, :Hq // 2].isnan().all()
    pg = int(table[0, 0])
    sk = ks.clone()
    sk[pg, 1, 0] = float("nan")
    got = run(kc, vc, sk, vs)
    assert got[:, Hq // 2:].isnan().all() and torch.isfinite(got[:, :Hq // 2]).all()


@pytest.mark.parametrize("q_len,Hq,D,dtype", [(1, 8, 128, BF), (4, 4, 256, BF), (2, 4, 64, BF), (33, 8, 64, BF),
                                              (1, 2, 128, F32)])
def test_paged8_scales_far_apart(q_len, Hq, D, dtype, cuda_device):
    """Blocks whose scales differ by 2^24, keys that a row prefers among the small ones; the
    largest and zero scales; scores of several hundred."""
    dev = cuda_device
    g = torch.Generator().manual_seed(q_len + D)
    L, Hkv, page, block = 700, 1, 64, 16
    c, (kc, ks, vc, vs, table) = make_cache8(g, [L], Hkv, D, page, block, dev, poison=False)
    vs *= torch.exp2(torch.randint(-12, 13, vs.shape, generator=g).float())
    ks *= torch.exp2(torch.randint(-2, 4, ks.shape, generator=g).float())
    vs[int(table[0, 3]), 0, 1] = 0.0
    ks[int(table[0, 4]), 0, 2] = 0.0
    q = randn(g, q_len, Hq, D, dtype=dtype, std=2.0)
    q[0, 0] *= 2.0 ** 60 if dtype == BF else 1.0       # one key takes all
    q[0, 1] *= 2.0 ** -60
    out = torch.empty(q_len, Hq, D, dtype=dtype, device=dev)
    lse = torch.empty(q_len, Hq, device=dev)
    kv = torch.tensor([L], dtype=torch.int32, device=dev)
    B.gdn_attn8_paged(q.to(dev), c["k_cache"], c["v_cache"], ks.to(dev), vs.to(dev), c["block_table"], kv,
                      cu_of([q_len], dev), out, lse=lse)
    B.gdn_read_device_status()
    ro, rl, pieces = Q.paged(q, kc, ks, vc, vs, table, [L], [q_len], D ** -0.5)
    # The row with a score error above 1 says nothing but which key wins.
    ok = pieces[1] < 0.1
    assert ok.sum() >= ok.size - 1
    R.check(R.f64(out)[ok], ro[ok], bounds(pieces, ro, dtype)[ok], "out")
    R.check(R.f64(lse)[ok], rl[ok], R.lse_bound(rl, pieces)[ok], "lse")


def test_paged8_bad_pages(cuda_device):
    """A page outside the cache reads as zeros: the same as a page of zeros, and raised."""
    dev = cuda_device
    for dtype, q_len, Hq in ((BF, 1, 8), (BF, 40, 8), (F32, 1, 4)):
        g = torch.Generator().manual_seed(4)
        D, page, block, L = 128, 32, 32, 200
        c, (kc, ks, vc, vs, table) = make_cache8(g, [L, L], 1, D, page, block, dev)
        q = randn(g, 2 * q_len, Hq, D, dtype=dtype).to(dev)
        kv = torch.tensor([L, L], dtype=torch.int32, device=dev)
        outs = []
        for bad in (True, False):
            t = table.clone()
            ksd, vsd = ks.clone(), vs.clone()
            if bad:
                t[0, 2], t[1, 6] = 10 ** 8, -1
            for s, i in ((0, 2), (1, 6)):
                ksd[int(table[s, i])] = 0.0
                vsd[int(table[s, i])] = 0.0
            out = torch.empty(2 * q_len, Hq, D, dtype=dtype, device=dev)
            B.gdn_attn8_paged(q, c["k_cache"], c["v_cache"], ksd.to(dev),
                              vsd.to(dev), t.to(dev), kv, cu_of([q_len, q_len], dev), out, max_q_len=q_len)
            if bad:
                with pytest.raises(B.GdnError):
                    B.gdn_read_device_status()
            else:
                B.gdn_read_device_status()
            outs.append(out.float().cpu())
        # (a page of zeros by its scales: 0 times a code; stale NaN codes past L are not seen)
        torch.testing.assert_close(outs[0], outs[1], rtol=2.0 ** -7, atol=1e-3)


@pytest.mark.parametrize("dtype,q_len", [(BF, 1), (BF, 3), (BF, 40), (BF, 70), (F32, 1)])
def test_paged8_repeats_streams_and_graphs(dtype, q_len, cuda_device):
    """Bit for bit the same on another stream, in a graph replayed over changed inputs, and
    beside another call in flight."""
    dev = cuda_device
    g = torch.Generator().manual_seed(11)
    Hq, Hkv, D, page, block = 8, 2, 128, 32, 32
    lens = [700, 33, 1500, 260]
    c, _ = make_cache8(g, lens, Hkv, D, page, block, dev)
    T = q_len * len(lens)
    q = randn(g, T, Hq, D, dtype=dtype).to(dev)
    other = randn(g, T, Hq, D, dtype=dtype).to(dev)
    kv = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = cu_of([q_len] * len(lens), dev)
    dt = B.GDN_DTYPE_BF16 if dtype == BF else B.GDN_DTYPE_F32
    nbytes = B.gdn_attn8_paged_workspace_bytes(T, len(lens), Hq, Hkv, D, q_len, dt, c["block_table"].shape[1], page)

    def run(x, out, ws=None, stream=None):
        B.gdn_attn8_paged(x, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["block_table"], kv, cu,
                          out, max_q_len=q_len, workspace=ws, stream=stream)

    want, want2 = torch.empty_like(q), torch.empty_like(q)
    run(q, want)
    run(other, want2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = torch.empty_like(q), torch.empty_like(q)
    for _ in range(3):
        run(q, a)
        run(other, b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want2)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    x, out = q.clone(), torch.empty_like(q)
    run(x, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(x, out, ws)
    for src, w in ((other, want2), (q, want)):
        x.copy_(src)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    B.gdn_read_device_status()
