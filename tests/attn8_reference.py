"""Plain forms of the 8-bit cache: its quantisation step by step on the CPU (exact: a
value divided by a power of two, torch's rounding to e4m3), and the values it stands
for, for the 64-bit attention of attn_reference.py."""
import numpy as np
import torch

import attn_reference as R

E4M3 = torch.float8_e4m3fn


def need(amax):
    """The smallest power of two, 2^-64 at least, with amax <= 448 times it (f64 in)."""
    s = 2.0 ** -64
    while amax > 448.0 * s:
        s *= 2.0
    return s


def encode(x, scale):
    """f32 values to e4m3 codes of x / scale; what is not finite becomes NaN."""
    y = (x.double() / scale).float()
    y[~torch.isfinite(x)] = float("nan")
    return y.to(E4M3)


def write_rows(codes, scales, table_row, first, x, block):
    """Rows x [n, Hkv, D] (f32) at positions first.. of one sequence, into codes [pages,
    Hkv, page, D] and scales [pages, Hkv, page / block] (CPU tensors, in place)."""
    page = codes.shape[2]
    n, Hkv, _ = x.shape
    at = 0
    while at < n:
        pos = first + at
        m = min(n - at, block - pos % block)
        if pos < 0:
            at += min(n - at, -pos)
            continue
        pg, row, b, r = int(table_row[pos // page]), pos % page, pos % page // block, pos % block
        for h in range(Hkv):
            new = x[at:at + m, h]
            fin = new[torch.isfinite(new)]
            s = need(float(fin.abs().max()) if fin.numel() else 0.0)
            if r > 0:
                old = float(scales[pg, h, b])
                if s > old:
                    c = codes[pg, h, row - r:row].float()
                    codes[pg, h, row - r:row] = (c.double() * (old / s)).float().to(E4M3)
                s = max(s, old)
            scales[pg, h, b] = s
            codes[pg, h, row:row + m] = encode(new, s)
        at += m


def values(codes, scales):
    """The values that a cache stands for, f64 [pages, Hkv, page, D]."""
    P, H, page, D = codes.shape
    nb = scales.shape[2]
    c = R.f64(codes.cpu().float()).reshape(P, H, nb, page // nb, D)
    return (c * R.f64(scales)[..., None, None]).reshape(P, H, page, D)


def paged(q, kc, ks, vc, vs, table, kv_lens, q_lens, scale, gate=None):
    k, v, table = values(kc, ks), values(vc, vs), table.cpu().numpy()
    page = k.shape[2]
    ctx = []
    for s, L in enumerate(kv_lens):
        pos = np.arange(L)
        pg = table[s][pos // page]
        ctx.append((k[pg, :, pos % page], v[pg, :, pos % page], L - q_lens[s]))
    return R._packed(R.f64(q), ctx, q_lens, scale, None if gate is None else R.f64(gate))


def half_code(y):
    """Half a step of e4m3 at magnitude y (below 2^-6: of its subnormals)."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return np.exp2(e - 4)
