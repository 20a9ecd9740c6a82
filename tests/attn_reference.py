"""Plain 64-bit forms of the full-attention operators, one row at a time in
numpy, and the error bounds the kernels are held to.

A bound is computed per element from the reference's own values, with u =
2^-24 (half a step of f32) and h = half a step of the stored type:
  score   s = scale q.k over D products: |ds| <= scale (D + 4) u sum_d |q_d k_d|
          (any order of f32 additions; tensor cores may cut instead of round:
          2 u per addition)
  weight  e^(s - m) with |s - m| <= S relative to the row maximum: relative
          2 |ds| + (S + 8) u: the exponent's argument, the exponential's own
          two ulp, and the rounded maximum that cancels in the quotient
  sums    n terms: (n + 8) 2 u relative to sum_j w_j |v_j|
  P       a weight stored in bf16 for the product with v: 2^-8 more (the sum l
          takes the weight before that rounding)
  store   h |out|
so |d out| <= A (2 max|ds| + (2 n + S + 64) u + P) + h |out|, A = sum w_j |v_j|.
"""
import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def attention_rows(q, k, v, first, scale, gate=None):
    """q [n, Hq, D] at positions first.. over k, v [L, Hkv, D] (f64 arrays).
    Returns out, lse, and the pieces of the bound (A, max|ds|, S, keys)."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    A = np.zeros((n, Hq, D))
    ds = np.zeros((n, Hq))
    S = np.zeros((n, Hq))
    keys = np.zeros((n, Hq))
    for i in range(n):
        m = first + i + 1
        if m <= 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // G], v[:m, h // G]
            s = scale * (kk @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            z = w.sum()
            out[i, h] = w @ vv / z
            lse[i, h] = top + np.log(z)
            A[i, h] = w @ np.abs(vv) / z
            # Scores whose weight is negligible do not matter: the relevant
            # score error is that of the weights' own mean.
            e = abs(scale) * (D + 4) * 2 * U * (np.abs(kk) @ np.abs(q[i, h]))
            ds[i, h] = e.max()
            S[i, h] = min((top - s).max(), 104.0)
            keys[i, h] = m
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-gate))
        out = out * sg
        A = A * sg
    return out, lse, (A, ds, S, keys)


def bound(out, pieces, dtype, p_bf16):
    A, ds, S, keys = pieces
    rel = 2 * ds + (2 * keys + S + 64) * U + (2.0 ** -8 if p_bf16 else 0.0)
    return A * rel[..., None] + half_step(dtype) * np.abs(out) + 1e-37


def lse_bound(lse, pieces):
    _, ds, S, keys = pieces
    return ds + (2 * keys + S + 64) * U + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def varlen(q, k, v, lens, scale, gate=None):
    """Packed prompts; torch tensors in, arrays out (out, lse, pieces)."""
    return _packed(f64(q), [(f64(k)[a:b], f64(v)[a:b], 0) for a, b in _ranges(lens)], lens, scale,
                   None if gate is None else f64(gate))


def paged(q, kc, vc, table, kv_lens, q_lens, scale, gate=None):
    kc, vc, table = f64(kc), f64(vc), table.cpu().numpy()
    page = kc.shape[2]
    ctx = []
    for s, L in enumerate(kv_lens):
        pos = np.arange(L)
        pg = table[s][pos // page]
        ctx.append((kc[pg, :, pos % page], vc[pg, :, pos % page], L - q_lens[s]))
    return _packed(f64(q), ctx, q_lens, scale, None if gate is None else f64(gate))


def _ranges(lens):
    a = 0
    for n in lens:
        yield a, a + n
        a += n


def _packed(q, ctx, lens, scale, gate):
    outs, lses, pieces = [], [], []
    for (a, b), (k, v, first) in zip(_ranges(lens), ctx):
        o, l, p = attention_rows(q[a:b], k, v, first, scale, None if gate is None else gate[a:b])
        outs.append(o)
        lses.append(l)
        pieces.append(p)
    return (np.concatenate(outs), np.concatenate(lses),
            tuple(np.concatenate([p[i] for p in pieces]) for i in range(4)))


def check(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    assert np.isfinite(got[~inf]).all(), f"{what}: non-finite"
    err = np.abs(got[~inf] - ref[~inf])
    t = np.broadcast_to(tol, ref.shape)[~inf]
    worst = float((err / t).max()) if err.size else 0.0
    print(f"{what}: worst error {worst:.3f} of its bound, max |err| {err.max() if err.size else 0:.2e}")
    assert worst <= 1.0, f"{what}: error {worst:.2f} times its bound"


# ---- prepare ------------------------------------------------------------------

def norm_rotate(x, w, eps, cos, sin):
    """x [T, H, D] f64; cos, sin [T, R/2] (None: no rotary).  Returns y and the
    magnitude its rounding errors are relative to."""
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if cos is None:
        return y, np.abs(y)
    h = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    a, b = y[..., :h], y[..., h:2 * h]
    rot = np.concatenate([a * c - b * s, b * c + a * s, y[..., 2 * h:]], -1)
    mag = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s),
                          np.abs(y[..., 2 * h:])], -1)
    return rot, mag


def prepare_bound(y, mag, D, dtype):
    """The mean of D squares, its root and three products (half the sum's
    relative error reaches the root): (D / 2 + 16) u; then the store."""
    return mag * (D / 2 + 16) * 2 * U + half_step(dtype) * np.abs(y) + 1e-37
