"""Measured workloads, and plain forms, of the operators for an 8-bit cache and for
searches over several continuations of a prompt:

  prepare8  per-head RMS norm of q and k, rotary positions, k and v written in
            8 bits into a paged cache                       (gdn_attn8_prepare)
  paged8    attention of new tokens (one, a few drafts, a chunk) over that cache
                                                            (gdn_attn8_paged)
  beam      the best continuations over beams and vocabulary (gdn_beam_select)
  slots     states reordered by the chosen parents, pages copied for a fork
                                                            (gdn_copy_slots)

``own = False`` computes them with elementary torch operations in 32 bits (64 for
the beams' scores, whose order decides), rounded once at the end; ``own = True``
calls the library.

The cache holds e4m3 codes [pages, Hkv, page, D] and f32 scales [pages, Hkv,
page / block]: a value is its code times the scale of its block of tokens and head.
A block's scale is the smallest power of two (2^-64 at least) that brings its values
within 448; rows that join a block raise it where they have to, and the codes that
were there are then rounded again.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------

def _prep(q_lens, kv_lens, Hq, Hkv, D, rot, page, block, dtype, gated):
    return dict(op="prepare8", q_lens=q_lens, kv_lens=kv_lens, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                page=page, block=block, dtype=dtype, gated=gated)


def _paged(q_lens, kv_lens, Hq, Hkv, D, page, block, dtype, gated):
    return dict(op="paged8", q_lens=q_lens, kv_lens=kv_lens, Hq=Hq, Hkv=Hkv, D=D, page=page,
                block=block, dtype=dtype, gated=gated)


def _beam(B, W, V, K, dtype, ended):
    return dict(op="beam", B=B, W=W, V=V, K=K, dtype=dtype, ended=ended)


def _reorder(B, W, layers, Hv, Dk, Dv, conv):
    return dict(op="slots", form="groups", B=B, W=W, layers=layers, Hv=Hv, Dk=Dk, Dv=Dv, conv=conv)


def _fork(n, pages, layers, Hkv, page, block, D):
    return dict(op="slots", form="list", n=n, pages=pages, layers=layers, Hkv=Hkv, page=page,
                block=block, D=D)


def _text(lens):
    """Lengths as a plain value of a case: 'n*len' runs joined by commas."""
    out, i = [], 0
    while i < len(lens):
        j = i
        while j < len(lens) and lens[j] == lens[i]:
            j += 1
        out.append(f"{j - i}*{lens[i]}" if j - i > 1 else str(lens[i]))
        i = j
    return ",".join(out)


def _lens(text):
    out = []
    for part in text.split(","):
        n, _, v = part.rpartition("*")
        out += [int(v)] * (int(n) if n else 1)
    return out


def _uniform(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def listed():
    cases = []

    def add(name, case):
        cases.append(dict(name=name, **case))

    # One new token for each of 512 decoding sequences: latency counts.
    add("prepare8_decode_512", _prep("512*1", _text(_uniform(11, 512, 1, 4096)), 32, 4, 128, 128,
                                     64, 32, "bf16", False))
    # Four new 2048-token prompts, q projected together with its output gate
    # (strided rows), a quarter of the head rotated.
    add("prepare8_prompts_4x2048", _prep("4*2048", "4*2048", 16, 2, 256, 64, 64, 64, "bf16", True))
    # Odd chunk lengths in 32 bits that begin and end inside blocks.
    add("prepare8_ragged_f32", _prep("1,333,64,379", "77,333,2113,1379", 12, 3, 64, 64, 16, 16,
                                     "f32", False))
    # Decode of 256 sequences over contexts of 1 to 16384 tokens.
    add("paged8_decode_256", _paged("256*1", _text(_uniform(5, 256, 1, 16384)), 32, 4, 128, 64, 32,
                                    "bf16", False))
    # One sequence, one token, a long context: the latency of a lone user.
    add("paged8_decode_1_long", _paged("1", "200003", 16, 2, 256, 64, 64, "bf16", True))
    # Speculative decode: 128 requests verifying 1 to 4 drafts, small pages.
    add("paged8_drafts_128", _paged(_text(_uniform(7, 128, 1, 4)), _text(_uniform(8, 128, 64, 8192)),
                                    32, 8, 128, 16, 16, "bf16", False))
    # A chunk of a long prompt over what is in the cache already, beside two
    # shorter ones.
    add("paged8_chunk_2048_over_32k", _paged("2048,333,7", "32768,5001,7", 32, 4, 128, 128, 64,
                                             "bf16", False))
    # Decode in 32 bits.
    add("paged8_decode_8_f32", _paged("8*1", "1000,1,4097,333,2048,17,0,4000", 8, 2, 128, 16, 16,
                                      "f32", False))
    # A batch of searches with eight beams each over a large vocabulary, twice as
    # many continuations kept as beams (some of them will end).
    add("beam_64x8", _beam(64, 8, 131072, 16, "bf16", False))
    # One search with four beams, one of them ended, an odd vocabulary, 32 bits.
    add("beam_1x4_f32", _beam(1, 4, 32003, 4, "f32", True))
    # The recurrence states and conv tails of three linear layers follow the chosen
    # beams of 16 searches of four.
    add("reorder_16x4", _reorder(16, 4, 3, 32, 128, 128, 8192))
    # Pages of two layers' 8-bit caches copied for forked sequences.
    add("fork_1001_pages", _fork(1001, 4000, 2, 4, 64, 32, 128))
    return cases


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total, n):
    """n positive lengths that sum to total."""
    n = min(n, total)
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["prepare8", "paged8", "paged8", "beam", "slots"])
    if op == "beam":
        W = rng.choice([1, 2, 3, 4, 5, 8, 16])
        V = _log_int(rng, 200, 131072)
        B = _log_int(rng, 1, max(1, min(64, 64 * 8 // W)))
        return _beam(B, W, V, W * rng.choice([1, 2]), rng.choice(["bf16", "f32"]) if B * W * V < 3e7 else "bf16",
                     rng.random() < 0.5)
    if op == "slots":
        if rng.random() < 0.5:
            B, W = _log_int(rng, 1, 32), rng.choice([2, 3, 4, 5, 8])
            B = max(1, min(B, 64 // W))
            return _reorder(B, W, rng.choice([1, 2, 3]), rng.choice([2, 4, 16, 32]), 128, 128,
                            rng.choice([512, 1024, 8192]))
        n = _log_int(rng, 1, 1000)
        return _fork(n, 3 * n + 7, rng.choice([1, 2]), rng.choice([1, 2, 4]), 64, 32, rng.choice([64, 128]))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    while Hkv * G > 32:
        G = max(1, G // 2)
    gated = rng.random() < 0.4
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    small = dtype == "f32"
    if op == "prepare8":
        T = _log_int(rng, 1, 2048 if small else 8192)
        ql = _split(rng, T, rng.choice([1, 2, 5, T, max(1, T // 100)]))
        kl = [q + rng.choice([0, rng.randint(0, 4096)]) for q in ql]
        return _prep(_text(ql), _text(kl), Hkv * G, Hkv, D, rng.choice([D, D // 2, D // 4]), page,
                     block, dtype, gated)
    kind = rng.choice(["decode", "drafts", "chunk"])
    top = 4096 if small else 16384
    if kind == "chunk":
        n = rng.choice([1, 2, 4])
        ql = [_log_int(rng, 1, 256 if small else 1024) for _ in range(n)]
    else:
        n = _log_int(rng, 1, 16 if small else 128)
        ql = [1 if kind == "decode" else rng.randint(1, 8) for _ in range(n)]
    kl = [q + rng.choice([0, _log_int(rng, 1, top)]) for q in ql]
    return _paged(_text(ql), _text(kl), Hkv * G, Hkv, D, page, block, dtype, gated)


# ---- inputs -----------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cumulative(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)


def _rotary_table(positions, rot, dev):
    """[cos | sin] rows of `rot` values, angles in 64 bits."""
    inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _need(amax):
    """The smallest power of two, 2^-64 at least, that brings amax within 448 = 0.875 2^9."""
    f, e = torch.frexp(amax)
    e = e - 9 + (f > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, -64).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def _pool(gen, case, pages, dev):
    """Random pages in 8 bits with the scales of their blocks (unused places hold
    other requests' old values); magnitudes differ from block to block."""
    shape = (pages, case["Hkv"], case["page"] // case["block"], case["block"], case["D"])
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    x *= torch.randn(shape[:3] + (1, 1), generator=gen, device=dev).mul_(0.3).exp_().to(x.dtype)
    scale = _need(x.abs().amax((-1, -2)).float())
    x /= scale[..., None, None].to(x.dtype)
    return x.to(E4M3).view(pages, case["Hkv"], case["page"], case["D"]), scale


def _cache(gen, case, kv_lens, dev):
    """A shuffled paged cache and its block table."""
    page = case["page"]
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + 3
    kc, ks = _pool(gen, case, pages, dev)
    vc, vs = _pool(gen, case, pages, dev)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.zeros((len(kv_lens), max(1, max(need))), dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return dict(kc=kc, ks=ks, vc=vc, vs=vs, table=table.to(dev))


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "beam":
        return _prepare_beam(case, gen, dev)
    if case["op"] == "slots":
        return _prepare_slots(case, gen, dev)
    dt = _dtype(case)
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    T, Hq, Hkv, D = sum(ql), case["Hq"], case["Hkv"], case["D"]
    st = dict(case=case, ql=ql, kl=kl, cu=_cumulative(ql, dev), T=T, Hq=Hq, Hkv=Hkv, D=D, dt=dt,
              kv=torch.tensor(kl, dtype=torch.int32).to(dev), **_cache(gen, case, kl, dev))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    if case["op"] == "prepare8":
        # One packed projection row per token: q heads (each followed by its
        # gate where gated), k heads, v heads.
        per = 2 * D if case["gated"] else D
        row = randn(T, Hq * per + 2 * Hkv * D)
        st["q_in"] = row[:, :Hq * per].view(T, Hq, per)[:, :, :D]
        st["k_in"] = row[:, Hq * per:Hq * per + Hkv * D].view(T, Hkv, D)
        st["v_in"] = row[:, Hq * per + Hkv * D:].view(T, Hkv, D)
        st["qw"] = torch.rand(D, generator=gen, device=dev).add_(0.5).to(dt)
        st["kw"] = torch.rand(D, generator=gen, device=dev).add_(0.5).to(dt)
        st["cs"] = _rotary_table(max(kl + [1]), case["rot"], dev)
        st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device=dev)
        return st
    st["q"] = (1.5 * torch.randn((T, Hq, D), generator=gen, device=dev)).to(dt)
    wide = randn(T, (Hq + Hkv) * D)       # the projection row that holds the gate
    st["gate"] = wide[:, :Hq * D].view(T, Hq, D) if case["gated"] else None
    st["out"] = torch.empty((T, Hq, D), dtype=dt, device=dev)
    return st


def _prepare_beam(case, gen, dev):
    B, W, V, K = case["B"], case["W"], case["V"], case["K"]
    # Logits with the head of likely tokens that a model's have.
    x = torch.randn((B, W, V), generator=gen, device=dev)
    x = (x.mul_(2.0) + x.abs().pow(2.0).mul_(0.25)).to(_dtype(case))
    scores = -torch.rand((B, W), generator=gen, device=dev) * 8.0
    ended = torch.rand((B, W), generator=gen, device=dev) < 0.3 if case["ended"] else None
    return dict(case=case, logits=x, scores=scores,
                ended=None if ended is None else ended.to(torch.uint8),
                parents=torch.empty((B, K), dtype=torch.int32, device=dev),
                tokens=torch.empty((B, K), dtype=torch.int32, device=dev),
                best=torch.empty((B, K), dtype=torch.float32, device=dev))


def _prepare_slots(case, gen, dev):
    pools = []
    if case["form"] == "groups":
        B, W = case["B"], case["W"]
        slots = B * W + 1
        for _ in range(case["layers"]):
            pools.append(torch.randn((slots, case["Hv"], case["Dv"], case["Dk"]), generator=gen,
                                     device=dev))
            pools.append(torch.randn((slots, case["conv"], 3), generator=gen, device=dev))
        dst = torch.randperm(slots, generator=gen, device=dev)[:B * W].to(torch.int32).view(B, W)
        # A good beam has several children, a bad one none.
        u = torch.rand((B, W), generator=gen, device=dev)
        return dict(case=case, pools=pools, dst=dst, src=(u * u * W).to(torch.int32).clamp_(max=W - 1))
    for _ in range(case["layers"]):
        kc, ks = _pool(gen, case, case["pages"], dev)
        vc, vs = _pool(gen, case, case["pages"], dev)
        pools += [kc, ks, vc, vs]
    n = case["n"]
    order = torch.randperm(case["pages"], generator=gen, device=dev).to(torch.int32)
    # Several forks copy the last page of one sequence.
    src = order[n:][torch.randint(0, max(1, n), (n,), generator=gen, device=dev)]
    return dict(case=case, pools=pools, dst=order[:n].contiguous(), src=src)


# ---- one pass ---------------------------------------------------------------

def run(st):
    return {"prepare8": _run_prepare, "paged8": _run_paged, "beam": _run_beam,
            "slots": _run_slots}[st["case"]["op"]](st)


def _positions(st):
    """Each token's sequence and its position there."""
    ids = torch.arange(st["T"], device=st["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu"][1:], ids, right=True)
    return seq, (st["kv"][seq] - (st["cu"][seq + 1] - ids)).long()


def _run_prepare(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_attn8_prepare(st["q_in"], st["k_in"], st["v_in"], st["cu"], st["q_out"],
                            kv_lens=st["kv"], block_table=st["table"], k_cache=st["kc"],
                            v_cache=st["vc"], k_scale=st["ks"], v_scale=st["vs"],
                            q_norm_weight=st["qw"], k_norm_weight=st["kw"], norm_eps=EPS,
                            cos_sin=st["cs"])
        return st["q_out"], st["kc"], st["ks"], st["vc"], st["vs"]
    rot = st["case"]["rot"]
    seq, pos = _positions(st)

    def norm_rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        cos, sin = st["cs"][pos][:, None, :rot // 2], st["cs"][pos][:, None, rot // 2:]
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)

    q = norm_rotate(st["q_in"], st["qw"]).to(st["dt"])
    _write8(st, seq, pos, norm_rotate(st["k_in"], st["kw"]), st["kc"], st["ks"])
    _write8(st, seq, pos, st["v_in"].float(), st["vc"], st["vs"])
    return q, st["kc"], st["ks"], st["vc"], st["vs"]


def _write8(st, seq, pos, x, codes, scales):
    """Rows x [T, Hkv, D] into their places of the cache."""
    page, block, Hkv = st["case"]["page"], st["case"]["block"], st["Hkv"]
    bytes_ = codes.view(torch.uint8)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    first = st["kv"].long() - n                     # position of a sequence's first new token
    where = st["table"][seq, pos // page].long()
    blk = pos % page // block
    flat = where * (page // block) + blk            # the block's number in the pool
    amax = torch.zeros((scales.shape[0] * (page // block), Hkv), device=x.device)
    amax.scatter_reduce_(0, flat[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    need = _need(amax)
    old = scales.permute(0, 2, 1).reshape(-1, Hkv)
    # Blocks that hold rows from before: the first of a sequence, where it begins inside.
    r = first % block
    mine = (r > 0) & (n > 0)
    s_page = st["table"][torch.arange(len(n), device=x.device), first.clamp(min=0) // page].long()
    s_flat = s_page * (page // block) + first % page // block
    joined = torch.zeros(amax.shape[0], dtype=torch.bool, device=x.device)
    joined[s_flat[mine]] = True
    new = torch.where(joined[:, None], torch.maximum(old, need), need)
    j = torch.arange(block, device=x.device)
    at = (first // block * block % page)[:, None] + j[None, :]      # rows of that block
    live = mine[:, None] & (j[None, :] < r[:, None])
    pg, row = s_page[:, None].expand(-1, block)[live], at[live]
    ratio = (old / new)[s_flat][:, None, :].expand(-1, block, -1)[live]
    c = bytes_[pg, :, row].view(E4M3).float() * ratio[..., None]
    bytes_[pg, :, row] = c.to(E4M3).view(torch.uint8)
    bytes_[where, :, pos % page] = (x / new[flat][..., None]).to(E4M3).view(torch.uint8)
    scales[where, :, blk] = new[flat]


def _run_paged(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_attn8_paged(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["table"], st["kv"],
                          st["cu"], st["out"], max_q_len=max(st["ql"]), gate=st["gate"])
        return st["out"]
    page, block = st["case"]["page"], st["case"]["block"]
    Hq, Hkv, D = st["Hq"], st["Hkv"], st["D"]
    N, Lq, L = len(st["ql"]), max(st["ql"]), max(max(st["kl"]), 1)
    width = -(-L // page)
    table = st["table"][:, :width].long()

    def rows(codes, scales):               # [N, Hkv, keys, D]
        c = codes.view(torch.uint8)[table].view(E4M3).float()
        c = c.view(N, width, Hkv, page // block, block, D) * scales[table][..., None, None]
        return c.view(N, width, Hkv, page, D).transpose(1, 2).reshape(N, Hkv, width * page, D)[:, :, :L]

    seq, pos = _positions(st)
    i = torch.arange(st["T"], device=seq.device) - st["cu"][seq]     # place among the sequence's new tokens
    q = torch.zeros((N, Lq, Hq, D), device=seq.device)
    q[seq, i] = st["q"].float()
    q = q.view(N, Lq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, -1, D)
    last = torch.full((N, Lq), -1, device=seq.device, dtype=torch.int64)
    last[seq, i] = pos
    hides = torch.arange(L, device=seq.device)[None, None, :] > last[:, :, None]
    s = torch.matmul(q, rows(st["kc"], st["ks"]).transpose(-1, -2))
    s = s.view(N, Hkv, Hq // Hkv, Lq, L)
    s *= 1.0 / math.sqrt(D)
    s.masked_fill_(hides[:, None, None], float("-inf"))
    s -= s.amax(-1, keepdim=True).clamp(min=-1e30)                   # (a row that sees nothing)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    # Pages past a sequence's end may hold anything: their weight is 0, and so is theirs here.
    past = torch.arange(L, device=seq.device)[None, :] >= st["kv"][:, None]
    v = rows(st["vc"], st["vs"]).masked_fill(past[:, None, :, None], 0.0)
    o = torch.matmul(s.view(N, Hkv, -1, L), v).view(N, Hkv, Hq // Hkv, Lq, D)
    o = o / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(N, Lq, Hq, D)[seq, i]
    if st["gate"] is not None:
        o = o * torch.sigmoid(st["gate"].float())
    return o.to(st["dt"])


def _run_beam(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_beam_select(st["logits"], st["scores"], st["parents"], st["tokens"], st["best"],
                          finished=st["ended"], pad_token=0)
        return st["parents"], st["tokens"], st["best"]
    B_, W, V, K = (st["case"][k] for k in "BWVK")
    x = st["logits"].double()
    x -= x.amax(-1, keepdim=True)
    x += st["scores"].double()[..., None] - x.exp().sum(-1, keepdim=True).log()
    if st["ended"] is not None:            # an ended beam goes on as it is, with the padding token 0
        x.masked_fill_(st["ended"][..., None] > 0, float("-inf"))
        x[..., 0] = torch.where(st["ended"] > 0, st["scores"].double(), x[..., 0])
    best, at = torch.sort(x.view(B_, W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    none = best == float("-inf")
    return ((at // V).masked_fill(none, -1).to(torch.int32),
            (at % V).masked_fill(none, -1).to(torch.int32), best.float())


def _run_slots(st):
    groups = st["case"]["form"] == "groups"
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_copy_slots(st["pools"], st["dst"], st["src"], groups=groups)
        return st["pools"]
    src = torch.gather(st["dst"], 1, st["src"].long()) if groups else st["src"]
    dst, src = st["dst"].reshape(-1).long(), src.reshape(-1).long()
    for pool in st["pools"]:
        bits = pool.view(torch.uint8)
        bits[dst] = bits[src]
    return st["pools"]


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    if case["op"] == "beam":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["B"] * case["W"] * case["V"]
        return {"bytes": n * e + case["B"] * (case["W"] * 4 + case["K"] * 12), "flops": 3 * n}
    if case["op"] == "slots":
        if case["form"] == "groups":
            # Of W children with parents u^2 W, those that stay where they are move nothing, and a
            # parent of several is read once.
            W = case["W"]
            cut = [math.sqrt(i / W) for i in range(W + 1)]
            p = [b - a for a, b in zip(cut, cut[1:])]
            moved = W - sum(p)
            read = sum(1 - (1 - x) ** (W - 1) for x in p)
            slot = case["layers"] * 4 * (case["Hv"] * case["Dk"] * case["Dv"] + case["conv"] * 3)
            return {"bytes": case["B"] * (moved + read) * slot, "flops": 0}
        n = case["n"]
        page = 2 * case["layers"] * case["Hkv"] * (case["page"] * case["D"] + 4 * case["page"] // case["block"])
        return {"bytes": (n + n * (1 - (1 - 1 / n) ** n)) * page, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    T, Hq, Hkv, D = sum(ql), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "prepare8":
        blocks = sum(-(-L // case["block"]) - max(L - n, 0) // case["block"] for n, L in zip(ql, kl))
        return {"bytes": T * (2 * Hq + 2 * Hkv) * D * e + 2 * T * Hkv * D + T * case["rot"] * 4 +
                blocks * Hkv * 8,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"]) + 2 * T * Hkv * D * 2}
    pairs = sum(n * max(L - n, 0) + min(n, L) * (min(n, L) + 1) // 2 for n, L in zip(ql, kl))
    byts = (T * Hq * D * e * (3 if case["gated"] else 2) + sum(kl) * 2 * Hkv * D +
            sum(-(-L // case["block"]) for L in kl) * Hkv * 8)
    return {"bytes": byts, "flops": 4 * D * Hq * pairs}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    if case["op"] == "slots":
        return None                        # bits that move
    st = prepare(case, seed)
    if case["op"] == "beam":
        return _exact_beam(st)
    if case["op"] == "prepare8":
        return _exact_prepare(st)
    T, Hq, Hkv, D = st["T"], st["Hq"], st["Hkv"], st["D"]
    page, block = case["page"], case["block"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=st["q"].device)
    start = 0
    for s, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        for g in range(Hkv if L > 0 else 0):
            j = torch.arange(L, device=out.device)
            pg = st["table"][s].long()[j // page]
            bl = j % page // block
            k = st["kc"].view(torch.uint8)[pg, g, j % page].view(E4M3).double() * st["ks"][pg, g, bl].double()[:, None]
            v = st["vc"].view(torch.uint8)[pg, g, j % page].view(E4M3).double() * st["vs"][pg, g, bl].double()[:, None]
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                for i0 in range(0, n, 2048):
                    i1 = min(n, i0 + 2048)
                    hi = max(L - n + i1, 0)      # keys that any of these rows sees
                    if hi == 0:
                        continue
                    sc = st["q"][start + i0:start + i1, h].double() @ k[:hi].T / D ** 0.5
                    sees = (torch.arange(hi, device=out.device)[None, :]
                            <= torch.arange(L - n + i0, L - n + i1, device=out.device)[:, None])
                    sc = torch.where(sees, sc, torch.full_like(sc, -math.inf))
                    out[start + i0:start + i1, h] = torch.softmax(sc, 1).nan_to_num(0.0) @ v[:hi]
        start += n
    if st["gate"] is not None:
        out = out / (1.0 + torch.exp(-st["gate"].double()))
    return out


def _exact_prepare(st):
    case = st["case"]
    page, block, half = case["page"], case["block"], case["rot"] // 2
    kc, ks, vc, vs = st["kc"].double(), st["ks"].double(), st["vc"].double(), st["vs"].double()
    q = torch.empty(st["q_out"].shape, dtype=torch.float64, device=kc.device)
    grid = torch.arange(127, dtype=torch.uint8, device=kc.device).view(E4M3).double()   # 0 .. 448

    def nearest(x):
        a = x.abs()
        i = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
        lo, hi = grid[i - 1], grid[i]
        up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))       # ties to the even code
        return torch.where(up, hi, lo) * x.sign()

    def put(x, codes, scales, s, first):
        """x [n, Hkv, D] at positions first, first + 1, ... of sequence s."""
        at = 0
        while at < x.shape[0]:
            p = first + at
            m = min(x.shape[0] - at, block - p % block)
            pg, b, row = int(table[s, p // page]), p % page // block, p % page
            new = x[at:at + m]
            top = new.abs().amax((0, 2))
            need = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448.0).clamp(min=-64.0))),
                               torch.full_like(top, 2.0 ** -64))
            r = p % block
            if r > 0:
                old = scales[pg, :, b].clone()
                need = torch.maximum(need, old)
                codes[pg, :, row - r:row] = nearest(codes[pg, :, row - r:row] * (old / need)[:, None, None])
            scales[pg, :, b] = need
            codes[pg, :, row:row + m] = nearest((new / need[None, :, None]).transpose(0, 1))
            at += m

    table = st["table"].cpu()
    start = 0
    for s, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        p = torch.arange(L - n, L, device=kc.device)
        c, sn = st["cs"].double()[p, :half][:, None], st["cs"].double()[p, half:][:, None]

        def turned(x, w):
            x = x[start:start + n].double()
            x = x / ((x * x).sum(2, keepdim=True) / st["D"] + EPS).sqrt() * w.double()
            y = x.clone()
            y[..., :half] = x[..., :half] * c - x[..., half:2 * half] * sn
            y[..., half:2 * half] = x[..., half:2 * half] * c + x[..., :half] * sn
            return y

        q[start:start + n] = turned(st["q_in"], st["qw"])
        put(turned(st["k_in"], st["kw"]), kc, ks, s, L - n)
        put(st["v_in"][start:start + n].double(), vc, vs, s, L - n)
        start += n
    return q, kc, ks, vc, vs


def _exact_beam(st):
    B_, W, V, K = (st["case"][k] for k in "BWVK")
    best = torch.empty((B_, K), dtype=torch.float64, device=st["scores"].device)
    for b in range(B_):
        found = []
        for w in range(W):
            if st["ended"] is not None and int(st["ended"][b, w]):
                found.append(st["scores"][b, w].double()[None])
                continue
            x = st["logits"][b, w].double()
            found.append(torch.log_softmax(x, 0).topk(min(K, V)).values + st["scores"][b, w].double())
        top = torch.cat(found).sort(descending=True).values[:K]
        best[b] = -math.inf
        best[b, :len(top)] = top
    return None, None, best
