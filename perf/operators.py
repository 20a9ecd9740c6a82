"""The full-attention operators' measured workloads, and their plain forms.

Three operators of the softmax-attention layers that stand between the
gated-delta-rule layers of a hybrid model:

  prepare   per-head RMS norm of q and k, rotary positions, k and v written
            into a paged cache                              (gdn_attn_prepare)
  prompt    causal attention over packed prompts            (gdn_attn_varlen)
  paged     attention of new tokens (one, a few drafts, a chunk) over a paged
            cache                                           (gdn_attn_paged)

``own = False`` computes them with elementary torch operations in 32 bits,
rounded once at the end; ``own = True`` calls the library.

A sequence with q_len new tokens and a context of kv_len tokens (the new ones
included) has its new token i at position kv_len - q_len + i; query head h
reads kv head h // (Hq // Hkv).  Cache pages are [pages, Hkv, page, D].
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def _prep(q_lens, kv_lens, Hq, Hkv, D, rot, page, dtype, gated):
    return dict(op="prepare", q_lens=q_lens, kv_lens=kv_lens, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                page=page, dtype=dtype, gated=gated)


def _prompt(lens, Hq, Hkv, D, dtype, gated):
    return dict(op="prompt", q_lens=lens, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, gated=gated)


def _paged(q_lens, kv_lens, Hq, Hkv, D, page, dtype, gated):
    return dict(op="paged", q_lens=q_lens, kv_lens=kv_lens, Hq=Hq, Hkv=Hkv, D=D, page=page,
                dtype=dtype, gated=gated)


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

    # One new token for each of the 512 decoding sequences of the mixed serving
    # step: latency counts.
    add("prepare_decode_512", _prep("512*1", _text(_uniform(11, 512, 1, 4096)), 32, 4, 128, 128,
                                    64, "bf16", False))
    # The four new 2048-token prompts of the mixed step, q projected together
    # with its output gate (strided rows), a quarter of the head rotated.
    add("prepare_prompts_4x2048", _prep("4*2048", "4*2048", 16, 2, 256, 64, 64, "bf16", True))
    # Odd chunk lengths in 32 bits, pages that end inside a chunk.
    add("prepare_ragged_f32", _prep("1,333,64,379", "77,333,2113,1379", 12, 3, 64, 64, 16, "f32",
                                    False))
    # One 4096-token prompt.
    add("prompt_4096", _prompt("4096", 32, 4, 128, "bf16", False))
    # Eight packed prompts of 512 to 8192 tokens, wide heads, gated output.
    add("prompt_varlen_8", _prompt(_text(_uniform(3, 8, 512, 8192)), 16, 2, 256, "bf16", True))
    # A batch of short ragged prompts, one token among them.
    add("prompt_short_ragged", _prompt("1,17,129,255,64,300,2,513", 24, 8, 64, "bf16", False))
    # 32-bit activations.
    add("prompt_1024_f32", _prompt("1024", 8, 2, 128, "f32", True))
    # Decode of 256 sequences over contexts of 1 to 16384 tokens.
    add("decode_256", _paged("256*1", _text(_uniform(5, 256, 1, 16384)), 32, 4, 128, 64, "bf16",
                             False))
    # One sequence, one token, a long context: the latency of a lone user.
    add("decode_1_long", _paged("1", "200003", 16, 2, 256, 64, "bf16", True))
    # Speculative decode: 128 requests verifying 1 to 4 drafts, small pages.
    add("drafts_128", _paged(_text(_uniform(7, 128, 1, 4)), _text(_uniform(8, 128, 64, 8192)), 32,
                             8, 128, 16, "bf16", False))
    # A chunk of a long prompt over what is in the cache already, beside two
    # shorter ones.
    add("chunk_2048_over_32k", _paged("2048,333,7", "32768,5001,7", 32, 4, 128, 128, "bf16",
                                      False))
    # Decode in 32 bits.
    add("decode_8_f32", _paged("8*1", "1000,1,4097,333,2048,17,0,4000", 8, 2, 128, 16, "f32",
                               False))
    return cases


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, total, n):
    """n positive lengths that sum to total."""
    n = min(n, total)
    cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["prepare", "prompt", "paged", "paged"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    while Hkv * G > 32:
        G = max(1, G // 2)
    gated = rng.random() < 0.4
    page = rng.choice([16, 32, 64, 128])
    small = dtype == "f32"
    if op == "prepare":
        T = _log_int(rng, 1, 2048 if small else 8192)
        ql = _split(rng, T, rng.choice([1, 2, 5, T, max(1, T // 100)]))
        kl = [q + rng.choice([0, rng.randint(0, 4096)]) for q in ql]
        return _prep(_text(ql), _text(kl), Hkv * G, Hkv, D, rng.choice([D, D // 2, D // 4]), page,
                     dtype, gated)
    if op == "prompt":
        T = _log_int(rng, 1, 1536 if small else 8192)
        ql = _split(rng, T, rng.choice([1, 1, 3, 8, 20]))
        return _prompt(_text(ql), Hkv * G, Hkv, D, dtype, gated)
    kind = rng.choice(["decode", "drafts", "chunk"])
    top = 4096 if small else 16384
    if kind == "chunk":
        n = rng.choice([1, 2, 4])
        ql = [_log_int(rng, 1, 256 if small else 1024) for _ in range(n)]
    else:
        n = _log_int(rng, 1, 16 if small else 128)
        ql = [1 if kind == "decode" else rng.randint(1, 8) for _ in range(n)]
    kl = [q + rng.choice([0, _log_int(rng, 1, top)]) for q in ql]
    return _paged(_text(ql), _text(kl), Hkv * G, Hkv, D, page, dtype, gated)


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


def _cache(gen, case, kv_lens, dt, dev):
    """A shuffled paged cache of random values (unused places hold other
    requests' old values) and its block table."""
    page = case["page"]
    need = [-(-n // page) for n in kv_lens]
    width = max(1, max(need))
    pages = sum(need) + 3
    shape = (pages, case["Hkv"], page, case["D"])
    k = torch.randn(shape, generator=gen, device=dev, dtype=dt)
    v = torch.randn(shape, generator=gen, device=dev, dtype=dt)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.zeros((len(kv_lens), width), dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return k, v, table.to(dev)


def prepare(case, seed):
    dev, dt = _device(), _dtype(case)
    gen = torch.Generator(device=dev).manual_seed(seed)
    ql = _lens(case["q_lens"])
    T, Hq, Hkv, D = sum(ql), case["Hq"], case["Hkv"], case["D"]
    st = dict(case=case, ql=ql, cu=_cumulative(ql, dev), T=T, Hq=Hq, Hkv=Hkv, D=D, dt=dt)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt)

    if case["op"] != "prompt":
        st["kl"] = _lens(case["kv_lens"])
        st["kv"] = torch.tensor(st["kl"], dtype=torch.int32).to(dev)
        st["kc"], st["vc"], st["table"] = _cache(gen, case, st["kl"], dt, dev)
    if case["op"] == "prepare":
        # One packed projection row per token: q heads (each followed by its
        # gate where gated), k heads, v heads.
        per = 2 * D if case["gated"] else D
        row = randn(T, Hq * per + 2 * Hkv * D)
        st["row"] = row
        st["q_in"] = row[:, :Hq * per].view(T, Hq, per)[:, :, :D]
        st["k_in"] = row[:, Hq * per:Hq * per + Hkv * D].view(T, Hkv, D)
        st["v_in"] = row[:, Hq * per + Hkv * D:].view(T, Hkv, D)
        st["qw"] = torch.rand(D, generator=gen, device=dev).add_(0.5).to(dt)
        st["kw"] = torch.rand(D, generator=gen, device=dev).add_(0.5).to(dt)
        st["cs"] = _rotary_table(max(st["kl"] + [1]), case["rot"], dev)
        st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device=dev)
        return st
    st["q"] = (1.5 * torch.randn((T, Hq, D), generator=gen, device=dev)).to(dt)
    wide = randn(T, (Hq + Hkv) * D)       # the projection row that holds gate and v
    st["gate"] = wide[:, :Hq * D].view(T, Hq, D) if case["gated"] else None
    if case["op"] == "prompt":
        st["k"] = randn(T, Hkv, D)
        st["v"] = wide[:, Hq * D:].view(T, Hkv, D)
    st["out"] = torch.empty((T, Hq, D), dtype=dt, device=dev)
    if own and case["op"] == "paged":
        from gated_delta_rule_44_gb300 import binding as B
        n = B.gdn_attn_paged_workspace_bytes(T, len(ql), Hq, Hkv, D, max(ql), B._dt(st["q"]))
        st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    return st


# ---- one pass ---------------------------------------------------------------

def run(st):
    return {"prepare": _run_prepare, "prompt": _run_prompt, "paged": _run_paged}[
        st["case"]["op"]](st)


def _run_prepare(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_attn_prepare(st["q_in"], st["k_in"], st["v_in"], st["cu"], st["q_out"],
                           kv_lens=st["kv"], block_table=st["table"], k_cache=st["kc"],
                           v_cache=st["vc"], q_norm_weight=st["qw"], k_norm_weight=st["kw"],
                           norm_eps=EPS, cos_sin=st["cs"])
        return st["q_out"], st["kc"], st["vc"]
    page, rot = st["case"]["page"], st["case"]["rot"]
    ids = torch.arange(st["T"], device=st["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu"][1:], ids, right=True)
    pos = (st["kv"][seq] - (st["cu"][seq + 1] - ids)).long()

    def norm_rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        cos, sin = st["cs"][pos][:, None, :rot // 2], st["cs"][pos][:, None, rot // 2:]
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1).to(st["dt"])

    q = norm_rotate(st["q_in"], st["qw"])
    k = norm_rotate(st["k_in"], st["kw"])
    where = st["table"][seq, pos // page].long()
    st["kc"][where, :, pos % page] = k
    st["vc"][where, :, pos % page] = st["v_in"]
    return q, st["kc"], st["vc"]


def _attend(q, k, v, first, out_dtype, gate):
    """q [Lq, Hq, D] at positions first, first + 1, ... over k, v [L, Hkv, D]."""
    Lq, Hq, D = q.shape
    L, Hkv, _ = k.shape
    if L == 0:
        return torch.zeros((Lq, Hq, D), dtype=out_dtype, device=q.device)
    qg = q.float().view(Lq, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
    s = torch.matmul(qg, k.float().permute(1, 2, 0)[:, None]) * (1.0 / math.sqrt(D))
    if Lq > 1:
        p = torch.arange(L, device=q.device)
        s.masked_fill_(p[None, :] > first + torch.arange(Lq, device=q.device)[:, None],
                       float("-inf"))
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    o = torch.matmul(s, v.float().permute(1, 0, 2)[:, None]) / s.sum(-1, keepdim=True)
    o = o.permute(2, 0, 1, 3).reshape(Lq, Hq, D)
    if gate is not None:
        o = o * torch.sigmoid(gate.float())
    return o.to(out_dtype)


def _run_prompt(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_attn_varlen(st["q"], st["k"], st["v"], st["cu"], st["out"], gate=st["gate"])
        return st["out"]
    outs, a = [], 0
    for n in st["ql"]:
        b = a + n
        outs.append(_attend(st["q"][a:b], st["k"][a:b], st["v"][a:b], 0, st["dt"],
                            None if st["gate"] is None else st["gate"][a:b]))
        a = b
    return torch.cat(outs)


def _run_paged(st):
    if own:
        from gated_delta_rule_44_gb300 import binding as B
        B.gdn_attn_paged(st["q"], st["kc"], st["vc"], st["table"], st["kv"], st["cu"], st["out"],
                         max_q_len=max(st["ql"]), gate=st["gate"], workspace=st["workspace"])
        return st["out"]
    outs, a, page = [], 0, st["case"]["page"]
    for s, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        b = a + n
        idx = st["table"][s, :-(-L // page)].long()
        k = st["kc"][idx].transpose(1, 2).flatten(0, 1)[:L]
        v = st["vc"][idx].transpose(1, 2).flatten(0, 1)[:L]
        outs.append(_attend(st["q"][a:b], k, v, L - n, st["dt"],
                            None if st["gate"] is None else st["gate"][a:b]))
        a = b
    return torch.cat(outs)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    ql = _lens(case["q_lens"])
    T, Hq, Hkv, D = sum(ql), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "prepare":
        tokens = T * (Hq + 2 * Hkv) * D
        return {"bytes": 2 * tokens * e + T * case["rot"] * 4,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    kl = ql if case["op"] == "prompt" else _lens(case["kv_lens"])
    pairs = sum(n * max(L - n, 0) + min(n, L) * (min(n, L) + 1) // 2 for n, L in zip(ql, kl))
    byts = T * Hq * D * e * (3 if case["gated"] else 2) + sum(kl) * 2 * Hkv * D * e
    return {"bytes": byts, "flops": 4 * D * Hq * pairs}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prepare":
        return _exact_prepare(st)
    T, Hq, Hkv, D = st["T"], st["Hq"], st["Hkv"], st["D"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=st["q"].device)
    kl = st["ql"] if case["op"] == "prompt" else st["kl"]
    start = 0
    for s, (n, L) in enumerate(zip(st["ql"], kl)):
        for g in range(Hkv if L > 0 else 0):
            if case["op"] == "prompt":
                k = st["k"][start:start + L, g].double()
                v = st["v"][start:start + L, g].double()
            else:
                j = torch.arange(L, device=out.device)
                pg = st["table"][s].long()[j // case["page"]]
                k = st["kc"][pg, g, j % case["page"]].double()
                v = st["vc"][pg, g, j % case["page"]].double()
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
    page, half = st["case"]["page"], st["case"]["rot"] // 2
    kc, vc = st["kc"].double(), st["vc"].double()
    q = torch.empty(st["q_out"].shape, dtype=torch.float64, device=kc.device)
    start = 0
    for s, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        p = torch.arange(L - n, L, device=kc.device)
        c, sn = st["cs"].double()[p, :half], st["cs"].double()[p, half:]
        rows = st["table"][s].long()[p // page]
        for src, w, H, put in ((st["q_in"], st["qw"], st["Hq"], None),
                               (st["k_in"], st["kw"], st["Hkv"], kc)):
            for h in range(H):
                x = src[start:start + n, h].double()
                x = x / ((x * x).sum(1, keepdim=True) / st["D"] + EPS).sqrt() * w.double()
                y = x.clone()
                y[:, :half] = x[:, :half] * c - x[:, half:2 * half] * sn
                y[:, half:2 * half] = x[:, half:2 * half] * c + x[:, :half] * sn
                if put is None:
                    q[start:start + n, h] = y
                else:
                    put[rows, h, p % page] = y
        for h in range(st["Hkv"]):
            vc[rows, h, p % page] = st["v_in"][start:start + n, h].double()
        start += n
    return q, kc, vc
