"""A small hybrid stack, served: three gated-delta-rule layers and one full-attention
layer, random weights, prompts first and then single tokens.

    python -m gated_delta_rule_44_gb300.hybrid_example

Each layer projects the hidden rows with one matrix, runs its step on views of
the projection, and projects back; a residual joins them.  The prompts go through
``GdnStep`` and ``AttnStep`` as one packed batch; every further token is a decode
batch over the state pool, the conv pool and the paged cache that the prompts
left.  ``generate`` returns every hidden row, so that serving in steps can be
compared with the whole sequences in one batch.

``beam_search`` keeps several continuations of each prompt: a prompt is computed once
and forked, and every step's best continuations take the states and cache pages of the
beams that they continue.  With ``cache_bits=8`` keys and values are cached in 8 bits.
"""
from __future__ import annotations

from typing import List

import torch

from . import binding as B
from .layer import AttnStep, GdnStep


class HybridStack:
    """Weights, pools and cache of the stack for up to `slots` sequences."""

    HID, HK, HV, DK, DV, K = 256, 2, 4, 128, 128, 4     # linear layers
    HQ, HKV, D, ROT, PAGE = 8, 2, 128, 64, 16           # attention layer

    def __init__(self, slots: int, max_tokens: int, device, seed: int = 0,
                 dtype: torch.dtype = torch.bfloat16, cache_bits: int = 16):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.dt, self.slots = torch.device(device), dtype, slots

        def w(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(self.dev)

        C = 2 * self.HK * self.DK + self.HV * self.DV
        h = self.HID ** -0.5
        self.linear = []
        for _ in range(3):
            self.linear.append(dict(
                w_in=w(self.HID, C + 2 * self.HV, std=h).to(dtype),
                w_out=w(self.HV * self.DV, self.HID, std=0.5 * (self.HV * self.DV) ** -0.5).to(dtype),
                conv=w(C, self.K, std=0.25), A_log=w(self.HV, std=0.5), dt_bias=w(self.HV, std=0.5),
                state=torch.zeros(slots, self.HV, self.DV, self.DK, device=self.dev),
                tail=torch.zeros(slots, C, self.K - 1, device=self.dev)))
        rows = (2 * self.HQ + 2 * self.HKV) * self.D      # q and gate interleaved, k, v
        self.attn = dict(w_in=w(self.HID, rows, std=h).to(dtype),
                         w_out=w(self.HQ * self.D, self.HID, std=0.5 * (self.HQ * self.D) ** -0.5).to(dtype),
                         q_norm=(1 + w(self.D, std=0.1)).to(dtype),
                         k_norm=(1 + w(self.D, std=0.1)).to(dtype))
        width = -(-max_tokens // self.PAGE)
        shape = (slots * width, self.HKV, self.PAGE, self.D)
        kind = torch.uint8 if cache_bits == 8 else dtype
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=kind, device=self.dev) for _ in range(2))
        self.scales = {}
        if cache_bits == 8:        # a scale for each page and head
            self.k_cache, self.v_cache = (t.view(torch.float8_e4m3fn) for t in (self.k_cache, self.v_cache))
            self.scales = {n: torch.zeros(slots * width, self.HKV, 1, device=self.dev)
                           for n in ("k_scale", "v_scale")}
        self.table = torch.randperm(slots * width, generator=g).to(torch.int32).view(slots, width).to(self.dev)
        inv = 1e4 ** (-torch.arange(0, self.ROT, 2, dtype=torch.float64) / self.ROT)
        ang = torch.arange(max_tokens, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().to(self.dev)

    def step(self, x, lens: List[int], kv_lens: List[int], new: bool, slots=None):
        """Hidden rows x [T, HID] of sequences with `lens` new tokens each, in `slots`
        (int32, default 0 .. N-1), their contexts `kv_lens` long afterwards; new: they
        start here."""
        T, N = x.shape[0], len(lens)
        nd = 0 if new else N
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(self.dev)
        kv = torch.tensor(kv_lens, dtype=torch.int32, device=self.dev)
        if slots is None:
            slots = torch.arange(N, dtype=torch.int32, device=self.dev)
        begun = torch.full((N,), 0 if new else 1, dtype=torch.uint8, device=self.dev)
        C = 2 * self.HK * self.DK + self.HV * self.DV
        gdn = GdnStep(T, N, nd, self.HK, self.HV, self.DK, self.DV, self.K, self.dt, self.dev)
        attn = AttnStep(T, N, nd, self.HQ, self.HKV, self.D, self.dt, self.dev, new_prompts=new)
        for i, L in enumerate(self.linear + [self.attn]):
            row = x @ L["w_in"]
            if i < len(self.linear):
                y = gdn.run(row, row[:, C:C + self.HV], row[:, C + self.HV:], L["conv"], L["A_log"],
                            L["dt_bias"], cu, slots, begun, L["state"], L["tail"],
                            cu_seqlens_prefill=cu)
            else:
                q = row[:, :2 * self.HQ * self.D].view(T, self.HQ, 2 * self.D)
                kvr = row[:, 2 * self.HQ * self.D:].view(T, 2 * self.HKV, self.D)
                y = attn.run(q[..., :self.D], kvr[:, :self.HKV], kvr[:, self.HKV:], cu, kv,
                             self.table[slots.long()], self.k_cache, self.v_cache,
                             cu_seqlens_prefill=cu, gate=q[..., self.D:], q_norm_weight=L["q_norm"],
                             k_norm_weight=L["k_norm"], cos_sin=self.cos_sin, **self.scales)
            x = x + y.reshape(T, -1) @ L["w_out"]
        return x

    def _states(self):
        return [p for L in self.linear for p in (L["state"], L["tail"])]

    def _pages(self):
        return [self.k_cache, self.v_cache, *self.scales.values()]

    def fork(self, src, dst):
        """Slots dst become copies of slots src (int32, equal lengths)."""
        B.gdn_copy_slots(self._states(), dst, src)
        B.gdn_copy_slots(self._pages(), self.table[dst.long()].reshape(-1),
                         self.table[src.long()].reshape(-1))

    def reorder(self, parents, first: int, tokens: int):
        """Slots in groups of W: place j of a group continues its place parents[g, j]
        (int32 [groups, W]).  Contexts are the same before position `first` and `tokens`
        long."""
        groups, W = parents.shape
        slots = torch.arange(groups * W, dtype=torch.int32, device=self.dev).view(groups, W)
        B.gdn_copy_slots(self._states(), slots, parents, groups=True)
        p0, p1 = first // self.PAGE, -(-tokens // self.PAGE)
        pages = self.table[:groups * W, p0:p1].t().contiguous().view(-1, W)    # [pages * groups, W]
        B.gdn_copy_slots(self._pages(), pages, parents.repeat(p1 - p0, 1), groups=True)


def generate(stack: HybridStack, x, prompt_lens: List[int], total_lens: List[int]):
    """Rows x (the sequences packed, total_lens each) through the stack: the first
    prompt_lens of each as one batch of prompts, the others token by token, one of
    every sequence a step: each has as many of them as the others."""
    steps = total_lens[0] - prompt_lens[0]
    if any(t - n != steps for t, n in zip(total_lens, prompt_lens)) or steps < 0:
        raise ValueError(f"sequences with unequal numbers of further tokens: prompts of {list(prompt_lens)} "
                         f"tokens in sequences of {list(total_lens)}")
    if len(total_lens) != len(prompt_lens) or sum(total_lens) != x.shape[0]:
        raise ValueError(f"{len(prompt_lens)} prompts and sequences of {list(total_lens)} tokens do not "
                         f"make {x.shape[0]} rows")
    starts = [sum(total_lens[:i]) for i in range(len(total_lens))]
    first = torch.cat([x[a:a + n] for a, n in zip(starts, prompt_lens)])
    y = stack.step(first, list(prompt_lens), list(prompt_lens), True)
    out, at = torch.empty_like(x), 0
    for a, n in zip(starts, prompt_lens):
        out[a:a + n] = y[at:at + n]
        at += n
    for i in range(steps):
        rows = torch.tensor([a + n + i for a, n in zip(starts, prompt_lens)], device=x.device)
        out[rows] = stack.step(x[rows], [1] * len(rows), [n + i + 1 for n in prompt_lens], False)
    return out


def beam_search(stack: HybridStack, vocab, prompts, beams: int, steps: int, end: int = -1):
    """The `beams` best continuations of `steps` tokens for each prompt (token tensors).
    vocab [V, HID]: a token's row, and the projection to the logits; end: the token that
    ends a continuation.  Returns tokens [prompts, beams, steps], their log-probabilities
    [prompts, beams], and each one's last hidden row [prompts, beams, HID]."""
    dev, n, W = stack.dev, len(prompts), beams
    lens = [len(p) for p in prompts]
    slots = torch.arange(n * W, dtype=torch.int32, device=dev).view(n, W)
    rows = stack.step(vocab[torch.cat(list(prompts)).to(dev)], lens, lens, True,
                      slots=slots[:, 0].contiguous())
    rows = rows[torch.tensor(lens).cumsum(0).to(dev) - 1]
    if W > 1:
        stack.fork(slots[:, :1].repeat(1, W - 1).view(-1), slots[:, 1:].contiguous().view(-1))
    rows = rows[:, None].repeat(1, W, 1)
    scores = torch.full((n, W), float("-inf"), device=dev)
    scores[:, 0] = 0.0                                   # one beam is alive at first
    ended = torch.zeros((n, W), dtype=torch.bool, device=dev)
    tokens = torch.zeros((n, W, 0), dtype=torch.int32, device=dev)
    for i in range(steps):
        parents, new = (torch.empty((n, W), dtype=torch.int32, device=dev) for _ in range(2))
        B.gdn_beam_select(rows.reshape(n * W, -1).matmul(vocab.t()).view(n, W, -1), scores, parents,
                          new, scores, finished=ended, pad_token=max(end, 0))
        at = parents.clamp(min=0).long()                 # (-1: fewer continuations than beams)
        ended = torch.gather(ended, 1, at) | (new == end)
        tokens = torch.cat([torch.gather(tokens, 1, at[..., None].expand(-1, -1, i)), new[..., None]], 2)
        kv = [m + i + 1 for m in lens for _ in range(W)]
        stack.reorder(parents, min(lens), max(kv) - 1)
        rows = stack.step(vocab[new.clamp(min=0).view(-1).long()], [1] * (n * W), kv, False).view(n, W, -1)
    return tokens, scores, rows


def main() -> None:
    dev = torch.device("cuda:0")
    prompts, more = [37, 130, 1], 9
    total = [n + more for n in prompts]
    g = torch.Generator().manual_seed(1)
    x = torch.randn(sum(total), HybridStack.HID, generator=g).to(torch.bfloat16).to(dev)
    served = generate(HybridStack(len(total), max(total), dev), x, prompts, total)
    whole = generate(HybridStack(len(total), max(total), dev), x, total, total)
    diff = (served.float() - whole.float()).abs().max().item()
    print(f"{len(total)} sequences, {sum(total)} tokens: prompts and {more} single tokens each, "
          f"against whole sequences: max difference {diff:.3f} of rows of rms "
          f"{whole.float().square().mean().sqrt().item():.2f}")
    vocab = (torch.randn(500, HybridStack.HID, generator=g) * 0.3).to(torch.bfloat16).to(dev)
    asked = [torch.randint(0, 500, (n,), generator=g) for n in (19, 40)]
    for bits in (16, 8):
        stack = HybridStack(8, 60, dev, cache_bits=bits)
        tokens, scores, _ = beam_search(stack, vocab, asked, beams=4, steps=8)
        print(f"cache in {bits} bits, best of 4 beams: "
              + "; ".join(f"{t.tolist()} ({s:.2f})" for t, s in zip(tokens[:, 0], scores[:, 0])))


if __name__ == "__main__":
    main()
