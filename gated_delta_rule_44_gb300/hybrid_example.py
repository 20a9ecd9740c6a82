"""A small hybrid stack, served: three gated-delta-rule layers and one full-attention
layer, random weights, prompts first and then single tokens.

    python -m gated_delta_rule_44_gb300.hybrid_example

Each layer projects the hidden rows with one matrix, runs its step on views of
the projection, and projects back; a residual joins them.  The prompts go through
``GdnStep`` and ``AttnStep`` as one packed batch; every further token is a decode
batch over the state pool, the conv pool and the paged cache that the prompts
left.  ``generate`` returns every hidden row, so that serving in steps can be
compared with the whole sequences in one batch.
"""
from __future__ import annotations

from typing import List

import torch

from .layer import AttnStep, GdnStep


class HybridStack:
    """Weights, pools and cache of the stack for up to `slots` sequences."""

    HID, HK, HV, DK, DV, K = 256, 2, 4, 128, 128, 4     # linear layers
    HQ, HKV, D, ROT, PAGE = 8, 2, 128, 64, 16           # attention layer

    def __init__(self, slots: int, max_tokens: int, device, seed: int = 0,
                 dtype: torch.dtype = torch.bfloat16):
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
        self.k_cache = torch.zeros(slots * width, self.HKV, self.PAGE, self.D, dtype=dtype,
                                   device=self.dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.randperm(slots * width, generator=g).to(torch.int32).view(slots, width).to(self.dev)
        inv = 1e4 ** (-torch.arange(0, self.ROT, 2, dtype=torch.float64) / self.ROT)
        ang = torch.arange(max_tokens, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().to(self.dev)

    def step(self, x, lens: List[int], kv_lens: List[int], new: bool):
        """Hidden rows x [T, HID] of sequences 0 .. N-1 with `lens` new tokens each,
        their contexts `kv_lens` long afterwards; new: they start here."""
        T, N = x.shape[0], len(lens)
        nd = 0 if new else N
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(self.dev)
        kv = torch.tensor(kv_lens, dtype=torch.int32, device=self.dev)
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
                             self.table[:N], self.k_cache, self.v_cache, cu_seqlens_prefill=cu,
                             gate=q[..., self.D:], q_norm_weight=L["q_norm"],
                             k_norm_weight=L["k_norm"], cos_sin=self.cos_sin)
            x = x + y.reshape(T, -1) @ L["w_out"]
        return x


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


if __name__ == "__main__":
    main()
