"""GPU: the selection, the forks and reorders, and the cache in either width together, as a
beam search over the hybrid stack runs them; the step helper on a cache in 8 bits."""
import pytest
import torch

import attn8_reference as Q
import attn_reference as R
from gated_delta_rule_44_gb300 import binding as B
from gated_delta_rule_44_gb300 import hybrid_example as E
from gated_delta_rule_44_gb300.layer import AttnStep
from test_gpu_attn8 import E4M3, bounds, make_cache8

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("lens,beams,steps", [([19, 40], 4, 7), ([5], 3, 20), ([17, 16, 1], 2, 4)])
def test_beams_have_their_own_histories(bits, lens, beams, steps, cuda_device):
    """Every beam's last row is that of its tokens served by themselves: states, conv tails and
    pages followed the selection.  (The batches differ, so that sums are split elsewhere: rows
    may differ by a few 2^-8 after eight stored projections.)  Its score is the sum of its
    tokens' log-probabilities there."""
    dev = cuda_device
    g = torch.Generator().manual_seed(sum(lens) + bits)
    V = 300
    vocab = (torch.randn(V, E.HybridStack.HID, generator=g) * 0.3).to(BF).to(dev)
    prompts = [torch.randint(0, V, (n,), generator=g) for n in lens]
    n, top = len(lens), max(lens) + steps
    tokens, scores, rows = E.beam_search(E.HybridStack(n * beams, top, dev, cache_bits=bits), vocab, prompts,
                                         beams, steps)
    B.gdn_read_device_status()
    assert tokens.shape == (n, beams, steps) and (tokens >= 0).all()
    assert (scores[:, :-1] >= scores[:, 1:]).all()
    for b in range(n):        # beams of a search differ
        assert len({tuple(t) for t in tokens[b].tolist()}) == beams
    seqs = [torch.cat([prompts[b].to(dev), tokens[b, w].long()]) for b in range(n) for w in range(beams)]
    own = E.generate(E.HybridStack(n * beams, top, dev, cache_bits=bits), vocab[torch.cat(seqs)],
                     [m for m in lens for _ in range(beams)], [m + steps for m in lens for _ in range(beams)])
    B.gdn_read_device_status()
    at = 0
    rms = rows.float().square().mean().sqrt().item()
    for b in range(n):
        for w in range(beams):
            mine = own[at:at + lens[b] + steps].float()
            at += lens[b] + steps
            err = (mine[-1] - rows[b, w].float()).square().mean().sqrt().item()
            assert err <= 16 * 2.0 ** -8 * rms, (b, w, err, rms)
            logp = torch.log_softmax(mine[lens[b] - 1:-1] @ vocab.float().t(), -1)
            total = logp.gather(1, tokens[b, w].long()[:, None]).sum().item()
            # a row off by e moves a logit by |vocab row| e sqrt(HID) / sqrt(HID) at the most
            slack = steps * 2 * 16 * 2.0 ** -8 * rms * vocab.float().norm(dim=1).max().item()
            assert abs(total - scores[b, w].item()) <= slack


def test_ended_beams_stay(cuda_device):
    """A beam that ends goes on as padding with its score; the search's best stays sorted."""
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    V, W, steps = 40, 4, 6
    vocab = (torch.randn(V, E.HybridStack.HID, generator=g) * 0.2).to(BF).to(dev)
    prompts = [torch.randint(0, V, (n,), generator=g) for n in (9, 21)]
    for end in (0, 3, 7):
        tokens, scores, _ = E.beam_search(E.HybridStack(2 * W, 40, dev), vocab, prompts, W, steps, end=end)
        B.gdn_read_device_status()
        assert (scores[:, :-1] >= scores[:, 1:]).all()
        for seq in tokens.view(-1, steps).tolist():
            if end in seq:
                assert all(t == end for t in seq[seq.index(end):])


@pytest.mark.parametrize("new_prompts", [True, False])
def test_step_on_a_cache_in_8_bits(new_prompts, cuda_device):
    """Three decode rows and two prompts (or chunks over an earlier context) in one batch,
    against the 64-bit forms on the rows and codes that the step stored."""
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    Hq, Hkv, D, page, block = 8, 2, 128, 32, 16
    ql = [1, 1, 1, 40, 150]
    before = [4, 299, 0, 0, 0] if new_prompts else [4, 299, 0, 50, 20]
    kl = [a + b for a, b in zip(before, ql)]
    T, N, nd = sum(ql), 5, 3
    c, _ = make_cache8(g, kl, Hkv, D, page, block, dev)
    row = torch.randn(T, (2 * Hq + 2 * Hkv) * D, generator=g).to(BF).to(dev)
    qg = row[:, :2 * Hq * D].view(T, Hq, 2 * D)
    kv = row[:, 2 * Hq * D:].view(T, 2 * Hkv, D)
    cs = torch.randn(320, 64, generator=g).to(dev)
    cu = torch.tensor([0] + ql).cumsum(0).to(torch.int32).to(dev)
    step = AttnStep(T, N, nd, Hq, Hkv, D, BF, dev, max_q_len=150, new_prompts=new_prompts)
    out = step.run(qg[..., :D], kv[:, :Hkv], kv[:, Hkv:], cu, torch.tensor(kl, dtype=torch.int32, device=dev),
                   c["block_table"], c["k_cache"], c["v_cache"], cu_seqlens_prefill=(cu[nd:] - nd).contiguous(),
                   gate=qg[..., D:], cos_sin=cs, k_scale=c["k_scale"], v_scale=c["v_scale"])
    B.gdn_read_device_status()
    cpu = [c[n].cpu() for n in ("k_cache", "k_scale", "v_cache", "v_scale", "block_table")]
    ro, _, pieces = Q.paged(step.q, *cpu, kl, ql, D ** -0.5, qg[..., D:])
    got, tol = R.f64(out), bounds(pieces, ro, BF)
    R.check(got[:nd], ro[:nd], tol[:nd], "decode")
    if new_prompts:        # prompts attend to their keys as they are
        kk, vv = R.f64(step.k)[nd:], R.f64(kv[nd:, Hkv:])
        rp, _, pp = R._packed(R.f64(step.q)[nd:], [(kk[:40], vv[:40], 0), (kk[40:], vv[40:], 0)], ql[nd:],
                              D ** -0.5, R.f64(qg[nd:, :, D:]))
        R.check(got[nd:], rp, R.bound(rp, pp, BF, True), "prompts")
    else:
        R.check(got[nd:], ro[nd:], tol[nd:], "chunks")
    with pytest.raises(ValueError):
        step.run(qg[..., :D], kv[:, :Hkv], kv[:, Hkv:], cu, None, c["block_table"], c["k_cache"], c["v_cache"],
                 k_scale=c["k_scale"])


def test_step_captured_before_a_wider_table(cuda_device):
    """A graph keeps the workspace that it was captured with, after the step has grown another for
    a wider table and the memory around it has been written."""
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    T, Hq, Hkv, D = 300, 8, 2, 128            # 300 tokens of 4 heads each: contexts are widened
    c, _ = make_cache8(g, [700], Hkv, D, 32, 16, dev)
    q, k = (torch.randn(T, h, D, generator=g).to(BF).to(dev) for h in (Hq, Hkv))
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    kv = torch.tensor([700], dtype=torch.int32, device=dev)
    step = AttnStep(T, 1, 0, Hq, Hkv, D, BF, dev, max_q_len=T)
    wide = torch.cat([c["block_table"], torch.full((1, 500), -1, dtype=torch.int32, device=dev)], 1)

    def run(table, stream=None):
        return step.run(q, k, k, cu, kv, table, c["k_cache"], c["v_cache"], cu_seqlens_prefill=cu,
                        k_scale=c["k_scale"], v_scale=c["v_scale"], stream=stream)

    want = run(c["block_table"]).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c["block_table"], torch.cuda.current_stream())
    size = step.workspace.numel()
    # (The widened form cuts its keys by the table's width: other sums, within a rounding or two of
    # the weights, 2^-8, and of the result.)
    assert torch.allclose(run(wide).float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * want.float().abs().max().item())
    assert step.workspace.numel() > size
    junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(4)]
    keep = [j.clone() for j in junk]
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, want)
    for a, b in zip(junk, keep):
        assert torch.equal(a, b)
    B.gdn_read_device_status()


@pytest.mark.parametrize("dtype,q_len,Hq", [(torch.bfloat16, 1, 8), (torch.bfloat16, 70, 8), (torch.float32, 1, 2)])
def test_captured_together(dtype, q_len, Hq, cuda_device):
    """The calls of a step in one graph, on a side stream, between kernels of others: bit for bit
    as one after another, each replay from changed inputs."""
    dev, n, W, Hkv, D, page, V = cuda_device, 2, 2, 2, 128, 32, 5000
    g = torch.Generator(device=dev).manual_seed(q_len + Hq)
    N = n * W
    lens = [300, 90, 128, 701][:N]
    pages = N * 24
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(N, 24)
    kv = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = torch.arange(0, N * q_len + 1, q_len, dtype=torch.int32, device=dev)
    T = N * q_len
    start = dict(k_cache=torch.randn(pages, Hkv, page, D, generator=g, device=dev).to(torch.float8_e4m3fn),
                 v_cache=torch.randn(pages, Hkv, page, D, generator=g, device=dev).to(torch.float8_e4m3fn),
                 k_scale=torch.ones(pages, Hkv, 2, device=dev), v_scale=torch.ones(pages, Hkv, 2, device=dev))
    inputs = [(torch.randn(T, Hq, D, generator=g, device=dev).to(dtype), torch.randn(T, Hkv, D, generator=g, device=dev).to(dtype),
               torch.randn(n, W, V, generator=g, device=dev).to(dtype)) for _ in range(3)]
    cos_sin = torch.randn(800, 64, generator=g, device=dev)
    slots = torch.arange(N, dtype=torch.int32, device=dev).view(n, W)
    q, k, logits = (t.clone() for t in inputs[0])
    c = {m: t.clone() for m, t in start.items()}
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    scores = torch.zeros(n, W, device=dev)
    par, tok = (torch.empty(n, W, dtype=torch.int32, device=dev) for _ in range(2))
    state = torch.zeros(N, T * Hq * D // N, dtype=dtype, device=dev)
    need = B.gdn_attn8_paged_workspace_bytes(T, N, Hq, Hkv, D, q_len, B._dt(q), 24, page)
    ws = [torch.empty(max(1, b), dtype=torch.uint8, device=dev)
          for b in (need, B.gdn_beam_select_workspace_bytes(n, W, V, W))]

    def step(stream):
        B.gdn_attn8_prepare(q, k, k, cu, q_out, kv_lens=kv, block_table=table, cos_sin=cos_sin, stream=stream, **c)
        B.gdn_attn8_paged(q_out, *c.values(), table, kv, cu, out, max_q_len=q_len, workspace=ws[0], stream=stream)
        state.copy_(out.view(N, -1))
        B.gdn_beam_select(logits, scores, par, tok, scores, workspace=ws[1], stream=stream)
        B.gdn_copy_slots([state, c["k_scale"][:N], table], slots, par, groups=True, stream=stream)

    tab0 = table.clone()

    def reset(i):
        for t, s in zip((q, k, logits), inputs[i]):
            t.copy_(s)
        for m, t in start.items():
            c[m].copy_(t)
        table.copy_(tab0)
        scores.zero_()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (q_out, out, state, scores, par, tok, table, *(x.view(torch.uint8) for x in c.values()))]

    want = []
    for i in range(3):
        reset(i)
        torch.cuda.synchronize()
        step(None)
        want.append(results())
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream())
    for i in (1, 0, 2, 1):
        reset(i)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        got = results()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
    B.gdn_read_device_status()
