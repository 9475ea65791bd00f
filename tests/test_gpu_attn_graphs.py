"""Attention of many and few rows captured into graphs and replayed, over values of all sizes."""

import pytest
import torch

from bit_group_quantized_gb300 import lib
from tests.test_gpu_attn import Case, attn_close, bf16
from tests.test_gpu_attn_ranges import KEYS, VALUES, times

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_replays_follow_the_lengths(cuda_device, d, new):
    """One captured call serves lengths, pages and rows that change on the device; some of the values and keys leave the usual range.
    Two graphs share a workspace, one after the other."""
    c = Case(cuda_device, [300, 210], [new, new], 2, d, 16, seed=80)
    times(c, VALUES, range(40, 300, 7), 2.0 ** -30)
    times(c, VALUES, range(100, 140), 2.0 ** 12, b=1)
    times(c, KEYS, range(3, 300, 50), 2.0 ** -24)
    q = bf16(c.rng, c.rows, 8, d, dev=cuda_device, scale=1.5)
    cache, seqs = c.cache(), c.seqs()
    ws = lib.kv4_attention_workspace(cache, seqs, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for causal in (True, False):
            out, lse = torch.empty_like(q), torch.empty(c.rows, 8, device=cuda_device)
            lib.bgq_kv4_attention(cache, seqs, q, causal=causal, out=out, lse=lse, ws=ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                lib.bgq_kv4_attention(cache, seqs, q, causal=causal, out=out, lse=lse, ws=ws)
            graphs.append(g)
            outs.append((out, lse))
    torch.cuda.current_stream().wait_stream(side)
    for kv, rows in (([300, 210], [new, new]), ([17, 210], [new, 1]), ([299, 0], [new, 0]), ([300, 99], [1, new])):
        c.kv, c.new = kv, rows
        c.q_start = [0, rows[0], rows[0] + rows[1]]
        seqs.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        seqs.q_start.copy_(torch.tensor(c.q_start, dtype=torch.int32))
        for g, (out, lse), causal in zip(graphs, outs, (True, False)):
            g.replay()
            attn_close(c, q, out, lse, causal=causal)
            live = slice(0, c.q_start[-1])
            eager, l = lib.bgq_kv4_attention(cache, seqs, q, causal=causal, want_lse=True)
            assert torch.equal(eager[live], out[live]) and torch.equal(l[live], lse[live])
    assert lib.read_device_status(ws) == lib.OK and not ws[256:4096].any()


def test_prompts_side_by_side(cuda_device):
    """Two prompts on two streams, with workspaces of their own and values that are summed apart, give the bits of calls in turn."""
    jobs = []
    for seed, d in ((81, 128), (82, 256)):
        c = Case(cuda_device, [500], [400], 2, d, 16, seed=seed)
        times(c, VALUES, range(0, 500, 3), 2.0 ** -26)
        times(c, VALUES, range(0, 500, 4), 2.0 ** 20, group=0)
        jobs.append((c.cache(), c.seqs(), bf16(c.rng, c.rows, 8, d, dev=cuda_device)))
    want = [lib.bgq_kv4_attention(*j)[0] for j in jobs]
    ws = [lib.kv4_attention_workspace(j[0], j[1], 8) for j in jobs]
    outs = [[torch.empty_like(j[2]) for _ in range(6)] for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(6):
        for j, w, o, s in zip(jobs, ws, outs, streams):
            lib.bgq_kv4_attention(*j, out=o[i], ws=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)
