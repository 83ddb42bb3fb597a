"""Calls on a stream other than the current one: what they allocate comes from that stream's memory, so that writes
still queued on the current stream for a block freed there do not reach it."""

import numpy as np
import pytest
import torch

from block_sparse_long_dual_b200 import sfa

pytestmark = pytest.mark.gpu


def segment_stream(t):
    """The stream from whose memory the allocator made a tensor."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def tensors(x):
    return [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]


def make_calls():
    """Every call that allocates its outputs, with inputs of a small layer and a small decode cache; each gives its
    outputs (the workspaces, whose contents are not results, left out)."""
    g = torch.Generator().manual_seed(5)
    L, d, block = 1024, 128, 128
    Q, K, V = (torch.randn((1, h, L, d), generator=g).bfloat16().cuda() for h in (4, 2, 2))
    cos, sin = sfa.rope_table(10000.0, L, d)
    kw = dict(band_split=d // 4, block=block)
    Q_rot, K_rot, probs, _ = sfa.block_scores(Q, K, cos, sin, **kw)
    shape = sfa.make_shape(Q, K)
    counts, idx = sfa.select(probs, shape, block=block, k=3)
    q = torch.randn((1, 4, d), generator=g).bfloat16().cuda()
    fc = np.tile(np.arange(8), (2, 1))
    K_fc = sfa.decode_fc_gather(K, fc)
    near = sfa.decode_select(q, K_fc, fc, L, k=40)
    return {
        "rope_table": lambda **s: sfa.rope_table(10000.0, L, d, **s),
        "block_scores": lambda **s: sfa.block_scores(Q, K, cos, sin, **kw, **s)[:3],
        "block_scores_select": lambda **s: sfa.block_scores_select(Q, K, cos, sin, k=3, want_probs=True, **kw, **s)[:5],
        "select": lambda **s: sfa.select(probs, shape, block=block, k=3, **s),
        "block_sparse_attn": lambda **s: sfa.block_sparse_attn(Q_rot, K_rot, V, counts, idx, block=block, **s),
        "block_sparse_attn_rope": lambda **s: sfa.block_sparse_attn_rope(Q, cos, sin, K_rot, V, counts, idx, block=block,
                                                                         **s),
        "decode_fc_gather": lambda **s: sfa.decode_fc_gather(K, fc, **s),
        "decode_select": lambda **s: sfa.decode_select(q, K_fc, fc, L, k=40, **s),
        "decode_attn": lambda **s: sfa.decode_attn(q, K, V, near, **s),
    }


@pytest.mark.parametrize("name", ["rope_table", "block_scores", "block_scores_select", "select", "block_sparse_attn",
                                  "block_sparse_attn_rope", "decode_fc_gather", "decode_select", "decode_attn"])
def test_buffers_made_for_a_call_on_another_stream(name):
    call = make_calls()[name]
    want = tensors(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)  # 10 ms before the current stream writes to the blocks that it frees here
    for t in late:
        t.view(torch.uint8).fill_(0x55)
    del late, t
    got = tensors(call(stream=side))
    assert [segment_stream(t) for t in got] == [side.cuda_stream] * len(got)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        if a.dtype == torch.int32 and a.dim() == 4:  # lists: up to each row's count
            n = got[-2] if name != "select" else got[0]
            here = torch.arange(a.shape[-1], device=a.device) < n[..., None]
            a, b = torch.where(here, a, -1), torch.where(here, b, -1)
        assert torch.equal(a, b)


def test_a_step_from_host_memory_runs_on_the_stream_it_is_given():
    """Its copies too: a busy current stream does not hold them up, nor let them overtake the kernels."""
    g = torch.Generator().manual_seed(6)
    host = [torch.randn((1, h, 1024, 128), generator=g).bfloat16().pin_memory() for h in (4, 2, 2)]
    m = sfa.PrismAttention(batch=1, heads_q=4, heads_kv=2, seq_len=1024, head_dim=128, dtype="bf16", block=128,
                           rope_base=10000.0, band_split=32, k=3)
    out, want = (torch.zeros((1, 4, 1024, 128), dtype=torch.bfloat16).pin_memory() for _ in range(2))
    m.run_host(*host, want)
    torch.cuda.synchronize()
    m.O.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)  # half a second
    m.run_host(*host, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    assert not torch.cuda.current_stream().query()  # the current stream is still busy
    torch.cuda.synchronize()
