"""The 8-bit KV cache on the GPU against its float64 oracle, through the public binding.

Stored codes, scales, lengths, index lists and compact keys must be equal (NaN codes as NaN).  Attention
is held to bounds counted in roundings:
  score     |ds| <= sk * ((d + 8) * 2^-24 + 2^-21): d products and sums in float32 and the factors' roundings,
            plus the query's two-part 8-bit form (its parts leave at most 2^-21 of the row's largest element)
  lse       ds + 2^-22 |lse| + 2^-20 (exp2 / log2 and a float32 sum)
  o         2^-8 |o| (one bf16 rounding) + a (2^-8 + 2 ds + 2^-18) with a = sum p |v|: probabilities in two
            8-bit parts (2^-8), moved scores, float32 sums; + 2^-23 a1 with a1 = max p * sum |v|: the parts end
            2^-23 below the largest probability beside them, so what lies under that is lost; + 2^-100: float32
            probabilities end at 2^-149
  weight    W (2 ds + 2^-19) + 2^-22 (w_in + W)
"""

import numpy as np
import pytest
import torch

from block_sparse_long_dual_b200 import sfa
from block_sparse_long_dual_b200.synthetic import make_decode_inputs
from block_sparse_long_dual_b200.workloads import DecodeWorkload
from oracle import cache8_oracle as co
from oracle import fasa_oracle as fo

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def dev():
    return torch.device("cuda")


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=dev())


def same_codes(got, want):
    a, b = co.VALUES[got], co.VALUES[want]
    np.testing.assert_array_equal(a, b)


class Arrays:
    """A random cache held twice: as numpy arrays and as a KvCache8."""

    def __init__(self, rng, B, H, cap, d, block, lens, weight=True, spread=0, behind=True):
        nb = -(-cap // block)
        self.block = block
        x = rng.normal(size=(2, B, H, cap, d)) * np.exp2(rng.integers(-spread, spread + 1, (2, B, H, cap, 1)))
        out = []
        for y in x:
            pad = np.zeros((B, H, nb * block, d))
            pad[:, :, :cap] = y
            top = np.abs(pad.reshape(B, H, nb, block * d)).max(-1)
            f = np.exp2(np.ceil(np.log2(np.maximum(top, 1e-30) / 448.0))).astype(np.float32)
            c = torch.from_numpy(y / np.repeat(f, block, -1)[:, :, :cap, None]).float().to(E4M3)
            out += [c.view(torch.uint8).numpy().copy(), f]
        self.k, self.ks, self.v, self.vs = out
        self.lens = np.asarray(lens, dtype=np.int32)
        self.w = (rng.random((B, H, cap)).astype(np.float32) if weight else None)
        if behind:  # rows that hold nothing hold NaN
            for b in range(B):
                n = min(max(int(lens[b]), 0), cap)
                self.k[b, :, n:], self.v[b, :, n:] = 0x7F, 0xFF
                blk = -(-n // block)
                self.ks[b, :, blk:], self.vs[b, :, blk:] = np.nan, np.nan

    def gpu(self):
        t = lambda x: torch.from_numpy(x.copy()).to(dev())  # noqa: E731
        return sfa.KvCache8(k=t(self.k).view(E4M3), v=t(self.v).view(E4M3), k_scale=t(self.ks), v_scale=t(self.vs),
                            lens=t(self.lens), weight=None if self.w is None else t(self.w), block=self.block)


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def bounds(o, lse, err, d):
    a, a1, sk = err
    ds = sk * ((d + 8) * 2.0 ** -24 + 2.0 ** -21)
    lse_tol = ds + 2.0 ** -20 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0)
    o_tol = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -18) + 2.0 ** -23 * a1 + 2.0 ** -100
    return o_tol, lse_tol, ds


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    np.testing.assert_array_equal(np.isfinite(got), np.isfinite(want), err_msg=what)
    f = np.isfinite(want)
    np.testing.assert_array_equal(got[~f], want[~f])
    err = np.abs(got[f] - want[f])
    lim = np.broadcast_to(tol, want.shape)[f]
    bad = err > lim
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err - lim):.3e} over"


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPENDS = [  # B, Hkv, cap, d, block, n, lens, at, counts
    (2, 2, 200, 128, 128, 1, (0, 127), None, None),
    (2, 1, 300, 64, 64, 130, (63, 64), None, (130, 0)),
    (1, 3, 77, 128, 64, 77, (0,), None, None),
    (3, 2, 500, 64, 128, 257, (10, 200, 243), None, (257, 1, 257)),
    (2, 2, 400, 128, 64, 33, (300, 5), (31, 5), (33, 32)),
    (1, 1, 1, 64, 64, 1, (0,), None, None),
    (4, 8, 1100, 128, 128, 1000, (1, 100, 37, 0), None, (999, 1000, 3, 128)),
]


@pytest.mark.parametrize("c", APPENDS, ids=lambda c: "-".join(map(str, c[:6])))
def test_append(c):
    B, H, cap, d, block, n, lens, at, counts = c
    rng = np.random.default_rng(n + cap)
    arr = Arrays(rng, B, H, cap, d, block, lens, behind=False)
    cache = arr.gpu()
    K = bf16(rng.normal(size=(B, H, n, d)) * np.exp2(rng.integers(-4, 5, (B, H, n, 1))))
    V = bf16(rng.normal(size=(B, H, n, d)) * 7)
    K[0, 0, 0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    V[-1, -1, -1] = 0
    cache.append(K.to(dev()), V.to(dev()), at=None if at is None else i32(at),
                 counts=None if counts is None else i32(counts))
    torch.cuda.synchronize()
    assert int(cache.status.item()) == 0
    w = arr.w.copy()
    for b in range(B):
        p, m = (lens if at is None else at)[b], n if counts is None else counts[b]
        w[b, :, p: p + m] = 0
    for got, got_s, src, cs, ss in ((cache.k, cache.k_scale, K, arr.k, arr.ks), (cache.v, cache.v_scale, V, arr.v, arr.vs)):
        want, want_s, want_l = co.append(cs, ss, arr.lens, src.double().numpy(), block, at=at, counts=counts)
        np.testing.assert_array_equal(got_s.cpu().numpy(), want_s)
        same_codes(codes(got), want)
        np.testing.assert_array_equal(cache.lens.cpu().numpy(), want_l)
    np.testing.assert_array_equal(cache.weight.cpu().numpy(), w)


def test_append_extreme_values():
    """The largest bf16, denormals and an all-zero block; then a token that makes the block's scale jump."""
    cache = sfa.KvCache8.empty(batch=1, heads_kv=1, capacity=192, head_dim=64, block=64, weight=False)
    rng = np.random.default_rng(0)
    x = np.zeros((1, 1, 130, 64))
    x[0, 0, :64] = rng.normal(size=(64, 64)) * 1e37
    x[0, 0, 0, 0] = 3.38e38
    x[0, 0, 128:] = rng.normal(size=(2, 64)) * 2.0 ** -130
    K = bf16(x)
    state = [(np.zeros((1, 1, 192, 64), np.uint8), np.ones((1, 1, 3), np.float32), np.zeros(1, np.int32))] * 2
    for rows in (K, bf16(np.full((1, 1, 1, 64), 2.0 ** 100))):
        cache.append(rows.to(dev()), rows.to(dev()))
        state = [co.append(*s, rows.double().numpy(), 64) for s in state]
    torch.cuda.synchronize()
    for got, scale, s in ((cache.k, cache.k_scale, state[0]), (cache.v, cache.v_scale, state[1])):
        np.testing.assert_array_equal(scale.cpu().numpy(), s[1])
        same_codes(codes(got), s[0])
    assert cache.lens.tolist() == [131]


def test_append_token_by_token():
    rng = np.random.default_rng(3)
    cache = sfa.KvCache8.empty(batch=2, heads_kv=2, capacity=150, head_dim=64, block=64)
    want = [(np.zeros((2, 2, 150, 64), np.uint8), np.ones((2, 2, 3), np.float32), np.zeros(2, np.int32))] * 2
    for t in range(140):
        K, V = (bf16(rng.normal(size=(2, 2, 1, 64)) * 2.0 ** rng.integers(-6, 7)) for _ in range(2))
        cache.append(K.to(dev()), V.to(dev()))
        want = [co.append(*s, x.double().numpy(), 64) for s, x in zip(want, (K, V))]
    same_codes(codes(cache.k), want[0][0])
    same_codes(codes(cache.v), want[1][0])
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy(), want[0][1])
    np.testing.assert_array_equal(cache.v_scale.cpu().numpy(), want[1][1])


def test_append_refuses_bad_positions_on_the_device():
    rng = np.random.default_rng(4)
    arr = Arrays(rng, 5, 2, 100, 64, 64, (99, -1, 5, 6, 7), behind=False)
    K = bf16(rng.normal(size=(5, 2, 3, 64))).to(dev())
    cache = arr.gpu()
    cache.append(K, K, counts=i32((2, 1, 4, -1, 3)))  # past the end, negative length, count > n, negative count, fine
    assert int(cache.status.item()) == 8
    assert cache.lens.tolist() == [99, -1, 5, 6, 10]
    same_codes(codes(cache.k)[:4], arr.k[:4])
    np.testing.assert_array_equal(cache.v_scale.cpu().numpy()[:4], arr.vs[:4])
    want, _, _ = co.append(arr.k[4:], arr.ks[4:], arr.lens[4:], K.double().cpu().numpy()[4:], 64)
    same_codes(codes(cache.k)[4:], want)


# ---------------------------------------------------------------------------
# attention over the whole cache
# ---------------------------------------------------------------------------
ATTNS = [  # B, Hkv, G, cap, d, block, nq, back, lens, spread
    (1, 1, 1, 1, 128, 128, 1, 0, (1,), 0),
    (2, 1, 4, 300, 128, 128, 1, 0, (300, 0), 0),
    (3, 2, 8, 129, 128, 64, 1, 0, (127, 128, 129), 0),
    (3, 2, 1, 700, 64, 64, 1, 0, (1, 640, 511), 0),
    (2, 2, 2, 1000, 128, 128, 8, 0, (3, 999), 0),     # the first queries of a short sequence see nothing
    (2, 1, 8, 513, 64, 128, 2, 0, (513, 129), 0),     # a causal edge on a tile's border
    (2, 2, 4, 400, 128, 64, 4, 7, (400, 6), 0),       # back beyond one sequence's length
    (1, 1, 4, 5000, 128, 128, 1, 0, (4999,), 0),      # more pieces than units
    (40, 1, 2, 140, 64, 64, 1, 0, tuple(range(40)) , 0),  # a warp's worth of sequences and more
    (2, 2, 4, 600, 128, 64, 1, 0, (600, 333), 6),     # scales far apart between blocks
    (2, 2, 4, 600, 64, 128, 3, 0, (600, 333), 6),
    (9, 8, 4, 900, 128, 128, 1, 0, (900, 1, 2, 3, 500, 0, 700, 800, 31), 1),  # pieces that cross sequences
    (1, 1, 1, 1, 64, 64, 1, 0, (1,), 0),
    (2, 2, 8, 700, 64, 64, 2, 3, (700, 2), 2),        # 16 rows, small blocks
    (1, 2, 1, 600, 64, 128, 11, 0, (600,), 1),        # 11 rows: padded to 12
    (20, 8, 4, 200, 128, 64, 1, 0, tuple(range(0, 200, 10)), 0),   # more rows than joining CTAs fit at once
    (3, 1, 1, 300, 128, 128, 16, 0, (300, 15, 256), 0),
    (4, 2, 2, 50, 64, 64, 1, 0, (0, 0, 0, 0), 0),     # nothing anywhere
    (3, 2, 1, 600, 64, 64, 8, 0, (259, 512, 258), 2),  # the causal edge over two tiles of 256
    (3, 1, 1, 300, 128, 128, 8, 0, (130, 256, 263), 1),  # and of 128
    # more tiles than CTAs: shares that cross units
    (64, 8, 4, 500, 128, 64, 1, 0, tuple(i * 37 % 501 for i in range(64)), 1),
    (70, 8, 1, 700, 64, 64, 2, 0, tuple(i * 211 % 701 if i % 5 else 0 for i in range(70)), 1),
    (3, 8, 2, 2600, 128, 128, 4, 5, (2600, 1300, 2599), 1),
    (1, 1, 1, 38100, 128, 128, 1, 0, (38100,), 0),
]


def run_attn(arr, q, nq, back, w=True, **kw):
    cache = arr.gpu()
    qd = q.to(dev())
    lse = torch.full(q.shape[:-1], 7.0, device=dev())
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev())
    w_out = torch.full(arr.w.shape, 7.0, device=dev()) if w else None
    sfa.cache8_attn(qd, cache, back=back, o=o, lse=lse, weight_in=cache.weight if w else None, weight_out=w_out,
                    status=cache.status, **kw)
    torch.cuda.synchronize()
    return o, lse, w_out, cache


def check_attn(arr, q, nq, back, o, lse, w_out, scale=None):
    B, H, cap, d = arr.k.shape
    qn = q.double().numpy()
    want, wl, ww, errs = co.attn(qn, arr.k, arr.ks, arr.v, arr.vs, arr.lens, arr.block, back=back, scale=scale)
    o_tol, lse_tol, ds = bounds(want, wl, errs, d)
    close(lse, wl, lse_tol, "lse")
    close(o, want, o_tol, "o")
    if w_out is not None:
        got = w_out.double().cpu().numpy()
        G = q.shape[1] // H
        dsu = ds.reshape(B, H, G * nq).max(-1)[..., None]
        for b in range(B):
            n = max(int(arr.lens[b]) - back, 0)
            win = arr.w[b, :, :n].astype(np.float64)
            tol = ww[b, :, :n] * (2 * dsu[b] + 2.0 ** -19) + 2.0 ** -22 * (win + ww[b, :, :n])
            err = np.abs(got[b, :, :n] - win - ww[b, :, :n])
            assert np.all(err <= tol), f"weights of sequence {b}: {np.max(err - tol):.3e} over"
            assert np.all(got[b, :, n:] == 7.0)


@pytest.mark.parametrize("c", ATTNS, ids=lambda c: "-".join(map(str, c[:8])))
@pytest.mark.parametrize("weights", [False, True])
def test_attention(c, weights):
    B, H, G, cap, d, block, nq, back, lens, spread = c
    rng = np.random.default_rng(cap + d + nq)
    arr = Arrays(rng, B, H, cap, d, block, lens, spread=spread)
    q = bf16(rng.normal(size=(B, H * G, nq, d)) * 2)
    o, lse, w_out, cache = run_attn(arr, q, nq, back, w=weights)
    assert int(cache.status.item()) == 0
    check_attn(arr, q, nq, back, o, lse, w_out)


def test_attention_three_dim_q_scale_and_bits():
    """[B, Hq, d] queries, a scale of one's own, weights added in place, the same bits twice."""
    rng = np.random.default_rng(11)
    arr = Arrays(rng, 2, 2, 777, 128, 64, (777, 200))
    q = bf16(rng.normal(size=(2, 8, 128)))
    first = arr.gpu()
    lse = torch.empty((2, 8), device=dev())
    o = first.attend(q.to(dev()), scale=0.2, accumulate=True, lse=lse)
    w = first.weight.clone()
    w[0, :, 777:] = 7.0
    w[1, :, 200:] = 7.0
    check_attn(arr, q[:, :, None], 1, 0, o[:, :, None], lse[:, :, None], w, scale=0.2)
    second = arr.gpu()
    o2 = second.attend(q.to(dev()), scale=0.2, accumulate=True)
    assert torch.equal(o, o2) and torch.equal(first.weight, second.weight)


def test_attention_peaked_and_far_scores():
    """One token takes all the weight; scores hundreds apart."""
    rng = np.random.default_rng(12)
    arr = Arrays(rng, 1, 1, 500, 128, 128, (500,))
    q = np.zeros((1, 4, 1, 128))
    q[0, :, 0] = co.values(arr.k[0, 0], arr.ks[0, 0], 128)[[0, 130, 260, 499]] * 20
    q = bf16(q)
    o, lse, w_out, _ = run_attn(arr, q, 1, 0)
    check_attn(arr, q, 1, 0, o, lse, w_out)


def test_attention_nan_stays_where_it_is():
    """A NaN key or value of a visible token spoils its head's rows, nothing else; a NaN of a token that a query
    does not see yet does not reach that query."""
    rng = np.random.default_rng(13)
    for d, block in ((128, 128), (64, 64)):
        arr = Arrays(rng, 2, 2, 400, d, block, (300, 260))
        clean = bf16(rng.normal(size=(2, 4, 3, d)))
        arr.k[0, 1, 17, 5] = 0x7F
        arr.v[1, 0, 259, 3] = 0x7F   # the newest token: only the last query sees it
        arr.k[1, 1, 258, 3] = 0x7F   # the last but one: the last two queries
        o, lse, _, _ = run_attn(arr, clean, 3, 0, w=False)
        on, ln = torch.isnan(o).cpu(), torch.isnan(lse).cpu()
        assert not on[0, :2].any() and on[0, 2:].all() and ln[0, 2:].all()
        assert not on[1, :2, :2].any() and on[1, :2, 2, 3].all() and not ln[1, :2].any()
        assert not on[1, 2:, 0].any() and on[1, 2:, 1:].all()
        q = clean.clone()
        q[0, 0, 1, 0] = float("inf")
        o, _, _, _ = run_attn(arr, q, 3, 0, w=False)
        assert torch.isnan(o[0, 0, 1]).all() and not torch.isnan(o[0, 0, 0]).any() and not torch.isnan(o[0, 1]).any()


def test_attention_bad_lengths_count_as_empty():
    rng = np.random.default_rng(14)
    arr = Arrays(rng, 3, 1, 200, 64, 64, (201, 100, -5))
    q = bf16(rng.normal(size=(3, 2, 1, 64)))
    o, lse, w_out, cache = run_attn(arr, q, 1, 0)
    assert int(cache.status.item()) == 8
    assert torch.isneginf(lse[[0, 2]]).all() and torch.all(o[[0, 2]] == 0)
    arr.lens = np.array([0, 100, 0], np.int32)
    check_attn(arr, q, 1, 0, o, lse, w_out)


def test_attention_in_a_graph_follows_the_lengths():
    """Captured once with the append before it: replays read new rows, new lengths, new queries."""
    rng = np.random.default_rng(15)
    arr = Arrays(rng, 2, 2, 400, 128, 128, (126, 255), behind=False)
    cache = arr.gpu()
    ref = arr.gpu()
    K, V = (torch.zeros((2, 2, 1, 128), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device=dev())
    o = torch.empty_like(q)
    side = torch.cuda.Stream()
    scratch = arr.gpu()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        scratch.append(K, V)
        scratch.attend(q, accumulate=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(K, V)
        cache.attend(q, accumulate=True, o=o)
    for step in range(5):
        for t in (K, V, q):
            t.copy_(bf16(rng.normal(size=tuple(t.shape))))
        graph.replay()
        ref.append(K, V)
        want = ref.attend(q, accumulate=True)
        assert torch.equal(o, want)
    assert cache.lens.tolist() == [131, 260]
    assert torch.equal(cache.weight, ref.weight) and torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8))


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(16)
    arr = Arrays(rng, 2, 2, 5000, 128, 128, (5000, 4000))
    cache = arr.gpu()
    qs = [bf16(rng.normal(size=(2, 8, 128))).to(dev()) for _ in range(2)]
    want = [cache.attend(q) for q in qs]
    ws = [torch.empty(sfa.cache8_attn_workspace(q, cache), dtype=torch.uint8, device=dev()) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(10):
        for q, w, o, s in zip(qs, ws, outs, streams):
            sfa.cache8_attn(q, cache, workspace=w, o=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    for _ in range(10):  # the handle's own workspaces: one a stream
        got = [cache.attend(q, o=o, stream=s) for q, o, s in zip(qs, outs, streams)]
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o, w)


def test_two_graphs_of_one_cache_replayed_together():
    """Each captured attention has a workspace of its own, although the handle is shared."""
    rng = np.random.default_rng(18)
    arr = Arrays(rng, 2, 2, 6000, 128, 64, (6000, 3000))
    cache = arr.gpu()
    qs = [bf16(rng.normal(size=(2, 8, 128))).to(dev()) for _ in range(2)]
    want = [cache.attend(q) for q in qs]
    outs, graphs, streams = [torch.empty_like(q) for q in qs], [], [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                cache.attend(q, o=o)
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_attention_long_cache_sampled_rows():
    """131072 tokens of 8 heads: some rows against the oracle."""
    rng = np.random.default_rng(17)
    g = torch.Generator(device=dev()).manual_seed(3)
    n, cap = 131000, 131072
    cache = sfa.KvCache8.empty(batch=1, heads_kv=8, capacity=cap, head_dim=128)
    K, V = (torch.randn((1, 8, n, 128), generator=g, device=dev()).bfloat16() for _ in range(2))
    cache.append(K, V)
    q = torch.randn((1, 32, 128), generator=g, device=dev()).bfloat16()
    lse = torch.empty((1, 32), device=dev())
    o = cache.attend(q, accumulate=True, lse=lse)
    total = cache.weight.double().sum(-1).cpu().numpy()
    np.testing.assert_allclose(total, 4.0, rtol=1e-4)  # four heads' softmax each
    for h in rng.choice(32, 3, replace=False):
        u = int(h) // 4
        arrs = [codes(cache.k[:, u:u + 1]), cache.k_scale[:, u:u + 1].cpu().numpy(), codes(cache.v[:, u:u + 1]),
                cache.v_scale[:, u:u + 1].cpu().numpy()]
        want, wl, _, errs = co.attn(q[:, h:h + 1, None].double().cpu().numpy(), *arrs, np.array([n]), 128)
        o_tol, lse_tol, _ = bounds(want, wl, errs, 128)
        close(lse[:, h:h + 1, None], wl, lse_tol, "lse")
        close(o[:, h:h + 1, None], want, o_tol, "o")


# ---------------------------------------------------------------------------
# index lists
# ---------------------------------------------------------------------------
LISTS = [  # B, Hkv, G, cap, d, block, k, lens
    (2, 2, 4, 500, 128, 128, 256, (500, 300)),
    (1, 1, 1, 40, 64, 64, 1, (40,)),
    (3, 1, 8, 700, 64, 64, 77, (700, 0, 5)),
    (2, 2, 2, 900, 128, 64, 1023, (900, 899)),
    (40, 8, 1, 130, 128, 128, 33, tuple(range(1, 41))),
    (1, 1, 2, 5000, 64, 128, 4500, (5000,)),   # a list staged in parts
    # more rows than CTAs of whole rows are resident: two CTAs a row
    (75, 2, 2, 300, 64, 64, 1, tuple(i * 7 % 300 for i in range(75))),
    (38, 8, 1, 703, 128, 64, 601, tuple(i * 19 for i in range(38))),
    (38, 1, 8, 900, 64, 128, 4500, (900,) * 38),
]


@pytest.mark.parametrize("c", LISTS, ids=lambda c: "-".join(map(str, c[:7])))
def test_list_attention(c):
    """Unordered lists with repeats and gaps; some rows of gaps only."""
    B, H, G, cap, d, block, k, lens = c
    rng = np.random.default_rng(k)
    arr = Arrays(rng, B, H, cap, d, block, lens, spread=2)
    q = bf16(rng.normal(size=(B, H * G, d)) * 2)
    idx = np.stack([rng.integers(-1, max(n, 1), (H * G, k)) for n in lens]).astype(np.int32)
    idx[np.asarray(lens) == 0] = -1
    idx[0, 0] = -1
    cache = arr.gpu()
    lse = torch.empty((B, H * G), device=dev())
    o = cache.attend_list(q.to(dev()), torch.from_numpy(idx).to(dev()), lse=lse)
    assert int(cache.status.item()) == 0
    want, wl, errs = co.attn_list(q.double().numpy(), arr.k, arr.ks, arr.v, arr.vs, arr.lens, idx, block)
    o_tol, lse_tol, _ = bounds(want, wl, errs, d)
    close(lse, wl, lse_tol, "lse")
    close(o, want, o_tol, "o")


def test_list_attention_reports_bad_entries():
    rng = np.random.default_rng(21)
    arr = Arrays(rng, 1, 1, 200, 128, 128, (100,))
    cache = arr.gpu()
    q = bf16(rng.normal(size=(1, 4, 128))).to(dev())
    idx = torch.randint(0, 100, (1, 4, 50), dtype=torch.int32, device=dev())
    good = cache.attend_list(q, idx)
    idx[0, 1, 7] = 100   # behind the last token
    idx[0, 2, 49] = -2
    lse = torch.empty((1, 4), device=dev())
    o = cache.attend_list(q, idx, lse=lse)
    assert int(cache.status.item()) == 8
    assert torch.all(o[0, 1:3] == 0) and torch.isneginf(lse[0, 1:3]).all()
    assert torch.equal(o[0, [0, 3]], good[0, [0, 3]])


def test_list_attention_reports_bad_entries_of_either_half():
    """More rows than fit as whole rows: a list's halves are read by two CTAs, and one bad entry empties the row."""
    rng = np.random.default_rng(22)
    arr = Arrays(rng, 50, 2, 200, 128, 128, (100,) * 50)
    cache = arr.gpu()
    q = bf16(rng.normal(size=(50, 8, 128))).to(dev())
    idx = torch.randint(0, 100, (50, 8, 51), dtype=torch.int32, device=dev())
    good = cache.attend_list(q, idx)
    assert int(cache.status.item()) == 0
    idx[3, 1, 0], idx[20, 7, 50], idx[49, 0, 26] = 100, -2, 150
    lse = torch.empty((50, 8), device=dev())
    o = cache.attend_list(q, idx, lse=lse)
    assert int(cache.status.item()) == 8
    fine = torch.ones((50, 8), dtype=torch.bool, device=dev())
    for at in ((3, 1), (20, 7), (49, 0)):
        assert torch.all(o[at] == 0) and torch.isneginf(lse[at])
        fine[at] = False
    assert torch.equal(o[fine], good[fine]) and torch.isfinite(lse[fine]).all()


# ---------------------------------------------------------------------------
# eviction and the compact keys
# ---------------------------------------------------------------------------
EVICTS = [  # B, Hkv, cap, d, block, keep, recent, dst capacity, lens
    (2, 2, 500, 128, 128, 200, 50, 200, (500, 150)),
    (1, 1, 5, 64, 64, 1, 0, 1, (5,)),
    (1, 1, 5, 64, 64, 1, 1, 3, (5,)),
    (3, 2, 1000, 64, 64, 65, 65, 100, (1000, 66, 0)),
    (2, 1, 700, 128, 64, 333, 0, 400, (700, 334)),
    (1, 8, 9000, 128, 128, 1100, 128, 1200, (9000,)),
    (2, 1, 300, 64, 128, 400, 7, 450, (300, 299)),
    (2, 1, 20000, 64, 64, 1500, 100, 1600, (20000, 17)),     # slices over a cluster of CTAs
    (1, 1, 140000, 64, 128, 2000, 31, 2000, (139999,)),      # longer than the clusters' shared memory holds
    # heads whose weights start at every remainder of 16 bytes
    (2, 2, 333, 64, 64, 100, 9, 100, (333, 331)),
    (1, 4, 20003, 64, 128, 700, 50, 700, (20003,)),
    (1, 2, 131079, 64, 128, 300, 0, 300, (131079,)),
]


@pytest.mark.parametrize("c", EVICTS, ids=lambda c: "-".join(map(str, c[:8])))
def test_eviction(c):
    B, H, cap, d, block, keep, recent, dcap, lens = c
    rng = np.random.default_rng(keep + cap)
    arr = Arrays(rng, B, H, cap, d, block, lens, spread=5, behind=False)
    arr.w = np.where(rng.random(arr.w.shape) < 0.3, np.float32(0.25), arr.w)  # ties
    arr.w[0, 0, : min(3, cap)] = [np.nan, -0.0, np.inf][: min(3, cap)]
    arr.k[0, 0, 0, 0] = 0x7F
    to = Arrays(rng, B, H, dcap, d, block, [0] * B, behind=False)
    src, dst = arr.gpu(), to.gpu()
    idx = src.evict(dst, keep=keep, recent=recent)
    assert int(src.status.item()) == 0
    held = dict(k=to.k, ks=to.ks, v=to.v, vs=to.vs, lens=to.lens, weight=to.w)
    want, widx = co.evict(arr.k, arr.ks, arr.v, arr.vs, arr.lens, arr.w, block, keep, recent, held)
    np.testing.assert_array_equal(idx.cpu().numpy(), widx)
    np.testing.assert_array_equal(dst.lens.cpu().numpy(), want["lens"])
    np.testing.assert_array_equal(dst.k_scale.cpu().numpy(), want["ks"])
    np.testing.assert_array_equal(dst.v_scale.cpu().numpy(), want["vs"])
    same_codes(codes(dst.k), want["k"])
    same_codes(codes(dst.v), want["v"])
    np.testing.assert_array_equal(dst.weight.cpu().numpy(), want["weight"])
    np.testing.assert_array_equal(src.lens.cpu().numpy(), arr.lens)


def test_eviction_bad_length_and_no_list():
    """A bad length counts as an empty sequence; without idx the list lives in the workspace."""
    rng = np.random.default_rng(31)
    arr = Arrays(rng, 3, 1, 300, 64, 64, (301, 300, -2), behind=False)
    src, dst = arr.gpu(), Arrays(rng, 3, 1, 64, 64, 64, (0, 0, 0), behind=False).gpu()
    lib = sfa.load()
    import ctypes
    ws = torch.empty(sfa.cache8_evict_workspace(src, 50), dtype=torch.uint8, device=dev())
    assert lib.sfa_cache8_evict(ctypes.byref(src.shape(1)), ctypes.byref(src._c), ctypes.byref(dst._c), 64, 50, 10, None,
                                ctypes.c_void_p(ws.data_ptr()), ws.numel(), ctypes.c_void_p(src.status.data_ptr()),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert int(src.status.item()) == 8
    assert dst.lens.tolist() == [0, 50, 0]
    other = Arrays(rng, 3, 1, 64, 64, 64, (0, 0, 0), behind=False).gpu()
    idx = src.evict(other, keep=50, recent=10)
    assert torch.all(idx[[0, 2]] == -1) and idx[1, 0].tolist() == co.kept_tokens(arr.w[1, 0], 300, 50, 10)
    assert torch.equal(other.k[1].view(torch.uint8)[:, :50], dst.k[1].view(torch.uint8)[:, :50])


@pytest.mark.parametrize("nfc,d", [(4, 64), (12, 128), (32, 64), (64, 128)])
def test_compact_keys(nfc, d):
    rng = np.random.default_rng(nfc)
    arr = Arrays(rng, 2, 3, 333, d, 64, (333, 333), spread=8)
    fc = np.stack([rng.permutation(d // 2)[:nfc] for _ in range(3)])
    out = torch.full((2, 3, 333, 2 * nfc), 7.0, dtype=torch.bfloat16, device=dev())
    sfa.cache8_fc_gather(arr.gpu(), fc, K_fc=out, pos0=60, npos=201)
    want = np.full(out.shape, 7.0)
    want[:, :, 60:261] = co.fc_gather(arr.k, arr.ks, fc, 64)[:, :, 60:261]
    np.testing.assert_array_equal(out.double().cpu().numpy(), want)


def test_offsets_beyond_32_bits():
    """Twelve heads of 2 million tokens (3 GB of keys, as much of values): rows at the end of the last head.  All
    tokens but the last 300 are zero, so the softmax has a closed form."""
    n, cap, m = 1_999_990, 2_000_000, 300
    rng = np.random.default_rng(51)
    cache = sfa.KvCache8.empty(batch=1, heads_kv=12, capacity=cap, head_dim=128)
    K, V = (bf16(rng.normal(size=(1, 12, m, 128))) for _ in range(2))
    cache.append(K.to(dev()), V.to(dev()), at=i32([n - m]))
    assert cache.lens.tolist() == [n]
    tail = slice((n - m) // 128 * 128, cap)
    held = [codes(x[:, 11:, tail]) for x in (cache.k, cache.v)] + [x[0, 11, tail.start // 128:].cpu().numpy()
                                                                 for x in (cache.k_scale, cache.v_scale)]
    off = n - m - tail.start
    k = co.values(held[0][0, 0], held[2], 128)[off: off + m]
    v = co.values(held[1][0, 0], held[3], 128)[off: off + m]
    close(torch.from_numpy(k), K[0, 11].double().numpy(), 2.0 ** -4 * np.abs(K[0, 11].double().numpy()) + 2.0 ** -10, "k")
    q = bf16(rng.normal(size=(1, 12, 128)) * 3)
    lse = torch.empty((1, 12), device=dev())
    o = cache.attend(q.to(dev()), accumulate=True, lse=lse)
    e = np.exp(k @ q[0, 11].double().numpy() / 128 ** 0.5)
    z = e.sum() + n - m
    assert abs(lse[0, 11].item() - np.log(z)) < 1e-5
    # a probability's two parts end 2^-23 under its block's largest; sums of 300 terms
    tol = (2.0 ** -8 + 2.0 ** -12) * (e @ np.abs(v)) / z + 2.0 ** -22 * e.max() / z * np.abs(v).sum(0) + 2.0 ** -30
    assert np.all(np.abs(o[0, 11].double().cpu().numpy() - e @ v / z) <= tol + 2.0 ** -8 * np.abs(e @ v / z))
    idx = torch.arange(n - m, n, dtype=torch.int32, device=dev()).expand(1, 12, m).contiguous()
    ol = cache.attend_list(q.to(dev()), idx)
    np.testing.assert_allclose(ol[0, 11].double().cpu().numpy(), e @ v / e.sum(), rtol=2e-2, atol=1e-2)
    fc = np.tile(np.arange(4), (12, 1))
    K_fc = sfa.cache8_fc_gather(cache, fc, pos0=n - m, npos=m)
    np.testing.assert_array_equal(K_fc[0, 11, n - m:n].double().cpu().numpy(), k[:, [0, 1, 2, 3, 64, 65, 66, 67]])
    cache.weight[0, 11, n - m] = 5.0
    small = sfa.KvCache8.empty(batch=1, heads_kv=12, capacity=128, head_dim=128)
    kept = cache.evict(small, keep=100, recent=99)
    assert kept[0, 11].tolist() == [n - m] + list(range(n - 99, n))
    got = co.values(codes(small.k)[0, 11], small.k_scale[0, 11].cpu().numpy(), 128)[:100]
    want = k[[0] + list(range(m - 99, m))]
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9)
    assert int(cache.status.item()) == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_run_of_them_together():
    """A prompt joins, its last queries are observed, tokens are decoded with the weights accumulated, the cache is
    evicted to its budget, and decoding goes on in the smaller cache."""
    rng = np.random.default_rng(41)
    B, H, G, d, T, n = 2, 2, 4, 128, 128, 600
    cache = sfa.KvCache8.empty(batch=B, heads_kv=H, capacity=700, head_dim=d, block=T)
    k = v = np.zeros((B, H, 700, d), np.uint8)
    ks = vs = np.ones((B, H, 6), np.float32)
    lens = np.zeros(B, np.int32)
    w = np.zeros((B, H, 700))

    def join(K, V, counts=None):
        nonlocal k, ks, v, vs, lens
        cache.append(K.to(dev()), V.to(dev()), counts=None if counts is None else i32(counts))
        k, ks, _ = co.append(k, ks, lens, K.double().numpy(), T, counts=counts)
        v, vs, lens = co.append(v, vs, lens, V.double().numpy(), T, counts=counts)

    def attend(q, back=0):
        nonlocal w
        nq = q.shape[2]
        lse = torch.empty(q.shape[:-1], device=dev())
        o = cache.attend(q.to(dev()), back=back, accumulate=True, lse=lse)
        want, wl, ww, errs = co.attn(q.double().numpy(), k, ks, v, vs, lens, T, back=back)
        o_tol, lse_tol, _ = bounds(want, wl, errs, d)
        close(o, want, o_tol, "o")
        close(lse, wl, lse_tol, "lse")
        w = w + ww

    join(bf16(rng.normal(size=(B, H, n, d))), bf16(rng.normal(size=(B, H, n, d))), counts=(600, 471))
    window = bf16(rng.normal(size=(B, H * G, 12, d)))
    for c in range(0, 12, 4):  # the prompt's last twelve queries, four at a time
        attend(window[:, :, c:c + 4].contiguous(), back=12 - 4 - c)
    for _ in range(5):
        join(bf16(rng.normal(size=(B, H, 1, d))), bf16(rng.normal(size=(B, H, 1, d))))
        attend(bf16(rng.normal(size=(B, H * G, 1, d))))
    np.testing.assert_allclose(cache.weight.double().cpu().numpy(), w, rtol=1e-4, atol=1e-6)
    small = sfa.KvCache8.empty(batch=B, heads_kv=H, capacity=300, head_dim=d, block=T)
    idx = cache.evict(small, keep=256, recent=64)
    held = dict(k=np.zeros((B, H, 300, d), np.uint8), ks=np.ones((B, H, 3), np.float32),
                v=np.zeros((B, H, 300, d), np.uint8), vs=np.ones((B, H, 3), np.float32), lens=np.zeros(B, np.int32),
                weight=np.zeros((B, H, 300), np.float32))
    got_w = cache.weight.cpu().numpy()
    held, widx = co.evict(k, ks, v, vs, lens, got_w, T, 256, 64, held)
    np.testing.assert_array_equal(idx.cpu().numpy(), widx)
    cache, (k, ks, v, vs, lens) = small, (held[x] for x in ("k", "ks", "v", "vs", "lens"))
    w = np.zeros((B, H, 300))
    join(bf16(rng.normal(size=(B, H, 1, d))), bf16(rng.normal(size=(B, H, 1, d))))
    attend(bf16(rng.normal(size=(B, H * G, 1, d))))
    assert cache.lens.tolist() == [257, 257] and int(cache.status.item()) == 0


def test_fasa_decode_on_the_8_bit_cache():
    """FasaDecode given the 8-bit cache: compact keys, selection and attention all see the stored values; its graph
    step gives the eager bits."""
    wl = DecodeWorkload(name="fasa8", batch=2, heads_q=8, heads_kv=2, seq_len=5000, head_dim=128, nfc=12, k=256)
    q, K, V, fc = make_decode_inputs(wl, seed=2)
    cache = sfa.KvCache8.empty(batch=2, heads_kv=2, capacity=5000, head_dim=128, weight=False)
    cache.append(K.to(dev()), V.to(dev()))
    m = sfa.FasaDecode(batch=2, heads_q=8, heads_kv=2, seq_len=5000, head_dim=128, fc=fc, k=256)
    m.refresh_keys(cache)
    qd = q.to(dev())
    o = m(qd, cache).clone()
    idx = m.idx.clone()
    ck, cks, cv, cvs = codes(cache.k), cache.k_scale.cpu().numpy(), codes(cache.v), cache.v_scale.cpu().numpy()
    stored = np.stack([[co.values(ck[b, g], cks[b, g], 128) for g in range(2)] for b in range(2)])
    _, widx, _, _ = fo.decode_step(q.double().numpy(), stored, stored, fc, 256)
    assert (idx.cpu().numpy() == widx).all(-1).mean() > 0.99
    want, wl_, errs = co.attn_list(q.double().numpy(), ck, cks, cv, cvs, cache.lens.cpu().numpy(), idx.cpu().numpy(),
                                    128)
    o_tol, lse_tol, _ = bounds(want, wl_, errs, 128)
    close(o, want, o_tol, "o")
    close(m.lse, wl_, lse_tol, "lse")
    for _ in range(2):
        m.idx.fill_(-7)
        m.step(qd, cache, pos=4999)
        assert torch.equal(m.idx, idx) and torch.equal(m.o, o)
    assert int(m.status.item()) == 0


def test_graph_step_follows_the_cache_it_is_given():
    """Caches over the same codes and lengths with other scales, and with other blocks: each step reads its own."""
    rng = np.random.default_rng(61)
    arr = Arrays(rng, 1, 2, 1000, 64, 64, (1000,), weight=False)
    a = arr.gpu()
    other = [torch.from_numpy(np.ldexp(x, rng.integers(-3, 4, x.shape)).astype(np.float32)).to(dev()) for x in (arr.ks, arr.vs)]
    same = dict(k=a.k, v=a.v, lens=a.lens)
    caches = [a, sfa.KvCache8(**same, k_scale=other[0], v_scale=a.v_scale, block=64),
              sfa.KvCache8(**same, k_scale=a.k_scale, v_scale=other[1], block=64),
              sfa.KvCache8(**same, k_scale=other[0][:, :, :8].contiguous(), v_scale=other[1][:, :, :8].contiguous())]
    fc = np.tile(np.arange(8), (2, 1))
    m, ref = (sfa.FasaDecode(batch=1, heads_q=8, heads_kv=2, seq_len=1000, head_dim=64, fc=fc, k=40) for _ in range(2))
    q = bf16(rng.normal(size=(1, 8, 64))).to(dev())
    outs = []
    for c in caches + caches[::-1]:
        for x in (m, ref):
            x.refresh_keys(c)
        got = m.step(q, c, pos=999)
        want = ref(q, c)
        assert torch.equal(got, want) and torch.equal(m.idx, ref.idx) and torch.equal(m.lse, ref.lse)
        outs.append(want.clone())
    assert not any(torch.equal(outs[0], o) for o in outs[1:4])
    assert int(m.status.item()) == 0


def test_threads_share_a_handle():
    """Four host threads on the default stream: attentions with partial results to join, and appended tokens."""
    import threading

    rng = np.random.default_rng(62)
    arr = Arrays(rng, 1, 2, 6000, 128, 128, (6000,))
    cache, grown = arr.gpu(), sfa.KvCache8.empty(batch=1, heads_kv=2, capacity=400, head_dim=128)
    qs = [bf16(rng.normal(size=(1, 8, 128))).to(dev()) for _ in range(4)]
    want = [cache.attend(q) for q in qs]
    outs = [torch.zeros((100, 1, 8, 128), dtype=torch.bfloat16, device=dev()) for _ in qs]
    rows = [torch.full((1, 2, 1, 128), float(i + 1), dtype=torch.bfloat16, device=dev()) for i in range(4)]
    start = threading.Barrier(4)

    def work(i):
        start.wait()
        for k in range(100):
            cache.attend(qs[i], o=outs[i][k])
            grown.append(rows[i], rows[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w.expand_as(o))
    held = co.values(codes(grown.k)[0, 0], grown.k_scale[0, 0].cpu().numpy(), 128)
    assert grown.lens.tolist() == [400] and all((held[:, 0] == i + 1).sum() == 100 for i in range(4))
    assert int(cache.status.item()) == 0 and int(grown.status.item()) == 0


def segment_stream(t):
    """The stream from whose memory the allocator made a tensor."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_buffers_made_for_a_call_on_another_stream():
    """Outputs and workspaces that a call makes come from its own stream's memory: what the current stream has still
    to write to a block that was freed there does not reach them."""
    rng = np.random.default_rng(63)
    arr = Arrays(rng, 2, 2, 3000, 128, 128, (3000, 2000))
    cache = arr.gpu()
    q = bf16(rng.normal(size=(2, 8, 128))).to(dev())
    idx = torch.randint(0, 2000, (2, 8, 64), dtype=torch.int32, device=dev())
    fc = np.tile(np.arange(4), (2, 1))
    small = [sfa.KvCache8.empty(batch=2, heads_kv=2, capacity=300, head_dim=128) for _ in range(2)]
    calls = [lambda **kw: cache.attend(q, **kw), lambda **kw: sfa.cache8_attn(q, cache, **kw),
             lambda **kw: cache.attend_list(q, idx, **kw), lambda **kw: sfa.cache8_fc_gather(cache, fc, **kw),
             lambda **kw: cache.evict(small[len(kw)], keep=300, recent=20, **kw)]
    want = [call() for call in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        late = torch.empty_like(w)
        torch.cuda._sleep(20_000_000)  # 10 ms before the current stream writes to the block that it frees here
        late.view(torch.uint8).fill_(0x55)
        del late
        got = call(stream=side)
        assert segment_stream(got) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))  # (rows that hold nothing are NaN)
    streams = {segment_stream(w) for w in cache._workspaces.values()}
    assert streams == {torch.cuda.current_stream().cuda_stream, side.cuda_stream}


def test_eviction_with_its_list_in_the_workspace():
    rng = np.random.default_rng(64)
    arr = Arrays(rng, 2, 2, 700, 64, 64, (700, 90), behind=False)
    src = arr.gpu()
    empty = [Arrays(rng, 2, 2, 128, 64, 64, (0, 0), behind=False).gpu() for _ in range(2)]
    ws = torch.full((sfa.cache8_evict_workspace(src, 100),), 0x55, dtype=torch.uint8, device=dev())
    idx = sfa.cache8_evict(src, empty[0], keep=100, recent=10, workspace=ws)
    want = src.evict(empty[1], keep=100, recent=10)
    assert idx.data_ptr() == ws.data_ptr() and torch.equal(idx, want)
    for b in range(2):
        n = int(empty[0].lens[b])
        assert n == min(100, int(arr.lens[b]))
        assert torch.equal(empty[0].k[b, :, :n].view(torch.uint8), empty[1].k[b, :, :n].view(torch.uint8))
    with pytest.raises(sfa.SfaError, match="WORKSPACE"):
        sfa.cache8_evict(src, empty[0], keep=100, recent=10, workspace=ws[:1536])


def test_weights_without_earlier_ones_and_eviction_into_a_cache_without():
    """weight_out alone starts from zero; a destination that keeps no weights gets the rows all the same."""
    rng = np.random.default_rng(65)
    arr = Arrays(rng, 2, 2, 500, 64, 64, (500, 77))
    cache = arr.gpu()
    q = bf16(rng.normal(size=(2, 4, 2, 64)))
    w = torch.full(arr.w.shape, 7.0, device=dev())
    o = sfa.cache8_attn(q.to(dev()), cache, weight_out=w)
    arr.w = np.zeros_like(arr.w)
    lse = torch.empty((2, 4, 2), device=dev())
    assert torch.equal(o, cache.attend(q.to(dev()), lse=lse))
    check_attn(arr, q, 2, 0, o, lse, w)
    with_w, without = (sfa.KvCache8.empty(batch=2, heads_kv=2, capacity=90, head_dim=64, block=64, weight=x)
                       for x in (True, False))
    assert torch.equal(cache.evict(with_w, keep=80, recent=9), cache.evict(without, keep=80, recent=9))
    for name in ("k", "v", "k_scale", "v_scale", "lens"):
        a, b = (getattr(c, name).view(torch.uint8) for c in (with_w, without))
        assert torch.equal(a, b)
    assert int(cache.status.item()) == 0
