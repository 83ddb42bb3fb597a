"""Pins of the 8-bit cache's oracle against torch, closed forms and properties (CPU)."""

import math

import numpy as np
import pytest
import torch

from oracle import cache8_oracle as co

NAN_CODES = (0x7F, 0xFF)


def test_values_are_torch_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(co.VALUES, t)
    assert co.VALUES[126] == 448.0 and co.VALUES[1] == 2.0 ** -9


def test_encode_is_the_torch_cast():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(size=4000) * 2.0 ** rng.integers(-12, 7, 4000)])
    mid = (co.VALUES[:126] + co.VALUES[1:127]) / 2  # every tie
    x = np.concatenate([x, mid, -mid, co.VALUES[~np.isnan(co.VALUES)]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(co.encode(x), want)
    assert list(co.encode([math.nan, math.inf, -math.inf])) == [0x7F] * 3


@pytest.mark.parametrize("a", [0.0, 1e-45, 2.0 ** -126, 448.0, np.nextafter(448.0, 500.0), 1.0, 3.4e38, 0.4375])
def test_need_is_the_smallest_power(a):
    f = co.need(a)
    assert a <= 448.0 * f and (f == 2.0 ** -126 or a > 224.0 * f)
    assert math.frexp(f)[0] == 0.5


def _cache(B, H, L, d, block):
    nb = -(-L // block)
    return np.zeros((B, H, L, d), np.uint8), np.ones((B, H, nb), np.float32), np.zeros(B, np.int32)


def _bf16(rng, shape):
    return torch.from_numpy(rng.normal(size=shape)).bfloat16().double().numpy()


def test_token_by_token_equals_at_once_for_normal_codes():
    """Powers of two: growing a block's scale keeps every code value that stays in e4m3's normal range."""
    rng = np.random.default_rng(1)
    x = _bf16(rng, (1, 2, 150, 8)) * np.exp2(rng.integers(0, 3, (1, 2, 150, 1)))
    x = np.where(np.abs(x) < 2.0 ** -3, 0.5, x)
    once = co.append(*_cache(1, 2, 200, 8, 64), x, 64)
    c = _cache(1, 2, 200, 8, 64)
    for t in range(150):
        c = co.append(*c, x[:, :, t: t + 1], 64)
    for a, b in zip(c, once):
        np.testing.assert_array_equal(a, b)


def test_append_rounds_once_and_uses_the_range():
    rng = np.random.default_rng(2)
    x = _bf16(rng, (2, 1, 70, 16))
    codes, scale, lens = co.append(*_cache(2, 1, 100, 16, 64), x, 64, counts=np.array([70, 3]))
    assert list(lens) == [70, 3]
    for b, m in ((0, 70), (1, 3)):
        back = co.values(codes[b, 0, :m], scale[b, 0], 64)
        f = np.repeat(scale[b, 0], 64)[:m, None].astype(np.float64)
        # half a step: 2^-4 of the value, or half the smallest code's value
        assert np.all(np.abs(back - x[b, 0, :m]) <= np.maximum(np.abs(x[b, 0, :m]) * 2.0 ** -4, f * 2.0 ** -10))
    assert np.all(codes[1, 0, 3:] == 0)
    bad = co.append(codes, scale, lens, x, 64, at=np.array([40, -1]))  # past the end, negative: nothing moves
    for a, b in zip(bad, (codes, scale, lens)):
        np.testing.assert_array_equal(a, b)


def test_nan_and_infinity_are_nan_codes_outside_the_scale():
    x = np.array([1.0, math.nan, math.inf, -2.0]).reshape(1, 1, 1, 4)
    codes, scale, _ = co.append(*_cache(1, 1, 64, 4, 64), x, 64)
    assert scale[0, 0, 0] == co.need(2.0)
    assert codes[0, 0, 0, 1] in NAN_CODES and codes[0, 0, 0, 2] in NAN_CODES
    assert VAL(codes[0, 0, 0, 3]) * scale[0, 0, 0] == -2.0


def VAL(c):
    return co.VALUES[c]


def test_attention_is_torch_softmax_attention():
    rng = np.random.default_rng(3)
    B, G, Hkv, nq, L, d = 2, 2, 2, 3, 40, 16
    x, y = _bf16(rng, (B, Hkv, L, d)), _bf16(rng, (B, Hkv, L, d))
    k, ks, lens = co.append(*_cache(B, Hkv, L, d, 64), x, 64, counts=np.array([40, 25]))
    v, vs, _ = co.append(*_cache(B, Hkv, L, d, 64), y, 64, counts=np.array([40, 25]))
    q = _bf16(rng, (B, G * Hkv, nq, d))
    o, lse, w, (a, a1, _) = co.attn(q, k, ks, v, vs, lens, 64, back=2)
    for b in range(B):
        n = int(lens[b]) - 2
        kk = torch.from_numpy(np.stack([co.values(k[b, h, :n], ks[b, h], 64) for h in range(Hkv)]))
        vv = torch.from_numpy(np.stack([co.values(v[b, h, :n], vs[b, h], 64) for h in range(Hkv)]))
        kk, vv = kk.repeat_interleave(G, 0), vv.repeat_interleave(G, 0)
        mask = torch.arange(n)[None, :] <= torch.arange(nq)[:, None] + n - nq
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b]), kk, vv, attn_mask=mask)
        np.testing.assert_allclose(o[b], want.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(w.sum((1, 2)), G * Hkv * nq, rtol=1e-12)
    assert np.all(w[1, :, 23:] == 0) and np.all(a >= np.abs(o) - 1e-15) and np.all(a1 >= a - 1e-15)
    # the whole cache as a list gives the one-query result
    idx = np.where(np.arange(L)[None, None] < lens[:, None, None], np.arange(L), -1)
    idx = np.broadcast_to(idx, (B, G * Hkv, L))
    ol, lsel, _ = co.attn_list(q[:, :, 0], k, ks, v, vs, lens, idx, 64)
    o1, lse1, _, _ = co.attn(q[:, :, :1], k, ks, v, vs, lens, 64)
    np.testing.assert_allclose(ol, o1[:, :, 0], rtol=1e-12)
    np.testing.assert_allclose(lsel, lse1[:, :, 0], rtol=1e-12)


def test_empty_rows():
    rng = np.random.default_rng(4)
    k, ks, lens = _cache(1, 1, 8, 4, 64)
    lens[0] = 1
    o, lse, w, _ = co.attn(_bf16(rng, (1, 2, 3, 4)), k, ks, k, ks, lens, 64)
    assert np.all(np.isneginf(lse[:, :, :2])) and np.all(o[:, :, :2] == 0)
    assert np.all(w[0, 0, 0] == 2.0) and np.all(w[0, 0, 1:] == 0)  # each head's last query on the only token


def test_eviction_keeps_a_dominant_set():
    rng = np.random.default_rng(5)
    for _ in range(60):
        n, keep = int(rng.integers(0, 30)), int(rng.integers(1, 30))
        recent = int(rng.integers(0, keep + 1))
        w = rng.integers(0, 4, 32).astype(np.float64)  # many ties
        t = co.kept_tokens(w, n, keep, recent)
        assert t == sorted(set(t)) and len(t) == min(n, keep)
        if n <= keep:
            continue
        assert set(range(n - recent, n)) <= set(t)
        out = [i for i in range(n - recent) if i not in t]
        for i in t:
            for j in out:
                assert i >= n - recent or (w[i], -i) > (w[j], -j)
    w = np.array([1.0, math.nan, math.inf, -0.0, 0.0, 2.0])
    assert co.kept_tokens(w, 6, 1, 0) == [1]
    assert co.kept_tokens(w, 6, 2, 0) == [1, 2]
    assert co.kept_tokens(w, 6, 5, 0) == [0, 1, 2, 3, 5]  # -0.0 ties with 0.0: the lower row


def test_evicted_rows_keep_their_values():
    rng = np.random.default_rng(6)
    x = _bf16(rng, (1, 1, 200, 8))
    x = np.where(np.abs(x) < 0.25, 0.25, x)  # far above the smallest normal code of any block here
    k, ks, lens = co.append(*_cache(1, 1, 200, 8, 64), x, 64)
    w = rng.random((1, 1, 200))
    z = _cache(1, 1, 100, 8, 64)
    dst = dict(k=z[0], ks=z[1], v=z[0], vs=z[1], lens=z[2], weight=np.zeros((1, 1, 100)))
    out, idx = co.evict(k, ks, k, ks, lens, w, 64, 90, 20, dst)
    assert out["lens"][0] == 90 and list(idx[0, 0, -20:]) == list(range(180, 200))
    np.testing.assert_array_equal(co.values(out["k"][0, 0, :90], out["ks"][0, 0], 64),
                                  co.values(k[0, 0], ks[0, 0], 64)[idx[0, 0]])
    np.testing.assert_array_equal(out["weight"][0, 0, :90], w[0, 0, idx[0, 0]])


def test_fc_gather_is_exact_in_bf16():
    rng = np.random.default_rng(7)
    k, ks, _ = co.append(*_cache(1, 2, 70, 16, 64), _bf16(rng, (1, 2, 70, 16)) * 100, 64)
    fc = np.array([[0, 3, 5, 7], [1, 2, 4, 6]])
    out = co.fc_gather(k, ks, fc, 64)
    np.testing.assert_array_equal(torch.from_numpy(out).bfloat16().double().numpy(), out)
    assert out[0, 1, 69, 1] == co.values(k[0, 1], ks[0, 1], 64)[69, 2]
    assert out[0, 0, 0, 6] == co.values(k[0, 0], ks[0, 0], 64)[0, 5 + 8]
